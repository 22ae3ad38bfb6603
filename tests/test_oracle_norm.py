"""The norm's oracle against torch autograd in 64 bits and finite differences."""
import numpy as np
import torch

from oracle import norm as ON
from oracle.numerics import bf16_rne


def _data(seed, R, C):
    rng = np.random.default_rng(seed)
    b = lambda *s: bf16_rne(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    return b(R, C), b(R, C), b(C), b(R, C), b(R, C)


def test_backward_is_autograd_of_the_forward():
    x, res, g, dy, dsum = _data(1, 5, 40)
    s, y, r = ON.forward(x, g, 1e-6, res)
    ts = torch.tensor(s, dtype=torch.float64, requires_grad=True)
    tg = torch.tensor(g, dtype=torch.float64, requires_grad=True)
    ty = ts * tg / torch.sqrt((ts * ts).mean(-1, keepdim=True) + 1e-6)
    np.testing.assert_array_equal(y, bf16_rne(ty.detach().numpy().astype(np.float32)))
    ((ty * torch.tensor(dy)).sum() + (ts * torch.tensor(dsum)).sum()).backward()
    dx, dg = ON.backward(s, g, r, dy, dsum)
    np.testing.assert_allclose(dx, ts.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dg, tg.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_backward_matches_differences():
    x, _, g, dy, _ = _data(2, 3, 24)
    s, _, r = ON.forward(x, g, 1e-3)
    dx, _ = ON.backward(s, g, r, dy)
    rng = np.random.default_rng(3)
    u = rng.standard_normal(s.shape)

    def f(h):
        z = s.astype(np.float64) + h * u
        return np.sum(dy * z * g / np.sqrt(np.mean(z * z, -1, keepdims=True) + 1e-3))
    h = 1e-5
    np.testing.assert_allclose((f(h) - f(-h)) / (2 * h), np.sum(dx * u), rtol=1e-7, atol=1e-9)


def test_zero_rows_and_the_residual():
    s, y, r = ON.forward(np.zeros((2, 8), np.float32), np.ones(8, np.float32), 1e-6)
    assert not y.any() and np.allclose(r, 1e3)
    x, res, g, _, _ = _data(4, 2, 16)
    s, _, _ = ON.forward(x, g, 1e-6, res)
    np.testing.assert_array_equal(s, bf16_rne(x + res))
