"""The head loss's oracle against torch autograd in 64 bits, the logits' loss of
oracle/distill.py, and finite differences."""
import numpy as np
import pytest
import torch

from oracle.distill import distill
from oracle.head import head


def _data(seed, T=6, H=16, V=40, k=5):
    rng = np.random.default_rng(seed)
    h, w = rng.standard_normal((T, H)), rng.standard_normal((V, H)) * 0.5
    ti = np.stack([rng.permutation(V)[:k] for _ in range(T)]).astype(np.int32)
    return h, w, rng.standard_normal((T, k)) * 2, ti, rng.integers(0, V, T).astype(np.int32)


def test_equals_the_loss_on_logits():
    h, w, tv, ti, lab = _data(1)
    loss, rows, grad, _ = head(h, w, tv, ti, lab, 0.7, 1.3)
    ref, ref_rows, gz = distill("topk_kl", h @ w.T, top_v=tv, top_i=ti, labels=lab, lm_weight=0.7, distill_weight=1.3)
    assert loss == pytest.approx(ref, rel=1e-12)
    np.testing.assert_allclose(rows, ref_rows, rtol=1e-10)
    np.testing.assert_allclose(grad, gz @ w, rtol=1e-9, atol=1e-14)


def test_masked_rows_and_absent_ids():
    h, w, tv, ti, lab = _data(2)
    lab[1], lab[4] = -1, 40                      # padding and a label past the vocabulary: rows that do not count
    ti[0, 2], ti[2] = -1, 99                     # one absent id, and a row with none left
    loss, rows, grad, _ = head(h, w, tv, ti, lab, 0.5, 1.0)
    live = [0, 2, 3, 5]
    assert rows[1] == rows[4] == 0 and not grad[[1, 4]].any()
    keep = np.ones(5, bool)
    keep[2] = False
    _, r0, _ = distill("topk_kl", h[:1] @ w.T, top_v=tv[:1, keep], top_i=ti[:1, keep], labels=lab[:1], lm_weight=0.5)
    assert rows[0] == pytest.approx(r0[0])
    lse = np.log(np.exp(h[2] @ w.T).sum())
    assert rows[2] == pytest.approx(0.5 * (lse - h[2] @ w[lab[2]]))
    assert loss == pytest.approx(rows[live].mean())
    assert head(h, w, tv, ti, np.full(6, -1, np.int32))[0] == 0.0


def test_repeated_ids_and_autograd():
    h, w, tv, ti, lab = _data(3)
    ti[:, 1] = ti[:, 0]
    ti[:, 2] = lab
    loss, _, grad, _ = head(h, w, tv, ti, lab, 0.8, 1.2)
    x = torch.tensor(h, requires_grad=True)
    lq = torch.log_softmax(x @ torch.tensor(w).T, -1)
    lp = torch.log_softmax(torch.tensor(tv), -1)
    t = 0.8 * -lq.gather(1, torch.tensor(lab).long()[:, None])[:, 0]
    t = t + 1.2 * (lp.exp() * (lp - lq.gather(1, torch.tensor(ti).long()))).sum(-1)
    t.mean().backward()
    assert loss == pytest.approx(t.mean().item(), rel=1e-12)
    np.testing.assert_allclose(grad, x.grad.numpy(), rtol=1e-9, atol=1e-13)


def test_differences():
    h, w, tv, ti, lab = _data(4)
    lab[3] = -1
    u = np.random.default_rng(5).standard_normal(h.shape)
    f = lambda e: head(h + e * u, w, tv, ti, lab, 0.8, 1.2)[0]  # noqa: E731
    d = (f(1e-5) - f(-1e-5)) / 2e-5
    assert d == pytest.approx(np.sum(head(h, w, tv, ti, lab, 0.8, 1.2)[2] * u), rel=1e-7)
