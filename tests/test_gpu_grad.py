"""GPU parity of the norm over many gradients and the clipping by it (fq_grad_norm, fq_grad_clip) with float64."""
import numpy as np
import pytest

from tests.fq_testutil import torch

pytestmark = pytest.mark.gpu


def _F():
    from scale_only_quantization_amd import fqlib
    return fqlib


def _tensors(spec, seed=1, scale=1.0):
    """spec: (length, bf16, offset in elements from a 256-byte boundary)."""
    T_ = torch()
    g = T_.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for n, bf, off in spec:
        x = T_.randn(n + off, generator=g, device="cuda") * scale
        out.append((x.to(T_.bfloat16) if bf else x)[off:])
    return out


def _norm(F, grads, ws=True):
    T_ = torch()
    G = F.grad_list(grads)
    norm = T_.full((1,), 9.0, device="cuda")
    n = F.grad_norm_workspace_size(G)
    # 0xFF: a NaN wherever something would be read before it is written
    F.grad_norm(G, norm, T_.full((n,), 255, dtype=T_.uint8, device="cuda") if n else None)
    T_.cuda.synchronize()
    return norm


def _exact(grads):
    return float(np.sqrt(sum(float((g.double() ** 2).sum()) for g in grads)))


SPECS = {
    "one": [(1, False, 0)],
    "one bf16": [(1, True, 1)],
    "empty ones": [(0, False, 0), (5, False, 0), (0, True, 0), (3, True, 0), (0, False, 0)],
    "all empty": [(0, False, 0)] * 3,
    "offsets": [(n, bf, o) for n in (7, 8, 9, 255, 4097) for bf in (False, True) for o in (0, 1, 2, 3, 5, 7)],
    "chunks": [(16384, False, 0), (16385, True, 0), (16383, False, 1), (32768, True, 3), (163847, False, 0)],
    "short": [(1024, i % 2 == 0, i % 3) for i in range(32)],
    "short, one more element": [(1024, i % 2 == 0, i % 3) for i in range(32)] + [(1, False, 0)],
    "64 short": [(512, i % 2 == 0, i % 3) for i in range(64)] + [(0, False, 0)],
    "65 short": [(500, i % 2 == 0, i % 3) for i in range(65)],
    "95": [(100 + i, i % 2 == 0, i % 4) for i in range(95)],
    "96": [(100 + i, i % 2 == 0, i % 4) for i in range(96)],
    "97": [(100 + i, i % 2 == 0, i % 4) for i in range(97)],
    "136": [(2000 + i, i % 2 == 0, i % 4) for i in range(136)],
    "137": [(2000 + i, i % 2 == 0, i % 4) for i in range(137)],
    "192": [(2000 + i, i % 2 == 0, i % 4) for i in range(192)],
    "193": [(2000 + i, i % 2 == 0, i % 4) for i in range(193)],
    "500 with empty ones": [((i * 37) % 301, i % 3 == 0, i % 3) for i in range(500)],
    "long": [(128 * 1536 * 128, False, 0), (3_000_001, True, 1), (128, False, 0)],
}


@pytest.mark.parametrize("name", list(SPECS))
def test_norm_and_clip(name):
    F, T_ = _F(), torch()
    grads = _tensors(SPECS[name])
    ref = _exact(grads)
    norm = _norm(F, grads)
    # fp64 sums of at most 2^25 squares, then one rounding to fp32
    assert abs(norm.item() - ref) <= ref * (2.0 ** -24 + 1e-8)
    limit = 0.37 * ref if ref else 1.0
    outs = [T_.full_like(g, 7.0) for g in grads]
    keep = [g.clone() for g in grads]
    F.grad_clip(F.grad_list(grads, outs), limit, norm)
    T_.cuda.synchronize()
    c = np.float32(min(1.0, float(np.float32(limit)) / (norm.double().item() + 1e-6)))
    for g, k, o in zip(grads, keep, outs):
        assert T_.equal(g, k)                                              # the gradients stay
        assert T_.equal(o, (k.float() * float(c)).to(k.dtype))             # one rounding of the fp32 product
    F.grad_clip(F.grad_list(grads), limit, norm)                           # in place
    T_.cuda.synchronize()
    for g, o in zip(grads, outs):
        assert T_.equal(g, o)


def test_neighbours_are_left_alone():
    """Clipped views of one buffer: what lies between them keeps its values."""
    F, T_ = _F(), torch()
    for dt in (T_.float32, T_.bfloat16):
        buf = T_.ones(100_000, dtype=dt, device="cuda")
        views = [buf[3:10], buf[11:12], buf[13:17000], buf[17001:50_003], buf[50_004:99_999]]
        norm = _norm(F, views)
        F.grad_clip(F.grad_list(views), 0.5 * norm.item(), norm)
        T_.cuda.synchronize()
        for at in (0, 1, 2, 10, 12, 17000, 50_003, 99_999):
            assert buf[at].item() == 1.0, at
        for v in views:
            assert bool((v == 0.5).all())


def test_no_clipping_leaves_or_copies():
    F, T_ = _F(), torch()
    grads = _tensors([(1000, False, 0), (1000, True, 1)])
    keep = [g.clone() for g in grads]
    norm = _norm(F, grads)
    outs = [T_.zeros_like(g) for g in grads]
    F.grad_clip(F.grad_list(grads), norm.item() * 2, norm)
    F.grad_clip(F.grad_list(grads, outs), norm.item() * 2, norm)
    T_.cuda.synchronize()
    for g, k, o in zip(grads, keep, outs):
        assert T_.equal(g, k) and T_.equal(o, k)


def test_norms_that_are_not_finite():
    F, T_ = _F(), torch()
    grads = _tensors([(1000, False, 0), (50, True, 0)])
    grads[0][17] = float("inf")
    norm = _norm(F, grads)
    assert norm.item() == float("inf")
    F.grad_clip(F.grad_list(grads), 1.0, norm)
    T_.cuda.synchronize()
    assert bool(T_.isnan(grads[0][17])) and bool((grads[0][18:] == 0).all()) and bool((grads[1] == 0).all())
    grads = _tensors([(1000, False, 0)])
    grads[0][3] = float("nan")
    norm = _norm(F, grads)
    assert bool(T_.isnan(norm).all())
    F.grad_clip(F.grad_list(grads), 1.0, norm)
    T_.cuda.synchronize()
    assert bool(T_.isnan(grads[0]).all())


def test_squares_past_fp32():
    F = _F()
    grads = _tensors([(5000, False, 0)], scale=1e30) + _tensors([(5000, True, 0)], scale=1e-30)
    ref = _exact(grads)
    assert abs(_norm(F, grads).item() - ref) <= ref * 2.0 ** -23


def test_no_tensors():
    F, T_ = _F(), torch()
    assert _norm(F, []).item() == 0.0
    F.grad_clip(F.grad_list([]), 1.0, T_.zeros(1, device="cuda"))


def test_same_result_every_time_and_past_2_31():
    """More than 2^31 elements in one tensor (bf16), and bitwise the same norm twice."""
    F, T_ = _F(), torch()
    n = (1 << 31) + 4099
    x = T_.full((n,), 0.5, dtype=T_.bfloat16, device="cuda")
    x[-1] = 3.0
    a, b = _norm(F, [x]), _norm(F, [x])
    assert T_.equal(a, b)
    ref = np.sqrt((n - 1) * 0.25 + 9.0)
    assert abs(a.item() - ref) <= ref * 2.0 ** -23
    F.grad_clip(F.grad_list([x]), a.item() / 2, a)
    T_.cuda.synchronize()
    assert x[-1].item() == 1.5 and x[-2].item() == 0.25 and x[0].item() == 0.25 and x[1 << 31].item() == 0.25


def test_joint_clipping_equals_the_optimisers():
    """fq_grad_norm and fq_grad_clip over the tensors of several layers, then fq_scale_adamw layer by layer without a
    clip, against one fq_scale_adamw call that clips all of them."""
    F, T_ = _F(), torch()
    g = T_.Generator(device="cuda")
    g.manual_seed(4)
    size = [5000, 128, 2500, 128] * 3
    r = lambda n, f: T_.randn(n, generator=g, device="cuda") * f  # noqa: E731
    state = [(r(n, 1e-3).abs() + 1e-3, r(n, 0.5), r(n, 1e-3), r(n, 1e-3).abs() * 1e-3) for n in size]
    copy = [tuple(x.clone() for x in s) for s in state]
    hp = F.adamw_defaults()
    ps = [F.scale_param(*s) for s in state]
    want = T_.zeros(1, device="cuda")
    F.scale_adamw(ps, hp, 1, grad_norm=want,
                  workspace=T_.empty(F.scale_adamw_workspace_size(ps), dtype=T_.uint8, device="cuda"))
    norm = _norm(F, [s[1] for s in copy])
    # both are one rounding of sums in fp64
    assert abs(norm.item() - want.item()) <= want.item() * 2.0 ** -23
    F.grad_clip(F.grad_list([s[1] for s in copy]), hp.max_grad_norm, norm)
    hp0 = F.adamw_defaults(max_grad_norm=0.0)
    for i in range(0, len(copy), 4):
        ps = [F.scale_param(*s) for s in copy[i:i + 4]]
        F.scale_adamw(ps, hp0, 1, workspace=T_.empty(F.scale_adamw_workspace_size(ps), dtype=T_.uint8, device="cuda"))
    T_.cuda.synchronize()
    for a, b in zip(state, copy):
        # the clip factor may differ by an fp32 ulp: two half ulps on g', four on its square
        assert T_.allclose(a[2], b[2], rtol=2.0 ** -21, atol=1e-9)
        assert T_.allclose(a[3], b[3], rtol=2.0 ** -20, atol=1e-12)
        assert T_.allclose(a[0], b[0], rtol=2.0 ** -18, atol=0.0)
