"""GPU parity of the RMS norm (fq_rms_norm_fwd, fq_rms_norm_bwd) with the
oracle: the stream, y, codes and scales bit for bit, gradients within the
stated rounding bounds."""
import numpy as np
import pytest

from oracle import norm as ON
from oracle.numerics import bf16_rne
from tests.fq_testutil import assert_bits_equal, from_dev, to_dev, to_dev_bf16, torch

pytestmark = pytest.mark.gpu
EPS = 1e-6

# one wave per row (with 1, 2 and 4 vectors a lane, ragged ends), one block per
# row of every kind, the longest row, a single element vector
SHAPES = [(1, 8), (1, 2048), (3, 1000), (1025, 64), (1030, 520), (1027, 1000), (2047, 2048), (2049, 64), (2051, 520),
          (2053, 1000), (2050, 2048), (77, 2056), (5, 8192),
          (3, 16384), (2, 65536)]


def _F():
    from scale_only_quantization_amd import fqlib
    return fqlib


def _data(seed, R, C):
    rng = np.random.default_rng(seed)
    size = np.exp(rng.standard_normal((R, 1)) * 2)
    b = lambda a: bf16_rne(a.astype(np.float32))  # noqa: E731
    x = b(rng.standard_normal((R, C)) * size)
    res = b(rng.standard_normal((R, C)) * size)
    g = b(1 + 0.3 * rng.standard_normal(C))
    if R > 2:
        x[1] = 0.0
        res[1] = 0.0                                   # an empty row
    return x, res, g, b(rng.standard_normal((R, C)) * 0.01), b(rng.standard_normal((R, C)) * 0.01)


def _quants(F, C):
    q = [("none", None), ("fp8_row", F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_ROW, 0, F.FQ_DYNAMIC)),
         ("int8_row", F.qdesc(F.FQ_INT, F.FQ_PER_ROW, 0, F.FQ_DYNAMIC, -128, 127)),
         ("fp8_tensor", F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_TENSOR, 0, F.FQ_STATIC)),
         ("int8_g8", F.qdesc(F.FQ_INT, F.FQ_PER_GROUP, 8, F.FQ_DYNAMIC, -127, 127))]
    for g in (64, 512):
        if C % g == 0:
            q.append((f"fp8_g{g}", F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_GROUP, g, F.FQ_DYNAMIC)))
    return q


def _forward(F, x, res, g, q, want_y=True):
    T = torch()
    R, C = x.shape
    new = lambda dt, *s: T.full(s, 7, dtype=dt, device="cuda")  # noqa: E731
    o = dict(sum=new(T.bfloat16, R, C) if res is not None else None, y=new(T.bfloat16, R, C) if want_y else None,
             rstd=new(T.float32, R), codes=None, scale=None)
    if q is not None:
        o["codes"] = new(T.uint8, R, C)
        o["scale"] = (T.full((1,), 0.013, device="cuda") if q.gran == F.FQ_PER_TENSOR
                      else new(T.float32, R) if q.gran == F.FQ_PER_ROW else new(T.float32, R, C // q.group))
    F.rms_norm_fwd(to_dev_bf16(x), to_dev_bf16(g), EPS, residual=None if res is None else to_dev_bf16(res),
                   q=q, **o)
    T.cuda.synchronize()
    return o


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("with_res", [False, True], ids=["plain", "residual"])
def test_forward_bits(R, C, with_res):
    F, T = _F(), torch()
    x, res, g, _, _ = _data(R + C, R, C)
    s, y, r = ON.forward(x, g, EPS, res if with_res else None)
    for name, q in _quants(F, C):
        o = _forward(F, x, res if with_res else None, g, q, want_y=name != "fp8_row")
        if with_res:
            assert_bits_equal(from_dev(o["sum"]), s, f"{name} sum")
        if o["y"] is not None:
            assert_bits_equal(from_dev(o["y"]), y, f"{name} y")
        np.testing.assert_allclose(from_dev(o["rstd"]), r, rtol=2.0 ** -23, err_msg=name)
        if q is None:
            continue
        # the codes fq_tensor gives on y, and the definition's scale
        yd = to_dev_bf16(y)
        codes = T.empty((R, C), dtype=T.uint8, device="cuda")
        F.fq_tensor(q, yd, scale=o["scale"] if q.gran == F.FQ_PER_TENSOR else None, codes=codes)
        T.cuda.synchronize()
        np.testing.assert_array_equal(from_dev(o["codes"]), from_dev(codes), err_msg=name)
        if q.gran != F.FQ_PER_TENSOR:
            b = np.abs(y).reshape(R, -1, q.group if q.gran == F.FQ_PER_GROUP else C).max(-1)
            div = np.float32(448.0 if q.kind == F.FQ_FP8E4M3 else q.qmax)
            assert_bits_equal(from_dev(o["scale"]), (b / div).reshape(o["scale"].shape), f"{name} scale")


def test_forward_in_place_and_nothing_past_the_end():
    F, T = _F(), torch()
    x, res, g, _, _ = _data(5, 37, 1000)
    s, y, _ = ON.forward(x, g, EPS, res)
    # the stream over the residual, and one row more behind every output
    pad = lambda a: T.cat([to_dev_bf16(a), T.full((1, 1000), 5.0, dtype=T.bfloat16, device="cuda")])  # noqa: E731
    dx, dr, dy = pad(x), pad(res), pad(x)
    F.rms_norm_fwd(dx[:37], to_dev_bf16(g), EPS, residual=dr[:37], sum=dr[:37], y=dy[:37])
    T.cuda.synchronize()
    assert_bits_equal(from_dev(dr[:37]), s, "sum over the residual")
    assert_bits_equal(from_dev(dy[:37]), y, "y")
    assert bool((dr[37:] == 5).all()) and bool((dy[37:] == 5).all())
    # y over x
    _, y1, _ = ON.forward(x, g, EPS)
    F.rms_norm_fwd(dx[:37], to_dev_bf16(g), EPS, y=dx[:37])
    assert_bits_equal(from_dev(dx[:37]), y1, "y over x")


def test_not_finite_rows_stay_their_own():
    F, T = _F(), torch()
    x, _, g, _, _ = _data(6, 9, 520)
    x[2, 7] = np.inf
    x[4, 0] = np.nan
    o = _forward(F, x, None, g, None)
    y = from_dev(o["y"])
    keep = [i for i in range(9) if i not in (2, 4)]
    assert_bits_equal(y[keep], ON.forward(x[keep], g, EPS)[1], "finite rows")
    assert np.isnan(y[4]).all() and np.isnan(y[2, 7])


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("extra", [False, True], ids=["dx", "dsum_dgamma"])
def test_backward(R, C, extra):
    F, T = _F(), torch()
    x, _, g, dy, dsum = _data(R * 3 + C, R, C)
    _, _, r = ON.forward(x, g, EPS)
    r32 = r.astype(np.float32)
    dx_ref, dg_ref = ON.backward(x, g, r32, dy, dsum if extra else None)
    dx = T.empty((R, C), dtype=T.bfloat16, device="cuda")
    dg = T.empty(C, dtype=T.float32, device="cuda") if extra else None
    ws = T.empty(F.rms_norm_bwd_workspace_size(R, C), dtype=T.uint8, device="cuda") if extra else None
    args = [to_dev_bf16(x), to_dev_bf16(g), to_dev(r32), to_dev_bf16(dy), dx]
    kw = dict(dsum=to_dev_bf16(dsum) if extra else None, dgamma=dg, workspace=ws)
    F.rms_norm_bwd(*args, **kw)
    T.cuda.synchronize()
    # one bf16 rounding; in fp32, half an ulp for each of the few operations on
    # the largest terms, and of the row's sum of at most 128 steps per thread
    # and 12 more across threads
    a, rr = np.abs(dy.astype(np.float64) * g), r32.astype(np.float64)[:, None]
    s = np.abs(x.astype(np.float64))
    terms = rr * (a + s * rr * rr * np.mean(a * s, -1, keepdims=True)) + (np.abs(dsum) if extra else 0)
    err = np.abs(from_dev(dx) - dx_ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(dx_ref) + 160 * 2.0 ** -24 * terms), f"dx off by {err.max()}"
    if extra:
        # a sum over the rows in fp32: at most R + 40 roundings of the running sum
        tot = np.sum(np.abs(dy.astype(np.float64) * x * rr), 0)
        err = np.abs(from_dev(dg) - dg_ref)
        assert np.all(err <= (R + 40) * 2.0 ** -24 * tot), f"dgamma off by {err.max()}"
        one = (from_dev(dx), from_dev(dg))
        F.rms_norm_bwd(*args, **kw)
        np.testing.assert_array_equal(from_dev(dx), one[0])
        np.testing.assert_array_equal(from_dev(dg), one[1])


def test_backward_matches_differences():
    # the directional derivative of the 64-bit forward against the kernel's dx
    F, T = _F(), torch()
    x, _, g, dy, _ = _data(11, 1, 4096)
    _, _, r = ON.forward(x, g, EPS)
    dx = T.empty((1, 4096), dtype=T.bfloat16, device="cuda")
    F.rms_norm_bwd(to_dev_bf16(x), to_dev_bf16(g), to_dev(r.astype(np.float32)), to_dev_bf16(dy), dx)
    u = np.random.default_rng(0).standard_normal(x.shape)

    def f(h):
        z = x.astype(np.float64) + h * u
        return np.sum(dy * z * g / np.sqrt(np.mean(z * z, -1, keepdims=True) + EPS))
    h = 1e-5 * float(np.abs(x).max())
    d = from_dev(dx).astype(np.float64)
    # each dx is off by at most 2^-8 of itself (bf16): the sum by the root of the squares, five times over
    tol = 5 * 2.0 ** -8 * np.linalg.norm(d * u)
    assert abs((f(h) - f(-h)) / (2 * h) - np.sum(d * u)) <= tol


def test_zero_rows():
    F, T = _F(), torch()
    z = T.empty((0, 64), dtype=T.bfloat16, device="cuda")
    g = T.ones(64, dtype=T.bfloat16, device="cuda")
    F.rms_norm_fwd(z, g, EPS, y=z)
    dg = T.full((64,), 3.0, device="cuda")
    F.rms_norm_bwd(z, g, T.empty(0, device="cuda"), z, z, dgamma=dg,
                   workspace=T.empty(64, dtype=T.float32, device="cuda"))
    T.cuda.synchronize()
    assert not from_dev(dg).any()


def test_more_blocks_than_one_grid_row():
    # 2^26 + 7 short rows: four rows a block of 256 threads are more than 2^32 threads
    F, T = _F(), torch()
    R, C = (1 << 26) + 7, 8
    x = T.randn((R, C), device="cuda", dtype=T.bfloat16)
    g = T.linspace(0.5, 1.5, C, device="cuda").to(T.bfloat16)
    y, r = T.full_like(x, 7), T.full((R + 1,), -1.0, device="cuda")
    F.rms_norm_fwd(x, g, EPS, y=y, rstd=r[:R])
    T.cuda.synchronize()
    rng = np.random.default_rng(1)
    edge = [(i << 22) + j for i in range(17) for j in range(-5, 6)]        # where the grid's rows of blocks meet
    pick = np.unique(np.clip(np.concatenate([edge, rng.integers(0, R, 5000), [0, R - 1, R - 5, R - 6]]), 0, R - 1))
    at = to_dev(pick.astype(np.int64))
    _, ref, rr = ON.forward(from_dev(x[at]), from_dev(g), EPS)
    assert_bits_equal(from_dev(y[at]), ref, "y")
    np.testing.assert_allclose(from_dev(r[at]), rr, rtol=2.0 ** -23)
    assert float(r[R]) == -1.0 and bool((r[:R] > 0).all())                 # no row left out, none past the end
