"""GPU parity of log probabilities, entropy, the most likely tokens and their
gradient (fq_logprob_*, fq_head_logprob_*) with the oracle.

Ids are compared as whole numbers.  From logits they are exact by definition
(comparisons of bf16 values).  From hidden states the inputs lie on grids of
powers of two on which every partial sum is exact in fp32, so that the logits
do not depend on the order of the sum."""
import numpy as np
import pytest

from oracle import logprob as O
from oracle.numerics import bf16_rne
from tests.fq_testutil import from_dev, to_dev, to_dev_bf16, torch

pytestmark = pytest.mark.gpu
H32 = 2.0 ** -24          # half an ulp of fp32, relative
H16 = 2.0 ** -8           # of bf16


def _F():
    from scale_only_quantization_amd import fqlib
    return fqlib


def _padded(z, pad, fill):
    """bf16 device tensor of z's rows with a stride of V rounded up to 8, and pad more, filled with `fill`."""
    T_ = torch()
    T, V = z.shape
    buf = T_.full((T, (V + 7) // 8 * 8 + pad), fill, dtype=T_.bfloat16, device="cuda")
    buf[:, :V] = to_dev_bf16(z)
    return buf, buf[:, :V]


def _out(T, m, k):
    T_ = torch()
    f = lambda *s: T_.full(s, 9.0, device="cuda")  # noqa: E731
    return dict(lse=f(T), entropy=f(T), logp=f(T, m) if m else None, top_logp=f(T, k) if k else None,
                top_ids=T_.full((T, k), -9, dtype=T_.int32, device="cuda") if k else None)


def _workspace(n):
    T_ = torch()
    # 0xFF: a NaN wherever something would be read before it is written
    return T_.full((n,), 255, dtype=T_.uint8, device="cuda") if n else None


def _ids(rng, T, V, m):
    """Given tokens: any, with padding, ids past the vocabulary and repeated ones among them."""
    ids = rng.integers(0, V, (T, m)).astype(np.int32)
    if m > 1:
        ids[::2, 1] = ids[::2, 0]
    if T > 2 and m:
        ids[1, 0], ids[2, m - 1] = -1, V
    return ids


def _check_forward(got, z, ids, k, zerr=0.0, what=""):
    """z in float64, known to zerr.  The kernel's s and u are sums of positive (negative) terms: an element enters by
    three roundings (z - M, times log2 e, the exponential's ulp; the first two move it by |d| 2 half ulps, and
    |d| e^d stays below e^d / (1 - 1/e) in a sum whose largest term is 1), then at most 128 sequential additions and
    32 of trees and chunks."""
    ref = O.forward(z, ids, k)
    lse, ent = from_dev(got["lse"]).astype(np.float64), from_dev(got["entropy"])
    fin = np.isfinite(ref["lse"])
    assert np.array_equal(lse[~fin], ref["lse"][~fin]), what
    lp = np.where(np.isfinite(ref["lse"])[:, None], z - np.where(fin, ref["lse"], 0.0)[:, None], -np.inf)
    p = np.exp(lp)
    with np.errstate(invalid="ignore"):
        spread = np.sum(p * np.where(p > 0, np.abs(z - np.where(fin, z.max(-1), 0.0)[:, None]), 0.0), -1)  # E |z - M|
    rel = (160 + 8 + 2 * spread) * H32
    with np.errstate(invalid="ignore"):
        tol = rel + 3 * H32 * np.abs(ref["lse"]) + zerr
        assert np.all(np.abs(lse - ref["lse"])[fin] <= tol[fin]), (what, np.abs(lse - ref["lse"])[fin].max())
        etol = rel * (1 + 2 * spread) + 4 * H32 * (spread + np.abs(ref["entropy"]) + 1) + 2 * zerr * (1 + spread)
    assert np.all(np.abs(ent - ref["entropy"])[fin] <= etol[fin]), (what, np.abs(ent - ref["entropy"]).max())
    assert np.all(ent[~fin] == 0.0)

    def close(x, r):
        inf = np.isinf(r)
        assert np.array_equal(x[inf], r[inf]), what
        t = np.broadcast_to(np.where(fin, tol, 0.0)[:, None] + zerr, r.shape)[~inf] + H32 * np.abs(r[~inf])
        assert np.all(np.abs(x[~inf] - r[~inf]) <= t), (what, np.abs(x[~inf] - r[~inf]).max())
        assert np.all(x <= 0.0), what

    if ids is not None and ids.shape[1]:
        close(from_dev(got["logp"]).astype(np.float64), ref["logp"])
    if k:
        assert np.array_equal(from_dev(got["top_ids"]), ref["top_ids"]), what
        close(from_dev(got["top_logp"]).astype(np.float64), ref["top_logp"])
    return ref


def _logits_fwd(z, ids, k, pad=0, fill=np.nan):
    F, T_ = _F(), torch()
    T, V = z.shape
    m = 0 if ids is None else ids.shape[1]
    d = F.logprob_desc(T, V, given=m, top=k)
    out = _out(T, m, k)
    F.logprob_fwd(d, _padded(z, pad, fill)[1], ids=to_dev(ids) if m else None,
                  workspace=_workspace(F.logprob_workspace_size(d)), **out)
    T_.cuda.synchronize()
    return out


@pytest.mark.parametrize("T,V,m,k,pad", [
    (1, 1, 1, 1, 0), (1, 7, 0, 3, 0), (3, 8, 2, 8, 8), (5, 63, 1, 5, 0), (2, 64, 64, 64, 0), (4, 65, 1, 64, 16),
    (33, 4099, 3, 64, 0), (3, 4096, 1, 33, 0), (1, 32003, 1, 20, 0), (4, 16384, 0, 64, 8), (7, 16385, 64, 33, 0),
    (530, 700, 1, 64, 0), (520, 17001, 2, 64, 0), (600, 4104, 1, 0, 0), (6, 151936, 1, 64, 0)])
def test_logits(T, V, m, k, pad):
    rng = np.random.default_rng(T * 1000 + V + k)
    z = bf16_rne((rng.standard_normal((T, V)) * 2 + rng.random((T, 1)) * 20 - 10).astype(np.float32))
    ids = _ids(rng, T, V, m) if m else None
    _check_forward(_logits_fwd(z, ids, k, pad), z.astype(np.float64), ids, k, what=f"{T}x{V}")


KINDS = ("equal", "zeros of both signs", "rising", "falling", "two values", "ruled out", "nothing", "few", "lowest",
         "sure", "wide")


def _row(kind, V, rng):
    z = rng.standard_normal(V) * 2
    if kind == "equal":
        z[:] = 1.5
    elif kind == "zeros of both signs":
        z = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    elif kind == "rising":
        z = np.linspace(-8, 8, V)
    elif kind == "falling":
        z = np.linspace(8, -8, V)
    elif kind == "two values":
        z = np.where(rng.random(V) < 0.3, 2.0, 1.0)
    elif kind == "ruled out":
        z[rng.random(V) < 0.9] = -np.inf
    elif kind == "nothing":
        z[:] = -np.inf
    elif kind == "few":
        keep = rng.choice(V, 5, replace=False)
        y = z[keep]
        z[:] = -np.inf
        z[keep] = y
    elif kind == "lowest":
        z[rng.random(V) < 0.999] = -3.3895313892515355e38
    elif kind == "sure":
        z[rng.integers(V)] = 60.0
    elif kind == "wide":
        z *= 3e4
    return z


@pytest.mark.parametrize("V", [300, 5000, 40001])
@pytest.mark.parametrize("many", [False, True])
def test_logits_of_every_kind(V, many):
    """Rows that tie everywhere, are sorted, ruled out, all but sure; long chunks (many rows) and short ones."""
    rng = np.random.default_rng(V)
    z = np.stack([_row(kind, V, rng) for kind in KINDS])
    z = bf16_rne(np.tile(z, (50 if many else 1, 1)).astype(np.float32))
    ids = _ids(rng, z.shape[0], V, 3)
    got = _logits_fwd(z, ids, 64)
    _check_forward(got, z.astype(np.float64), ids, 64, what=f"V={V}")
    # the same row wherever it stands
    for n in ("lse", "entropy", "top_ids", "top_logp"):
        x = from_dev(got[n])
        assert np.array_equal(x, np.tile(x[:len(KINDS)], (z.shape[0] // len(KINDS),) + (1,) * (x.ndim - 1))), n


@pytest.mark.parametrize("V", [300, 5000, 40001])
@pytest.mark.parametrize("many", [False, True])
def test_logits_masked_by_the_lowest_value(V, many):
    """Masks of the type's lowest value over whole chunks, over all of a row but a few entries, over a whole row, with
    ruled-out entries among them; and entries at the other end of the type's range."""
    rng = np.random.default_rng(V + 7)
    low = -3.3895313892515355e38
    z = np.full((6, V), low)
    z[0, V // 2:V // 2 + 7] = rng.standard_normal(7)             # chunks of nothing but masks beside one with entries
    z[1, :2] = rng.standard_normal(2) * 1e4
    z[3, V // 3:] = -np.inf                                       # (2: a row of masks)
    z[4, rng.choice(V, 9, replace=False)] = -low
    z[5] = 2.0 ** 126 * (1 + rng.integers(0, 2, V) / 128)
    z = bf16_rne(np.tile(z, (100 if many else 1, 1)).astype(np.float32))
    ids = np.stack([np.zeros(len(z)), np.full(len(z), V // 2), np.full(len(z), V - 1)], 1).astype(np.int32)
    got = _logits_fwd(z, ids, 64)
    zz = z.astype(np.float64)
    near = np.arange(len(z)) % 6 < 2
    _check_forward({n: v[to_dev(near)] for n, v in got.items()}, zz[near], ids[near], 64, what=f"V={V}")
    # far rows: what is below the maximum is 2^118 and more below it, so p is uniform over the n largest (float64
    # loses log n beside the maximum, so it is taken apart here); counts below 2^24 are exact, a logarithm of fp32
    # is within 2 ulps
    far = ~near
    ref = O.forward(zz[far], ids[far], 64)
    top = zz[far].max(-1, keepdims=True)
    n = (zz[far] == top).sum(-1)
    with np.errstate(over="ignore"):
        lp = (zz[far] - top - np.log(n)[:, None]).astype(np.float32).astype(np.float64)    # past fp32: -inf
    lse, ent = from_dev(got["lse"])[far], from_dev(got["entropy"])[far]
    assert np.array_equal(lse, z[far].max(-1))
    assert np.all(np.abs(ent - np.log(n)) <= 4 * H32 * np.log(n))
    assert np.array_equal(from_dev(got["top_ids"])[far], ref["top_ids"])
    lt = np.where(ref["top_ids"] >= 0, np.take_along_axis(lp, np.maximum(ref["top_ids"], 0), 1), -np.inf)
    for x, r in ((from_dev(got["logp"])[far], np.take_along_axis(lp, ids[far], 1)), (from_dev(got["top_logp"])[far], lt)):
        finite = np.isfinite(r)
        assert np.array_equal(x[~finite], r[~finite])
        assert np.all(np.abs(x[finite] - r[finite]) <= 8 * H32 * np.abs(r[finite]))


def test_logits_nan_stays_in_its_row():
    rng = np.random.default_rng(5)
    z = bf16_rne(rng.standard_normal((3, 9000)).astype(np.float32))
    z[1, 4321] = np.nan
    got = _logits_fwd(z, None, 4)
    assert np.isnan(from_dev(got["lse"])[1]) and np.isnan(from_dev(got["entropy"])[1])
    ids = from_dev(got["top_ids"])
    assert np.all((ids >= -1) & (ids < 9000))
    ok = [0, 2]
    ref = O.forward(z[ok].astype(np.float64), None, 4)
    assert np.array_equal(ids[ok], ref["top_ids"]) and np.allclose(from_dev(got["lse"])[ok], ref["lse"], rtol=1e-5)


def _bwd_tolerance(g, part, z, a_abs, rnd, a):
    """bf16 of the result, and of p (A + b (log p + entropy)): the exponential's argument is known to a few half ulps
    of |z| + |lse|, and log p + entropy to as much.  A p below fp32's normal range, 2^-126, may be 0; what it is
    multiplied by is at most 30 a there (|log p| <= 200 where p > 0 in fp32)."""
    zmax = np.where(np.isfinite(z), np.abs(z), 0.0).max(-1, keepdims=True)
    rel = (16 + 6 * zmax) * H32
    return rnd * np.abs(g) * (1 + 1e-3) + rel * (part + np.exp(-1) * a_abs) + 2.0 ** -126 * 30 * a


@pytest.mark.parametrize("T,V,m,ent,place", [
    (1, 1, 1, True, "own"), (3, 8, 2, True, "in place"), (5, 77, 1, False, "own"), (4, 8193, 3, True, "in place"),
    (9, 20001, 64, True, "own"), (2, 16384, 0, True, "in place"), (40, 5000, 1, True, "own")])
def test_logits_gradient(T, V, m, ent, place):
    F, T_ = _F(), torch()
    rng = np.random.default_rng(V + m)
    z = np.stack([_row(KINDS[t % len(KINDS)], V, rng) if V > 10 else rng.standard_normal(V) for t in range(T)])
    z = bf16_rne(np.clip(z, -1e4, 1e4).astype(np.float32) * np.where(np.isinf(z), np.inf, 1.0).astype(np.float32))
    ids = _ids(rng, T, V, m) if m else None
    dl = rng.standard_normal((T, m)).astype(np.float32)
    de = (rng.standard_normal(T) * 0.3).astype(np.float32) if ent else None
    fwd = _logits_fwd(z, None, 0)
    ref, part = O.backward(z.astype(np.float64), ids, dl if m else None, de)
    buf, zv = _padded(z, 8, 3.0)
    if place == "own":
        gbuf, gv = _padded(np.full((T, V), 7.0, np.float32), 16, 5.0)
    else:
        gbuf, gv = buf, zv
    d = F.logprob_desc(T, V, given=m)
    F.logprob_bwd(d, zv, fwd["lse"], gv, ids=to_dev(ids) if m else None, dlogp=to_dev(dl) if m else None,
                  entropy=fwd["entropy"] if ent else None, dentropy=to_dev(de) if ent else None)
    T_.cuda.synchronize()
    g = from_dev(gv).astype(np.float64)
    lp = O.forward(z.astype(np.float64))
    sure = np.exp(z.astype(np.float64) - np.where(np.isfinite(lp["lse"]), lp["lse"], 0.0)[:, None])
    sure[~np.isfinite(lp["lse"])] = 0.0
    a = np.abs(dl).sum(-1)[:, None] + (np.abs(de)[:, None] * 12 if ent else 0.0)
    tol = _bwd_tolerance(ref, part, z, sure * a, H16, a)
    bad = np.abs(g - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], g[bad][:5], ref[bad][:5])
    assert np.all(from_dev(gbuf)[:, V:] == (5.0 if place == "own" else 3.0))       # what lies beyond the vocabulary


@pytest.mark.parametrize("m,ent", [(0, True), (1, False), (2, True)])
def test_logits_gradient_of_masks_and_nan(m, ent):
    """Rows of the type's lowest value have gradient 0 like ruled-out ones, a row with a NaN is NaN throughout, and the
    rows beside them are what they are alone."""
    F, T_ = _F(), torch()
    rng = np.random.default_rng(17 + m)
    V = 9001
    z = bf16_rne((rng.standard_normal((5, V)) * 2).astype(np.float32))
    z[1] = bf16_rne(np.full(V, -3.3895313892515355e38, np.float32))
    z[2, 8000] = np.inf if m == 1 else np.nan
    z[3] = -np.inf
    ids = np.tile(np.array([8000, 3][:m], np.int32), (5, 1)) if m else None
    dl, de = rng.standard_normal((5, m)).astype(np.float32), rng.standard_normal(5).astype(np.float32)

    def grad(rows):
        fwd = _logits_fwd(z[rows], None, 0)
        g = T_.full((len(rows), V + 7), 9.0, dtype=T_.bfloat16, device="cuda")[:, :V]
        zb = _padded(z[rows], 8, 0.0)[1]
        F.logprob_bwd(F.logprob_desc(len(rows), V, given=m), zb, fwd["lse"], g, ids=to_dev(ids[rows]) if m else None,
                      dlogp=to_dev(dl[rows]) if m else None, entropy=fwd["entropy"] if ent else None,
                      dentropy=to_dev(de[rows]) if ent else None)
        T_.cuda.synchronize()
        return from_dev(g)

    got = grad([0, 1, 2, 3, 4])
    assert np.all(got[[1, 3]] == 0.0)
    assert np.all(np.isnan(got[2]))
    assert np.array_equal(got[[0, 4]], grad([0, 4])) and np.all(np.isfinite(got[[0, 4]])) and np.any(got[0] != 0.0)


@pytest.mark.parametrize("T,m", [(3, 1), (20, 1), (70, 2), (300, 0)])
def test_head_nan_stays_in_its_row(T, m):
    """A NaN in a token's hidden state: its lse, entropy and gradient are NaN, ids stay in range, the others as alone."""
    F, T_ = _F(), torch()
    H, V, bad = 128, 5003, T // 2
    h, w, ids, _ = _hidden(T, T, H, V, m)
    rng = np.random.default_rng(1)
    dl, de = to_dev(rng.standard_normal((T, m)).astype(np.float32)), to_dev(rng.standard_normal(T).astype(np.float32))

    def run(h):
        fwd = _head_fwd(h, w, ids, 5)
        g = T_.empty((T, H), dtype=T_.bfloat16, device="cuda")
        d = F.logprob_desc(T, V, given=m, hidden=H)
        F.head_logprob_bwd(d, to_dev_bf16(h), to_dev_bf16(w), fwd["lse"], g, ids=to_dev(ids) if m else None,
                           dlogp=dl if m else None, entropy=fwd["entropy"], dentropy=de,
                           workspace=_workspace(F.head_logprob_workspace_size(d, True)))
        T_.cuda.synchronize()
        return {n: from_dev(v) for n, v in dict(fwd, g=g).items() if v is not None}

    good = run(h)
    h = h.copy()
    h[bad, 7] = np.nan
    got = run(h)
    assert np.isnan(got["lse"][bad]) and np.isnan(got["entropy"][bad]) and np.all(np.isnan(got["g"][bad]))
    assert np.all((got["top_ids"][bad] >= -1) & (got["top_ids"][bad] < V))
    rest = np.arange(T) != bad
    for n in good:
        assert np.array_equal(got[n][rest], good[n][rest]), n


def test_logits_past_4gb():
    """Offsets past 32 bits, in bytes and in elements; the last rows are checked."""
    F, T_ = _F(), torch()
    T, V = 30000, 151936
    z = T_.empty((T, V), dtype=T_.bfloat16, device="cuda")
    g = T_.Generator(device="cuda")
    g.manual_seed(3)
    for r in range(0, T, 1000):
        z[r:r + 1000] = T_.randn((1000, V), generator=g, device="cuda") * 2
    ids = T_.randint(0, V, (T, 1), generator=g, device="cuda").to(T_.int32)
    d = F.logprob_desc(T, V, given=1, top=8)
    out = _out(T, 1, 8)
    F.logprob_fwd(d, z, ids=ids, workspace=_workspace(F.logprob_workspace_size(d)), **out)
    rows = [0, 1, 14130, 14135, 28300, T - 2, T - 1]
    zr = from_dev(z[rows]).astype(np.float64)
    _check_forward({n: v[rows] for n, v in out.items()}, zr, from_dev(ids[rows]), 8)
    dl = T_.randn((T, 1), generator=g, device="cuda")
    F.logprob_bwd(F.logprob_desc(T, V, given=1), z, out["lse"], z, ids=ids, dlogp=dl)
    T_.cuda.synchronize()
    ref, part = O.backward(zr, from_dev(ids[rows]), from_dev(dl[rows]))
    got = from_dev(z[rows]).astype(np.float64)
    sure = np.exp(zr - O.forward(zr)["lse"][:, None]) * np.abs(from_dev(dl[rows]))
    assert np.all(np.abs(got - ref) <= _bwd_tolerance(ref, part, zr, sure, H16, np.abs(from_dev(dl[rows]))))


# ------------------------------------------------------- from hidden states --
def _hidden(seed, T, H, V, m, spread=2.0):
    """Hidden states and weight on grids of powers of two (whole numbers up to 127 times a unit), given tokens of
    which the first stands out in most rows."""
    rng = np.random.default_rng(seed)
    unit = 2.0 ** np.round(np.log2(spread / (1024 * np.sqrt(H))))
    wq = np.clip(np.rint(rng.standard_normal((V, H)) * 32), -127, 127)
    ids = _ids(rng, T, V, m) if m else None
    hq = rng.standard_normal((T, H)) * 32
    if m:
        hq += rng.random((T, 1)) * 12 / (unit * 1024 * H) * wq[np.clip(ids[:, 0], 0, V - 1)]
    hq = np.clip(np.rint(hq), -127, 127)
    assert np.abs(hq).max() * 127 * H < 2 ** 31
    z = hq @ wq.T                                                       # whole numbers: exact in float64
    assert np.abs(z).max() < 2 ** 23
    return (hq / 32).astype(np.float32), (wq * (unit * 32)).astype(np.float32), ids, z * unit


def _head_fwd(h, w, ids, k, entropy=True):
    F, T_ = _F(), torch()
    T, H = h.shape
    m = 0 if ids is None else ids.shape[1]
    d = F.logprob_desc(T, w.shape[0], given=m, top=k, hidden=H)
    out = _out(T, m, k)
    if not entropy:
        out["entropy"] = None
    F.head_logprob_fwd(d, to_dev_bf16(h), to_dev_bf16(w), ids=to_dev(ids) if m else None,
                       workspace=_workspace(F.head_logprob_workspace_size(d)), **out)
    T_.cuda.synchronize()
    return out


HEAD = [(1, 64, 1, 1, 1), (1, 64, 300, 1, 20), (1, 2048, 20011, 1, 20), (2, 128, 257, 0, 64), (17, 320, 5003, 2, 5),
        (33, 192, 4096, 64, 64), (65, 128, 40001, 1, 64), (100, 64, 255, 1, 33), (257, 192, 1000, 3, 5),
        (16, 2048, 5001, 1, 20), (9, 4096, 3001, 1, 20), (32, 2048, 3001, 1, 5), (64, 1024, 3003, 2, 64),
        (1, 16384, 300, 1, 1), (4, 16384, 301, 0, 3), (333, 1024, 32003, 1, 64), (700, 128, 33000, 1, 64), (1030, 64, 20000, 0, 1), (513, 256, 9001, 1, 0),
        (2100, 64, 100000, 1, 64), (40, 64, 4200000, 1, 64)]


@pytest.mark.parametrize("T,H,V,m,k", HEAD)
def test_head(T, H, V, m, k):
    h, w, ids, z = _hidden(T + V, T, H, V, m)
    _check_forward(_head_fwd(h, w, ids, k), z, ids, k, what=f"{T}x{H}x{V}")


@pytest.mark.parametrize("T,V", [(3, 9000), (70, 30000), (600, 30000)])
def test_head_ties_and_orders(T, V):
    """Equal logits everywhere (hidden states of zero), logits that rise or fall with the id over the whole
    vocabulary, and a few entries that stand out at its ends."""
    H = 64
    rng = np.random.default_rng(V)
    w = np.zeros((V, H), np.float32)
    w[:, 0] = bf16_rne(np.linspace(-1, 1, V).astype(np.float32))
    w[:, 1] = bf16_rne(np.linspace(1, -1, V).astype(np.float32))
    w[:, 2] = 0.0
    w[[0, 1, V // 2, V - 1], 2] = 1.0
    w[:, 3] = rng.integers(0, 3, V)
    h = np.zeros((T, H), np.float32)
    for t in range(T):
        h[t, t % 5 if t % 5 < 4 else 63] = 8.0            # column 63 of w is zero: all equal
    z = h.astype(np.float64) @ w.astype(np.float64).T
    ids = rng.integers(0, V, (T, 1)).astype(np.int32)
    _check_forward(_head_fwd(h, w, ids, 64), z, ids, 64)


def test_head_without_some_outputs_and_repeatable():
    h, w, ids, z = _hidden(11, 300, 128, 20000, 1)
    a, b = _head_fwd(h, w, ids, 16), _head_fwd(h, w, ids, 16, entropy=False)
    for n in ("lse", "logp", "top_ids", "top_logp"):
        assert torch().equal(a[n], b[n]), n
    c = _head_fwd(h, w, ids, 16)
    for n in a:
        assert torch().equal(a[n], c[n]), n


@pytest.mark.parametrize("T,H,V,m,ent", [
    (1, 64, 1, 1, True), (1, 64, 300, 1, True), (5, 128, 257, 2, True), (17, 320, 5003, 64, True), (257, 192, 1000, 1, False),
    (333, 512, 20003, 1, True), (130, 64, 70001, 0, True), (700, 128, 33000, 1, True)])
def test_head_gradient(T, H, V, m, ent):
    F, T_ = _F(), torch()
    h, w, ids, z = _hidden(T + V + 1, T, H, V, m)
    rng = np.random.default_rng(2)
    dl = rng.standard_normal((T, m)).astype(np.float32)
    de = (rng.standard_normal(T) * 0.3).astype(np.float32) if ent else None
    fwd = _head_fwd(h, w, None, 0)
    d = F.logprob_desc(T, V, given=m, hidden=H)
    hd = to_dev_bf16(h)
    F.head_logprob_bwd(d, hd, to_dev_bf16(w), fwd["lse"], hd, ids=to_dev(ids) if m else None,
                       dlogp=to_dev(dl) if m else None, entropy=fwd["entropy"] if ent else None,
                       dentropy=to_dev(de) if ent else None,
                       workspace=_workspace(F.head_logprob_workspace_size(d, True)))
    T_.cuda.synchronize()
    got = from_dev(hd).astype(np.float64)
    dz, part = O.backward(z, ids, dl if m else None, de)
    W = w.astype(np.float64)
    ref = dz @ W
    given = np.zeros((T, V), bool)
    if m:
        for t in range(T):
            given[t, ids[t][(ids[t] >= 0) & (ids[t] < V)]] = True
    # P is rounded to bf16 beside the given tokens' entries; its exponential's argument and log p + entropy are known
    # to a few half ulps of |z| + |lse|; sums of V terms in fp32 (H does not enter: z is exact)
    zmax = np.abs(z).max(-1, keepdims=True)
    f = np.abs(dl).sum(-1)[:, None] + (np.abs(de)[:, None] * (2 * zmax + 12) if ent else 0.0)
    p = np.exp(z - O.forward(z)["lse"][:, None])
    aw = np.abs(W)
    terms = (part + np.abs(dz)) @ aw
    tol = (H16 * np.abs(ref) * 1.001 + H16 * (np.where(given, 0.0, part) @ aw) * 1.001 + (16 + 6 * zmax) * H32 * ((p * f) @ aw)
           + (V / 64 + 64) * H32 * terms)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])
