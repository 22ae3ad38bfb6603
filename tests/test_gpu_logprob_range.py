"""Log probabilities over the whole range of logits: masks of any finite size over chunks and over rows, logits far
from 0, infinities, and hidden states that lie on no grid."""
import numpy as np
import pytest

from oracle.numerics import bf16_rne
from tests.fq_testutil import from_dev, to_dev, to_dev_bf16, torch
from tests.test_gpu_logprob import _head_fwd, _hidden, _logits_fwd, _padded, _workspace

pytestmark = pytest.mark.gpu
H32 = 2.0 ** -24          # half an ulp of fp32, relative
H16 = 2.0 ** -8           # of bf16
LOWEST = 3.3895313892515355e38


def _F():
    from scale_only_quantization_amd import fqlib
    return fqlib


def _bf(z):
    with np.errstate(over="ignore"):
        return bf16_rne(np.asarray(z, np.float32))


def _ref(z, ids, k):
    """The definitions in float64, from the distance to the largest logit, so that log n is not lost beside it."""
    z = np.asarray(z, np.float64)
    M = z.max(-1, keepdims=True)
    none = M == -np.inf
    with np.errstate(invalid="ignore", divide="ignore"):
        d = np.where(none, -np.inf, z - np.where(none, 0.0, M))
        ls = np.log(np.exp(d).sum(-1, keepdims=True))
        lp = np.where(none, -np.inf, d - ls)
        p = np.exp(lp)
        out = dict(M=M[:, 0], ls=ls[:, 0], lse=np.where(none, -np.inf, M + ls)[:, 0], lp=lp, p=p, none=none[:, 0],
                   entropy=-np.where(p > 0, p * lp, 0.0).sum(-1), spread=np.where(p > 0, -p * d, 0.0).sum(-1))
    if ids is not None:
        ok = (ids >= 0) & (ids < z.shape[1])
        out["logp"] = np.where(ok, np.take_along_axis(lp, np.where(ok, ids, 0).astype(np.int64), 1), 0.0)
    if k:
        order = np.argsort(-z, axis=-1, kind="stable")[:, :k]
        there = np.take_along_axis(z, order, 1) > -np.inf
        out["top_ids"] = np.where(there, order, -1)
        out["top_logp"] = np.where(there, np.take_along_axis(lp, order, 1), -np.inf)
    return out


def _check(got, z, ids, k, zerr=0.0, what="", sums=True):
    """An element enters the sums by three roundings and the exponential's ulp; a frame's rounding is taken off to
    2^-26; at most 128 sequential additions and 32 of trees and chunks: as the tests near 0, and not in terms of |z|.
    Only lse itself is a number of the size of z: one rounding of it, and one of the largest logit plus its log sum.
    zerr: how well the logits are known; sums: lse and entropy too."""
    with np.errstate(over="ignore", invalid="ignore"):
        r = _ref(z, ids, k)
        rel = (160 + 8 + 4 + 2 * r["spread"]) * H32 + 2 * zerr
        lse, ent = from_dev(got["lse"]).astype(np.float64), from_dev(got["entropy"]).astype(np.float64)
        assert np.all(np.isneginf(lse[r["none"]])) and np.all(ent[r["none"]] == 0.0), what
        live = ~r["none"] & sums
        t = rel + 4 * H32 * np.abs(r["ls"]) + 2 * H32 * np.abs(r["lse"])
        bad = live & ~(np.abs(lse - r["lse"]) <= t)
        assert not bad.any(), (what, "lse", np.nonzero(bad)[0][:8], lse[bad][:8], r["lse"][bad][:8])
        t = rel * (1 + 2 * r["spread"]) + 4 * H32 * (r["spread"] + r["entropy"] + 1)
        bad = live & ~(np.abs(ent - r["entropy"]) <= t)
        assert not bad.any(), (what, "entropy", np.nonzero(bad)[0][:8], ent[bad][:8], r["entropy"][bad][:8])
        for n in ("logp", "top_logp"):
            if n not in r:
                continue
            x, y = from_dev(got[n]).astype(np.float64), r[n]
            y32 = y.astype(np.float32)
            inf = np.isinf(y32)
            assert np.array_equal(x[inf], y32[inf].astype(np.float64)), (what, n)
            t = (rel + 4 * H32 * np.abs(r["ls"]))[:, None] + 3 * H32 * np.abs(np.where(inf, 0.0, y))
            bad = ~inf & ~(np.abs(x - y) <= t)
            assert not bad.any() and np.all(x <= 0.0), (what, n, np.argwhere(bad)[:6], x[bad][:6], y[bad][:6])
        if k:
            assert np.array_equal(from_dev(got["top_ids"]), r["top_ids"]), (what, "ids")
    return r


SIZES = (1e4, 1e5, 1e7, 1e9, 1e10, 1e12, 1e15, 1e18, 1e20, 1e25, 1e30, 1e35, 1e37, LOWEST)


def _masked(size, V, rng):
    """Rows masked by -size: all but a stretch, all but the last entry, half of them, all; rows about +size, and a few
    entries there."""
    z = np.full((7, V), -size)
    z[0, V // 2:V // 2 + 7] = rng.standard_normal(7)
    z[1, V - 1] = 1.0
    keep = rng.random(V) < 0.5
    z[2, keep] = rng.standard_normal(keep.sum())
    z[4] = size
    z[5] = rng.standard_normal(V) * 2
    z[5, rng.choice(V, 9, replace=False)] = size
    z[6, V // 3:] = -np.inf
    return z


@pytest.mark.parametrize("V", [300, 5000, 40001])
@pytest.mark.parametrize("many", [False, True])
def test_logits_masked_by_finite_values(V, many):
    """Masks of any size over whole chunks beside live ones, and over whole rows; long chunks and short ones."""
    rng = np.random.default_rng(V + 11)
    z = np.concatenate([_masked(s, V, rng) for s in SIZES])
    z = _bf(np.tile(z, (6 if many else 1, 1)))
    n = 256 if many else 25                                          # 25 rows of 40001 are short chunks
    ids = np.stack([np.zeros(len(z)), np.full(len(z), V // 2), np.full(len(z), V - 1)], 1).astype(np.int32)
    for r in range(0, len(z), n):
        _check(_logits_fwd(z[r:r + n], ids[r:r + n], 20), z[r:r + n], ids[r:r + n], 20, what=(V, r))


def _offset(T, H, V, m, base, seed=0):
    """Hidden states and weight whose logits stand about `base`, exact in fp32 (steps of 2^-12, below 2^12)."""
    h, w, ids, _ = _hidden(T + V + seed, T, H, V, m, spread=2.0 ** -12 * 1024 * np.sqrt(H))
    h[:, -1] = 32.0
    w[:, -1] = _bf(base / 32.0)
    z = h.astype(np.float64) @ w.astype(np.float64).T
    assert np.abs(z).max() < 4096 and np.array_equal(z * 4096, np.rint(z * 4096))
    return h, w, ids, z


BASES = (-3500.0, -1000.0, 500.0, 1500.0, 2500.0, 3000.0, 3500.0)


@pytest.mark.parametrize("T", [1, 5, 20])
@pytest.mark.parametrize("base", BASES)
def test_hidden_states_of_a_few_tokens_with_logits_far_from_0(T, base):
    """The frame's rounding is up to 2^-12 here: it is taken off both sums, the entropy's too."""
    h, w, ids, z = _offset(T, 64, 9001, 2, base)
    _check(_head_fwd(h, w, ids, 20), z, ids, 20, what=(T, base))


@pytest.mark.parametrize("T", [72, 300])
@pytest.mark.parametrize("base", BASES)
def test_log_probabilities_of_hidden_states_with_logits_far_from_0(T, base):
    """They are as exact as near 0, where lse is rounded by 2^-13."""
    h, w, ids, z = _offset(T, 64, 9001, 2, base)
    _check(_head_fwd(h, w, ids, 20), z, ids, 20, what=(T, base), sums=False)


def _kinds(H, V, size, seed):
    """12 hidden states and a weight whose logits are exact: general ones; the same with two thirds of the vocabulary, in
    one piece and scattered, masked by -size; every logit -size; every logit +size; the first half -size, 0 beyond; +size
    at 9 entries, 0 elsewhere."""
    h, w, _, _ = _hidden(seed, 12, H, V, 0)
    rng = np.random.default_rng(seed)
    w[:, :4] = 0.0
    h[:, :4] = 0.0
    masked = np.arange(V) < V // 2
    masked[V // 2:] = rng.random(V - V // 2) < 0.3
    w[masked] = 0.0                                       # so that -size is not rounded with what is left
    w[masked, 0] = -size
    w[:, 1] = size
    w[:V // 2, 2] = -size
    w[rng.choice(V, 9, replace=False), 3] = size
    h[2:4, 0] = 1.0
    h[4:] = 0.0
    h[4:6, 1], h[6:8, 1], h[8:10, 2], h[10:, 3] = -1.0, 1.0, 1.0, 1.0
    w = _bf(w)
    return h, w, h.astype(np.float64) @ w.astype(np.float64).T


def _tiled(T, h, w, z, k, what):
    """The rows of h repeated to T: the first ones against the definitions, the others equal to them."""
    n = len(h)
    ids = np.stack([np.arange(n) * 7, z.shape[1] - 1 - np.arange(n)], 1).astype(np.int32)
    tile = lambda x: np.concatenate([np.tile(x, (T // n,) + (1,) * (x.ndim - 1)), x[:T % n]])  # noqa: E731
    got = _head_fwd(tile(h), w, tile(ids), k)
    _check({name: None if v is None else v[:n] for name, v in got.items()}, z, ids, k, what=what)
    for name, v in got.items():
        if v is not None:
            x = from_dev(v)
            assert np.array_equal(x, tile(x[:n])), (what, name)


@pytest.mark.parametrize("T", [12, 72, 300, 4104])
@pytest.mark.parametrize("V", [1000, 20001])
@pytest.mark.parametrize("size", [1e4, 1e7, 1e9, 1e10, 1e15, 1e20, 1e29])
def test_hidden_states_masked_by_finite_values(T, V, size):
    """Whole strips and whole rows of masks, in every form (few tokens, one and two waves a token)."""
    h, w, z = _kinds(128, V, size, V)
    _tiled(T, h, w, z, 20, (T, V, size))
    if T > 12:
        _tiled(T, h, w, z, 0, (T, V, size, "no alternatives"))


@pytest.mark.parametrize("T", [72, 300])
@pytest.mark.parametrize("base", BASES)
def test_sums_of_hidden_states_with_logits_far_from_0(T, base):
    h, w, ids, z = _offset(T, 64, 9001, 2, base)
    _check(_head_fwd(h, w, ids, 20), z, ids, 20, what=(T, base))


@pytest.mark.parametrize("T", [12, 72, 300, 4104])
@pytest.mark.parametrize("V", [1024, 20480])
@pytest.mark.parametrize("how", ["some", "strips", "all but one", "all"])
def test_hidden_states_with_ruled_out_entries(T, V, how):
    """Logits of -inf (a weight of -inf where every hidden state is 1): in the midst of others, over whole strips and
    pieces, all but one, all."""
    h, w, _, z = _hidden(V, 12, 512, V, 0)
    rng = np.random.default_rng(V)
    out = dict(some=rng.random(V) < 0.3, strips=np.arange(V) // 200 % 2 == 0)
    out["all"] = np.ones(V, bool)
    out["all but one"] = np.arange(V) != V - 2
    h[:, 7], w[:, 7] = 1.0, 0.0
    z = h.astype(np.float64) @ w.astype(np.float64).T
    w[out[how], 7] = -np.inf
    z[:, out[how]] = -np.inf
    _tiled(T, h, w, z, 20, (T, V, how))
    if T > 12:
        _tiled(T, h, w, z, 0, (T, V, how, "no alternatives"))


@pytest.mark.parametrize("T", [72, 300])
@pytest.mark.parametrize("V", [1000, 20001, 65])
@pytest.mark.parametrize("size", [1e30, 1e32, LOWEST, np.inf])
def test_columns_past_the_vocabulary_are_below_every_logit(T, V, size):
    """A vocabulary that ends inside a strip, with rows of nothing but large masks or ruled-out entries."""
    h, w, z = _kinds(128, V, 1.0 if np.isinf(size) else size, V)
    if np.isinf(size):
        h[:, 7], w[:, 7] = 1.0, -np.inf
        z = np.full_like(z, -np.inf)
    _tiled(T, h, w, z, 20, (T, V, size))
    _tiled(T, h, w, z, 0, (T, V, size, "no alternatives"))


@pytest.mark.parametrize("T", [1, 2, 3, 8, 12])
@pytest.mark.parametrize("H", [64, 320, 576])
def test_ruled_out_entries_of_rows_that_end_inside_512_columns(T, H):
    """A weight of -inf in a row's first columns, which stand in for those past its end."""
    h, w, _, _ = _hidden(T, T, H, 3001, 0)
    h[:, 2], w[:, 2] = 1.0, 0.0
    z = h.astype(np.float64) @ w.astype(np.float64).T
    out = np.random.default_rng(T).random(3001) < 0.5
    w[out, 2] = -np.inf
    z[:, out] = -np.inf
    ids = np.arange(T, dtype=np.int32)[:, None]
    _check(_head_fwd(h, w, ids, 20), z, ids, 20, what=(T, H))


def _grad_ref(z, ids, dl, de):
    """d L / d z, p and the size of what p is multiplied by, from the distance to the largest logit; rows below -2^20 have
    gradient 0."""
    r = _ref(z, None, 0)
    T, V = z.shape
    live = (r["lse"] > -2.0 ** 20)[:, None]
    p = np.where(live, r["p"], 0.0)
    lp = np.where(p > 0, r["lp"], 0.0)
    g, A, size = np.zeros((T, V)), np.zeros(T), np.zeros(T)
    if dl is not None:
        for t in range(T):
            for i, a in zip(ids[t], dl[t].astype(np.float64)):
                if 0 <= i < V and live[t]:
                    A[t] += a
                    size[t] += abs(a)
                    g[t, i] += a
    f, a = np.broadcast_to(A[:, None], (T, V)), np.broadcast_to(size[:, None], (T, V))
    if de is not None:
        b, H = de.astype(np.float64)[:, None], r["entropy"][:, None]
        f, a = f + b * (lp + H), a + np.abs(b) * (np.abs(lp) + H + 1)
    with np.errstate(invalid="ignore"):
        # of log p, in lse; past 2^20 entries are the largest or far below it
        err = np.where(np.abs(r["lse"]) <= 2.0 ** 20, np.abs(r["lse"]), 0.0)[:, None] * 2 * H32
        # log p: also its own rounding and the product with log2 e; what p is multiplied by: an error like log p's and sums
        perr = np.expm1(err + (3 * np.abs(lp) + 16) * H32)
    return r, g - p * f, p, p * a * 3 * perr + 2.0 ** -126 * 30 * a


@pytest.mark.parametrize("V", [300, 20001])
@pytest.mark.parametrize("m,ent", [(0, True), (1, False), (2, True)])
def test_logits_gradient_masked_by_finite_values(V, m, ent):
    """Masks of any size beside live entries, and rows of nothing else, through forward and backward."""
    F, T_ = _F(), torch()
    rng = np.random.default_rng(V + m)
    z = _bf(np.concatenate([_masked(s, V, rng)[[0, 1, 2, 3]] for s in SIZES]))
    T = len(z)
    ids = rng.integers(0, V, (T, m)).astype(np.int32)
    dl, de = rng.standard_normal((T, m)).astype(np.float32), rng.standard_normal(T).astype(np.float32)
    fwd = _logits_fwd(z, None, 0)
    grad = T_.full((T, (V + 7) // 8 * 8), 9.0, dtype=T_.bfloat16, device="cuda")[:, :V]
    F.logprob_bwd(F.logprob_desc(T, V, given=m), _padded(z, 0, 0.0)[1], fwd["lse"], grad, ids=to_dev(ids) if m else None,
                  dlogp=to_dev(dl) if m else None, entropy=fwd["entropy"] if ent else None,
                  dentropy=to_dev(de) if ent else None)
    T_.cuda.synchronize()
    got = from_dev(grad).astype(np.float64)
    _, ref, _, tol = _grad_ref(z.astype(np.float64), ids, dl if m else None, de if ent else None)
    bad = ~(np.abs(got - ref) <= H16 * np.abs(ref) * 1.001 + tol)
    assert not bad.any(), (np.argwhere(bad)[:6], got[bad][:6], ref[bad][:6])
    whole = np.arange(T) % 4 == 3
    assert np.all(got[whole & (np.repeat(SIZES, 4) > 2.0 ** 20)] == 0.0)


def _head_grad_check(h, w, z, ids, T, what):
    """The gradient of the rows of h, repeated to T, from their forward's lse and entropy; z exact."""
    F, T_ = _F(), torch()
    n, V, H, m = len(h), z.shape[1], h.shape[1], ids.shape[1]
    rng = np.random.default_rng(T + V)
    dl, de = rng.standard_normal((n, m)).astype(np.float32), rng.standard_normal(n).astype(np.float32)
    tile = lambda x: np.concatenate([np.tile(x, (T // n, 1)), x[:T % n]])  # noqa: E731
    fwd = _head_fwd(tile(h), w, None, 0)
    d = F.logprob_desc(T, V, given=m, hidden=H)
    g = T_.full((T, H), 9.0, dtype=T_.bfloat16, device="cuda")
    F.head_logprob_bwd(d, to_dev_bf16(tile(h)), to_dev_bf16(w), fwd["lse"], g, ids=to_dev(tile(ids)),
                       dlogp=to_dev(tile(dl)), entropy=fwd["entropy"], dentropy=to_dev(tile(de[:, None])[:, 0]),
                       workspace=_workspace(F.head_logprob_workspace_size(d, True)))
    T_.cuda.synchronize()
    got = from_dev(g)
    assert np.array_equal(got, tile(got[:n])), what
    got = got[:n].astype(np.float64)
    _, dz, p, tol = _grad_ref(z, ids, dl, de)
    aw = np.abs(w.astype(np.float64))
    ref = dz @ w.astype(np.float64)
    given = np.zeros(z.shape, bool)
    for t in range(n):
        given[t, ids[t][(ids[t] >= 0) & (ids[t] < V)]] = True
    part = np.where(p > 0, np.abs(dz), 0.0)
    # the result's rounding, that of dL/dz beside the given tokens, and fp32 sums
    tol = (H16 * (np.abs(ref) + np.where(given, 0.0, part) @ aw) * 1.001 + tol @ aw + (V / 64 + 64) * H32 * (np.abs(dz) @ aw)
           + (V / 64 + 64) * H32 * (p @ aw) * np.abs(dl).sum(-1, keepdims=True))
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:6], got[bad][:6], ref[bad][:6], tol[bad][:6])
    return got


@pytest.mark.parametrize("T", [12, 300])
@pytest.mark.parametrize("m", [1, 3])
@pytest.mark.parametrize("size", [1e4, 1e7, 1e9, 1e10, 1e20, 1e30, 1e37])
def test_hidden_states_gradient_masked_by_finite_values(T, m, size):
    """Masked entries beside live ones, rows of nothing but masks, and one entry far above all others."""
    h, w, z = _kinds(128, 5003, size, 3)
    one = int(np.argmax(w[:, 3]))
    w[:, 3] = 0.0
    w[one, 3] = _bf(size)
    h[6:8], z = h[10:], None                                         # (no row of equal logits past 2^20)
    z = h.astype(np.float64) @ w.astype(np.float64).T
    rng = np.random.default_rng(m)
    ids = rng.integers(0, 5003, (12, m)).astype(np.int32)
    ids[6, 0] = one
    got = _head_grad_check(h, w, z, ids, T, (T, m, size))
    if size > 2.0 ** 20:
        assert np.all(got[4:6] == 0.0)


@pytest.mark.parametrize("T", [12, 300])
@pytest.mark.parametrize("m", [1, 3])
@pytest.mark.parametrize("base", [-3500.0, -1000.0, 1500.0, 3500.0])
def test_hidden_states_gradient_far_from_0(T, m, base):
    h, w, ids, z = _offset(12, 64, 5003, m, base)
    _head_grad_check(h, w, z, ids, T, (T, m, base))


@pytest.mark.parametrize("m", [1, 2])
def test_hidden_states_gradient_of_logits_past_fp32(m):
    """Finite hidden states and weights whose logits are -inf in fp32: some of a row, a given one among them (p = 0), and
    all of a row (gradient 0)."""
    h, w, _, _ = _hidden(4, 12, 128, 2000, 0)
    h[:, 0], h[8:] = 2.0 ** 100, 0.0
    h[8:, 1] = 2.0 ** 100
    w[:, 0] = np.where(np.arange(2000) % 3 == 0, -2.0 ** 60, 0.0)
    w[:, 1] = -2.0 ** 60
    h[:8, 1] = 0.0
    z = h.astype(np.float64) @ w.astype(np.float64).T
    z = np.where(z < -1e39, -np.inf, z)
    ids = np.tile(np.array([[3, 4][:m]], np.int32), (12, 1))
    got = _head_grad_check(h, w, z, ids, 12, m)
    assert np.all(got[8:] == 0.0)
    _head_grad_check(h, w, z, ids, 300, m)


def _general(T, H, V, seed):
    """bf16 normal values on no grid, and how well fp32 knows a logit: a product enters at most 32 additions inside a
    matrix instruction, or H / 64 of a lane's and 6 of the lanes', then one per instruction of its wave, H / 16 at most;
    each has an error of an ulp (two halves) at most."""
    rng = np.random.default_rng(seed)
    h, w = _bf(rng.standard_normal((T, H))), _bf(rng.standard_normal((V, H)) * 2 / np.sqrt(H))
    h[:, :4] *= 8
    hd, wd = h.astype(np.float64), w.astype(np.float64)
    return h, w, hd @ wd.T, (64 + H / 8) * H32 * (np.abs(hd) @ np.abs(wd).T).max(-1)


FORMS = [(1, 2048), (2, 320), (4, 2048), (8, 1024), (12, 2048), (30, 512), (64, 512), (40, 2048), (300, 192), (300, 2048)]


@pytest.mark.parametrize("T,H", FORMS)
def test_hidden_states_on_no_grid(T, H):
    """Every form on general values: the products' own rounding is in the results.  Alternatives are compared by what
    their logits are, as neighbours may change places."""
    V, k = 5003, 20
    h, w, z, zerr = _general(T, H, V, T + H)
    top = np.argsort(-z, axis=-1, kind="stable")
    ids = np.concatenate([top[:, :2], top[:, V // 2:V // 2 + 1]], 1).astype(np.int32)
    got = _head_fwd(h, w, ids, k)
    r = _check({n: v for n, v in got.items() if n != "top_ids" and n != "top_logp"}, z, ids, 0, zerr=zerr, what=(T, H))
    tid, tlp = from_dev(got["top_ids"]), from_dev(got["top_logp"]).astype(np.float64)
    assert np.all((tid >= 0) & (tid < V)) and all(len(set(row)) == k for row in tid)
    at = np.take_along_axis(z, tid.astype(np.int64), 1)
    kth = np.take_along_axis(z, top[:, k - 1:k], 1)
    assert np.all(at >= kth - 2 * zerr[:, None]) and np.all(np.diff(at, axis=1) <= 2 * zerr[:, None])
    sure = np.take_along_axis(z, top[:, :k], 1) > kth + 2 * zerr[:, None]
    assert all(set(top[t, :k][sure[t]]) <= set(tid[t]) for t in range(T))
    tol = ((160 + 8 + 4 + 2 * r["spread"]) * H32 + 2 * zerr)[:, None] + 8 * H32 * (np.abs(r["ls"])[:, None] + np.abs(tlp))
    assert np.all(np.abs(tlp - np.take_along_axis(r["lp"], tid.astype(np.int64), 1)) <= tol)
    # a given token and the same one among the alternatives: two sums of one logit
    lp = from_dev(got["logp"]).astype(np.float64)
    for j in range(2):
        t, at = np.nonzero(tid == ids[:, j:j + 1])
        assert np.all(np.abs(lp[t, j] - tlp[t, at]) <= 2 * zerr[t] + 4 * H32 * np.abs(lp[t, j]))


@pytest.mark.parametrize("T,H", FORMS)
@pytest.mark.parametrize("m,ent", [(1, True), (2, False)])
def test_hidden_states_gradient_on_no_grid(T, H, m, ent):
    F, T_ = _F(), torch()
    V = 5003
    h, w, z, zerr = _general(T, H, V, T + H + 1)
    rng = np.random.default_rng(T)
    ids = rng.integers(0, V, (T, m)).astype(np.int32)
    ids[::2, 0] = np.argmax(z, -1)[::2]
    dl = rng.standard_normal((T, m)).astype(np.float32)
    de = rng.standard_normal(T).astype(np.float32) if ent else None
    fwd = _head_fwd(h, w, None, 0)
    d = F.logprob_desc(T, V, given=m, hidden=H)
    g = T_.full((T, H), 9.0, dtype=T_.bfloat16, device="cuda")
    F.head_logprob_bwd(d, to_dev_bf16(h), to_dev_bf16(w), fwd["lse"], g, ids=to_dev(ids), dlogp=to_dev(dl),
                       entropy=fwd["entropy"] if ent else None, dentropy=to_dev(de) if ent else None,
                       workspace=_workspace(F.head_logprob_workspace_size(d, True)))
    T_.cuda.synchronize()
    got = from_dev(g).astype(np.float64)
    r, dz, p, tol = _grad_ref(z, ids, dl, de)
    W, aw = w.astype(np.float64), np.abs(w.astype(np.float64))
    given = np.zeros(z.shape, bool)
    np.put_along_axis(given, ids.astype(np.int64), True, 1)
    a = np.abs(dl).sum(-1, keepdims=True)
    size = p * (a + (np.abs(de)[:, None] * (np.abs(r["lp"]) + r["entropy"][:, None] + 1) if ent else 0.0))
    # the result's rounding, that of dL/dz beside the given tokens, the logits' own error (theirs and lse's: 2 zerr in
    # log p, as much again in log p + entropy times its spread), fp32 sums over the vocabulary
    z2 = (2 * zerr * (2 + r["spread"]))[:, None]
    tol = (H16 * (np.abs(dz @ W) + np.where(given, 0.0, np.abs(dz)) @ aw) * 1.01 + (tol + size * np.expm1(z2) * 2) @ aw
           + (V / 64 + 64) * H32 * ((np.abs(dz) + size) @ aw))
    bad = ~(np.abs(got - dz @ W) <= tol)
    assert not bad.any(), ((T, H), np.argwhere(bad)[:6], got[bad][:6], (dz @ W)[bad][:6], tol[bad][:6])


@pytest.mark.parametrize("far", [3e4, 1e30, np.inf])
def test_a_tokens_sums_do_not_depend_on_its_neighbours(far):
    """Bitwise the same beside tokens whose logits are far from 0 or infinite."""
    T, H, V = 300, 128, 5003
    h, w, ids, _ = _hidden(5, T, H, V, 1)
    h[:, 3], w[:, 3] = 0.0, 1.0
    alone = _head_fwd(h, w, ids, 5)
    there = np.random.default_rng(1).random(T) < 0.3
    h[there, 3] = _bf(far)
    got = _head_fwd(h, w, ids, 5)
    for n in alone:
        assert np.array_equal(from_dev(got[n])[~there], from_dev(alone[n])[~there]), n


@pytest.mark.parametrize("T", [12, 300])
def test_entropies_are_never_negative(T):
    """Rows that are sure of one entry: a sum of 1 and little else."""
    rng = np.random.default_rng(T)
    z = np.full((T, 300), -np.inf)
    z[np.arange(T), rng.integers(0, 300, T)] = rng.standard_normal(T) * np.exp(rng.random(T) * 8)
    got = _logits_fwd(_bf(z), None, 0)
    assert np.all(from_dev(got["entropy"]) >= 0.0) and np.all(from_dev(got["entropy"]) <= 2 * H32)
    assert np.all(np.abs(from_dev(got["lse"]) - _bf(z).max(-1)) <= 4 * H32 * (1 + np.abs(_bf(z).max(-1))))
    h, w, _, _ = _hidden(1, T, 64, 300, 0)
    h[:] = 0.0
    h[:, 0] = _bf(np.abs(rng.standard_normal(T)) * np.exp(rng.random(T) * 6) + 1)
    w[:] = 0.0
    w[7, 0], w[np.arange(300) != 7, 0] = 3.0, -256.0
    got = _head_fwd(h, w, None, 0)
    ent = from_dev(got["entropy"])
    assert np.all(ent >= 0.0) and np.all(ent <= 2 * H32)


@pytest.mark.parametrize("T", [12, 300])
@pytest.mark.parametrize("k", [0, 20])
def test_logits_without_the_entropy(T, k):
    """The same bits with and without it, near 0 and far."""
    F, T_ = _F(), torch()
    V = 9001
    rng = np.random.default_rng(T)
    z = _bf(np.concatenate([_masked(s, V, rng) for s in (1e4, 1e9, 1e30, LOWEST)] * 11)[:T])
    ids = rng.integers(0, V, (T, 2)).astype(np.int32)
    want = _logits_fwd(z, ids, k)
    got = {n: None if v is None or n == "entropy" else T_.full_like(v, 9) for n, v in want.items()}
    d = F.logprob_desc(T, V, given=2, top=k)
    F.logprob_fwd(d, _padded(z, 0, np.nan)[1], ids=to_dev(ids), workspace=_workspace(F.logprob_workspace_size(d)), **got)
    T_.cuda.synchronize()
    for n, v in got.items():
        assert v is None or T_.equal(v, want[n]), n


def test_as_many_rows_as_the_contract_takes():
    """2^24 - 1 rows, from logits and from hidden states, forward and backward: rows of the same kind, at every place,
    equal the first of their kind."""
    F, T_ = _F(), torch()
    T, V, H, kinds = (1 << 24) - 1, 40, 64, 5

    def spread(x):
        return to_dev_bf16(x)[T_.arange(T, device="cuda") % kinds].contiguous()

    def same(x):
        n = T // kinds * kinds
        assert bool((x[:n].reshape(n // kinds, kinds, -1) == x[:kinds].reshape(1, kinds, -1)).all())
        assert T_.equal(x[n:], x[:T - n])

    h, w, _, z = _hidden(3, kinds, H, V, 0)
    at = (T_.arange(T, device="cuda") % kinds).int()
    ids = (at * 7)[:, None].contiguous()
    dl, de = (at.float() - 1.5)[:, None].contiguous(), (at.float() * 0.1)
    for hidden in (0, H):
        zz = z if hidden else _bf(z)
        d = F.logprob_desc(T, V, given=1, top=3, hidden=hidden)
        out = dict(lse=T_.empty(T, device="cuda"), entropy=T_.empty(T, device="cuda"), logp=T_.empty((T, 1), device="cuda"),
                   top_ids=T_.empty((T, 3), dtype=T_.int32, device="cuda"), top_logp=T_.empty((T, 3), device="cuda"))
        x = spread(h if hidden else zz)
        if hidden:
            wd = to_dev_bf16(w)
            F.head_logprob_fwd(d, x, wd, ids=ids, workspace=_workspace(F.head_logprob_workspace_size(d)), **out)
            F.head_logprob_bwd(d, x, wd, out["lse"], x, ids=ids, dlogp=dl, entropy=out["entropy"], dentropy=de,
                               workspace=_workspace(F.head_logprob_workspace_size(d, True)))
        else:
            F.logprob_fwd(d, x, ids=ids, workspace=_workspace(F.logprob_workspace_size(d)), **out)
            F.logprob_bwd(d, x, out["lse"], x, ids=ids, dlogp=dl, entropy=out["entropy"], dentropy=de)
        T_.cuda.synchronize()
        first = np.arange(kinds)
        _check({n: v[:kinds] for n, v in out.items()}, zz, (first * 7).astype(np.int32)[:, None], 3, what=hidden)
        for v in out.values():
            same(v)
        same(x)
        _, dz, p, tol = _grad_ref(zz.astype(np.float64), (first * 7)[:, None], from_dev(dl[:kinds]), from_dev(de[:kinds]))
        aw = np.abs(w.astype(np.float64)) if hidden else np.eye(V)
        ref = dz @ w.astype(np.float64) if hidden else dz
        tol = H16 * (np.abs(ref) + (np.abs(dz) @ aw if hidden else 0.0)) * 1.001 + tol @ aw + 64 * H32 * (np.abs(dz) @ aw)
        assert np.all(np.abs(from_dev(x[:kinds]) - ref) <= tol)
        del x, out
        T_.cuda.empty_cache()
