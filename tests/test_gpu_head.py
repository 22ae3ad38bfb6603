"""GPU parity of the output layer's loss from hidden states (fq_head_loss) with
the oracle: row losses, their mean and the gradient within bounds that follow
from the roundings the header states."""
import numpy as np
import pytest

from oracle.head import head
from oracle.numerics import bf16_rne
from tests.fq_testutil import from_dev, to_dev, to_dev_bf16, torch

pytestmark = pytest.mark.gpu


def _F():
    from scale_only_quantization_amd import fqlib
    return fqlib


def _data(seed, T, H, V, k, spread=2.0):
    """Hidden states, weight (logits of standard deviation `spread`), the teacher's k distinct ids and logits
    (the label among them in half the rows), labels."""
    rng = np.random.default_rng(seed)
    w = bf16_rne((rng.standard_normal((V, H)) * (spread / np.sqrt(H))).astype(np.float32))
    lab = rng.integers(0, V, T).astype(np.int32)
    h = rng.standard_normal((T, H)) + rng.random((T, 1)) * 3 * w[lab] / spread
    h = bf16_rne(h.astype(np.float32))
    ti = np.zeros((T, k), np.int32)
    for t in range(T):
        ids = rng.choice(V, size=k, replace=False)
        if k and t % 2 and lab[t] not in ids:
            ids[0] = lab[t]
        ti[t] = ids
    return h, w, (rng.standard_normal((T, k)) * 2).astype(np.float32), ti, lab


def _run(h, w, tv, ti, lab, lm=0.8, dist=1.2, want_grad=True, rows=True):
    F, T_ = _F(), torch()
    T, H = h.shape
    k = 0 if ti is None else ti.shape[1]
    d = F.head_desc(T, H, w.shape[0], k, lm, dist)
    loss = T_.full((1,), 9.0, device="cuda")
    row = T_.full((T,), 9.0, device="cuda") if rows else None
    grad = T_.full((T, H), 9.0, dtype=T_.bfloat16, device="cuda") if want_grad else None
    # 0xFF: a NaN wherever something would be read before it is written
    ws = T_.full((F.head_loss_workspace_size(d, want_grad),), 255, dtype=T_.uint8, device="cuda")
    F.head_loss(d, to_dev_bf16(h), to_dev_bf16(w), loss, top_v=None if ti is None else to_dev(tv),
                top_i=None if ti is None else to_dev(ti), labels=None if lab is None else to_dev(lab), row_loss=row,
                grad=grad, workspace=ws)
    T_.cuda.synchronize()
    return from_dev(loss)[0], from_dev(row) if rows else None, from_dev(grad) if want_grad else None


def _check(got, h, w, tv, ti, lab, lm=0.8, dist=1.2, what=""):
    loss, rows, grad = got
    ref, ref_rows, ref_grad, (rest, full) = head(h, w, tv, ti, lab, lm, dist)
    H = h.shape[1]
    # a logit: exact bf16 products, H/16 sums of 16 products in fp32 (and the
    # sparse ones H/64 steps and 6 more), so at most H/16 + 16 half ulps of the
    # sum of the absolute products; the base-2 frame and log2 e: 2 half ulps of |z|
    za = (np.abs(h.astype(np.float64)) @ np.abs(w.astype(np.float64)).T).max(-1)
    ez = (H / 16 + 18) * 2.0 ** -24 * za
    # e^x in fp32: a few ulps per term, and as many in the sum of V (pairwise by
    # strips: 32 + 6 + strips / 16 steps): 2^-20 covers up to 2^4 ulps
    wsum = abs(lm) + abs(dist)
    tol = wsum * (2 * ez + 2.0 ** -20 + 4 * 2.0 ** -24 * np.abs(ref_rows)) + 2.0 ** -22
    np.testing.assert_array_less(np.abs(rows - ref_rows), tol, err_msg=f"{what} rows")
    assert abs(loss - ref) <= tol.max() + 2.0 ** -22 * abs(ref), f"{what} loss {loss} {ref}"
    if grad is not None:
        # the output's bf16 rounding, the probabilities' in the product (2^-8
        # each), and the logits' errors in every probability
        tol = (2.0 ** -8 * np.abs(ref_grad) + 2.0 ** -8 * rest + (4 * ez[:, None] + 2.0 ** -18) * full + 1e-38)
        bad = np.abs(grad - ref_grad) > tol
        assert not bad.any(), (f"{what} grad: {bad.sum()} of {bad.size} beyond tolerance, worst "
                               f"{(np.abs(grad - ref_grad) / tol).max():.2f}")


# one token; one tile with ragged rows; several row tiles; a vocabulary smaller
# than a tile, of one entry, odd; every hidden size class (one step, odd number
# of steps, more columns than a tile)
@pytest.mark.parametrize("T,H,V,k", [(1, 64, 300, 4), (37, 128, 1000, 16), (300, 192, 777, 64), (513, 320, 2049, 1),
                                     (5, 64, 1, 0), (9, 64, 1, 1), (70, 640, 63, 33), (256, 64, 256, 64),
                                     (129, 1024, 5003, 0),
                                     (300, 128, 40000, 16), (700, 256, 30001, 4)])   # more tiles than CUs
@pytest.mark.parametrize("what", ["both", "lm", "distill"])
def test_matches_the_oracle(T, H, V, k, what):
    if what == "distill" and k == 0 or what == "lm" and k > 0 and T > 100:
        pytest.skip("covered by another combination")
    h, w, tv, ti, lab = _data(T + V, T, H, V, k)
    if k == 0 or what == "lm":
        tv = ti = None
    if what == "distill":
        lab = None
    elif T > 4:
        lab[[1, T - 1]] = -1, V                                # rows that do not count
    got = _run(h, w, tv, ti, lab)
    _check(got, h, w, tv, ti, lab, what=f"{T}x{H}x{V} k={k} {what}")
    if lab is not None and T > 4:
        assert got[1][1] == 0 and not got[2][1].any() and got[1][T - 1] == 0 and not got[2][T - 1].any()
    # the loss alone: the same rows, bit for bit
    alone = _run(h, w, tv, ti, lab, want_grad=False)
    assert alone[0] == got[0]
    np.testing.assert_array_equal(alone[1], got[1])
    assert _run(h, w, tv, ti, lab, want_grad=False, rows=False)[0] == got[0]


def test_absent_repeated_and_impossible_ids():
    T, H, V, k = 40, 128, 500, 8
    h, w, tv, ti, lab = _data(3, T, H, V, k)
    ti[0] = -1                                                 # none left
    ti[1] = [V, V + 7, -5, 2 ** 31 - 1, -2 ** 31, V, V, V]
    ti[2, 3:] = 1 << 20                                        # some left
    tv[3] = -np.inf                                            # the teacher rules all out
    tv[4, 1:] = -np.inf                                        # all but one
    ti[5] = ti[5, 0]                                           # one id eight times
    ti[6] = lab[6]                                             # the label eight times
    ti[7, 1] = ti[7, 0]
    tv[8] = [80, -80, 0, 0, 0, 0, 0, 0]
    tv[9] = -3.0e38
    for labels in (lab, None):
        got = _run(h, w, tv, ti, labels)
        _check(got, h, w, tv, ti, labels, what="ids")
    assert got[1][0] == 0 and not got[2][0].any()              # no label, no id: nothing to learn from


def test_every_row_masked_and_no_rows():
    h, w, tv, ti, lab = _data(4, 11, 64, 100, 4)
    loss, rows, grad = _run(h, w, tv, ti, np.full(11, -1, np.int32))
    assert loss == 0 and not rows.any() and not grad.any()
    F, T_ = _F(), torch()
    d = F.head_desc(0, 64, 100, 4)
    out = T_.full((1,), 9.0, device="cuda")
    z = T_.empty((0, 64), dtype=T_.bfloat16, device="cuda")
    F.head_loss(d, z, to_dev_bf16(w), out, top_v=T_.empty((0, 4), device="cuda"),
                top_i=T_.empty((0, 4), dtype=T_.int32, device="cuda"),
                workspace=T_.empty(F.head_loss_workspace_size(d), dtype=T_.uint8, device="cuda"))
    assert from_dev(out)[0] == 0


def test_student_that_has_learned():
    # the teacher's logits are the student's own over the whole vocabulary: q - p
    # cancels, and what is left must be small against the terms, not against 2^-8 of them
    h, w, _, _, _ = _data(5, 33, 256, 64, 0)
    ti = np.tile(np.arange(64, dtype=np.int32), (33, 1))
    tv = (h.astype(np.float64) @ w.astype(np.float64).T).astype(np.float32)
    got = _run(h, w, tv, ti, None, dist=1.0)
    _check(got, h, w, tv, ti, None, dist=1.0, what="learned")
    full = head(h, w, tv, ti, None)[3][1]
    assert np.all(np.abs(got[2]) <= 2.0 ** -12 * full.max())


@pytest.mark.parametrize("spread", [30.0, 300.0])
def test_far_logits_move_the_frame(spread):
    # logits hundreds of binary orders apart, the largest ones anywhere in the
    # vocabulary, and labels far below them; two pieces of the vocabulary
    T_ = torch()
    T, H, V = 4200, 64, 80000
    F = _F()
    g = T_.Generator(device="cuda")
    g.manual_seed(8)
    w = T_.randn((V, H), generator=g, device="cuda") * (spread / 8)
    w *= T_.linspace(0.2, 1.0, V, device="cuda")[:, None]      # later entries reach higher
    w = w.to(T_.bfloat16)
    h = T_.randn((T, H), generator=g, device="cuda").to(T_.bfloat16)
    lab = T_.randint(0, V // 10, (T,), generator=g, device="cuda").to(T_.int32)
    d = F.head_desc(T, H, V)
    assert F.head_loss_workspace_size(d) < 2 * T * V           # fewer bytes than the bf16 logits: several pieces
    loss, rows = T_.empty(1, device="cuda"), T_.empty(T, device="cuda")
    grad = T_.empty((T, H), dtype=T_.bfloat16, device="cuda")
    ws = T_.full((F.head_loss_workspace_size(d),), 255, dtype=T_.uint8, device="cuda")
    F.head_loss(d, h, w, loss, labels=lab, row_loss=rows, grad=grad, workspace=ws)
    T_.cuda.synchronize()
    pick = np.random.default_rng(1).permutation(T)[:60]
    hh, ww, ll = from_dev(h[pick.tolist()]), from_dev(w), from_dev(lab[pick.tolist()])
    _, ref_rows, ref_grad, (rest, full) = head(hh, ww, labels=ll)
    za = (np.abs(hh.astype(np.float64)) @ np.abs(ww.astype(np.float64)).T).max(-1)
    ez = (H / 16 + 18) * 2.0 ** -24 * za
    err = np.abs(from_dev(rows)[pick] - ref_rows)
    assert np.all(err <= 2 * ez + 2.0 ** -20 + 4 * 2.0 ** -24 * ref_rows), err.max()
    n = T / 60.0                                               # the oracle's mean is over the 60 rows
    tol = (2.0 ** -8 * np.abs(ref_grad) + 2.0 ** -8 * rest + (4 * ez[:, None] + 2.0 ** -18) * full) / n + 1e-38
    assert np.all(np.abs(from_dev(grad)[pick] - ref_grad / n) <= tol)
    assert abs(from_dev(loss)[0] - from_dev(rows).astype(np.float64).mean()) <= 1e-6 * from_dev(loss)[0]


def test_deterministic_and_rows_of_their_own():
    # the same call twice, bit for bit; and a NaN in one token's state stays in its row
    h, w, tv, ti, lab = _data(6, 300, 128, 3000, 16)
    a, b = _run(h, w, tv, ti, lab), _run(h, w, tv, ti, lab)
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x, y)
    h[7, 3] = np.nan
    c = _run(h, w, tv, ti, lab)
    keep = np.arange(300) != 7
    np.testing.assert_array_equal(c[1][keep], a[1][keep])
    np.testing.assert_array_equal(c[2][keep], a[2][keep])
    assert np.isnan(c[1][7]) and np.isnan(c[0]) and np.isnan(c[2][7]).all()


def test_gradient_matches_differences():
    h, w, tv, ti, lab = _data(9, 20, 128, 400, 8)
    got = _run(h, w, tv, ti, lab)
    u = np.random.default_rng(2).standard_normal(h.shape)
    f = lambda e: head(h + e * u, w, tv, ti, lab, 0.8, 1.2)[0]  # noqa: E731
    d = (f(1e-4) - f(-1e-4)) / 2e-4
    g = got[2].astype(np.float64)
    _, _, _, (rest, _) = head(h, w, tv, ti, lab, 0.8, 1.2)
    # roundings of 2^-8 of each entry and of its terms, taken as independent, five times over
    tol = 5 * 2.0 ** -8 * np.linalg.norm((np.abs(g) + rest) * u) + 1e-6 * abs(d)
    assert abs(d - np.sum(g * u)) <= tol


def test_no_tokens_without_workspace():
    F, T_ = _F(), torch()
    w = T_.zeros((100, 64), dtype=T_.bfloat16, device="cuda")
    z = T_.empty((0, 64), dtype=T_.bfloat16, device="cuda")
    for k in (0, 4):
        out = T_.full((1,), 9.0, device="cuda")
        F.head_loss(F.head_desc(0, 64, 100, k), z, w, out, grad=z)
        assert from_dev(out)[0] == 0


def test_the_most_tokens():
    # 2^24 - 1 tokens, the most of the contract: their sparse logits and the
    # count of rows take 2^24 blocks, 2^32 threads; two pieces of the vocabulary
    F, T_ = _F(), torch()
    T, H, V, k = (1 << 24) - 1, 64, 300, 2
    g = T_.Generator(device="cuda")
    g.manual_seed(12)
    h = T_.randn((T, H), generator=g, device="cuda", dtype=T_.bfloat16)
    w = (T_.randn((V, H), generator=g, device="cuda") * 0.25).to(T_.bfloat16)
    lab = T_.randint(0, V, (T,), generator=g, device="cuda", dtype=T_.int32)
    lab[::7] = -1
    ti = T_.randint(0, V, (T, k), generator=g, device="cuda", dtype=T_.int32)
    tv = T_.randn((T, k), generator=g, device="cuda")
    d = F.head_desc(T, H, V, k, 0.8, 1.2)
    loss, rows = T_.empty(1, device="cuda"), T_.full((T,), -9.0, device="cuda")
    grad = T_.full((T, H), 9.0, dtype=T_.bfloat16, device="cuda")
    ws = T_.full((F.head_loss_workspace_size(d),), 255, dtype=T_.uint8, device="cuda")
    F.head_loss(d, h, w, loss, top_v=tv, top_i=ti, labels=lab, row_loss=rows, grad=grad, workspace=ws)
    T_.cuda.synchronize()
    counted = int((lab >= 0).sum())
    rng = np.random.default_rng(3)
    pick = np.unique(np.concatenate([rng.integers(0, T, 200), [0, 1, T - 1, T - 2, T - 3], (1 << 20) * np.arange(1, 16),
                                     (1 << 20) * np.arange(1, 16) - 1]))
    at = to_dev(pick.astype(np.int64))
    hh, ww, ll, vv, ii = from_dev(h[at]), from_dev(w), from_dev(lab[at]), from_dev(tv[at]), from_dev(ti[at])
    _, ref, ref_grad, (rest, full) = head(hh, ww, vv, ii, ll, 0.8, 1.2)
    live = ll >= 0
    n = counted / live.sum()                                   # the oracle's mean is over the picked rows that count
    ez = (H / 16 + 18) * 2.0 ** -24 * (np.abs(hh.astype(np.float64)) @ np.abs(ww.astype(np.float64)).T).max(-1)
    err = np.abs(from_dev(rows[at]) - ref)                     # the bounds of _check
    assert np.all(err <= 2.0 * (2 * ez + 2.0 ** -20 + 4 * 2.0 ** -24 * np.abs(ref)) + 2.0 ** -22)
    # and of 1/n: its own rounding and the count's, 2^-23 of each value, in the room of 2^-18 of the terms
    tol = (2.0 ** -8 * np.abs(ref_grad) + 2.0 ** -8 * rest + (4 * ez[:, None] + 2.0 ** -18) * full) / n + 1e-38
    assert np.all(np.abs(from_dev(grad[at]) - ref_grad / n) <= tol)
    assert bool((rows[::7] == 0).all()) and bool((rows >= -1e-3).all())
    mean = float(rows.double().sum() / counted)
    assert abs(from_dev(loss)[0] - mean) <= 2.0 ** -22 * mean  # 1/n and the loss, one rounding each


def _piece(F, T, H, V, k):
    """Vocabulary entries of a piece: without the gradient the workspace grows by 8 bytes per token and 64 entries
    of a piece, a piece has whole multiples of 256, and 256 where the vocabulary is no longer."""
    size = lambda v: F.head_loss_workspace_size(F.head_desc(T, H, v, k), grad=False)  # noqa: E731
    assert T * 32 % 256 == 0                                    # the parts' rounding up takes no share in the difference
    return 256 + (size(V) - size(max(k, 1))) * 64 // (8 * T)


def _many_pieces(seed, T, H, V, k, far):
    """Numpy inputs of several pieces: labels and teacher ids from 72 entries that lie at both ends of every piece
    and between, and whose logits stand out, so that each has about a hundredth of a token's probability; with `far`
    later entries reach ever higher instead, hundreds of binary orders above those."""
    F = _F()
    vc = _piece(F, T, H, V, k)
    ends = [e for p in range(0, V, vc) for e in (p, p + 1, min(p + vc, V) - 1, min(p + vc, V) - 2)]
    assert vc < V
    rng = np.random.default_rng(seed)
    special = np.array(sorted(set(ends) | set(rng.integers(0, V, 72 - len(set(ends))).tolist())), np.int32)
    w = rng.standard_normal((V, H)).astype(np.float32)
    h = rng.standard_normal((T, H)).astype(np.float32)
    if far:
        w *= np.linspace(1.0, 25.0, V, dtype=np.float32)[:, None]
    else:
        # logits of standard deviation 0.5; the special ones 8 and, in all, as much again as half of the others
        w *= np.float32(0.5 / np.sqrt(H))
        h[:, 0] = 4.0
        w[special, 0] = (8.0 + np.log(V / 7e4)) / 4.0
    w, h = bf16_rne(w), bf16_rne(h)
    pick = np.argsort(rng.random((T, special.size)), axis=1)[:, :k + 1]
    lab, ti = special[pick[:, -1]], special[pick[:, :k]]
    own = rng.random(T) < 0.5
    ti[own, 5 % max(k, 1)] = lab[own]                           # the label among the teacher's ids, in half the rows
    lab[::17] = -1
    return h, w, (rng.standard_normal((T, k)) * 2).astype(np.float32), np.ascontiguousarray(ti), lab, vc, special


# merges of 16 tokens and of 4 a block; 65 slots a token (16 * 65 are more than the block's threads); four to six
# pieces, moved frames with the teacher's entries among them.  Near, one slot's share counted twice would be beyond
# the bound in every row that counts, in three quarters of its elements
@pytest.mark.parametrize("T,V", [(4200, 250000), (1024, 700000), (1000, 700000)])
@pytest.mark.parametrize("far", [False, True], ids=["near", "far"])
def test_a_teacher_over_several_pieces(T, V, far):
    F, T_ = _F(), torch()
    H, k = 64, 64
    h, w, tv, ti, lab, vc, special = _many_pieces(T, T, H, V, k, far)
    loss, rows, grad = _run(h, w, tv, ti, lab)
    pick = np.random.default_rng(7).permutation(T)[:40]
    pick[0] = 0                                                # a row that does not count
    _, ref_rows, ref_grad, (rest, full) = head(h[pick], w, tv[pick], ti[pick], lab[pick], 0.8, 1.2)
    n = (lab >= 0).sum() / (lab[pick] >= 0).sum()              # the oracle's mean is over the picked rows that count
    ez = (H / 16 + 18) * 2.0 ** -24 * (np.abs(h[pick].astype(np.float64)) @ np.abs(w.astype(np.float64)).T).max(-1)
    # the bounds of _check
    assert np.all(np.abs(rows[pick] - ref_rows) <= 2.0 * (2 * ez + 2.0 ** -20 + 4 * 2.0 ** -24 * np.abs(ref_rows)) + 2.0 ** -22)
    tol = (2.0 ** -8 * np.abs(ref_grad) + 2.0 ** -8 * rest + (4 * ez[:, None] + 2.0 ** -18) * full) / n + 1e-38
    bad = np.abs(grad[pick] - ref_grad / n) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {(np.abs(grad[pick] - ref_grad / n) / tol).max():.2f}"
    assert rows[0] == 0 and not grad[0].any()
    mean = rows.astype(np.float64).sum() / (lab >= 0).sum()
    assert abs(loss - mean) <= 2.0 ** -22 * abs(mean)
    alone = _run(h, w, tv, ti, lab, want_grad=False)           # the loss alone: bit for bit
    assert alone[0] == loss
    np.testing.assert_array_equal(alone[1], rows)


@pytest.mark.parametrize("T", [7, 300])
@pytest.mark.parametrize("spread", [30.0, 300.0])
def test_far_logits_with_few_tokens(T, spread):
    # as above in one piece with merges of 4 tokens a block: every row and element against the oracle
    rng = np.random.default_rng(T)
    H, V, k = 64, 20000, 9
    w = rng.standard_normal((V, H)) * (spread / 8) * np.linspace(0.2, 1.0, V)[:, None]
    w, h = bf16_rne(w.astype(np.float32)), bf16_rne(rng.standard_normal((T, H)).astype(np.float32))
    lab = rng.integers(0, V // 10, T).astype(np.int32)
    ti = np.stack([np.append(rng.permutation(V // 10)[:k - 1], rng.integers(0, V)) for _ in range(T)]).astype(np.int32)
    tv = (rng.standard_normal((T, k)) * 2).astype(np.float32)
    for args in ((tv, ti, lab), (None, None, lab), (tv, ti, None)):
        _check(_run(h, w, *args), h, w, *args, what=f"{T} spread {spread}")
