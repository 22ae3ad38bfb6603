"""Log probabilities and the gradients' norm run with the operators that they stand beside, as they are used: a
teacher's pass that feeds the distillation loss, a sequence trained on its log probabilities and entropies, a served
token beside a batch; on streams of their own, captured into graphs and replayed on other inputs, two calls at once;
many rows, and weights past 4 GB."""
import numpy as np
import pytest

from oracle import logprob as O
from oracle.head import head
from oracle.numerics import bf16_rne
from tests.fq_testutil import from_dev, to_dev, to_dev_bf16, torch
from tests.test_gpu_logprob import _hidden, _out, _workspace

pytestmark = pytest.mark.gpu


def _F():
    from scale_only_quantization_amd import fqlib
    return fqlib


def _same(a, b, what=""):
    for n in a:
        if a[n] is not None:
            assert torch().equal(a[n], b[n]), (what, n)


class Scorer:
    """Buffers of a forward and a backward pass from hidden states."""

    def __init__(self, T, H, V, m, k):
        F, T_ = _F(), torch()
        self.F, self.d = F, F.logprob_desc(T, V, given=m, top=k, hidden=H)
        self.out = _out(T, m, k)
        self.grad = T_.zeros((T, H), dtype=T_.bfloat16, device="cuda")
        self.ws = _workspace(F.head_logprob_workspace_size(self.d))
        self.wsb = _workspace(F.head_logprob_workspace_size(self.d, True))

    def run(self, h, w, ids, dl, de):
        self.F.head_logprob_fwd(self.d, h, w, ids=ids, workspace=self.ws, **self.out)
        self.F.head_logprob_bwd(self.d, h, w, self.out["lse"], self.grad, ids=ids, dlogp=dl, entropy=self.out["entropy"],
                                dentropy=de, workspace=self.wsb)
        return dict(self.out, grad=self.grad)


def test_teachers_pass_feeds_the_distillation_loss():
    """Top 16 of a teacher's hidden states -> fq_head_loss of the student's -> its loss and gradient, and the student's
    gradients clipped beside others."""
    F, T_ = _F(), torch()
    T, H, V, k = 300, 256, 9001, 16
    ht, w, lab, zt = _hidden(1, T, H, V, 1)
    rng = np.random.default_rng(8)
    hs = bf16_rne((ht + 0.2 * rng.standard_normal(ht.shape)).astype(np.float32))
    d = F.logprob_desc(T, V, top=k, hidden=H)
    wd = to_dev_bf16(w)
    tv, ti = T_.zeros((T, k), device="cuda"), T_.zeros((T, k), dtype=T_.int32, device="cuda")
    F.head_logprob_fwd(d, to_dev_bf16(ht), wd, top_ids=ti, top_logp=tv, workspace=_workspace(F.head_logprob_workspace_size(d)))
    hd = F.head_desc(T, H, V, k, 0.8, 1.2)
    loss, grad = T_.zeros(1, device="cuda"), T_.zeros((T, H), dtype=T_.bfloat16, device="cuda")
    F.head_loss(hd, to_dev_bf16(hs), wd, loss, top_v=tv, top_i=ti, labels=to_dev(lab[:, 0].copy()), grad=grad,
                workspace=_workspace(F.head_loss_workspace_size(hd)))
    ref = O.forward(zt, None, k)
    assert np.array_equal(from_dev(ti), ref["top_ids"])
    want, _, wgrad, (rest, full) = head(hs, w, ref["top_logp"], ref["top_ids"], lab[:, 0], 0.8, 1.2)
    assert abs(loss.item() - want) <= 1e-5 * (1 + abs(want))
    g = from_dev(grad).astype(np.float64)
    # the output's rounding and the probabilities', both half a bf16 step, and fp32 sums
    assert np.all(np.abs(g - wgrad) <= 2.0 ** -8 * (np.abs(wgrad) + rest) * 1.01 + 2.0 ** -15 * full)
    others = [T_.randn(n, device="cuda") for n in (1000, 33)]
    G = F.grad_list([grad] + others)
    norm = T_.zeros(1, device="cuda")
    F.grad_norm(G, norm, _workspace(F.grad_norm_workspace_size(G)))
    before = [x.clone() for x in [grad] + others]
    F.grad_clip(G, 1.0, norm)
    T_.cuda.synchronize()
    total = np.sqrt(sum(float((x.double() ** 2).sum()) for x in before))
    after = np.sqrt(sum(float((x.double() ** 2).sum()) for x in [grad] + others))
    # bf16 rounding of the first tensor's share, far below the fp32 ones'
    assert abs(norm.item() - total) <= 1e-6 * total and abs(after - 1.0) <= 2.0 ** -8


@pytest.mark.parametrize("T,V,m", [(40, 700, 1), (270, 3001, 3)])
def test_gradient_against_differences(T, V, m):
    """d L / d h along random directions against differences of the loss in float64."""
    H = 128
    h, w, ids, _ = _hidden(3, T, H, V, m)
    rng = np.random.default_rng(1)
    dl = rng.standard_normal((T, m)).astype(np.float32)
    de = (rng.standard_normal(T) * 0.5).astype(np.float32)
    s = Scorer(T, H, V, m, 0)
    got = s.run(to_dev_bf16(h), to_dev_bf16(w), to_dev(ids), to_dev(dl), to_dev(de))
    g = from_dev(got["grad"]).astype(np.float64)

    def loss(x):
        r = O.forward(x @ w.astype(np.float64).T, ids)
        return np.sum(r["logp"] * dl, -1) + r["entropy"] * de

    z = h.astype(np.float64) @ w.astype(np.float64).T
    dz, part = O.backward(z, ids, dl, de)
    size = (np.abs(dz) + part) @ np.abs(w.astype(np.float64))
    for _ in range(3):
        v = rng.standard_normal(h.shape)
        e = 1e-4
        num = (loss(h + e * v) - loss(h - e * v)) / (2 * e)
        # half a bf16 step of the gradient and of each probability in it; the differences' own error is below 1e-6
        tol = np.sum((2.0 ** -8 * (np.abs(g) + size)) * np.abs(v), -1) * 1.01 + 1e-5
        assert np.all(np.abs(np.sum(g * v, -1) - num) <= tol)


def test_a_row_gives_the_same_in_every_form():
    """One row of hidden states alone, beside few others and in a batch: the same ids (the logits are exact here), the
    same values but for the order of the sums."""
    F, T_ = _F(), torch()
    H, V, k = 512, 30011, 20
    h, w, ids, z = _hidden(5, 600, H, V, 1)
    ref = O.forward(z[:1], ids[:1], k)
    wd, hd, idd = to_dev_bf16(w), to_dev_bf16(h), to_dev(ids)
    for T in (1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 256, 257, 600):
        d = F.logprob_desc(T, V, given=1, top=k, hidden=H)
        out = _out(T, 1, k)
        F.head_logprob_fwd(d, hd[:T], wd, ids=idd[:T], workspace=_workspace(F.head_logprob_workspace_size(d)), **out)
        T_.cuda.synchronize()
        assert np.array_equal(from_dev(out["top_ids"])[:1], ref["top_ids"]), T
        for n in ("lse", "entropy", "logp", "top_logp"):
            assert np.allclose(from_dev(out[n])[:1], ref[n], rtol=2e-6, atol=5e-6), (T, n)


def test_streams_and_two_calls_at_once():
    T_ = torch()
    args = []
    for i in range(2):
        T, H, V, m, k = (300, 256, 20000, 1, 16) if i == 0 else (500, 128, 33000, 2, 64)
        h, w, ids, _ = _hidden(20 + i, T, H, V, m)
        rng = np.random.default_rng(i)
        args.append((Scorer(T, H, V, m, k), Scorer(T, H, V, m, k),
                     (to_dev_bf16(h), to_dev_bf16(w), to_dev(ids), to_dev(rng.standard_normal((T, m)).astype(np.float32)),
                      to_dev(rng.standard_normal(T).astype(np.float32)))))
    want = [dict((n, None if v is None else v.clone()) for n, v in a.run(*x).items()) for a, _, x in args]
    T_.cuda.synchronize()
    streams = [T_.cuda.Stream(), T_.cuda.Stream()]
    for _ in range(3):
        for s, (_, b, x) in zip(streams, args):
            with T_.cuda.stream(s):
                b.run(*x)
    T_.cuda.synchronize()
    for w_, (_, b, _) in zip(want, args):
        _same(w_, dict(b.out, grad=b.grad))
    # a stream given to the call
    F = _F()
    _, b, x = args[0]
    b.out["lse"].fill_(0.0)
    T_.cuda.synchronize()
    F.head_logprob_fwd(b.d, x[0], x[1], ids=x[2], workspace=b.ws, stream=streams[0].cuda_stream, **b.out)
    streams[0].synchronize()
    _same({n: want[0][n] for n in b.out}, b.out)


@pytest.mark.parametrize("form", ["hidden few", "hidden", "logits", "clip"])
def test_captured_and_replayed_on_other_inputs(form):
    """A captured forward and backward, replayed with other inputs in the same buffers, eager work in between."""
    F, T_ = _F(), torch()
    rng = np.random.default_rng(9)
    if form == "clip":
        grads = [T_.randn(n, device="cuda") for n in (5, 20000, 1, 777)] + [T_.randn(333, device="cuda").bfloat16()]
        outs = [T_.zeros_like(g) for g in grads]
        G, norm = F.grad_list(grads, outs), T_.zeros(1, device="cuda")
        ws = _workspace(F.grad_norm_workspace_size(G))
        inputs, outputs = grads, outs + [norm]

        def run():
            F.grad_norm(G, norm, ws)
            F.grad_clip(G, 1.0, norm)
    elif form == "logits":
        T, V = 20, 20011
        z, grad = (T_.randn((T, (V + 7) // 8 * 8), device="cuda").bfloat16()[:, :V] for _ in range(2))
        ids, dl, de = T_.randint(0, V, (T, 2), device="cuda").to(T_.int32), T_.randn((T, 2), device="cuda"), T_.randn(T, device="cuda")
        d, out = F.logprob_desc(T, V, given=2, top=30), _out(T, 2, 30)
        ws = _workspace(F.logprob_workspace_size(d))
        inputs, outputs = [z, dl, de], [grad] + list(out.values())

        def run():
            F.logprob_fwd(d, z, ids=ids, workspace=ws, **out)
            F.logprob_bwd(d, z, out["lse"], grad, ids=ids, dlogp=dl, entropy=out["entropy"], dentropy=de)
    else:
        T, H, V, m, k = (3, 128, 9000, 1, 10) if form == "hidden few" else (300, 128, 20000, 1, 32)
        h, w, ids, _ = _hidden(2, T, H, V, m)
        s = Scorer(T, H, V, m, k)
        x = [to_dev_bf16(h), to_dev_bf16(w), to_dev(ids), to_dev(rng.standard_normal((T, m)).astype(np.float32)),
             to_dev(rng.standard_normal(T).astype(np.float32))]
        inputs, outputs = [x[0], x[3], x[4]], [s.grad] + [v for v in s.out.values() if v is not None]

        def run():
            s.run(*x)
    run()
    T_.cuda.synchronize()
    graph = T_.cuda.CUDAGraph()
    with T_.cuda.graph(graph):
        run()
    for i in range(4):
        for t in inputs:
            t.copy_(T_.roll(t, i + 1, 0) * (0.5 if i % 2 else 2.0))
        run()
        T_.cuda.synchronize()
        want = [o.clone() for o in outputs]
        for o in outputs:
            o.zero_()
        T_.randn(1000, device="cuda").sum().item()                          # eager work and a wait in between
        graph.replay()
        T_.cuda.synchronize()
        for o, e in zip(outputs, want):
            assert T_.equal(o, e), (form, i)


def test_more_rows_than_the_grids_second_axis():
    F, T_ = _F(), torch()
    g = T_.Generator(device="cuda")
    g.manual_seed(1)
    T, V, k = 70001, 41, 3
    buf = T_.zeros((T, 48), dtype=T_.bfloat16, device="cuda")
    z = buf[:, :V]
    z.copy_(T_.randn((T, V), generator=g, device="cuda") * 3)
    ids = T_.randint(-1, V, (T, 1), generator=g, device="cuda").to(T_.int32)
    dl = T_.randn((T, 1), generator=g, device="cuda")
    d, out = F.logprob_desc(T, V, given=1, top=k), _out(T, 1, k)
    F.logprob_fwd(d, z, ids=ids, workspace=_workspace(F.logprob_workspace_size(d)), **out)
    grad = T_.zeros_like(buf)[:, :V]
    F.logprob_bwd(d, z, out["lse"], grad, ids=ids, dlogp=dl)
    T_.cuda.synchronize()
    zn = from_dev(z).astype(np.float64)
    ref = O.forward(zn, from_dev(ids), k)
    assert np.array_equal(from_dev(out["top_ids"]), ref["top_ids"])
    for n in ("lse", "entropy", "logp", "top_logp"):
        assert np.allclose(from_dev(out[n]), ref[n], rtol=2e-6, atol=2e-5), n
    want, _ = O.backward(zn, from_dev(ids), from_dev(dl))
    assert np.allclose(from_dev(grad), want, rtol=2.0 ** -8 * 1.01, atol=1e-5)
    # from hidden states: 70001 rows of 64
    h, w, hid, zh = _hidden(4, T, 64, 300, 1)
    d, out = F.logprob_desc(T, 300, given=1, top=k, hidden=64), _out(T, 1, k)
    F.head_logprob_fwd(d, to_dev_bf16(h), to_dev_bf16(w), ids=to_dev(hid), workspace=_workspace(F.head_logprob_workspace_size(d)),
                       **out)
    T_.cuda.synchronize()
    ref = O.forward(zh, hid, k)
    assert np.array_equal(from_dev(out["top_ids"]), ref["top_ids"])
    assert np.allclose(from_dev(out["lse"]), ref["lse"], rtol=2e-6, atol=2e-5)
    assert np.allclose(from_dev(out["logp"]), ref["logp"], rtol=2e-6, atol=2e-5)


@pytest.mark.parametrize("T", [2, 20, 130])
def test_output_weight_past_4gb(T):
    """2.3 M rows of 1024 (4.7 GB): the largest logits stand near the end, and the gradient reaches there."""
    F, T_ = _F(), torch()
    V, H, k = 2_300_003, 1024, 8
    g = T_.Generator(device="cuda")
    g.manual_seed(6)
    w = T_.empty((V, H), dtype=T_.bfloat16, device="cuda")
    for r in range(0, V, 100_000):
        n = min(100_000, V - r)
        w[r:r + n] = T_.randint(-20, 21, (n, H), generator=g, device="cuda").bfloat16() / 1024
    h = T_.randint(-60, 61, (T, H), generator=g, device="cuda").float() / 32
    far = V - 1 - T_.arange(T, device="cuda") * 5
    h = (h + 24 * w[far].float()).mul(32).round().clamp(-127, 127).div(32).bfloat16()
    ids = far.to(T_.int32)[:, None].contiguous()
    s = Scorer(T, H, V, 1, k)
    dl, de = T_.randn((T, 1), generator=g, device="cuda"), T_.randn(T, generator=g, device="cuda") * 0.1
    got = s.run(h, w, ids, dl, de)
    T_.cuda.synchronize()
    for r in range(0, T, 26):
        rows = slice(r, min(r + 2, T))
        z = T_.cat([h[rows].double() @ w[c:c + 100_000].double().t() for c in range(0, V, 100_000)], 1)
        lse = T_.logsumexp(z, -1)
        order = T_.sort(z, dim=-1, descending=True, stable=True).indices[:, :k]
        assert T_.equal(got["top_ids"][rows], order.to(T_.int32))
        assert T_.allclose(got["lse"][rows].double(), lse, rtol=1e-6, atol=1e-5)
        lp = z - lse[:, None]
        p = lp.exp()
        ent = -(p * lp).sum(-1)
        assert T_.allclose(got["entropy"][rows].double(), ent, rtol=1e-5, atol=1e-5)
        at = T_.arange(z.shape[0], device="cuda")
        assert T_.allclose(got["logp"][rows, 0].double(), lp[at, far[rows]], rtol=1e-6, atol=2e-5)
        dz = -p * (dl[rows].double() + de[rows, None].double() * (lp + ent[:, None]))
        size = sum(dz[:, c:c + 100_000].abs() @ w[c:c + 100_000].double().abs() for c in range(0, V, 100_000))
        dz[at, far[rows]] += dl[rows, 0].double()
        ref = sum(dz[:, c:c + 100_000] @ w[c:c + 100_000].double() for c in range(0, V, 100_000))
        assert bool((T_.abs(got["grad"][rows].double() - ref) <= 2.0 ** -8 * (ref.abs() + size) * 1.01 + 1e-6).all())
