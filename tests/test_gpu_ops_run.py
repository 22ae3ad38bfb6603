"""The operators around the expert layer run together, as they are used: a
training step from the norm in front of the layer to the loss and back, and a
served token from the norm through the packed layer; on a stream of their own,
captured into graphs and replayed on other inputs; and tensors past 4 GB."""
import numpy as np
import pytest

import synth
from oracle import norm as ON
from oracle import packed as OPK
from oracle.head import head
from oracle.numerics import bf16_rne
from tests.fq_testutil import assert_bits_equal, from_dev, to_dev, to_dev_bf16, torch

pytestmark = pytest.mark.gpu
EPS = 1e-6
E, H, I, T, K, V, TOP = 8, 256, 128, 48, 2, 500, 8


def _F():
    from scale_only_quantization_amd import fqlib
    return fqlib


class Train:
    """s1 = x + res; y1 = norm(s1); o = experts(y1); s2 = s1 + o; y2 = norm(s2); loss(y2); and d loss / d x."""

    def __init__(self, fmt="none"):
        from scale_only_quantization_amd.layer import ExpertLayer, LayerDims
        F, T_ = _F(), torch()
        rng = np.random.default_rng(3)
        b = lambda *s, f=1.0: bf16_rne((rng.standard_normal(s) * f).astype(np.float32))  # noqa: E731
        self.n = dict(W1=b(E, 2 * I, H, f=0.08), W2=b(E, H, I, f=0.1), x=b(T, H), res=b(T, H), g1=bf16_rne(1 + 0.2 * b(H)),
                      g2=bf16_rne(1 + 0.2 * b(H)), w=b(V, H, f=0.12))
        n = self.n
        n["ids"] = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
        n["tw"] = rng.random((T, K)).astype(np.float32)
        n["lab"] = rng.integers(0, V, T).astype(np.int32)
        n["lab"][[2, 9]] = -1
        n["ti"] = np.stack([rng.permutation(V)[:TOP] for _ in range(T)]).astype(np.int32)
        n["tv"] = (rng.standard_normal((T, TOP)) * 2).astype(np.float32)
        none = F.qdesc()
        self.layer = ExpertLayer(LayerDims(E, H, I, T, K), (none,) * 4, n["W1"], n["W2"], n["x"], n["ids"], n["tw"],
                                 np.zeros((T, H), np.float32))
        d = {k: to_dev_bf16(n[k]) for k in ("x", "res", "g1", "g2", "w")}
        d.update({k: to_dev(n[k]) for k in ("lab", "ti", "tv")})
        new = lambda dt, *s: T_.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        bf, f32 = T_.bfloat16, T_.float32
        for k in ("s1", "s2", "y2", "dy2", "ds2", "dx"):
            d[k] = new(bf, T, H)
        d.update(r1=new(f32, T), r2=new(f32, T), loss=new(f32, 1), rows=new(f32, T), dg1=new(f32, H), dg2=new(f32, H))
        self.hd = F.head_desc(T, H, V, TOP, 0.8, 1.2)
        d["hws"] = new(T_.uint8, F.head_loss_workspace_size(self.hd))
        d["nws"] = new(T_.uint8, F.rms_norm_bwd_workspace_size(T, H))
        self.d, self.F = d, F

    def step(self):
        F, d, L = self.F, self.d, self.layer
        y1, dy1 = L.d["X"], L.dx                           # the layer's input and its gradient
        F.rms_norm_fwd(d["x"], d["g1"], EPS, residual=d["res"], sum=d["s1"], y=y1, rstd=d["r1"])
        L.forward()
        F.rms_norm_fwd(L.y, d["g2"], EPS, residual=d["s1"], sum=d["s2"], y=d["y2"], rstd=d["r2"])
        F.head_loss(self.hd, d["y2"], d["w"], d["loss"], top_v=d["tv"], top_i=d["ti"], labels=d["lab"],
                    row_loss=d["rows"], grad=d["dy2"], workspace=d["hws"])
        F.rms_norm_bwd(d["s2"], d["g2"], d["r2"], d["dy2"], L.d["dY"], dgamma=d["dg2"], workspace=d["nws"])
        L.backward()
        F.rms_norm_bwd(d["s1"], d["g1"], d["r1"], dy1, d["dx"], dsum=L.d["dY"], dgamma=d["dg1"], workspace=d["nws"])

    def outputs(self):
        return {k: self.d[k].clone() for k in ("loss", "rows", "dy2", "dx", "dg1", "dg2", "s2")}

    def loss64(self, x):
        """The loss of float64 x with no rounding on the way."""
        n = self.n
        s1 = x + n["res"]
        nrm = lambda s, g: s * g / np.sqrt(np.mean(s * s, -1, keepdims=True) + EPS)  # noqa: E731
        y1 = nrm(s1, n["g1"])
        o = np.zeros_like(s1)
        W1, W2 = n["W1"].astype(np.float64), n["W2"].astype(np.float64)
        for t in range(T):
            for j in range(K):
                e = n["ids"][t, j]
                z = W1[e] @ y1[t]
                o[t] += float(n["tw"][t, j]) * (W2[e] @ (z[:I] / (1 + np.exp(-z[:I])) * z[I:]))
        return head(nrm(s1 + o, n["g2"]), n["w"], n["tv"], n["ti"], n["lab"], 0.8, 1.2)[0]


def test_training_step_against_differences():
    m = Train()
    m.step()
    torch().cuda.synchronize()
    x = m.n["x"].astype(np.float64)
    ref = m.loss64(x)
    # bf16 streams on the way: each of a dozen roundings moves the hidden state
    # by up to 2^-9 rms, at random; the loss, a mean over 46 rows of terms of
    # order ten, by well under a hundredth
    assert abs(from_dev(m.d["loss"])[0] - ref) <= 1e-2 * ref
    dx = from_dev(m.d["dx"]).astype(np.float64)
    rng = np.random.default_rng(7)
    # along dx itself (the derivative is its squared norm) and along a random
    # direction; the gradient's roundings are of 2^-8 of entries, at random over
    # 12288 of them
    for u, scale in ((dx / np.linalg.norm(dx), 1.0), (rng.standard_normal(dx.shape) / np.sqrt(dx.size), 0.1)):
        h = 1e-4
        fd = (m.loss64(x + h * u) - m.loss64(x - h * u)) / (2 * h)
        assert abs(fd - np.sum(dx * u)) <= 0.03 * scale * np.linalg.norm(dx) + 1e-9, (fd, np.sum(dx * u))
    assert not from_dev(m.d["rows"])[[2, 9]].any()


def test_training_step_on_a_stream_and_as_a_graph():
    T_ = torch()
    m = Train()
    m.step()
    T_.cuda.synchronize()
    eager = m.outputs()
    side = T_.cuda.Stream()
    side.wait_stream(T_.cuda.current_stream())
    with T_.cuda.stream(side):                              # the current stream of the tensors' device is taken
        m.step()
    side.synchronize()
    for k, v in m.outputs().items():
        assert T_.equal(v, eager[k]), f"{k} on another stream"
    g = T_.cuda.CUDAGraph()
    with T_.cuda.graph(g):
        m.step()
    other = T_.randn((T, H), device="cuda").to(T_.bfloat16)
    first = m.d["x"].clone()
    for i in range(4):                                      # replays with eager work and other inputs between them
        m.d["x"].copy_(other if i % 2 else first)
        for k in ("loss", "rows", "dx", "dg1", "dg2"):
            m.d[k].fill_(3.0)
        g.replay()
        T_.cuda.synchronize()
        got = m.outputs()
        m.step()
        T_.cuda.synchronize()
        for k, v in m.outputs().items():
            assert T_.equal(v, got[k]), f"{k}, replay {i}"
        assert i % 2 or all(T_.equal(got[k], eager[k]) for k in got)


def test_served_tokens():
    """norm with codes -> packed layer -> norm -> a dense packed product, against the oracle stage by stage, and as
    a graph replayed on other tokens."""
    F, T_ = _F(), torch()
    case = synth.CASES["tiny"]
    data = synth.make_layer(case, T=6)
    P = synth.layer_params(data, "nvfp4")
    q = F.preset("nvfp4")
    ws = []
    for n in ("1", "2"):
        W = to_dev_bf16(data["W" + n])
        B, N, C = W.shape
        c, b = T_.empty((B, N, C // 2), dtype=T_.uint8, device="cuda"), T_.empty((B, N, C // 16), dtype=T_.uint8, device="cuda")
        t = to_dev(P["t_w" + n])
        F.fq_tensor(q[0], W, to_dev(P["s_w" + n]), t, codes=c, block_codes=b)
        ws.append(dict(codes=c, block_codes=b, tensor_scale=t))
    L = F.layer_desc(case.E, case.H, case.I, 6, case.k, *q)
    packed = F.packed_experts(*ws, to_dev(P["s_a1"]), to_dev(P["s_a2"]))
    rng = np.random.default_rng(5)
    gamma = bf16_rne((1 + 0.2 * rng.standard_normal(case.H)).astype(np.float32))
    new = lambda dt, *s: T_.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    bf = T_.bfloat16
    x, g, ids, tw = to_dev_bf16(data["X"]), to_dev_bf16(gamma), to_dev(data["ids"]), to_dev(data["w"])
    y1, o, s2, y2, out = (new(bf, 6, case.H) for _ in range(5))
    fp8 = F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_ROW, 0, F.FQ_DYNAMIC)
    codes, scale = new(T_.uint8, 6, case.H), new(T_.float32, 6)
    wsp = new(T_.uint8, F.packed_expert_workspace_size(L))
    i4 = F.qdesc(F.FQ_INT, F.FQ_PER_GROUP, 64, F.FQ_LEARNABLE, -8, 7)
    dc = rng.integers(0, 256, (1, case.H, case.H // 2)).astype(np.uint8)
    ds = (rng.random((1, case.H, case.H // 64)) * 0.01).astype(np.float32)
    dcd, dsd = to_dev(dc), to_dev(ds)

    def run():
        F.rms_norm_fwd(x, g, EPS, y=y1)
        F.packed_expert_fwd(L, packed, y1, ids, tw, o, wsp)
        F.rms_norm_fwd(o, g, EPS, residual=x, sum=s2, y=y2, q=fp8, codes=codes, scale=scale)
        F.packed_matvec(i4, dcd, y2, out, scale=dsd)

    run()
    T_.cuda.synchronize()
    assert_bits_equal(from_dev(y1), ON.forward(data["X"], gamma, EPS)[1], "y1")
    W = [OPK.dequant(*(from_dev(w[k]) if k in w else None for k in ("codes", "scale", "block_codes", "tensor_scale")))
         for w in ws]
    from oracle import presets as OP
    _, _, a1, a2 = OP.PRESETS["nvfp4"]
    ref = OPK.experts(*W, from_dev(y1), data["ids"], data["w"], a1, P["s_a1"], a2, P["s_a2"])
    assert np.linalg.norm(from_dev(o) - ref) <= 2.0 ** -7 * np.linalg.norm(ref)
    s, y, _ = ON.forward(from_dev(o), gamma, EPS, data["X"])
    assert_bits_equal(from_dev(s2), s, "s2")
    assert_bits_equal(from_dev(y2), y, "y2")
    Wd = OPK.dequant(dc, scale=ds)[0]
    ref = y.astype(np.float64) @ Wd.T
    assert np.linalg.norm(from_dev(out) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    graph = T_.cuda.CUDAGraph()
    with T_.cuda.graph(graph):
        run()
    for i in range(3):
        x.copy_(T_.randn((6, case.H), device="cuda").to(bf))
        ids.copy_(T_.rand((6, case.E), device="cuda").topk(case.k, -1).indices.to(T_.int32))
        out.fill_(9.0)
        codes.fill_(9)
        graph.replay()
        T_.cuda.synchronize()
        got = (out.clone(), codes.clone(), scale.clone(), s2.clone())
        run()
        T_.cuda.synchronize()
        for a, b in zip(got, (out, codes, scale, s2)):
            assert T_.equal(a, b), f"replay {i}"


def test_two_calls_at_once_with_their_own_workspaces():
    # two streams, each with its own buffers: neither's result depends on the other
    T_ = torch()
    a, b = Train(), Train()
    b.d["x"].copy_(T_.randn((T, H), device="cuda").to(T_.bfloat16))
    a.step(), b.step()
    T_.cuda.synchronize()
    want = a.outputs(), b.outputs()
    s = T_.cuda.Stream(), T_.cuda.Stream()
    T_.cuda.synchronize()
    for _ in range(3):
        for m, st in zip((a, b), s):
            with T_.cuda.stream(st):
                m.step()
    T_.cuda.synchronize()
    for m, w in zip((a, b), want):
        for k, v in m.outputs().items():
            assert T_.equal(v, w[k]), k


def test_past_four_gigabytes():
    F, T_ = _F(), torch()
    # a stack of matrices whose codes pass 2^32 bytes: the last matrix
    B, N, C = 1100, 1024, 8192
    codes = T_.zeros((B, N, C // 2), dtype=T_.uint8, device="cuda")
    scale = T_.zeros((B, N), device="cuda")
    rng = np.random.default_rng(1)
    c = rng.integers(0, 256, (1, N, C // 2)).astype(np.uint8)
    s = (rng.random((1, N)) * 0.01).astype(np.float32)
    codes[-1:] = to_dev(c)
    scale[-1:] = to_dev(s)
    x = bf16_rne(rng.standard_normal((2, C)).astype(np.float32))
    y = T_.empty((2, N), dtype=T_.bfloat16, device="cuda")
    F.packed_matvec(F.qdesc(F.FQ_INT, F.FQ_PER_ROW, 0, F.FQ_LEARNABLE, -8, 7), codes, to_dev_bf16(x), y, scale=scale,
                    which=to_dev(np.array([B - 1, 0], np.int32)))
    ref = x[0].astype(np.float64) @ OPK.dequant(c, scale=s)[0].T
    assert np.linalg.norm(from_dev(y)[0] - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    assert not from_dev(y)[1].any()
    del codes, scale
    # more than 2^31 elements through the norm and its gradient: the last rows
    R, C = 1_050_001, 2048
    x = T_.randn((R, C), device="cuda", dtype=T_.bfloat16)
    g = T_.ones(C, dtype=T_.bfloat16, device="cuda")
    y, r = T_.empty_like(x), T_.empty(R, device="cuda")
    F.rms_norm_fwd(x, g, EPS, y=y, rstd=r)
    last = from_dev(x[-3:])
    assert_bits_equal(from_dev(y[-3:]), ON.forward(last, np.ones(C, np.float32), EPS)[1], "last rows")
    dx = T_.empty_like(x)
    F.rms_norm_bwd(x, g, r, y, dx)
    ref, _ = ON.backward(last, np.ones(C), from_dev(r[-3:]), from_dev(y[-3:]))
    # y's own direction: the gradient cancels to eps-sized terms, so compare against the terms
    assert np.all(np.abs(from_dev(dx[-3:]) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-5)


def test_tensors_of_another_device_or_type_are_refused():
    F, T_ = _F(), torch()
    x = T_.zeros((4, 64), dtype=T_.bfloat16, device="cuda")
    g = T_.zeros(64, dtype=T_.bfloat16, device="cuda")
    for kw in (dict(y=x.float()), dict(y=x.cpu()), dict(y=x[:2]), dict(y=x.t().contiguous().t()), dict(rstd=T_.zeros(4, device="cuda").double())):
        with pytest.raises(ValueError, match="contiguous"):
            F.rms_norm_fwd(x, g, EPS, **kw)
    with pytest.raises(F.FqError, match="invalid argument"):
        F.rms_norm_fwd(x, g, EPS)
    d = F.head_desc(4, 64, 10)
    with pytest.raises(F.FqError, match="buffer too small"):
        F.head_loss(d, x, T_.zeros((10, 64), dtype=T_.bfloat16, device="cuda"), T_.zeros(1, device="cuda"),
                    labels=T_.zeros(4, dtype=T_.int32, device="cuda"), workspace=T_.zeros(64, dtype=T_.uint8, device="cuda"))


def test_gradient_over_the_hidden_states():
    F, T_ = _F(), torch()
    h = T_.randn((70, 128), device="cuda").to(T_.bfloat16)
    w = T_.randn((600, 128), device="cuda").to(T_.bfloat16)
    lab = T_.randint(0, 600, (70,), device="cuda", dtype=T_.int32)
    d = F.head_desc(70, 128, 600)
    ws = T_.empty(F.head_loss_workspace_size(d), dtype=T_.uint8, device="cuda")
    loss, grad = T_.empty(1, device="cuda"), T_.empty_like(h)
    F.head_loss(d, h, w, loss, labels=lab, grad=grad, workspace=ws)
    first = loss.clone()
    F.head_loss(d, h, w, loss, labels=lab, grad=h, workspace=ws)
    T_.cuda.synchronize()
    assert T_.equal(h, grad) and T_.equal(loss, first)


def test_packed_weights_under_another_format_are_refused():
    # the same codes, scales for groups of 64, then asked for with groups of 32 (twice as many scales)
    F, T_ = _F(), torch()
    E, H, I = 4, 256, 128
    none = F.qdesc()
    gr = [F.qdesc(F.FQ_INT, F.FQ_PER_GROUP, g, F.FQ_LEARNABLE, -8, 7) for g in (64, 32)]
    new = lambda dt, *s: T_.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    P = F.packed_experts(dict(codes=new(T_.uint8, E, 2 * I, H // 2), scale=new(T_.float32, E, 2 * I, H // 64)),
                         dict(codes=new(T_.uint8, E, H, I // 2), scale=new(T_.float32, E, H, I // 64)))
    x, ids, tw = new(T_.bfloat16, 2, H), new(T_.int32, 2, 1), new(T_.float32, 2, 1)
    y = T_.ones((2, H), dtype=T_.bfloat16, device="cuda")
    L = [F.layer_desc(E, H, I, 2, 1, q, q, none, none) for q in gr]
    ws = new(T_.uint8, F.packed_expert_workspace_size(L[0]))
    F.packed_expert_fwd(L[0], P, x, ids, tw, y, ws)
    T_.cuda.synchronize()
    assert not from_dev(y).any()
    with pytest.raises(ValueError, match="scale"):
        F.packed_expert_fwd(L[1], P, x, ids, tw, y, ws)
