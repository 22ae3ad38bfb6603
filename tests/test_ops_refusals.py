"""Refusals of the operators around the expert layer: every invalid call is
answered with its status before any HIP call (no GPU needed: no pointer passed
here is ever dereferenced), and the Python wrappers refuse tensors that the C
side cannot see to be wrong."""
import ctypes

import pytest

F = pytest.importorskip("scale_only_quantization_amd.fqlib")
torch = pytest.importorskip("torch")

FAKE = 0x100000
MIS = 0x100002
FP8_ROW = F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_ROW, 0, F.FQ_DYNAMIC)


def _nf(q=None, R=4, C=64, eps=1e-6, x=FAKE, res=None, g=FAKE, sum=None, y=FAKE, rstd=None, codes=None, scale=None):
    return F.lib().fq_rms_norm_fwd(None if q is None else ctypes.byref(q), R, C, eps, x, res, g, sum, y, rstd, codes,
                                   scale, None)


def test_rms_norm_fwd_refusals():
    assert _nf(R=-1) == F.FQ_E_SHAPE
    assert _nf(R=1 << 31) == F.FQ_E_SHAPE
    assert _nf(C=60) == F.FQ_E_SHAPE
    assert _nf(C=0) == F.FQ_E_SHAPE
    assert _nf(C=65544) == F.FQ_E_UNSUPPORTED
    for e in (-1.0, float("nan"), float("inf")):
        assert _nf(eps=e) == F.FQ_E_INVALID
    assert _nf(x=None) == F.FQ_E_INVALID
    assert _nf(g=None) == F.FQ_E_INVALID
    assert _nf(y=None) == F.FQ_E_INVALID                         # nothing to write
    assert _nf(res=FAKE) == F.FQ_E_INVALID                       # residual without sum
    assert _nf(sum=FAKE) == F.FQ_E_INVALID
    assert _nf(codes=FAKE) == F.FQ_E_INVALID                     # codes without a quantiser
    assert _nf(scale=FAKE) == F.FQ_E_INVALID
    assert _nf(q=FP8_ROW) == F.FQ_E_INVALID                      # quantiser without codes
    assert _nf(q=FP8_ROW, codes=FAKE) == F.FQ_E_INVALID
    for q in (F.qdesc(F.FQ_NVFP4, F.FQ_PER_GROUP, 16, F.FQ_DYNAMIC),
              F.qdesc(F.FQ_INT, F.FQ_PER_ROW, 0, F.FQ_DYNAMIC, -8, 7),
              F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_ROW, 0, F.FQ_STATIC),
              F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_TENSOR, 0, F.FQ_DYNAMIC)):
        assert _nf(q=q, codes=FAKE, scale=FAKE) == F.FQ_E_UNSUPPORTED, q
    assert _nf(q=F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_GROUP, 128, F.FQ_DYNAMIC), codes=FAKE, scale=FAKE) == F.FQ_E_SHAPE
    assert _nf(q=F.qdesc(kind=9), codes=FAKE, scale=FAKE) == F.FQ_E_INVALID
    for kw in (dict(x=MIS), dict(g=MIS), dict(y=MIS), dict(res=MIS, sum=FAKE), dict(res=FAKE, sum=MIS),
               dict(rstd=MIS), dict(q=FP8_ROW, codes=FAKE + 4, scale=FAKE), dict(q=FP8_ROW, codes=FAKE, scale=MIS)):
        assert _nf(**kw) == F.FQ_E_ALIGN, kw
    assert _nf(R=0, x=None, g=None, y=None) == F.FQ_OK


def _nb(R=4, C=64, s=FAKE, g=FAKE, r=FAKE, dy=FAKE, ds=None, dx=FAKE, dg=None, ws=None, wsb=0):
    return F.lib().fq_rms_norm_bwd(R, C, s, g, r, dy, ds, dx, dg, ws, wsb, None)


def test_rms_norm_bwd_refusals():
    assert _nb(R=-1) == F.FQ_E_SHAPE
    assert _nb(C=12) == F.FQ_E_SHAPE
    assert _nb(C=1 << 20) == F.FQ_E_UNSUPPORTED
    for n in ("s", "g", "r", "dy", "dx"):
        assert _nb(**{n: None}) == F.FQ_E_INVALID, n
        assert _nb(**{n: MIS}) == F.FQ_E_ALIGN, n
    assert _nb(ds=MIS) == F.FQ_E_ALIGN
    need = F.rms_norm_bwd_workspace_size(4, 64)
    assert need == 4 * 64 * 4
    assert F.rms_norm_bwd_workspace_size(4, 60) == 0
    assert _nb(dg=FAKE, wsb=need) == F.FQ_E_WORKSPACE
    assert _nb(dg=FAKE, ws=FAKE, wsb=need - 1) == F.FQ_E_WORKSPACE
    assert _nb(dg=FAKE, ws=FAKE + 8, wsb=need) == F.FQ_E_ALIGN
    assert _nb(R=0, s=None, g=None, r=None, dy=None, dx=None) == F.FQ_OK


def test_wrappers_refuse_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    g = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        F.rms_norm_fwd(x, g, 1e-6, y=x)
    with pytest.raises(ValueError, match="GPU"):
        F.rms_norm_bwd(x, g, torch.zeros(4), x, x)


def test_expect_checks_type_shape_layout_and_device():
    # the wrappers' one check, on CPU tensors
    dev = -1
    t = torch.zeros((4, 6), dtype=torch.bfloat16)
    assert F._expect("f", "t", t, torch.bfloat16, (4, 6), dev) == t.data_ptr()
    assert F._expect("f", "t", None, torch.bfloat16, (4, 6), dev) is None
    for bad, dt, shape, d in ((t, torch.float32, (4, 6), dev), (t, torch.bfloat16, (6, 4), dev),
                              (t.t(), torch.bfloat16, (6, 4), dev), (t[:, :3], torch.bfloat16, (4, 3), dev),
                              (t, torch.bfloat16, (4, 6), 0)):
        with pytest.raises(ValueError, match="contiguous"):
            F._expect("f", "t", bad, dt, shape, d)


def _hl(T=4, H=64, V=100, k=0, lm=1.0, dist=1.0, h=FAKE, w=FAKE, tv=None, ti=None, lab=FAKE, loss=FAKE, rows=None,
        grad=None, ws=FAKE, wsb=1 << 40, d=True):
    desc = F.head_desc(T, H, V, k, lm, dist)
    return F.lib().fq_head_loss(ctypes.byref(desc) if d else None, h, w, tv, ti, lab, loss, rows, grad, ws, wsb, None)


def test_head_loss_refusals():
    assert _hl(d=False) == F.FQ_E_INVALID
    for kw in (dict(T=-1), dict(T=1 << 24), dict(H=0), dict(H=96), dict(H=32), dict(V=0), dict(V=1 << 31)):
        assert _hl(**kw) == F.FQ_E_SHAPE, kw
        assert F.head_loss_workspace_size(F.head_desc(kw.get("T", 4), kw.get("H", 64), kw.get("V", 100))) == 0
    assert _hl(H=16448) == F.FQ_E_UNSUPPORTED
    for kw in (dict(k=-1), dict(k=65), dict(k=9, V=8), dict(lm=float("nan")), dict(dist=float("inf")), dict(h=None),
               dict(w=None), dict(loss=None), dict(lab=None), dict(k=4), dict(k=4, tv=FAKE), dict(k=4, ti=FAKE),
               dict(tv=FAKE), dict(ti=FAKE)):
        assert _hl(**kw) == F.FQ_E_INVALID, kw
    for kw in (dict(h=MIS), dict(w=MIS), dict(lab=MIS), dict(loss=MIS), dict(rows=MIS), dict(grad=MIS),
               dict(ws=FAKE + 128), dict(k=4, tv=MIS, ti=FAKE), dict(k=4, tv=FAKE, ti=MIS)):
        assert _hl(**kw) == F.FQ_E_ALIGN, kw
    need = F.head_loss_workspace_size(F.head_desc(4, 64, 100))
    alone = F.head_loss_workspace_size(F.head_desc(4, 64, 100), grad=False)
    assert 0 < alone < need
    assert _hl(grad=FAKE, wsb=need - 1) == F.FQ_E_WORKSPACE
    assert _hl(wsb=alone - 1) == F.FQ_E_WORKSPACE
    assert _hl(ws=None) == F.FQ_E_WORKSPACE


def test_head_loss_workspace_stays_small():
    # at the largest batch the workspace holds no [tokens, vocab] tensor: 15360 of 151936 entries at a time
    d = F.head_desc(16384, 2048, 151936, 64)
    assert F.head_loss_workspace_size(d) < 16384 * 151936 * 2 / 6
    # and a long vocabulary over few tokens stays within a buffer's reach
    assert F.head_loss_workspace_size(F.head_desc(1, 16384, 2 ** 31 - 1)) < 1 << 30


I4 = F.qdesc(F.FQ_INT, F.FQ_PER_GROUP, 128, F.FQ_LEARNABLE, -8, 7)
NV = F.qdesc(F.FQ_NVFP4, F.FQ_PER_GROUP, 16, F.FQ_LEARNABLE)


def _mv(q=I4, E=1, N=16, K=256, c=FAKE, b=None, s=FAKE, t=None, M=2, which=None, x=FAKE, y=FAKE):
    return F.lib().fq_packed_matvec(ctypes.byref(q), E, N, K, c, b, s, t, M, which, x, y, None)


def test_packed_matvec_refusals():
    for kw in (dict(E=0), dict(N=0), dict(N=1 << 31), dict(M=-1), dict(K=0), dict(K=48), dict(K=192),
               dict(q=NV, K=40, s=None, b=FAKE, t=FAKE)):
        assert _mv(**kw) == F.FQ_E_SHAPE, kw
    for q in (F.qdesc(F.FQ_INT, F.FQ_PER_ROW, 0, F.FQ_LEARNABLE, -128, 127), F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_ROW),
              F.qdesc(F.FQ_INT, F.FQ_PER_GROUP, 16, F.FQ_LEARNABLE, -8, 7),
              F.qdesc(F.FQ_INT, F.FQ_PER_TENSOR, 0, F.FQ_LEARNABLE, -8, 7),
              F.qdesc(F.FQ_INT, F.FQ_PER_ROW, 0, F.FQ_LEARNABLE, -9, 5), F.qdesc()):
        assert _mv(q=q) == F.FQ_E_UNSUPPORTED, q
    assert _mv(K=1 << 17) == F.FQ_E_UNSUPPORTED
    assert _mv(M=1025) == F.FQ_E_UNSUPPORTED
    assert _mv(q=F.qdesc(kind=7)) == F.FQ_E_INVALID
    for kw in (dict(c=None), dict(s=None), dict(b=FAKE), dict(t=FAKE), dict(x=None), dict(y=None), dict(E=2),
               dict(q=NV, s=None, b=FAKE), dict(q=NV, s=None, t=FAKE), dict(q=NV, b=FAKE, t=FAKE)):
        assert _mv(**kw) == F.FQ_E_INVALID, kw
    for kw in (dict(c=FAKE + 8), dict(s=MIS), dict(x=FAKE + 8), dict(y=FAKE + 1), dict(E=2, which=MIS),
               dict(q=NV, s=None, b=FAKE + 1, t=FAKE), dict(q=NV, s=None, b=FAKE, t=MIS)):
        assert _mv(**kw) == F.FQ_E_ALIGN, kw
    assert _mv(M=0, x=None, y=None) == F.FQ_OK
    assert _mv(K=256, N=256) == F.FQ_E_INVALID                          # y is x


def _pe(fmt="w4a16", E=8, H=256, I=128, T=4, k=2, P=None, x=FAKE, ids=FAKE, w=FAKE, y=FAKE, ws=FAKE, wsb=1 << 30,
        quants=None, **over):
    L = F.layer_desc(E, H, I, T, k, *(quants or F.preset(fmt)))
    if P is None:
        nv = fmt.startswith("nvfp4")
        act = fmt in ("nvfp4", "w4afp8")
        d = dict(w1_codes=FAKE, w2_codes=FAKE, s_a1=FAKE if act else None, s_a2=FAKE if act else None)
        for n in ("1", "2"):
            d.update({f"w{n}_block_codes": FAKE if nv else None, "t_w" + n: FAKE if nv else None,
                      "s_w" + n: None if nv else FAKE})
        d.update(over)
        P = F.PackedExperts(**d)
    return F.lib().fq_packed_expert_fwd(ctypes.byref(L), ctypes.byref(P), x, ids, w, y, ws, wsb, None)


def test_packed_expert_refusals():
    w1, w2, a1, a2 = F.preset("w4a16")
    tok = F.qdesc(F.FQ_INT, F.FQ_PER_ROW, 0, F.FQ_DYNAMIC, -128, 127)
    for kw in (dict(fmt="w8a8"), dict(fmt="fp8"), dict(T=513), dict(quants=(w1, w2, tok, a2)),
               dict(quants=(w1, w2, a1, tok)), dict(H=8320)):
        assert _pe(**kw) == F.FQ_E_UNSUPPORTED, kw
    assert F.packed_expert_workspace_size(F.layer_desc(8, 256, 128, 513, 2, w1, w2, a1, a2)) == 0
    for kw in (dict(H=192), dict(T=-1), dict(k=9), dict(E=0)):
        assert _pe(**kw) == F.FQ_E_SHAPE, kw
    for kw in (dict(w1_codes=None), dict(w2_codes=None), dict(s_w1=None), dict(t_w1=FAKE), dict(w2_block_codes=FAKE),
               dict(s_a1=FAKE), dict(fmt="nvfp4", s_a1=None), dict(fmt="nvfp4", s_a2=None), dict(fmt="nvfp4", t_w2=None),
               dict(x=None), dict(ids=None), dict(w=None), dict(y=None)):
        assert _pe(**kw) == F.FQ_E_INVALID, kw
    for kw in (dict(x=FAKE + 8), dict(ids=MIS), dict(w=MIS), dict(y=FAKE + 8), dict(ws=FAKE + 16),
               dict(w1_codes=FAKE + 4), dict(s_w2=MIS), dict(fmt="nvfp4", s_a1=MIS)):
        assert _pe(**kw) == F.FQ_E_ALIGN, kw
    need = F.packed_expert_workspace_size(F.layer_desc(8, 256, 128, 4, 2, w1, w2, a1, a2))
    assert need >= 8 * (128 * 2 + 256 * 4)
    assert _pe(wsb=need - 1) == F.FQ_E_WORKSPACE
    assert _pe(ws=None) == F.FQ_E_WORKSPACE
    assert _pe(T=0, x=None, ids=None, w=None, y=None, ws=None) == F.FQ_OK
    assert _pe() == F.FQ_E_INVALID                                      # y is x


def test_head_loss_of_no_tokens_needs_no_workspace():
    # with no tokens only `loss` has to be there; the call gets as far as its
    # launch, which has no GPU to go to here (with one, a GPU test makes the call)
    if torch.cuda.is_available():
        pytest.skip("no device memory behind the pointer")
    for kw in (dict(), dict(k=4), dict(lab=None), dict(grad=FAKE)):
        assert _hl(**{**dict(T=0, h=None, w=None, lab=None, ws=None, wsb=0), **kw}) == F.FQ_E_HIP, kw
    assert _hl(T=0, h=None, w=None, lab=None, ws=None, wsb=0, loss=None) == F.FQ_E_INVALID


def test_packed_expert_workspace_of_formats_that_the_layer_refuses():
    # 0 for every descriptor that the call itself refuses
    w1, w2, a1, a2 = F.preset("w4a16")
    row8 = F.qdesc(F.FQ_INT, F.FQ_PER_ROW, 0, F.FQ_LEARNABLE, -128, 127)
    g16 = F.qdesc(F.FQ_INT, F.FQ_PER_GROUP, 16, F.FQ_LEARNABLE, -8, 7)
    wide = F.qdesc(F.FQ_INT, F.FQ_PER_ROW, 0, F.FQ_LEARNABLE, -9, 5)
    for quants in ((row8, w2, a1, a2), (w1, row8, a1, a2), (g16, w2, a1, a2), (w1, wide, a1, a2), (F.qdesc(), w2, a1, a2),
                   (w1, F.qdesc(F.FQ_FP8E4M3, F.FQ_PER_ROW), a1, a2)):
        assert _pe(quants=quants) == F.FQ_E_UNSUPPORTED
        assert F.packed_expert_workspace_size(F.layer_desc(8, 256, 128, 4, 2, *quants)) == 0
    for fmt in ("nvfp4", "nvfp4a16", "w4a16", "w4afp8"):
        assert F.packed_expert_workspace_size(F.layer_desc(8, 256, 128, 4, 2, *F.preset(fmt))) > 0
