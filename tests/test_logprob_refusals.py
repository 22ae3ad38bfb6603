"""Refusals of the log probabilities and of the gradients' norm and clipping: every invalid call is answered with its
status before any HIP call (no GPU needed: no pointer passed here is ever dereferenced), and the Python wrappers
refuse tensors that the C side cannot see to be wrong."""
import ctypes

import pytest

F = pytest.importorskip("scale_only_quantization_amd.fqlib")
torch = pytest.importorskip("torch")

FAKE = 0x100000
MIS = 0x100002
BIG = 1 << 50


def _lf(T=4, V=100, m=1, k=5, H=0, z=FAKE, ld=104, ids=FAKE, logp=FAKE, lse=FAKE, ent=FAKE, ti=FAKE, tv=FAKE, ws=FAKE,
        wsb=BIG):
    d = F.logprob_desc(T, V, m, k, H)
    return F.lib().fq_logprob_fwd(ctypes.byref(d), z, ld, ids, logp, lse, ent, ti, tv, ws, wsb, None)


def _hf(T=4, V=100, m=1, k=5, H=128, h=FAKE, w=FAKE, ids=FAKE, logp=FAKE, lse=FAKE, ent=FAKE, ti=FAKE, tv=FAKE, ws=FAKE,
        wsb=BIG):
    d = F.logprob_desc(T, V, m, k, H)
    return F.lib().fq_head_logprob_fwd(ctypes.byref(d), h, w, ids, logp, lse, ent, ti, tv, ws, wsb, None)


@pytest.mark.parametrize("f", [_lf, _hf])
def test_forward_refusals(f):
    # the workspace is asked for last, so FQ_E_WORKSPACE says that all else was right
    ok = dict(ws=None)
    assert f(**ok) == F.FQ_E_WORKSPACE
    assert f(wsb=255) == F.FQ_E_WORKSPACE
    for kw in (dict(T=-1), dict(T=1 << 24), dict(V=0, k=0), dict(V=1 << 31), dict(H=64 if f is _lf else 0)):
        assert f(**kw, **ok) == F.FQ_E_SHAPE, kw
    for kw in (dict(m=-1), dict(m=65), dict(k=-1), dict(k=65), dict(V=4, k=5)):
        assert f(**kw, **ok) == F.FQ_E_INVALID, kw
    for kw in (dict(ids=None), dict(logp=None), dict(ti=None), dict(tv=None), dict(m=0), dict(k=0), dict(m=0, ids=None),
               dict(k=0, tv=None)):
        assert f(**kw, **ok) == F.FQ_E_INVALID, kw
    assert f(m=0, k=0, ids=None, logp=None, ti=None, tv=None, lse=None, ent=None, **ok) == F.FQ_E_INVALID
    for kw in (dict(m=0, ids=None, logp=None), dict(k=0, ti=None, tv=None), dict(lse=None, ent=None)):
        assert f(**kw, **ok) == F.FQ_E_WORKSPACE, kw
    for n in ("ids", "logp", "lse", "ent", "ti", "tv"):
        assert f(**{n: MIS}, **ok) == F.FQ_E_ALIGN, n
    assert f(ws=FAKE + 64) == F.FQ_E_ALIGN
    assert f(T=0, ids=None, logp=None, lse=None, ent=None, ti=None, tv=None, ws=None, wsb=0) == F.FQ_OK


def test_forward_refusals_of_rows_and_weights():
    for kw in (dict(ld=96), dict(ld=101), dict(ld=0)):
        assert _lf(ws=None, **kw) == F.FQ_E_SHAPE, kw
    assert _lf(z=None) == F.FQ_E_INVALID
    assert _lf(z=FAKE + 8) == F.FQ_E_ALIGN
    for n in ("h", "w"):
        assert _hf(**{n: None}) == F.FQ_E_INVALID
        assert _hf(**{n: FAKE + 8}) == F.FQ_E_ALIGN
    assert _hf(H=96) == F.FQ_E_SHAPE
    assert _hf(H=16448) == F.FQ_E_UNSUPPORTED
    assert F.lib().fq_logprob_fwd(None, FAKE, 104, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None) == F.FQ_E_INVALID


def _lb(T=4, V=100, m=1, H=0, z=FAKE, ld=104, ids=FAKE, lse=FAKE, ent=FAKE, dl=FAKE, de=FAKE, g=FAKE, gld=104):
    d = F.logprob_desc(T, V, m, 0, H)
    return F.lib().fq_logprob_bwd(ctypes.byref(d), z, ld, ids, lse, ent, dl, de, g, gld, None)


def _hb(T=4, V=100, m=1, H=128, h=FAKE, w=FAKE, ids=FAKE, lse=FAKE, ent=FAKE, dl=FAKE, de=FAKE, g=FAKE, ws=None, wsb=0):
    d = F.logprob_desc(T, V, m, 0, H)
    return F.lib().fq_head_logprob_bwd(ctypes.byref(d), h, w, ids, lse, ent, dl, de, g, ws, wsb, None)


@pytest.mark.parametrize("f", [_lb, _hb])
def test_backward_refusals(f):
    for kw in (dict(T=-1), dict(T=1 << 24), dict(V=0), dict(V=1 << 31), dict(H=64 if f is _lb else 0)):
        assert f(**kw) == F.FQ_E_SHAPE, kw
    for kw in (dict(m=65), dict(m=-1), dict(m=0), dict(ids=None), dict(dl=None), dict(lse=None), dict(g=None),
               dict(ent=None), dict(m=0, ids=None, dl=None, de=None)):
        assert f(**kw) == F.FQ_E_INVALID, kw
    for n in ("ids", "lse", "ent", "dl", "de", "g"):
        assert f(**{n: MIS}) == F.FQ_E_ALIGN, n
    assert f(T=0, ids=None, lse=None, ent=None, dl=None, de=None, g=None) == F.FQ_OK


def test_backward_refusals_of_rows_and_weights():
    for kw in (dict(ld=96), dict(gld=96), dict(gld=108 + 1), dict(g=FAKE, z=FAKE, gld=112)):
        assert _lb(**kw) == (F.FQ_E_INVALID if "z" in kw else F.FQ_E_SHAPE), kw
    assert _lb(z=None) == F.FQ_E_INVALID
    assert _lb(z=FAKE + 8, g=FAKE) == F.FQ_E_ALIGN
    assert _hb() == F.FQ_E_WORKSPACE                             # all else was right
    need = F.head_logprob_workspace_size(F.logprob_desc(4, 100, 1, 0, 128), True)
    assert need > 0 and _hb(ws=FAKE, wsb=need - 1) == F.FQ_E_WORKSPACE
    for n in ("h", "w"):
        assert _hb(**{n: None}) == F.FQ_E_INVALID
        assert _hb(**{n: FAKE + 8}) == F.FQ_E_ALIGN


def test_workspace_sizes():
    assert F.logprob_workspace_size(F.logprob_desc(0, 100, 1, 5)) == 0
    assert F.logprob_workspace_size(F.logprob_desc(4, 100, 1, 5)) > 0
    for d in (F.logprob_desc(4, 100, 65), F.logprob_desc(4, 100, 0, 101), F.logprob_desc(4, 0), F.logprob_desc(4, 100, hidden=64)):
        assert F.logprob_workspace_size(d) == 0
    for d in (F.logprob_desc(4, 100), F.logprob_desc(4, 100, hidden=100), F.logprob_desc(4, 100, 0, 65, hidden=128)):
        assert F.head_logprob_workspace_size(d) == 0 and F.head_logprob_workspace_size(d, True) == 0
    # a piece of about 640 MB, whatever the sizes, and what the header adds to it
    for T, H, V, k in ((1, 2048, 151936, 64), (64, 1024, 151936, 20), (64, 2048, 151936, 20), (2048, 2048, 151936, 64),
                       (16384, 2048, 151936, 64), (16384, 2048, 151936, 0), (100000, 4096, 151936, 64), (1, 64, 1 << 30, 64),
                       (64, 64, (1 << 31) - 1, 64), (300, 64, (1 << 31) - 1, 0), ((1 << 24) - 1, 64, 1000, 64)):
        d = F.logprob_desc(T, V, 1, k, H)
        size = F.head_logprob_workspace_size(d)
        assert size <= max(680 << 20, T * 256 * 5) + T * (20 + 8 * k) + 4096, (T, size)
        assert F.head_logprob_workspace_size(d, True) <= F.head_loss_workspace_size(F.head_desc(T, H, V, 0)) + T * 64 + 4096


def _grads(*t):
    return (F.GradTensor * len(t))(*[F.GradTensor(*x) for x in t])


def _gn(t, n=None, norm=FAKE, ws=FAKE, wsb=BIG):
    return F.lib().fq_grad_norm(t, len(t) if n is None else n, norm, ws, wsb, None)


def _gc(t, n=None, limit=1.0, norm=FAKE):
    return F.lib().fq_grad_clip(t, len(t) if n is None else n, limit, norm, None)


def test_grad_refusals():
    ok = _grads((FAKE, FAKE, 100, F.FQ_F32), (FAKE + 1024, FAKE + 1024, 100, F.FQ_BF16))
    need = F.lib().fq_grad_norm_workspace_size(ok, 2)
    assert need == 2 * 8
    for f in (_gn, _gc):
        assert f(ok, n=-1) == F.FQ_E_SHAPE
        assert f(ok, n=65537) == F.FQ_E_UNSUPPORTED
        assert f(None, n=1) == F.FQ_E_INVALID
        assert f(ok, norm=None) == F.FQ_E_INVALID
        assert f(ok, norm=MIS) == F.FQ_E_ALIGN
        for bad in ((None, FAKE, 1, 0), (FAKE, FAKE, -1, 0), (FAKE, FAKE, 1 << 40, 0), (FAKE, FAKE, 1, 2)):
            assert f(_grads(bad)) == F.FQ_E_INVALID, bad
        for bad in ((MIS, FAKE, 1, F.FQ_F32), (FAKE + 1, FAKE, 1, F.FQ_BF16)):
            assert f(_grads(bad)) == F.FQ_E_ALIGN, bad
    assert _gn(ok, ws=None) == F.FQ_E_WORKSPACE
    assert _gn(ok, wsb=need - 1) == F.FQ_E_WORKSPACE
    assert _gn(ok, ws=FAKE + 4) == F.FQ_E_ALIGN
    assert _gc(_grads((FAKE, None, 1, 0))) == F.FQ_E_INVALID
    assert _gc(_grads((FAKE, MIS, 1, F.FQ_F32))) == F.FQ_E_ALIGN
    for limit in (0.0, -1.0, float("inf"), float("nan")):
        assert _gc(ok, limit=limit) == F.FQ_E_INVALID
    assert F.lib().fq_grad_norm_workspace_size(None, 0) == 0
    assert F.lib().fq_grad_norm_workspace_size(_grads((FAKE, FAKE, -1, 0)), 1) == 0
    assert _gc(_grads((None, None, 0, 0))) == F.FQ_OK                # nothing to do
    assert _gc(None, n=0) == F.FQ_OK


def test_wrappers_refuse_tensors():
    z = torch.zeros((4, 64), dtype=torch.bfloat16)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        F.logprob_fwd(F.logprob_desc(4, 64), z, lse=f)
    with pytest.raises(ValueError, match="GPU"):
        F.logprob_bwd(F.logprob_desc(4, 64), z, f, z)
    with pytest.raises(ValueError, match="GPU"):
        F.head_logprob_fwd(F.logprob_desc(4, 64, hidden=64), z, z, lse=f)
    with pytest.raises(ValueError, match="GPU"):
        F.head_logprob_bwd(F.logprob_desc(4, 64, hidden=64), z, z, f, z)
    with pytest.raises(ValueError, match="GPU"):
        F.grad_list([f])
    with pytest.raises(ValueError, match="outputs"):
        F.grad_list([f], [])


def _strided(shape, dtype, stride=None):
    """A tensor on no device, as far as the checks of types, shapes and strides look."""
    class Fake:
        def __init__(self):
            self.t = torch.empty_strided(shape, stride, dtype=dtype) if stride else torch.empty(shape, dtype=dtype)

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return 0
    return Fake()


def test_rows_of_logits():
    bf = torch.bfloat16
    for t, ld in ((_strided((4, 64), bf), 64), (_strided((4, 64), bf, (72, 1)), 72), (_strided((1, 61), bf, (64, 1)), 64)):
        if t.shape[1] % 8 == 0:
            assert F._rows("x", "logits", t, t.shape, 0)[1] == ld
    for t in (_strided((4, 64), torch.float32), _strided((4, 64), bf, (1, 4)), _strided((4, 64), bf, (0, 1)),
              _strided((4, 64, 1), bf), _strided((4, 60), bf)):
        with pytest.raises(ValueError, match="logits"):
            F._rows("x", "logits", t, (4, 64), 0)
    with pytest.raises(ValueError, match="last row"):
        F._rows("x", "logits", _strided((3, 61), bf, (64, 1)), (3, 61), 0)
    full = _strided((3, 64), bf)
    full.t = full.t[:, :61]
    assert F._rows("x", "logits", full, (3, 61), 0)[1] == 64


def test_grad_list_refuses_overlaps():
    f, bf = torch.float32, torch.bfloat16

    class Fake:
        """A contiguous view of a buffer, said to be on GPU 0."""
        is_cuda = True

        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return 0

    buf, other = torch.zeros(100), torch.zeros(100)
    v = lambda lo, hi, b=buf: Fake(b[lo:hi])  # noqa: E731
    F.grad_list([v(0, 10), v(10, 20), v(20, 20), v(25, 100)])
    F.grad_list([v(0, 10), v(5, 15)], [v(0, 10, other), v(10, 20, other)])          # gradients that share memory
    F.grad_list([v(0, 10), v(10, 20)], [v(0, 10, other), v(10, 20)])                # one of them in place
    for g, o in (([v(0, 10), v(0, 10)], None), ([v(0, 10), v(9, 20)], None), ([v(0, 10)], [v(5, 15)]),
                 ([v(0, 10), v(20, 30)], [v(50, 60), v(0, 10)]), ([v(0, 10), v(20, 30)], [v(50, 60), v(55, 65)]),
                 ([v(0, 50), v(60, 70)], [v(0, 50), v(10, 20)])):
        with pytest.raises(ValueError, match="overlaps"):
            F.grad_list(g, o)
    with pytest.raises(ValueError, match="gradients must be"):
        F.grad_list([Fake(torch.zeros(4, dtype=torch.float64))])
    with pytest.raises(ValueError, match="output"):
        F.grad_list([v(0, 10)], [Fake(torch.zeros(10, dtype=bf))])
    with pytest.raises(ValueError, match="output"):
        F.grad_list([v(0, 10)], [v(0, 9, other)])
    with pytest.raises(ValueError, match="contiguous"):
        F.grad_list([Fake(torch.zeros((4, 4), dtype=f).t()[1:])])
