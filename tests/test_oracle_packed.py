"""The packed weights' oracle: code values from their closed forms, unpacking
against the codec's own codes, the layer against the layer oracle's W^."""
import numpy as np
import pytest
import torch

from oracle import packed as OPK
from oracle import presets as OP
from oracle.codec import QSpec, fake_quant
from oracle.numerics import bf16_rne


def test_e4m3_bytes():
    b = np.arange(256)
    b = b[(b & 127) != 127]
    ref = torch.tensor(b, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(OPK.e4m3_value(b), ref)


@pytest.mark.parametrize("q", [OP.NVFP4_W, OP.INT4_G128, QSpec("int", "row", 0, "learnable", -8, 7),
                               QSpec("int", "group", 32, "learnable", -8, 7)],
                         ids=["nvfp4", "g128", "row", "g32"])
def test_dequant_is_the_codec_before_its_rounding(q):
    rng = np.random.default_rng(1)
    W = bf16_rne((rng.standard_normal((2, 3, 256)) * 0.02).astype(np.float32))
    if q.kind == "nvfp4":
        t = np.array([0.02, 0.03], np.float32) / 400
        s = (np.abs(W).reshape(2, 3, 16, 16).max(-1) / 6).astype(np.float32)
        r = fake_quant(q, W, scale=s, tscale=t)
        got = OPK.dequant(r["codes"], block_codes=r["block_codes"], tensor_scale=t)
    else:
        g = 256 if q.gran == "row" else q.group
        s = (np.abs(W).reshape(2, 3, -1, g).max(-1) / 7).astype(np.float32)
        s = s[..., 0] if q.gran == "row" else s
        r = fake_quant(q, W, scale=s)
        got = OPK.dequant(r["codes"], scale=s)
    y = np.asarray(r["y"], np.float64).reshape(got.shape)
    np.testing.assert_array_less(np.abs(got - y), 2.0 ** -8 * np.abs(got) + 1e-12)


def test_experts_by_brute_force():
    rng = np.random.default_rng(2)
    E, H, I, T, k = 3, 8, 4, 2, 2
    W1, W2 = rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    x = bf16_rne(rng.standard_normal((T, H)).astype(np.float32))
    ids, tw = np.array([[2, 0], [1, 2]]), np.array([[0.25, 0.75], [0.5, 0.5]])
    y = OPK.experts(W1, W2, x, ids, tw)
    for t in range(T):
        ref = np.zeros(H)
        for j in range(k):
            h = []
            for i in range(I):
                g = sum(W1[ids[t, j], i, c] * float(x[t, c]) for c in range(H))
                u = sum(W1[ids[t, j], I + i, c] * float(x[t, c]) for c in range(H))
                h.append(float(bf16_rne(np.array([g / (1 + np.exp(-g)) * u], np.float32))[0]))
            ref += tw[t, j] * np.array([sum(W2[ids[t, j], n, i] * h[i] for i in range(I)) for n in range(H)])
        np.testing.assert_allclose(y[t], ref, rtol=1e-12)


@pytest.mark.parametrize("g", [32, 64, 128, 512, 0], ids=lambda g: f"g{g}" if g else "row")
@pytest.mark.parametrize("N,K,M", [(65, 8192, 13), (257, 2048, 3), (48, 512, 64)])
def test_the_int4_bound_sees_a_lost_segment_and_a_wrong_scale(N, K, M, g):
    # the bound that the GPU's INT4 products are held to, against results with
    # a mistake: 32 columns left out, and one group under its neighbour's scale
    from tests.fq_testutil import int4_bound
    rng = np.random.default_rng(N)
    codes = rng.integers(0, 256, (1, N, K // 2)).astype(np.uint8)
    s = (rng.random((1, N, K // g) if g else (1, N)) * 0.01 + 1e-3).astype(np.float32)
    x = bf16_rne((rng.standard_normal((M, K)) + 0.3).astype(np.float32)).astype(np.float64)
    W = OPK.dequant(codes, scale=s)[0]
    ref = x @ W.T
    tol = int4_bound(x, W, s[0], ref)
    assert np.all(np.abs(bf16_rne(ref.astype(np.float32)) - ref) <= tol)     # the right result, rounded
    lost = W.copy()
    lost[:, K - 32:] = 0
    # half of all results and more must be seen to be wrong: 32 columns are of the order of 5 s sqrt(32) = 28 s
    assert np.mean(np.abs(x @ lost.T - ref) > tol) > 0.5
    if g:
        swap = s.copy()
        swap[:, :, -1] = s[:, :, -2] if s.shape[2] > 1 else 0
        # neighbours differ by 0.004 of 0.006 (rms), at times by nearly nothing: with groups of 32 of 8192 columns
        # the change is 0.004 * 4.6 * sqrt(32) = 0.1 (rms) against bounds of 0.02 to 0.06, so a quarter must be seen
        assert np.mean(np.abs(x @ OPK.dequant(codes, scale=swap)[0].T - ref) > tol) > 0.25
