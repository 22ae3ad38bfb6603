"""Products of packed 4-bit weights and the expert layer on them, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring): nothing in the product
path may import or call this module.

Codes are two per byte, the even column in the low nibble: INT4 in two's
complement, NVFP4 a sign bit and an E2M1 magnitude; NVFP4 block codes are E4M3
bytes.  W = q s or q d t, not rounded to bf16.
"""
from __future__ import annotations

import numpy as np

from .codec import QSpec, fake_quant
from .numerics import bf16_rne

F64 = np.float64
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], F64)


def e4m3_value(b):
    b = np.asarray(b, np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(b & 128, -v, v)


def dequant(codes, scale=None, block_codes=None, tensor_scale=None):
    """W [E, N, K] float64 of codes [E, N, K/2]."""
    c = np.asarray(codes, np.int64)
    q = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1)
    E, N, K = q.shape
    if block_codes is None:
        v = np.where(q > 7, q - 16, q).astype(F64)
        s = np.asarray(scale, F64).reshape(E, N, -1)
    else:
        v = np.where(q & 8, -1.0, 1.0) * E2M1[q & 7]
        s = e4m3_value(block_codes) * np.asarray(tensor_scale, F64)[:, None, None]
    return (v.reshape(E, N, s.shape[-1], -1) * s[..., None]).reshape(E, N, K)


def act_quant(x, q: QSpec | None, s):
    """One bf16 row through an activation quantiser with scale s (None: as it is)."""
    if q is None or not q.enabled:
        return np.asarray(x, F64)
    s = np.array([s], np.float32)
    t = fake_quant(q, x[None, None, :], tscale=s) if q.kind == "nvfp4" else fake_quant(q, x[None, None, :], scale=s)
    return np.asarray(t["y"], F64).reshape(-1)


def experts(W1, W2, x, ids, tw, a1=None, s_a1=None, a2=None, s_a2=None):
    """y [T, H] float64 of the routed SwiGLU layer on dequantised W1 [E, 2I, H] and W2 [E, H, I]."""
    T, k = ids.shape
    I = W2.shape[2]
    y = np.zeros((T, W2.shape[1]))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            z = W1[e] @ act_quant(x[t], a1, None if s_a1 is None else s_a1[e])
            h = bf16_rne((z[:I] / (1.0 + np.exp(-z[:I])) * z[I:]).astype(np.float32))
            y[t] += F64(tw[t, j]) * (W2[e] @ act_quant(h, a2, None if s_a2 is None else s_a2[e]))
    return y
