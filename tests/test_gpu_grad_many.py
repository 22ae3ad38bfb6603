"""As many gradients as fq_grad_norm and fq_grad_clip take in a call."""
import numpy as np
import pytest

from tests.fq_testutil import torch

pytestmark = pytest.mark.gpu


def test_65536_tensors():
    from scale_only_quantization_amd import fqlib as F
    T_ = torch()
    n = 65536
    size = np.arange(n) % 4                               # empty ones among them
    at = np.concatenate([[0], np.cumsum(size)])
    g = T_.Generator(device="cuda")
    g.manual_seed(2)
    x = T_.randn(int(at[-1]), generator=g, device="cuda")
    keep = x.clone()
    G = F.grad_list(x[int(a):int(b)] for a, b in zip(at[:-1], at[1:]))
    norm = T_.zeros(1, device="cuda")
    ws = T_.full((F.grad_norm_workspace_size(G),), 255, dtype=T_.uint8, device="cuda")
    F.grad_norm(G, norm, ws)
    F.grad_clip(G, 1.0, norm)
    T_.cuda.synchronize()
    ref = float((keep.double() ** 2).sum().sqrt())
    assert abs(norm.item() - ref) <= ref * 2.0 ** -23     # fp64 sums and one rounding to fp32
    c = np.float32(1.0 / (norm.double().item() + 1e-6))
    assert T_.equal(x, keep * float(c))
