"""Attention over the 4-bit cache at the ends of the range of `scale`."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import require_gpu
from test_kv4_gpu import close, cu, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qv():
    require_gpu()
    from quantized_verification_gb300 import qv as _qv
    _qv.load()
    return _qv


@pytest.mark.parametrize("NB", [9, 400])
@pytest.mark.parametrize("D,T,Hq", [(128, 1, 2), (128, 5, 4), (128, 8, 4), (64, 5, 4)])
@pytest.mark.parametrize("scale,e", [(2.0e38, -120), (9e37, -120), (1e-30, 90), (1e-38, 112), (1e-30, 107)])
def test_largest_and_smallest_scales(qv, scale, e, NB, D, T, Hq):
    """Queries of +-2^e and keys of whole numbers times 2^-6, so that scores come to about +-100, or to
    nearly nothing: every product and every sum of them is exact, which leaves the
    scaled score's two roundings and the rest of test_kv4_gpu.py's bound."""
    n, g = 32 * NB - 5, gen(21)
    codes = torch.randint(-7, 8, (NB, 1, 64 * D), generator=g).numpy()
    codes[:, :, : 32 * D][codes[:, :, : 32 * D] == 0] = 1
    scales = np.full((NB, 1, 2 * D), 15 * 8, np.uint8)
    scales[:, :, :D] = 9 * 8                                   # 2^-6
    cache = np.concatenate([ref.pack(codes), scales], axis=2)
    qkv = torch.randn(T, (Hq + 2) * D, generator=g)
    qkv[:, : Hq * D] = torch.sign(qkv[:, : Hq * D]) * 2.0 ** e
    qkv[:, Hq * D: (Hq + 1) * D] = (torch.randint(1, 8, (T, D), generator=g) * torch.sign(qkv[:, Hq * D: (Hq + 1) * D])) / 64
    qkv = qkv.to(torch.bfloat16)
    ln = np.array([n], np.int32)
    scale = float(np.float32(scale))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(1, T, Hq, 1, D, NB), dtype=torch.uint8, device="cuda")
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, 1, D, NB, scale)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((T, Hq * D), float("nan"), dtype=dt, device="cuda")
        qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, 1, scale, out, ws)
        assert bool(out.isfinite().all())
        close(out, want, vmax, smax, D)
