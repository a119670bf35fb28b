"""Waits that run out in attention over the 4-bit cache: the call returns and says so, whatever its warps were doing, and
the next call on the same workspace is right. Tolerances are those of test_kv4_gpu.py."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import require_gpu
from test_kv4_gpu import attend_inputs, close, cu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qv():
    require_gpu()
    from quantized_verification_gb300 import qv as _qv
    _qv.load()
    return _qv


@pytest.mark.parametrize("B,T,Hq,Hkv,D,lens,out_dtype", [
    (1, 3, 8, 2, 128, [12800], torch.float32),                 # 12 rows a tile
    (12, 5, 8, 2, 128, None, torch.float32),                   # 20 rows, many tiles a thread block
    (12, 5, 8, 2, 128, None, torch.bfloat16),
    (3, 8, 8, 2, 128, [9000, 40, 12800], torch.float32),       # 32 rows
    (3, 8, 8, 2, 128, [9000, 40, 12800], torch.bfloat16),
    (2, 64, 2, 1, 128, [12800, 0], torch.float32),             # more own rows than a unit
    (4, 1, 8, 2, 128, None, torch.float32),                    # the mma.sync kernel's line
    (4, 6, 8, 2, 64, None, torch.bfloat16),
])
def test_calls_whose_records_never_come(qv, B, T, Hq, Hkv, D, lens, out_dtype):
    """Scores that grow along the cache, so that maxima move in most steps, and 20 calls without a single record."""
    NB = 400
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, lens, True)
    cache[:, :, 32 * D: 33 * D] = (8 * 9 + np.arange(len(cache)) // 64 % 40)[:, None, None]
    scale = float(np.float32(D ** -0.5))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    out = torch.empty(B * T, Hq * D, dtype=out_dtype, device="cuda")
    args, block_table = (qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out, ws), cu(table)
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, table)
    assert qv.qv_device_error() == 0
    qv.qv_attention_verify_kv4(*args, block_table=block_table)
    close(out, want, vmax, smax, D)
    good = out.clone()
    for _ in range(20):
        try:
            qv.qv_debug_set_slot_wait_ns(500_000)
            qv.qv_debug_hold_attention_loads(1)
            qv.qv_attention_verify_kv4(*args, block_table=block_table)
            assert qv.qv_device_error() == qv.QV_DEVICE_ERR_FULL_WAIT
        finally:
            qv.qv_debug_set_slot_wait_ns(0)
            qv.qv_debug_hold_attention_loads(0)
        assert int(ws[:4096].max()) == 0
        qv.qv_attention_verify_kv4(*args, block_table=block_table)
        assert torch.equal(out, good) and qv.qv_device_error() == 0
