"""Attention over the 4-bit cache for steps of more than 32 tokens, whose own rows are the work of several warps: each
way to share the work, contexts so short that most warps have nothing else to do, against 64 bits and bit for bit over
many calls. Tolerances are those of test_kv4_gpu.py."""
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


def run(qv, B, T, Hq, Hkv, D, NB, lens, out_dtype, calls):
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, lens, True)
    scale = float(np.float32(D ** -0.5))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    args = (qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale)
    block_table = cu(table)
    outs = torch.full((calls, B * T, Hq * D), float("nan"), dtype=out_dtype, device="cuda")
    for out in outs:
        qv.qv_attention_verify_kv4(*args, out, ws, block_table=block_table)
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, table)
    close(outs[0], want, vmax, smax, D)
    bits = outs.view(torch.int16 if out_dtype == torch.bfloat16 else torch.int32)
    assert bool((bits == bits[0]).all())
    assert int(ws[:4096].max()) == 0
    assert qv.qv_device_error() == 0


# Tables of 3 blocks: one or two thread blocks a tile. Of 40: larger clusters, ranks with own rows only among them.
# Of 400: the line of units (D = 64), the tcgen05 kernel (D = 128).
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("NB", [3, 40, 400])
@pytest.mark.parametrize("T,Hq", [(33, 1), (64, 1), (100, 3), (128, 1), (256, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_own_rows_of_many_warps(qv, D, T, Hq, NB, out_dtype):
    run(qv, 3, T, Hq, 1, D, NB, [0, 10, 90], out_dtype, calls=40)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,NB", [(170, 64, 1, 1, 64, 2), (90, 128, 2, 2, 64, 3), (60, 256, 1, 1, 64, 3),
                                             (160, 64, 1, 1, 128, 2), (100, 100, 1, 1, 64, 45)])
def test_own_rows_of_many_tiles(qv, B, T, Hq, Hkv, D, NB, out_dtype):
    """More tiles than the GPU holds thread blocks: one each (D = 64, short tables), or the line."""
    run(qv, B, T, Hq, Hkv, D, NB, None, out_dtype, calls=10)
