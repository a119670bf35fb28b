"""Prompts among very many empty sequences, as a batch with a fixed number of slots has them."""
import pytest
import torch

from gpu_util import require_gpu
from quantized_verification_gb300 import qv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    require_gpu()


def run(x, lens, Hq, Hkv, dtype):
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32).cuda()
    out = torch.full((x.shape[0], Hq * x.shape[1] // (Hq + 2 * Hkv)), 7.0, dtype=dtype, device="cuda")
    qv.qv_attention_prompt(x, cu, Hq, Hkv, 0.1, out)
    assert qv.qv_device_error() == 0
    return out


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (32, 8), (3, 1)])
@pytest.mark.parametrize("slots", [900, 1100, 5000, 70000, 1 << 22])
def test_empty_slots_change_nothing(slots, Hq, Hkv):
    D = 64
    g = torch.Generator().manual_seed(slots)
    lens = torch.randint(1, 60, (40,), generator=g)
    M = int(lens.sum())
    x = torch.randn(M, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16).cuda()
    want = run(x, lens, Hq, Hkv, torch.float32)
    many = torch.zeros(slots, dtype=torch.int64)
    many[torch.randperm(slots, generator=g)[:40].sort().values] = lens
    assert torch.equal(run(x, many, Hq, Hkv, torch.float32), want)
    # all of the empty ones between two
    one = torch.zeros(slots, dtype=torch.int64)
    one[0], one[-1] = M // 2, M - M // 2
    assert torch.equal(run(x, one, Hq, Hkv, torch.float32),
                       run(x, torch.tensor([M // 2, M - M // 2]), Hq, Hkv, torch.float32))
