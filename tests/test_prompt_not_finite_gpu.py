"""Keys and values that are not finite, in the rows that see them: the softmax's definition holds for the scores."""
import pytest
import torch

from gpu_util import require_gpu
from quantized_verification_gb300 import qv

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    require_gpu()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [2, 150])                          # few rows and many: two merges
@pytest.mark.parametrize("where", ["prefix", "cache", "own"])
def test_a_value_that_is_not_finite_under_scores_of_minus_infinity(where, B, dtype):
    # weight 0 times infinity is NaN, wherever the key lies and whatever else its part of the positions holds
    T, Hq, Hkv, D, P = 1, 16, 4, 64, 300
    g = torch.Generator(device="cuda").manual_seed(B)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = r(B, Hq + 2 * Hkv, D)
    x[:, :Hq] = x[:, :Hq].abs() + 0.25                           # positive queries
    x, pk, pv, kc, vc = (t.to(torch.bfloat16) for t in (x.view(B, -1), r(P, Hkv, D), r(P, Hkv, D), r(B, 4, Hkv, D), r(B, 4, Hkv, D)))
    own = x.view(B, Hq + 2 * Hkv, D)
    if where == "prefix":
        pk[:], pv[:, :, 5] = -float("inf"), float("inf")
    elif where == "cache":
        kc[:], vc[:, :, :, 5] = -float("inf"), float("inf")
    else:
        own[:, Hq:Hq + Hkv], own[:, Hq + Hkv:, 5] = -float("inf"), float("inf")
    out = torch.zeros(B, Hq * D, dtype=dtype, device="cuda")
    ws = torch.empty(qv.qv_attention_prefix_workspace_bytes(B, T, Hq, Hkv, D, P), dtype=torch.uint8, device="cuda")
    qv.qv_attention_verify_prefix(x, pk, pv, i32([P]), kc, vc, i32([4] * B), T, Hq, Hkv, 0.1, out, ws)
    out = out.view(B, Hq, D)
    assert torch.isnan(out[:, :, 5]).all()
    assert torch.isfinite(out[:, :, :5]).all() and torch.isfinite(out[:, :, 6:]).all()
    # without cached positions nothing of the caches is left to see
    if where == "cache":
        qv.qv_attention_verify_prefix(x, pk, pv, i32([P]), kc, vc, i32([0] * B), T, Hq, Hkv, 0.1, out.view(B, -1), ws)
        assert torch.isfinite(out).all()
    if where == "prefix":
        qv.qv_attention_verify_prefix(x, pk, pv, i32([0]), kc, vc, i32([4] * B), T, Hq, Hkv, 0.1, out.view(B, -1), ws)
        assert torch.isfinite(out).all()
