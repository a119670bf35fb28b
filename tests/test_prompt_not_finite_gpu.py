"""Keys and values that are not finite, in the rows that see them: the softmax's definition holds for the scores."""
import pytest
import torch

import prompt_ref as ref
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
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 300), (32, 8, 1300)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_key_that_is_not_finite_in_one_element(bad, Hq, Hkv, n, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(torch.bfloat16)
    y = x.view(n, Hq + 2 * Hkv, D)
    at, e = 140, 9
    y[:, :Hq, e] = torch.where(y[:, :Hq, e] == 0, 1.0, y[:, :Hq, e])
    clean = x.clone()
    y[at, Hq:Hq + Hkv, e] = bad
    out = torch.zeros(n, Hq * D, dtype=dtype, device="cuda")
    qv.qv_attention_prompt(x, i32([0, n]), Hq, Hkv, 0.1, out)
    out = out.view(n, Hq, D)
    # NaN and +inf scores make the row NaN; a score of -inf weighs nothing: as if the key were not there
    q = y[:, :Hq, e].double()
    low = (q * bad == -float("inf")) & (torch.arange(n, device="cuda") >= at)[:, None]
    before = (torch.arange(n, device="cuda") < at)[:, None].expand(n, Hq)
    assert torch.isnan(out[~low & ~before]).all()
    o, a = ref.prompt(clean, [0, n], Hq, Hkv, 0.1)
    o1, a1 = without(clean, at, Hq, Hkv, 0.1)
    got = out.double()
    assert ((got - o).abs() <= ref.bound(o, a, dtype))[before].all()
    assert ((got - o1).abs() <= ref.bound(o1, a1, dtype))[low].all()
    assert qv.qv_device_error() == 0


def without(qkv, at, Hq, Hkv, scale):
    """The definition in 64 bits for one sequence in which no row sees position `at`."""
    n = qkv.shape[0]
    x = qkv.double().view(n, Hq + 2 * Hkv, -1)
    see = torch.ones(n, n, dtype=torch.bool, device=qkv.device).tril()
    see[:, at] = False
    o = torch.empty(n, Hq, x.shape[2], dtype=torch.float64, device=qkv.device)
    a = torch.empty_like(o)
    for h in range(Hq):
        k, v = x[:, Hq + h // (Hq // Hkv)], x[:, Hq + Hkv + h // (Hq // Hkv)]
        p = torch.softmax(torch.where(see, (x[:, h] @ k.T) * scale, -float("inf")), -1)
        o[:, h], a[:, h] = p @ v, p @ v.abs()
    return o, a


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
