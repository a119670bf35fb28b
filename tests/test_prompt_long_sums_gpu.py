"""bf16 outputs over very long prompts and prefixes of values of one sign: the tensor cores cut their accumulator off at every
product, which must not add up."""
import pytest
import torch

from gpu_util import require_gpu
from quantized_verification_gb300 import qv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    require_gpu()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def positive(g, *shape):
    """Values of one sign whose mean differs from dim to dim, so that the outputs' own roundings do not all go one way."""
    D = shape[-1]
    return (torch.randn(*shape, generator=g, device="cuda").abs() * (1 + torch.arange(D, device="cuda") / D)).to(torch.bfloat16)


def near(out, want):
    """Equal scores: every weight is the same power of two, so the output's rounding (2^-8) and what the accumulator loses
    remain. Within a stretch of 32768 positions it takes 2048 products, cut off at 2^-23 of it at most, on a sum that grows
    from 0: 1.2e-4 of the sum; the sum of the weights and of the stretches is binary32's."""
    off = ((out.double() - want) / want).abs()
    assert float(off.max()) <= 2.0 ** -8 + 1.5e-4, float(off.max())
    assert qv.qv_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq,Hkv", [(1 << 20, 1, 1), (70001, 2, 1), (32769, 1, 1)])
def test_long_prompts(n, Hq, Hkv, D):
    g = torch.Generator(device="cuda").manual_seed(n)
    first, m = 77, 1000                                          # a short sequence before the long one
    x = torch.zeros(first + n, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda")
    v = x[:, (Hq + Hkv) * D:]
    v.copy_(positive(g, first + n, D))
    out = torch.zeros(first + n, Hq * D, dtype=torch.bfloat16, device="cuda")
    qv.qv_attention_prompt(x, i32([0, first, first + n]), Hq, Hkv, 0.1, out)
    sums = v[first:first + n].double().cumsum(0)
    count = torch.arange(1, n + 1, device="cuda")[:, None]
    for r in (slice(0, m), slice(n // 2, n // 2 + m), slice(n - m, n)):
        near(out[first:].view(n, Hq, D)[r], (sums[r] / count[r])[:, None])
    near(out[:first].view(first, Hq, D), (v[:first].double().cumsum(0) / count[:first])[:, None])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,half", [(80001, 40000), (38801, 33000)])       # blocks of two tiles and of one
def test_long_prompts_whose_scores_rise_late(n, half, D):
    # the reference moves after sums have been carried on: positions that then weigh 2^-29 each, and some that count
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.zeros(n, 3, D, device="cuda")
    x[:, 0, 0] = 1.0
    x[half:, 1, 0] = 20.0                                        # score 20: e^20 = 2^28.9
    x[:, 2] = positive(g, n, D).float()
    x = x.to(torch.bfloat16).view(n, 3 * D)
    out = torch.zeros(n, D, dtype=torch.bfloat16, device="cuda")
    qv.qv_attention_prompt(x, i32([0, n]), 1, 1, 1.0, out)
    w = torch.ones(n, 1, dtype=torch.float64, device="cuda")
    w[half:] = torch.exp(w[half:] * 20)
    want = (x[:, 2 * D:].double() * w).cumsum(0) / w.cumsum(0)
    # two different weights: each rounded to bf16 (2^-8) before the product, but not in the sum of the weights
    off = ((out.double() - want) / want).abs()
    assert float(off.max()) <= 2 * 2.0 ** -8 + 1.5e-4, float(off.max())
    assert qv.qv_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_long_prefix(D):
    # rows enough that the prefix is not cut into parts
    P, B, T = 1 << 20, 4864, 8
    g = torch.Generator(device="cuda").manual_seed(9)
    pv = positive(g, P, 1, D)
    pk, x = torch.zeros_like(pv), torch.zeros(B * T, 3 * D, dtype=torch.bfloat16, device="cuda")
    x[:, 2 * D:] = positive(g, B * T, D)
    kc = torch.empty(B, 0, 1, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(B * T, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(qv.qv_attention_prefix_workspace_bytes(B, T, 1, 1, D, P), dtype=torch.uint8, device="cuda")
    qv.qv_attention_verify_prefix(x, pk, pv, i32([P]), kc, kc, i32([0] * B), T, 1, 1, 0.1, out, ws)
    own = x[:, 2 * D:].double().view(B, T, D).cumsum(1)
    want = (pv.double().sum(0) + own) / (P + torch.arange(1, T + 1, device="cuda")[:, None])
    near(out.view(B, T, D), want)


@pytest.mark.parametrize("D", [64, 128])
def test_long_prefix_behind_few_rows(D):
    # blocks of one tile, again without a cut into parts; the scores rise where the sums have been written once
    P, H, rise = 40001, 152, 33000
    g = torch.Generator(device="cuda").manual_seed(10)
    pk, pv = torch.zeros(P, H, D, dtype=torch.bfloat16, device="cuda"), positive(g, P, H, D)
    x = torch.zeros(1, 3 * H, D, dtype=torch.bfloat16, device="cuda")
    x[:, :H, 0], pk[rise:, :, 0] = 1.0, 20.0
    x[:, H:2 * H, 0], x[:, 2 * H:] = 20.0, positive(g, 1, H, D)
    kc = torch.empty(1, 0, H, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(1, H * D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(qv.qv_attention_prefix_workspace_bytes(1, 1, H, H, D, P), dtype=torch.uint8, device="cuda")
    qv.qv_attention_verify_prefix(x.view(1, -1), pk, pv, i32([P]), kc, kc, i32([0]), 1, H, H, 1.0, out, ws)
    e = float(torch.exp(torch.tensor(20.0, dtype=torch.float64)))
    want = pv[:rise].double().sum(0) + e * (pv[rise:].double().sum(0) + x[0, 2 * H:].double())
    want = want / (rise + e * (P - rise + 1))
    off = ((out.view(H, D).double() - want) / want).abs()
    # as above: two different weights, and the output's rounding
    assert float(off.max()) <= 2 * 2.0 ** -8 + 1.5e-4, float(off.max())
    assert qv.qv_device_error() == 0
