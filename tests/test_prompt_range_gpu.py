"""Attention over prompts and behind a prefix with large values and scores that rise after the first keys: every weight is at
most 1 before the sums, so that they overflow no earlier than the largest value times the positions a row sees."""
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


def line(n, rise, g):
    """n keys' first element: rises by `rise` over the positions, in steps and with noise of 1."""
    return (torch.linspace(0, rise, n, device="cuda") + torch.rand(n, generator=g, device="cuda")) / 8


def near(out, o, a, rise):
    assert torch.isfinite(out).all()
    # (scores up to `rise`, which binary32 holds to 2^-24 of it each way)
    extra = (rise + 2) * 2.0 ** -22 * a
    got = out.double().view(o.shape)
    assert ((got - o).abs() <= ref.bound(o, a, out.dtype) + extra).all(), float(((got - o).abs() / a).max())
    assert qv.qv_device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rise", [5.0, 15.0, 27.0, 80.0])
@pytest.mark.parametrize("n,Hq,Hkv", [(400, 2, 1), (1300, 32, 8)])
def test_large_values_and_rising_scores_of_a_prompt(n, Hq, Hkv, rise, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(n)
    y = torch.randn(n, Hq + 2 * Hkv, D, generator=g, device="cuda")
    y[:, :Hq + Hkv] = 0
    y[:, :Hq, 0] = 8
    y[:, Hq:Hq + Hkv, 0] = line(n, rise, g)[:, None]
    # |randn| < 6: 6e34 times 1300 positions is within binary32
    x = torch.cat([y[:, :Hq + Hkv], y[:, Hq + Hkv:].clamp(-6, 6) * 1e34], 1).view(n, -1).to(torch.bfloat16)
    out = torch.zeros(n, Hq * D, dtype=dtype, device="cuda")
    qv.qv_attention_prompt(x, i32([0, n]), Hq, Hkv, 1.0, out)
    near(out, *ref.prompt(x, [0, n], Hq, Hkv, 1.0), rise)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rise", [15.0, 27.0])
@pytest.mark.parametrize("B,T,Hq,Hkv,D", [(100, 1, 32, 8, 128), (9, 2, 16, 16, 64)])       # many rows and few: two merges
def test_large_values_and_rising_scores_behind_a_prefix(B, T, Hq, Hkv, D, rise, dtype):
    P, L = 6000, 500
    g = torch.Generator(device="cuda").manual_seed(B)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").clamp(-6, 6)  # noqa: E731
    x = torch.zeros(B * T, Hq + 2 * Hkv, D, device="cuda")
    x[:, :Hq, 0] = 8
    x[:, Hq:Hq + Hkv, 0] = rise / 8
    x[:, Hq + Hkv:] = r(B * T, Hkv, D) * 1e33
    pk, kc = torch.zeros(P, Hkv, D, device="cuda"), torch.zeros(B, L, Hkv, D, device="cuda")
    pk[:, :, 0], kc[:, :, :, 0] = line(P, rise, g)[:, None], line(L, rise, g)[None, :, None]
    x, pk, pv, kc, vc = (t.to(torch.bfloat16) for t in (x.view(B * T, -1), pk, r(P, Hkv, D) * 1e33, kc, r(B, L, Hkv, D) * 1e33))
    lens = [L - 5 * b % L for b in range(B)]
    out = torch.zeros(B * T, Hq * D, dtype=dtype, device="cuda")
    ws = torch.empty(qv.qv_attention_prefix_workspace_bytes(B, T, Hq, Hkv, D, P), dtype=torch.uint8, device="cuda")
    qv.qv_attention_verify_prefix(x, pk, pv, i32([P]), kc, vc, i32(lens), T, Hq, Hkv, 1.0, out, ws)
    near(out, *ref.verify_prefix(x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 1.0), rise)
