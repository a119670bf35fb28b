"""qv_token_logprobs on rows of millions of logits, where a sum of one thread has thousands of terms, against 64 bits.

Tolerances. S's relative error E: a term's exponential 2^-22, its argument's roundings 2^-22 |z| ln 2, |z| at most log2 V
on the average over the terms' weights (ln V 2^-22 together); a group's sum of up to 32 terms at most 11 additions deep,
then a group for every 8192 logits of the row and 4 more, each an addition (above 2^19 logits a compensated sum: 3): n
additions, n 2^-24; rescalings: a few of a thread (at most one for every 8 that the maximum rises) count, 2^-22 each, 4
2^-22 together; the combination of threads, warps and thread blocks at most 13 steps of 1.5 2^-22. E = (25 + n / 4 + ln V)
2^-22. ln S is within E, the log probability within that and 2^-22 of its own and the logits' size; T has S's error, and
the entropy ln S - ln 2 T / S, with |ln 2 T / S| <= ln V, is within E (1 + 2 ln V) and 2^-22 of the logits' size."""
import math

import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qv():
    require_gpu()
    from quantized_verification_gb300 import qv as _qv
    _qv.load()
    return _qv


def sum_error(V):
    n = 14 if V > 2 ** 19 else 15 + V / 8192
    return (25 + n / 4 + math.log(V)) * 2.0 ** -22


def rows(V):
    """Rows that a running sum in 32 bits, or a rescaling at every new maximum, treats worst, and ordinary ones."""
    g = torch.Generator(device="cuda").manual_seed(V)
    half = torch.full((V,), math.log(0.5 + 2.0 ** -14), device="cuda")      # terms just above a half: the rest of each
    half[:16384] = 0.0                                                      # addition to a sum of thousands is lost
    third = torch.full((V,), math.log(1 / 3), device="cuda")
    third[:16384] = 0.0
    low = torch.full((V,), -20.2, device="cuda")
    low[V // 2] = 0.0
    return torch.stack([half, third, low, torch.full((V,), 1.3, device="cuda"),
                        torch.randn(V, device="cuda", generator=g) * 2.5, torch.linspace(0, 1, V, device="cuda"),
                        torch.linspace(-30, 30, V, device="cuda"), torch.linspace(0, 1, V, device="cuda") + 1000])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,M", [(1 << 22, 160), (1 << 24, 8), (151936, 320), (3 * 10 ** 6 + 1, 160), (1 << 19, 160),
                                 ((1 << 19) + 1, 160)])
def test_error_does_not_grow_with_the_row(qv, V, M, dtype):
    unique = rows(V).to(dtype)
    n, K = unique.shape[0], 3
    x = unique.repeat(M // n, 1)
    tok = torch.full((M,), V // 3, dtype=torch.int32, device="cuda")
    lp, ent = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    tt, tl = torch.empty(M, K, dtype=torch.int32, device="cuda"), torch.empty(M, K, device="cuda")
    qv.qv_token_logprobs(x, tok, lp, entropy=ent, top_tokens=tt, top_logprobs=tl)
    for got in (lp, ent, tt, tl):                              # equal rows, equal bits
        assert torch.equal(got.view(M // n, -1), got.view(M // n, -1)[:1].expand(M // n, -1))
    E = sum_error(V)
    for r in range(n):
        z = unique[r].double()
        size = float(z.abs().max())
        z = z - torch.logsumexp(z, 0)
        want = z[V // 3]
        assert abs(float(lp[r] - want)) <= E + 2.0 ** -22 * (abs(float(want)) + size), (r, float(lp[r] - want))
        h = -(z.exp() * z).sum()
        assert abs(float(ent[r] - h)) <= E * (1 + 2 * math.log(V)) + 2.0 ** -22 * size, (r, float(ent[r] - h))
        v, i = torch.sort(z, descending=True, stable=True)
        assert torch.equal(tt[r].long(), i[:K])
        assert bool(((tl[r] - v[:K]).abs() <= E + 2.0 ** -22 * (v[:K].abs() + size)).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [3001, 40000, 151936])
def test_probable_tokens_are_never_above_one(qv, V, dtype):
    """One token above the others by 0 to 30, at any place of the row: its log probability is 0 or less, and within the
    tolerance above."""
    g = torch.Generator(device="cuda").manual_seed(V + 1)
    M = 400
    x = torch.rand(M, V, device="cuda", generator=g)
    tok = torch.randint(0, V, (M,), device="cuda", generator=g, dtype=torch.int32)
    x.scatter_(1, tok.long()[:, None], torch.linspace(1, 31, M, device="cuda")[:, None])
    x = x.to(dtype)
    lp = torch.empty(M, device="cuda")
    qv.qv_token_logprobs(x, tok, lp)
    assert float(lp.max()) <= 0.0
    z = x.double()
    want = (z - torch.logsumexp(z, 1, keepdim=True)).gather(1, tok.long()[:, None])[:, 0]
    E = sum_error(V)
    assert bool(((lp - want).abs() <= E + 2.0 ** -22 * (want.abs() + 31)).all())
