"""How near qv_attention_verify_kv4's fp32 outputs come to 64 bits in the 2-norm: a bound that a missing part of the
probabilities (2^-12) or a merge weight off by 2^-15 breaks, where the worst case element by element of test_kv4_gpu.py
lets them pass.

The bound. A key i of a row has probability p, value v and a score s off by d: the output moves by p d (v - o). Values are
independent of scores and errors here, so the squares of p d |v| add up. d is at most
- (D / 16) 2^-23 of the partial sums: the tensor cores cut the sum off below its last bit at each of D / 16 products. The
  partial sums on the way to s are no larger than sqrt(s^2 + sigma^2), sigma the scores' own size (a random walk that
  ends at s);
- 2^-22 sqrt(s^2 + sigma^2) for the roundings of scale * log2 e and of its product;
- of the probability: 2^-21 ln 2 for its exponent, of 16 at most; 2^-22 for the exponential, 2^-22 for its two parts; 2^-23
  for sums and merges (rounded additions, at most 300 to a sum, that err both ways: 2^-24 sqrt(300 / 3) < 2^-20.6, taken
  once more on top): 2^-20 + 2^-20.6 together.
Own keys' scores are formed by the same products, or by 128 rounded additions that err both ways (less)."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import require_gpu
from test_kv4_gpu import ATTENDS, LINES, attend_inputs, cu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qv():
    require_gpu()
    from quantized_verification_gb300 import qv as _qv
    _qv.load()
    return _qv


def exact(qkv, cache, lens, T, Hq, Hkv, D, NB, scale, table):
    """(outputs in 64 bits [B*T, Hq*D], the bound on the 2-norm of their errors)."""
    B, G = len(lens), Hq // Hkv
    x = qkv.cuda().double().view(B, T, Hq + 2 * Hkv, D)
    kc, vc, ks, vs = ref.parts(cache, D)
    K = torch.from_numpy(ref.values(ref.unpack(kc), ks)).cuda()                   # [pages, Hkv, 32, D]
    V = torch.from_numpy(ref.values(ref.unpack(vc), vs)).cuda()
    later = torch.ones(T, T, device="cuda").triu(1).bool()
    out = torch.empty(B, T, Hq, D, dtype=torch.float64, device="cuda")
    by_score, plain = 0.0, 0.0
    for b in range(B):
        n = min(max(int(lens[b]), 0), 32 * NB)
        blocks = torch.from_numpy(np.arange(b * NB, (b + 1) * NB) if table is None else table[b].astype(np.int64)).cuda()
        for h in range(Hkv):
            k = torch.cat([K[blocks, h].reshape(-1, D)[:n], x[b, :, Hq + h]])
            v = torch.cat([V[blocks, h].reshape(-1, D)[:n], x[b, :, Hq + Hkv + h]])
            q = x[b, :, h * G:(h + 1) * G]
            s = torch.einsum("tgd,ld->gtl", q, k) * scale
            s[:, :, n:] = s[:, :, n:].masked_fill(later, -float("inf"))
            p = torch.softmax(s, -1)
            out[b, :, h * G:(h + 1) * G] = torch.einsum("gtl,ld->tgd", p, v)
            s2 = s.masked_fill(s == -float("inf"), 0.0) ** 2
            weight = (p * v.norm(dim=1)) ** 2
            by_score += float((weight * (s2 + s2.mean(-1, keepdim=True))).sum())
            plain += float(weight.sum())
    bound = (D / 16 + 2) * 2.0 ** -23 * by_score ** 0.5 + (2.0 ** -20 + 2.0 ** -20.6) * plain ** 0.5
    return out.reshape(B * T, Hq * D), bound


PARTS = [(1, 1, 4, 1, 128, 2000, [63990], True), (1, 5, 4, 1, 128, 2000, [63990], True), (1, 8, 4, 1, 128, 1400, [44800], True),
         (1, 6, 4, 1, 64, 2000, [64000], True), (2, 1, 8, 1, 64, 1500, [48000, 33], True),
         (3, 5, 4, 1, 128, 1500, [47000, 200, 48000], True), (2, 64, 2, 1, 128, 600, [19000, 5], True),
         (1, 5, 32, 8, 128, 1024, [32749], True), (2, 100, 3, 1, 64, 40, [0, 1250], False)]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,NB,lens,paged", ATTENDS + LINES + PARTS)
def test_error_in_the_2_norm(qv, B, T, Hq, Hkv, D, NB, lens, paged):
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, lens, paged)
    scale = float(np.float32(D ** -0.5))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    out = torch.full((B * T, Hq * D), float("nan"), device="cuda")
    qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out, ws, block_table=cu(table))
    want, bound = exact(qkv, cache, ln, T, Hq, Hkv, D, NB, scale, table)
    err, size = float((out.double() - want).norm()), float(want.norm())
    print(f"error {err / size:.2e}, bound {bound / size:.2e}")
    assert err <= bound
    assert bound <= 2.0 ** -16 * size                          # (the bound itself is of some use)
