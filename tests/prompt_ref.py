"""64-bit definitions of rotary positions and of attention over prompts and prefixes (plain torch, any device)."""
import math

import torch


def rotate(qkv, positions, inv_freq, Hq, Hkv, interleaved=False, magnitude=1.0, q_gamma=None, k_gamma=None, eps=1e-6):
    """What qv_rotary writes, in 64 bits, head by head and pair by pair."""
    M, heads = qkv.shape[0], Hq + 2 * Hkv
    D = qkv.shape[1] // heads
    x = qkv.double().reshape(M, heads, D).clone()
    rot = 2 * inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq.double()[None]
    c, s = magnitude * torch.cos(angle), magnitude * torch.sin(angle)
    for h in range(Hq + Hkv):
        y = x[:, h].clone()
        if q_gamma is not None:
            y = y / torch.sqrt((y * y).mean(1, keepdim=True) + eps) * (q_gamma if h < Hq else k_gamma).double()
        z = y.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            z[:, a] = y[:, a] * c[:, i] - y[:, b] * s[:, i]
            z[:, b] = y[:, b] * c[:, i] + y[:, a] * s[:, i]
        x[:, h] = z
    return x.reshape(M, -1)


def _attend(q, k, v, scale, see):
    """Outputs and the weighted mean of |v| (what rounding errors of the probabilities act on) of one head."""
    s = (q @ k.T) * scale
    s = torch.where(see, s, -math.inf)
    p = torch.softmax(s, -1)
    # a position that is not seen takes no part, whatever it holds
    o = torch.where(see[:, :, None], p[:, :, None] * v[None], 0.0).sum(1) if not torch.isfinite(v).all() else p @ v
    return o, p @ torch.nan_to_num(v, 0.0, 0.0, 0.0).abs()


def prompt(qkv, cu, Hq, Hkv, scale):
    """(outputs, weighted mean of |v|) [M, Hq, D] in 64 bits; rows of no sequence are NaN."""
    M = qkv.shape[0]
    x = qkv.double().reshape(M, Hq + 2 * Hkv, -1)
    o = torch.full((M, Hq, x.shape[2]), math.nan, dtype=torch.float64, device=qkv.device)
    a = o.clone()
    G = Hq // Hkv
    for f, e in zip(cu[:-1], cu[1:]):
        see = torch.ones(e - f, e - f, dtype=torch.bool, device=qkv.device).tril()
        for h in range(Hq):
            o[f:e, h], a[f:e, h] = _attend(x[f:e, h], x[f:e, Hq + h // G], x[f:e, Hq + Hkv + h // G], scale, see)
    return o, a


def verify_prefix(qkv, pk, pv, plen, kc, vc, lens, T, Hq, Hkv, scale):
    """The same for the rows of verify steps behind a shared prefix, [B * T, Hq, D]."""
    B, G = len(lens), Hq // Hkv
    x = qkv.double().reshape(B * T, Hq + 2 * Hkv, -1)
    o = torch.empty(B * T, Hq, x.shape[2], dtype=torch.float64, device=qkv.device)
    a = o.clone()
    for b, n in enumerate(lens):
        r = slice(b * T, (b + 1) * T)
        see = torch.ones(T, plen + n + T, dtype=torch.bool, device=qkv.device).tril(plen + n)
        for h in range(Hkv):
            k = torch.cat([pk[:plen, h].double(), kc[b, :n, h].double(), x[r, Hq + h]])
            v = torch.cat([pv[:plen, h].double(), vc[b, :n, h].double(), x[r, Hq + Hkv + h]])
            for g in range(G):
                o[r, h * G + g], a[r, h * G + g] = _attend(x[r, h * G + g], k, v, scale, see)
    return o, a


def bound(o, a, dtype):
    """How far an output may be from o. bf16: the probabilities' rounding (half a step, 2^-8 of each) acts on the mean
    of |v|, the output's own on itself. fp32: two bf16 parts leave 2^-17 of a probability; scores (sums of up to 128
    products, 2^-23 of their terms each) and the sums' truncation are covered by 1e-5."""
    if dtype == torch.bfloat16:
        return 2.0 ** -8 * (a + o.abs()) * 1.01 + 1e-5 * a
    return (2.0 ** -17 + 1e-5) * a


def norm_bound(dtype):
    """The same for the 2-norm of the difference over the 2-norm of the outputs. fp32: errors of single probabilities are
    independent, so that their share of the mean is that of one of them, whether or not the values cancel: the residue of
    two bf16 parts, at most 2^-17 of a probability, evenly spread, is 2^-17 / sqrt(3) = 4.4e-6; the sum of a score's 128
    products, cut off 8 times at 2^-24 of scores up to about 8, 2e-6; the cut sums of at most 128 products, 1.6e-8 each on a
    sum that grows from 0, 1e-6: 5e-6 together. bf16: half a step of the probabilities and of the outputs, evenly spread,
    2^-8 / sqrt(3) each: 3.2e-3."""
    return 4e-3 if dtype == torch.bfloat16 else 5e-6
