"""Cases of the 4-bit KV cache operators and of the token log probabilities.

Four operators, as a verify step uses them together:

  write      key/value rows of the qkv projection, quantized into the 4-bit
             paged cache, and the written rows read back as values
  read       positions of the cache read back as fp32 or bf16 values
  attend     attention of the verify tokens over the 4-bit cache and over the
             step's own keys and values
  logprobs   log probability of one given token per row of logits, the row's
             entropy and its most probable alternatives

The cache: blocks of 32 positions. One block of one key/value head is a record
of 34 * D bytes: key codes [32][D/2], value codes [32][D/2], key scales
[32][D/32], value scales [32][D/32]. A code is a 4-bit two's complement number
q in [-7, 7] (even element in the low nibble); a scale byte b, shared by 32
elements, stands for s = (1 + (b & 7) / 8) * 2^((b >> 3) - 15); the value is
q * s. With x a group's 32 elements: t = fl32(max |x| / 7), s the nearest scale
to t (ties to the even byte, clamped to the range), q = the integer nearest
fl32(x / s), ties to even, clamped to [-7, 7].
"""
import math

import torch

own = False

BLOCK = 32            # positions per cache block
GROUP = 32            # elements per scale
VOCAB = 151936        # the vocabulary of this repository's workloads


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence just after a short prompt: latency
        {"name": "attend_one_token_517", "op": "attend", "B": 1, "T": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "longest": 517, "shortest": 517, "paged": False, "out": "f32"},
        # the verify step of the benchmark: 5 tokens over about 2048 positions
        {"name": "attend_verify_2043", "op": "attend", "B": 1, "T": 5, "Hq": 32, "Hkv": 8, "D": 128,
         "longest": 2043, "shortest": 2043, "paged": False, "out": "f32"},
        # a serving batch of 24 sequences of very different lengths, paged
        {"name": "attend_verify_batch_paged", "op": "attend", "B": 24, "T": 5, "Hq": 32, "Hkv": 8, "D": 128,
         "longest": 16001, "shortest": 33, "paged": True, "out": "f32"},
        # single tokens over two long documents, eight query heads a key head
        {"name": "attend_one_token_131071", "op": "attend", "B": 2, "T": 1, "Hq": 64, "Hkv": 8, "D": 128,
         "longest": 131071, "shortest": 120000, "paged": True, "out": "bf16"},
        # heads of 64 values, 40 query rows a key head (more than one row tile)
        {"name": "attend_verify_heads_of_64", "op": "attend", "B": 6, "T": 5, "Hq": 32, "Hkv": 4, "D": 64,
         "longest": 7001, "shortest": 500, "paged": False, "out": "bf16"},
        # the accepted tokens of a verify step over a batch: 1 to 5 rows a sequence
        {"name": "write_accepted_rows", "op": "write", "B": 16, "T": 5, "Hq": 32, "Hkv": 8, "D": 128,
         "ragged": True, "start": 3001, "paged": True, "x": "bf16", "out": "bf16"},
        # two prompts written at once
        {"name": "write_two_prompts", "op": "write", "B": 2, "T": 8190, "Hq": 32, "Hkv": 8, "D": 128,
         "ragged": False, "start": 0, "paged": True, "x": "bf16", "out": "bf16"},
        # a short shared prefix read back in full precision
        {"name": "read_prefix_333", "op": "read", "B": 1, "T": 333, "Hkv": 8, "D": 64, "ragged": False,
         "start": 7, "paged": False, "out": "f32"},
        # whole caches turned back into bf16 ones
        {"name": "read_four_caches", "op": "read", "B": 4, "T": 16384, "Hkv": 8, "D": 128, "ragged": True,
         "start": 0, "paged": True, "out": "bf16"},
        # the rows of one verify step, with 20 alternatives each
        {"name": "logprobs_verify_rows", "op": "logprobs", "M": 5, "V": VOCAB, "K": 20, "x": "f32",
         "masked": 0.0},
        # one row of an odd, small vocabulary in bf16 (many equal logits)
        {"name": "logprobs_one_row_32003", "op": "logprobs", "M": 1, "V": 32003, "K": 5, "x": "bf16",
         "masked": 0.0},
        # a long text scored token by token under a vocabulary mask
        {"name": "logprobs_scored_text", "op": "logprobs", "M": 2000, "V": VOCAB, "K": 5, "x": "f32",
         "masked": 0.1},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "read", "logprobs"])
    if op == "logprobs":
        V = _log(rng, 1000, VOCAB)
        M = _log(rng, 1, max(1, min(4000, 2000 * VOCAB // V)))
        return {"op": op, "M": M, "V": V, "K": rng.choice([0, 1, 5, 20, 32]), "x": rng.choice(["f32", "bf16"]),
                "masked": rng.choice([0.0, 0.0, 0.1, 0.5])}
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    paged = rng.random() < 0.6
    if op == "attend":
        B = _log(rng, 1, 64)
        T = rng.choice([1, 1, 2, 3, 5, 8, 16])
        # positions of all sequences together, so that no draw is above the largest case
        longest = _log(rng, 1, max(64, min(131072, 262144 * 64 // (B * max(64, T * G * Hkv)))))
        return {"op": op, "B": B, "T": T, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "longest": longest,
                "shortest": rng.choice([0, longest, max(1, longest // 3)]), "paged": paged,
                "out": rng.choice(["f32", "bf16"])}
    if op == "write":
        B = _log(rng, 1, 32)
        T = _log(rng, 1, max(1, 16384 // B))
        return {"op": op, "B": B, "T": T, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "ragged": rng.random() < 0.5,
                "start": rng.choice([0, 1, rng.randint(0, 5000)]), "paged": paged,
                "x": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"])}
    B = _log(rng, 1, 16)
    T = _log(rng, 1, max(1, 32768 // B))
    return {"op": op, "B": B, "T": T, "Hkv": Hkv, "D": D, "ragged": rng.random() < 0.5,
            "start": rng.choice([0, rng.randint(0, 500)]), "paged": paged, "out": rng.choice(["bf16", "f32"])}


# ------------------------------------------------------------------- inputs
def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _spread(lo, hi, n, gen):
    """n lengths in [lo, hi], the first the longest, the rest spread over their logarithm."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    a, b = math.log(lo + 1), math.log(hi + 1)
    v = torch.exp(a + (b - a) * u).round().to(torch.int32) - 1
    v[0] = hi
    return v.clamp_(lo, hi)


def _table(B, NB, paged, gen):
    """Block tables over a pool with room to spare: shuffled pages, or None (page b * NB + i)."""
    if not paged:
        return None, B * NB
    pages = B * NB + 8
    return torch.randperm(pages, generator=gen, device="cuda")[: B * NB].to(torch.int32).view(B, NB).contiguous(), pages


def _random_cache(pages, Hkv, D, gen):
    """A filled cache: uniform codes in [-7, 7], scales of values between about 0.5 and 4 at most."""
    c = torch.randint(0, 225, (pages, Hkv, 32 * D), generator=gen, device="cuda", dtype=torch.int32)
    codes = ((c // 15 - 7) & 15) | (((c % 15 - 7) & 15) << 4)
    scales = torch.randint(11 * 8, 14 * 8, (pages, Hkv, 2 * D), generator=gen, device="cuda", dtype=torch.int32)
    return torch.cat([codes, scales], 2).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    st = dict(case)
    if case["op"] == "logprobs":
        M, V, K = case["M"], case["V"], case["K"]
        x = rnd(M, V).mul_(2.5)
        tok = torch.randint(0, V, (M,), generator=gen, device="cuda", dtype=torch.int32)
        if case["masked"]:
            x.masked_fill_(torch.rand(M, V, generator=gen, device="cuda") < case["masked"], -math.inf)
        likely = torch.randint(0, 2, (M,), generator=gen, device="cuda").to(torch.float32) * 6 + 4
        x.scatter_(1, tok.long()[:, None], likely[:, None] + rnd(M, 1))
        st.update(logits=x.to(_dt(case["x"])), tokens=tok,
                  logprob=torch.empty(M, device="cuda"), entropy=torch.empty(M, device="cuda"),
                  top_tokens=torch.empty(M, K, dtype=torch.int32, device="cuda") if K else None,
                  top_logprobs=torch.empty(M, K, device="cuda") if K else None)
        return st
    B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
    if case["op"] == "attend":
        NB = -(-max(case["longest"], 1) // BLOCK)
        st["len"] = _spread(case["shortest"], case["longest"], B, gen)
    else:
        NB = -(-(case["start"] + T) // BLOCK) + 1
        if case["ragged"]:
            st["count"] = _spread(1, T, B, gen)
        else:
            st["count"] = None
        st["first"] = torch.full((B,), case["start"], dtype=torch.int32, device="cuda")
        if B > 1 and case["start"] > 0:
            st["first"] -= torch.randint(0, min(case["start"], 31) + 1, (B,), generator=gen, device="cuda",
                                         dtype=torch.int32)
    st["NB"] = NB
    st["table"], st["pages"] = _table(B, NB, case["paged"], gen)
    st["cache"] = _random_cache(st["pages"], Hkv, D, gen)
    if case["op"] != "read":
        Hq = case["Hq"]
        x = rnd(B * T, (Hq + 2 * Hkv) * D)
        x[:, Hq * D: (Hq + Hkv) * D: 61] *= 4           # a few wide key channels
        st["qkv"] = x.to(_dt(case.get("x", "bf16")))
    if case["op"] == "attend":
        st["scale"] = 1.0 / math.sqrt(D)
        st["o"] = torch.empty(B * T, Hq * D, dtype=_dt(case["out"]), device="cuda")
    else:
        st["k"] = torch.zeros(B, T, Hkv, D, dtype=_dt(case["out"]), device="cuda")
        st["v"] = torch.zeros(B, T, Hkv, D, dtype=_dt(case["out"]), device="cuda")
    return st


# ------------------------------------------------------------ plain 32-bit forms
def _pages_of(st, blocks):
    """Page of each block index [B, n] of each sequence."""
    if st["table"] is None:
        return torch.arange(st["B"], device="cuda")[:, None] * st["NB"] + blocks
    return st["table"].long().gather(1, blocks)


def _fields(cache, D):
    """The four parts of every record, as views [pages, Hkv, 32, ...]."""
    cut = [0, 16 * D, 32 * D, 33 * D, 34 * D]
    return [cache[:, :, a:b].unflatten(2, (BLOCK, (b - a) // BLOCK)) for a, b in zip(cut, cut[1:])]


def _scale_value(b):
    return ((b.to(torch.int32) << 20) + (112 << 23)).view(torch.float32)      # exponent and mantissa put in place


def _values(codes, scales):
    """fp32 values [..., D] of codes [..., D/2] and scale bytes [..., D/32]."""
    c = codes.to(torch.int32)
    q = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    q = q - 16 * (q > 7)
    return (q.unflatten(-1, (-1, GROUP)).float() * _scale_value(scales)[..., None]).flatten(-2)


def _quantize(x):
    """Codes [..., D/2] and scale bytes [..., D/32] of fp32 values [..., D]."""
    g = x.unflatten(-1, (-1, GROUP))
    a = g.abs().amax(-1)
    t = a / torch.full_like(a, 7.0)               # a quotient: by a plain number it would be a product with 1 / 7
    bits = t.view(torch.int32)
    b = (((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - 896).clamp(0, 255)
    q = torch.round(g / _scale_value(b)[..., None]).clamp(-7, 7).to(torch.int32).flatten(-2)
    n = q & 15
    return (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8), b.to(torch.uint8)


def _rows(st):
    """Page and slot of every (sequence, row), and which rows there are."""
    j = torch.arange(st["T"], device="cuda")[None, :]
    pos = st["first"].long()[:, None] + j
    there = pos < st["NB"] * BLOCK
    if st["count"] is not None:
        there = there & (j < st["count"][:, None])
    return _pages_of(st, (pos // BLOCK).clamp(max=st["NB"] - 1)), pos % BLOCK, there


def _plain_write(st):
    B, T, Hq, Hkv, D = st["B"], st["T"], st["Hq"], st["Hkv"], st["D"]
    page, slot, there = _rows(st)
    at = there.nonzero(as_tuple=True)
    x = st["qkv"].view(B, T, -1)[at].float()
    k = x[:, Hq * D: (Hq + Hkv) * D].unflatten(1, (Hkv, D))
    v = x[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    kc, vc, ks, vs = _fields(st["cache"], D)
    p, s = page[at], slot[at]
    kq, kb = _quantize(k.contiguous())
    vq, vb = _quantize(v.contiguous())
    kc[p, :, s], ks[p, :, s] = kq, kb
    vc[p, :, s], vs[p, :, s] = vq, vb


def _plain_read(st):
    page, slot, there = _rows(st)
    kc, vc, ks, vs = _fields(st["cache"], st["D"])
    take = there[:, :, None, None]
    k = torch.where(take, _values(kc[page, :, slot], ks[page, :, slot]).to(st["k"].dtype), st["k"])
    v = torch.where(take, _values(vc[page, :, slot], vs[page, :, slot]).to(st["v"].dtype), st["v"])
    return k, v


def _plain_attend(st):
    B, T, Hq, Hkv, D, NB = st["B"], st["T"], st["Hq"], st["Hkv"], st["D"], st["NB"]
    G, L = Hq // Hkv, NB * BLOCK
    page = _pages_of(st, torch.arange(NB, device="cuda").expand(B, NB))
    kc, vc, ks, vs = [f[page] for f in _fields(st["cache"], D)]            # [B, NB, Hkv, 32, ...]
    K = _values(kc, ks).permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)
    V = _values(vc, vs).permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)
    x = st["qkv"].view(B, T, Hq + 2 * Hkv, D).float()
    q = x[:, :, :Hq].unflatten(2, (Hkv, G)).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    kn, vn = x[:, :, Hq:Hq + Hkv].permute(0, 2, 1, 3), x[:, :, Hq + Hkv:].permute(0, 2, 1, 3)
    s_old = torch.matmul(q, K.transpose(2, 3)) * st["scale"]
    s_old = s_old.masked_fill(torch.arange(L, device="cuda") >= st["len"][:, None, None, None], -math.inf)
    s_new = torch.matmul(q, kn.transpose(2, 3)) * st["scale"]
    j = torch.arange(T, device="cuda")
    s_new = s_new.masked_fill(j[None, :] > j.repeat_interleave(G)[:, None], -math.inf)
    m = torch.maximum(s_old.amax(-1), s_new.amax(-1))[..., None]
    p_old, p_new = torch.exp(s_old - m), torch.exp(s_new - m)
    o = torch.matmul(p_old, V) + torch.matmul(p_new, vn)
    o = o / (p_old.sum(-1) + p_new.sum(-1))[..., None]
    return o.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B * T, Hq * D).to(st["o"].dtype)


def _plain_logprobs(st):
    x = st["logits"].float()
    m = x.amax(1, keepdim=True)
    z = x - m
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    lse = torch.log(total)
    lp = (z.gather(1, st["tokens"].long()[:, None]) - lse)[:, 0]
    ent = lse[:, 0] - (torch.where(e > 0, z, 0.0) * e).sum(1) / total[:, 0]
    if not st["K"]:
        return {"logprob": lp, "entropy": ent}
    # order by value, then by the lower index: one whole number per entry
    i = (x + 0.0).view(torch.int32)
    key = ((i ^ ((i >> 31) & 0x7FFFFFFF)).long() << 32) | torch.arange(x.shape[1] - 1, -1, -1, device="cuda")
    best = torch.topk(key, st["K"], 1, sorted=True).values
    idx = x.shape[1] - 1 - (best & 0xFFFFFFFF)
    return {"logprob": lp, "entropy": ent, "top_tokens": idx.to(torch.int32), "top_logprobs": z.gather(1, idx) - lse}


# ------------------------------------------------------- this repository's calls
def _own(st):
    from quantized_verification_gb300 import qv
    op = st["op"]
    if op == "logprobs":
        qv.qv_token_logprobs(st["logits"], st["tokens"], st["logprob"], entropy=st["entropy"],
                             top_tokens=st["top_tokens"], top_logprobs=st["top_logprobs"])
        out = {"logprob": st["logprob"], "entropy": st["entropy"]}
        if st["K"]:
            out.update(top_tokens=st["top_tokens"], top_logprobs=st["top_logprobs"])
        return out
    if op == "attend":
        if "ws" not in st:                      # a program keeps one workspace for all its steps
            n = qv.qv_attention_kv4_workspace_bytes(st["B"], st["T"], st["Hq"], st["Hkv"], st["D"], st["NB"])
            st["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        qv.qv_attention_verify_kv4(st["qkv"], st["cache"], st["len"], st["T"], st["Hq"], st["Hkv"], st["scale"],
                                   st["o"], st["ws"], block_table=st["table"])
        return {"o": st["o"]}
    if op == "write":
        qv.qv_kv4_write(st["qkv"], st["first"], st["cache"], st["T"], st["Hq"], st["Hkv"], block_table=st["table"],
                        count=st["count"])
    qv.qv_kv4_read(st["cache"], st["first"], st["k"], st["v"], block_table=st["table"], count=st["count"])
    return {"k": st["k"], "v": st["v"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "logprobs":
        return _plain_logprobs(state)
    if op == "attend":
        return {"o": _plain_attend(state)}
    if op == "write":
        _plain_write(state)
    k, v = _plain_read(state)
    return {"k": k, "v": v}


# --------------------------------------------------------------------- work
def work(case):
    size = lambda n: 4 if n == "f32" else 2  # noqa: E731
    if case["op"] == "logprobs":
        M, V, K = case["M"], case["V"], case["K"]
        return {"bytes": M * V * size(case["x"]) + M * (4 + 8 + 8 * K), "flops": 5 * M * V}
    B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
    row = Hkv * D * 17 // 16                    # bytes of one position: keys and values, codes and scales
    if case["op"] == "attend":
        lo, hi, Hq = case["shortest"], case["longest"], case["Hq"]
        # the first sequence is the longest; the mean of the others, even over the logarithm
        mean = hi if lo == hi else (hi - lo) / math.log((hi + 1) / (lo + 1)) - 1
        positions = hi + (B - 1) * max(mean, 0)
        io = B * T * ((Hq + 2 * Hkv) * D * 2 + Hq * D * size(case["out"]))
        return {"bytes": int(positions * row + io), "flops": int(4 * T * Hq * D * (positions + B * (T + 1) / 2))}
    rows = B * T
    if case["ragged"] and T > 1:
        rows = int(T + (B - 1) * (T - 1) / math.log((T + 1) / 2))
    out = rows * 2 * Hkv * D * size(case["out"])
    if case["op"] == "read":
        return {"bytes": rows * row + out, "flops": rows * 2 * Hkv * D}
    return {"bytes": rows * 2 * Hkv * D * size(case["x"]) + rows * row + out, "flops": rows * 8 * Hkv * D}


# ------------------------------------------------------ the definition in 64 bits
def _power(n):
    """2^n in 64 bits for whole numbers n: exact, as a library's pow need not be."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_value(codes, scales):
    """Values in 64 bits, nibble by nibble from the definition."""
    lo, hi = (codes % 16).double(), (codes // 16).double()
    lo, hi = torch.where(lo < 8, lo, lo - 16), torch.where(hi < 8, hi, hi - 16)
    q = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    q[..., 0::2], q[..., 1::2] = lo, hi
    s = (8 + (scales % 8).double()) * _power(scales // 8 - 18)
    return q * s.repeat_interleave(GROUP, -1)


def _exact_rounded(x):
    """What x [..., D] becomes in the cache: the nearest scale and the nearest code, in 64 bits with the definition's two binary32 quotients."""
    D = x.shape[-1]
    g = x.double().reshape(*x.shape[:-1], D // GROUP, GROUP)
    t = (g.abs().max(-1).values / 7).float().double()
    step = _power(torch.frexp(t.clamp_min(2.0 ** -60)).exponent - 4)   # 8 scales an octave; torch.round takes ties to even
    s = (torch.round(t / step) * step).clamp(2.0 ** -15, 122880.0)
    q = torch.round((g / s[..., None]).float().double()).clamp(-7, 7)
    return (q * s[..., None]).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprobs":
        x, tok, K = st["logits"], st["tokens"].long(), case["K"]
        parts = []
        for r in range(0, case["M"], 256):
            z = x[r:r + 256].double()
            z = z - torch.logsumexp(z, 1, keepdim=True)
            p = torch.exp(z)
            part = [z.gather(1, tok[r:r + 256, None])[:, 0], -(p * z.masked_fill(p == 0, 0.0)).sum(1)]
            if K:
                v, i = torch.sort(z, dim=1, descending=True, stable=True)
                part += [i[:, :K].to(torch.int32), v[:, :K].contiguous()]
            parts.append(part)
        return dict(zip(("logprob", "entropy", "top_tokens", "top_logprobs"), [torch.cat(c) for c in zip(*parts)]))
    B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
    NB = st["NB"]
    table = st["table"] if st["table"] is not None else torch.arange(B * NB, device="cuda").view(B, NB)
    rec = st["cache"]
    if case["op"] in ("write", "read"):
        k, v = st["k"].double(), st["v"].double()
        for b in range(B):
            n = T if st["count"] is None else int(st["count"][b])
            f = int(st["first"][b])
            if case["op"] == "write":
                rows = st["qkv"].view(B, T, -1)[b, :n, case["Hq"] * D:].reshape(n, 2, Hkv, D)
                k[b, :n], v[b, :n] = _exact_rounded(rows[:, 0]), _exact_rounded(rows[:, 1])
                continue
            c = rec[table[b].long()].to(torch.int32).transpose(1, 2)          # [NB, 34 D, Hkv]
            part = lambda a, w: (c[:, a * D: a * D + BLOCK * w].reshape(NB * BLOCK, w, Hkv)  # noqa: E731
                                 .transpose(1, 2)[f:f + n])
            k[b, :n] = _exact_value(part(0, D // 2), part(32, D // GROUP))
            v[b, :n] = _exact_value(part(16, D // 2), part(33, D // GROUP))
        return {"k": k, "v": v}
    Hq = case["Hq"]
    G = Hq // Hkv
    o = torch.empty(B, T, Hq, D, dtype=torch.float64, device="cuda")
    x = st["qkv"].view(B, T, Hq + 2 * Hkv, D).double()
    later = torch.ones(T, T, device="cuda").triu(1).bool()
    for b in range(B):
        n = int(st["len"][b])
        for h in range(Hkv):
            r = rec[table[b, : -(-n // BLOCK)].long(), h].to(torch.int32)
            cut = lambda a, w: r[:, a * D: a * D + BLOCK * w].reshape(-1, w)[:n]  # noqa: E731
            K = torch.cat([_exact_value(cut(0, D // 2), cut(32, D // GROUP)), x[b, :, Hq + h]])
            V = torch.cat([_exact_value(cut(16, D // 2), cut(33, D // GROUP)), x[b, :, Hq + Hkv + h]])
            s = torch.einsum("tgd,ld->gtl", x[b, :, h * G:(h + 1) * G], K) * st["scale"]
            s[:, :, n:] = s[:, :, n:].masked_fill(later, -math.inf)
            o[b, :, h * G:(h + 1) * G] = torch.einsum("gtl,ld->tgd", torch.softmax(s, -1), V)
    return {"o": o.view(B * T, Hq * D)}
