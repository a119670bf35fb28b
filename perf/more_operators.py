"""Cases of rotary positions, attention over whole prompts and attention over a shared prefix.

Three operators, as a program that serves prompts uses them together:

  rotary     the query and key heads of qkv rows, normalised (or not) and rotated
             by their positions: half and interleaved pairs, part of the head,
             stretched frequencies
  prompt     causal grouped-query attention of packed prompts of different
             lengths: every row attends to its own sequence's rows up to itself
  prefix     attention of the verify tokens of a batch whose sequences all begin
             with the same long prefix: over the prefix (stored once), over each
             sequence's own cache and over the step's own keys and values

A qkv row holds Hq query heads, then Hkv key heads, then Hkv value heads, D
values each; query head h reads key/value head h / (Hq / Hkv).
Rotation of pair i by position p: angle p * inv_freq[i] (inv_freq in binary32,
the product not rounded), cos and sin times `magnitude`. Pairs are (i, i + rot /
2) or, interleaved, (2 i, 2 i + 1); dims from rot on are not rotated. With norm
weights a head x is first x * gamma / sqrt(mean(x^2) + eps). Value heads are
copied.
"""
import math

import torch

own = False

EPS = 1e-6


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the rows of one verify step far into a long context: latency
        {"name": "rotary_verify_rows", "op": "rotary", "M": 5, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "interleaved": False, "norm": True, "stretch": 1.0, "start": 131001, "x": "bf16"},
        # a partly rotated head of 64, pairs side by side, in full precision
        {"name": "rotary_part_of_the_head", "op": "rotary", "M": 2043, "Hq": 12, "Hkv": 4, "D": 64, "rot": 24,
         "interleaved": True, "norm": False, "stretch": 1.0, "start": 0, "x": "f32"},
        # a long prompt with frequencies stretched for long contexts
        {"name": "rotary_prompt_16001", "op": "rotary", "M": 16001, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "interleaved": False, "norm": True, "stretch": 4.0, "start": 0, "x": "bf16"},
        # one short prompt: latency
        {"name": "prompt_short_97", "op": "prompt", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "longest": 97,
         "shortest": 97, "spare": 0, "out": "bf16"},
        # one prompt of ordinary length
        {"name": "prompt_2043", "op": "prompt", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "longest": 2043,
         "shortest": 2043, "spare": 0, "out": "bf16"},
        # a batch of prompts of very different lengths in one buffer that is not full
        {"name": "prompt_packed_24", "op": "prompt", "B": 24, "Hq": 32, "Hkv": 8, "D": 128, "longest": 4001,
         "shortest": 33, "spare": 37, "out": "bf16"},
        # heads of 64, three query heads a key head, fp32 outputs, the shortest prompt a single token
        {"name": "prompt_heads_of_64", "op": "prompt", "B": 5, "Hq": 12, "Hkv": 4, "D": 64, "longest": 1500,
         "shortest": 1, "spare": 5, "out": "f32"},
        # one long document, eight query heads a key head
        {"name": "prompt_16001", "op": "prompt", "B": 1, "Hq": 64, "Hkv": 8, "D": 128, "longest": 16001,
         "shortest": 16001, "spare": 0, "out": "bf16"},
        # single tokens of two sequences behind a short system prompt: latency
        {"name": "prefix_two_517", "op": "prefix", "B": 2, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "prefix": 517,
         "longest": 40, "shortest": 1, "out": "f32"},
        # heads of 64, three query heads a key head
        {"name": "prefix_heads_of_64", "op": "prefix", "B": 7, "T": 3, "Hq": 12, "Hkv": 4, "D": 64, "prefix": 2999,
         "longest": 300, "shortest": 0, "out": "bf16"},
        # verify steps of a serving batch behind a prompt of 8190 tokens
        {"name": "prefix_verify_batch_8190", "op": "prefix", "B": 24, "T": 5, "Hq": 32, "Hkv": 8, "D": 128,
         "prefix": 8190, "longest": 700, "shortest": 1, "out": "f32"},
        # single tokens of 64 conversations about one long document
        {"name": "prefix_one_token_100001", "op": "prefix", "B": 64, "T": 1, "Hq": 64, "Hkv": 8, "D": 128,
         "prefix": 100001, "longest": 500, "shortest": 3, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rotary", "prompt", "prompt", "prefix", "prefix"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    case = {"op": op, "Hq": Hkv * G, "Hkv": Hkv, "D": D}
    if op == "rotary":
        case.update(M=_log(rng, 1, 16001), rot=rng.choice([D, D, D // 2, 24]), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.5, stretch=rng.choice([1.0, 1.0, 4.0, 8.0]),
                    start=rng.choice([0, 1, rng.randint(0, 1000000)]), x=rng.choice(["bf16", "f32"]))
        return case
    case["out"] = rng.choice(["bf16", "bf16", "f32"])
    if op == "prompt":
        # no more than 16001 rows of 64 heads of 128: the square of the longest counts
        B = _log(rng, 1, 48)
        most = min(16001.0, 16001.0 * math.sqrt(64 * 128 / (Hkv * G * D * B)))
        longest = _log(rng, 1, int(most))
        case.update(B=B, longest=longest, shortest=rng.choice([0, 1, longest, max(1, longest // 5)]),
                    spare=rng.choice([0, 0, rng.randint(1, 200)]))
        return case
    T = rng.choice([t for t in (1, 1, 2, 3, 5, 8) if t * G <= 32])
    B = _log(rng, 1, 96)
    case.update(B=B, T=T, prefix=_log(rng, 1, max(64, min(100001, 100001 * 4096 // max(4096, B * T * Hkv * G)))),
                longest=_log(rng, 1, 700))
    case["shortest"] = rng.choice([0, case["longest"], max(1, case["longest"] // 4)])
    return case


def lengths(case):
    """The lengths of a case's sequences, longest first: even over their logarithm."""
    B, hi, lo = case["B"], case["longest"], case["shortest"]
    if B == 1:
        return [hi]
    a, b = math.log(hi + 1), math.log(lo + 1)
    return [int(round(math.exp(a + (b - a) * i / (B - 1)))) - 1 for i in range(B)]


# ------------------------------------------------------------------- inputs
def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _frequencies(rot, stretch):
    """Rotary frequencies of base 1e6; stretched ones keep the fast pairs, divide the slow ones and blend between."""
    f = [1e6 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if stretch == 1.0:
        return f, 1.0
    turns = [8192 * v / (2 * math.pi) for v in f]                     # turns within the length that was trained
    keep = [min(1.0, max(0.0, (t - 1.0) / 31.0)) for t in turns]
    return [v * k + v / stretch * (1 - k) for v, k in zip(f, keep)], 0.1 * math.log(stretch) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    st = dict(case)
    op, Hq, Hkv, D = case["op"], case["Hq"], case["Hkv"], case["D"]
    W = (Hq + 2 * Hkv) * D
    if op == "rotary":
        M = case["M"]
        x = rnd(M, W)
        x[:, :(Hq + Hkv) * D:61] *= 4                                  # a few wide channels
        f, st["magnitude"] = _frequencies(case["rot"], case["stretch"])
        pos = case["start"] + torch.arange(M, device="cuda", dtype=torch.int32)
        pos[M // 2:] -= int(torch.randint(0, min(case["start"], 64) + 1, (1,), generator=gen, device="cuda"))
        st.update(qkv=x.to(_dt(case["x"])), positions=pos, inv_freq=torch.tensor(f, dtype=torch.float32, device="cuda"),
                  q_gamma=(1 + 0.1 * rnd(D)).to(torch.bfloat16) if case["norm"] else None,
                  k_gamma=(1 + 0.1 * rnd(D)).to(torch.bfloat16) if case["norm"] else None,
                  o=torch.empty(M, W, dtype=_dt(case["x"]), device="cuda"))
        return st
    n = torch.tensor(lengths(case), device="cuda")[torch.randperm(case["B"], generator=gen, device="cuda")]
    rows = sum(lengths(case)) + case["spare"] if op == "prompt" else case["B"] * case["T"]
    rows = max(rows, 1)
    x = rnd(rows, W)
    x[:, Hq * D:(Hq + Hkv) * D:61] *= 4                                # a few wide key channels
    st.update(qkv=x.to(torch.bfloat16), scale=1.0 / math.sqrt(D),
              o=torch.zeros(rows, Hq * D, dtype=_dt(case["out"]), device="cuda"))
    if op == "prompt":
        st["cu"] = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), n.cumsum(0)]).to(torch.int32)
        return st
    Lmax = max(case["longest"], 1)
    st["len"] = n.to(torch.int32)
    st["prefix_len"] = torch.full((1,), case["prefix"], dtype=torch.int32, device="cuda")
    for name, shape in (("pk", (case["prefix"] + 29, Hkv, D)), ("pv", (case["prefix"] + 29, Hkv, D)),
                        ("kc", (case["B"], Lmax, Hkv, D)), ("vc", (case["B"], Lmax, Hkv, D))):
        st[name] = rnd(*shape).to(torch.bfloat16)
    return st


# ------------------------------------------------------------ plain 32-bit forms
def _plain_rotary(st):
    M, Hq, Hkv, D, rot = st["M"], st["Hq"], st["Hkv"], st["D"], st["rot"]
    x = st["qkv"].float().view(M, Hq + 2 * Hkv, D)
    if st["norm"]:
        q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * st["q_gamma"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * st["k_gamma"].float()
        x = torch.cat([q, k, x[:, Hq + Hkv:]], 1)
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()       # far positions lose in 32 bits
    c = (torch.cos(angle) * st["magnitude"]).float()[:, None]
    s = (torch.sin(angle) * st["magnitude"]).float()[:, None]
    h = x[:, :Hq + Hkv]
    if st["interleaved"]:
        a, b = h[..., 0:rot:2], h[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = h[..., :rot // 2], h[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    h = torch.cat([turned, h[..., rot:]], -1)
    return torch.cat([h, x[:, Hq + Hkv:]], 1).view(M, -1).to(st["o"].dtype)


def _heads(x, Hq, Hkv, D):
    """Queries [Hkv, G, rows, D] and keys, values [Hkv, 1, rows, D] of qkv rows."""
    y = x.unflatten(-1, (Hq + 2 * Hkv, D)).transpose(0, 1)
    return y[:Hq].unflatten(0, (Hkv, -1)), y[Hq:Hq + Hkv, None], y[Hq + Hkv:, None]


def _plain_prompt(st):
    Hq, Hkv, D = st["Hq"], st["Hkv"], st["D"]
    out = torch.zeros_like(st["o"])
    at = 0
    for n in st["cu"].diff().tolist():
        if n == 0:
            continue
        q, k, v = _heads(st["qkv"][at:at + n].float(), Hq, Hkv, D)
        step = max(1, min(n, (1 << 28) // (Hq * n)))                   # query rows whose scores fit a gigabyte
        for i in range(0, n, step):
            e = min(n, i + step)
            s = torch.matmul(q[:, :, i:e], k[:, :, :e].transpose(2, 3)) * st["scale"]
            later = torch.arange(e, device="cuda")[None] > torch.arange(i, e, device="cuda")[:, None]
            s.masked_fill_(later, -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = torch.matmul(p, v[:, :, :e]) / p.sum(-1, keepdim=True)
            out[at + i:at + e] = o.flatten(0, 1).transpose(0, 1).flatten(1).to(out.dtype)
        at += n
    return out


def _plain_prefix(st):
    B, T, Hq, Hkv, D, P = st["B"], st["T"], st["Hq"], st["Hkv"], st["D"], st["prefix"]
    G, L = Hq // Hkv, st["kc"].shape[1]
    x = st["qkv"].view(B, T, Hq + 2 * Hkv, D).float()
    q = x[:, :, :Hq].unflatten(2, (Hkv, G)).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    kn, vn = x[:, :, Hq:Hq + Hkv].permute(0, 2, 1, 3), x[:, :, Hq + Hkv:].permute(0, 2, 1, 3)
    K, V = st["kc"].float().transpose(1, 2), st["vc"].float().transpose(1, 2)
    pk, pv = st["pk"][:P].float().transpose(0, 1), st["pv"][:P].float().transpose(0, 1)
    both = q.transpose(0, 1).reshape(Hkv, B * T * G, D)                # all sequences' rows over the prefix at once
    s_pre = torch.matmul(both, pk.transpose(1, 2)) * st["scale"]
    s_pre = s_pre.view(Hkv, B, T * G, P)
    s_old = torch.matmul(q, K.transpose(2, 3)) * st["scale"]
    s_old = s_old.masked_fill(torch.arange(L, device="cuda") >= st["len"][:, None, None, None], -math.inf)
    s_new = torch.matmul(q, kn.transpose(2, 3)) * st["scale"]
    j = torch.arange(T, device="cuda")
    s_new = s_new.masked_fill(j[None, :] > j.repeat_interleave(G)[:, None], -math.inf)
    m = torch.maximum(torch.maximum(s_old.amax(-1), s_new.amax(-1)), s_pre.amax(-1).transpose(0, 1))[..., None]
    p_pre = torch.exp(s_pre - m.transpose(0, 1))
    p_old, p_new = torch.exp(s_old - m), torch.exp(s_new - m)
    o = torch.matmul(p_pre.view(Hkv, B * T * G, P), pv).view(Hkv, B, T * G, D).transpose(0, 1)
    o = o + torch.matmul(p_old, V) + torch.matmul(p_new, vn)
    o = o / (p_pre.sum(-1).transpose(0, 1) + p_old.sum(-1) + p_new.sum(-1))[..., None]
    return o.reshape(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B * T, Hq * D).to(st["o"].dtype)


# ------------------------------------------------------- this repository's calls
def _own(st):
    from quantized_verification_gb300 import qv
    if st["op"] == "rotary":
        qv.qv_rotary(st["qkv"], st["positions"], st["inv_freq"], st["Hq"], st["Hkv"], out=st["o"],
                     interleaved=st["interleaved"], magnitude=st["magnitude"], q_gamma=st["q_gamma"],
                     k_gamma=st["k_gamma"], eps=EPS)
    elif st["op"] == "prompt":
        qv.qv_attention_prompt(st["qkv"], st["cu"], st["Hq"], st["Hkv"], st["scale"], st["o"])
    else:
        if "ws" not in st:                      # a program keeps one workspace for all its steps
            n = qv.qv_attention_prefix_workspace_bytes(st["B"], st["T"], st["Hq"], st["Hkv"], st["D"], st["pk"].shape[0])
            st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        qv.qv_attention_verify_prefix(st["qkv"], st["pk"], st["pv"], st["prefix_len"], st["kc"], st["vc"], st["len"],
                                      st["T"], st["Hq"], st["Hkv"], st["scale"], st["o"], st["ws"])
    return {"o": st["o"]}


def run(state):
    if own:
        return _own(state)
    return {"o": {"rotary": _plain_rotary, "prompt": _plain_prompt, "prefix": _plain_prefix}[state["op"]](state)}


# --------------------------------------------------------------------- work
def work(case):
    size = lambda n: 4 if n == "f32" else 2  # noqa: E731
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    W = (Hq + 2 * Hkv) * D
    if case["op"] == "rotary":
        return {"bytes": case["M"] * (2 * W * size(case["x"]) + 4), "flops": case["M"] * (Hq + Hkv) * D * 6}
    n = lengths(case)
    if case["op"] == "prompt":
        pairs = sum(v * (v + 1) // 2 for v in n)
        return {"bytes": sum(n) * (W * 2 + Hq * D * size(case["out"])), "flops": 4 * Hq * D * pairs}
    B, T = case["B"], case["T"]
    io = B * T * (W * 2 + Hq * D * size(case["out"]))
    return {"bytes": (case["prefix"] + sum(n)) * Hkv * D * 4 + io,
            "flops": 4 * Hq * D * T * (B * case["prefix"] + sum(n)) + 2 * Hq * D * B * T * (T + 1)}


# ------------------------------------------------------ the definition in 64 bits
def _softmax_product(q, k, v, scale, visible):
    """softmax(scale q k^T) v of one head; visible [rows, keys] or None."""
    s = (q @ k.mT) * scale
    if visible is not None:
        s = torch.where(visible, s, -math.inf)
    return torch.softmax(s, -1) @ v


def exact(case, seed):
    if case["op"] != "rotary" and work(case)["flops"] > 6e12:
        return None
    st = prepare(case, seed)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    if case["op"] == "rotary":
        M, rot = case["M"], case["rot"]
        x = st["qkv"].double().reshape(M, -1, D)
        o = x.clone()
        for first, count, gamma in ((0, Hq, st["q_gamma"]), (Hq, Hkv, st["k_gamma"])):
            y = x[:, first:first + count]
            if gamma is not None:
                y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / D + EPS) * gamma.double()
            # pairs as complex numbers, turned by magnitude * e^(i angle)
            r = y[..., :rot].contiguous()
            pairs = r.reshape(M, count, rot // 2, 2) if case["interleaved"] else r.reshape(M, count, 2, rot // 2).mT
            z = torch.view_as_complex(pairs.contiguous())
            angle = st["positions"].double().outer(st["inv_freq"].double())
            z = z * torch.polar(torch.full_like(angle, st["magnitude"]), angle)[:, None]
            back = torch.view_as_real(z)
            back = back if case["interleaved"] else back.mT
            o[:, first:first + count] = torch.cat([back.reshape(M, count, rot), y[..., rot:]], -1)
        return {"o": o.view(M, -1)}
    x = st["qkv"].double()
    x = x.view(x.shape[0], -1, D)
    o = torch.zeros(x.shape[0], Hq, D, dtype=torch.float64, device="cuda")
    if case["op"] == "prompt":
        cu = st["cu"].tolist()
        for a, b in zip(cu, cu[1:]):
            for h in range(Hq):
                k, v = x[a:b, Hq + h // G], x[a:b, Hq + Hkv + h // G]
                for i in range(a, b, 2000):
                    e = min(b, i + 2000)
                    see = torch.ones(e - i, e - a, dtype=torch.bool, device="cuda").tril(i - a)
                    o[i:e, h] = _softmax_product(x[i:e, h], k[:e - a], v[:e - a], st["scale"], see)
        return {"o": o.view(-1, Hq * D)}
    T, P = case["T"], case["prefix"]
    for h in range(Hkv):
        pk, pv = st["pk"][:P, h].double(), st["pv"][:P, h].double()
        for b in range(case["B"]):
            n = int(st["len"][b])
            r = slice(b * T, b * T + T)
            k = torch.cat([pk, st["kc"][b, :n, h].double(), x[r, Hq + h]])
            v = torch.cat([pv, st["vc"][b, :n, h].double(), x[r, Hq + Hkv + h]])
            see = torch.ones(T, P + n + T, dtype=torch.bool, device="cuda").tril(P + n)
            o[r, h * G:(h + 1) * G] = _softmax_product(x[r, h * G:(h + 1) * G].transpose(0, 1), k, v, st["scale"],
                                                       see).transpose(0, 1)
    return {"o": o.view(-1, Hq * D)}
