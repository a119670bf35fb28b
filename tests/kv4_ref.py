"""Plain references of the 4-bit KV cache and of the token log probabilities
(numpy, 64 bits), written from the definitions in include/qv.h; used by the
CPU pins and by the GPU tests. Caches are numpy uint8 [pages, Hkv, 34 * D]."""
import numpy as np

BLOCK, GROUP = 32, 32


def scale_of(byte):
    b = np.asarray(byte, dtype=np.int64)
    return (1.0 + (b & 7) / 8.0) * 2.0 ** ((b >> 3) - 15.0)


ALL_SCALES = scale_of(np.arange(256))


def quantize(x):
    """Rows x [..., D] -> (codes int [..., D], scale bytes [..., D/32])."""
    x = np.asarray(x, dtype=np.float32)
    big = np.float32(np.finfo(np.float32).max)
    x = np.clip(np.where(np.isnan(x), np.float32(0), x), -big, big)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    t = (np.abs(g).max(-1) / np.float32(7)).astype(np.float64)
    # the nearest of all 256 scales; a tie between neighbours goes to the even byte
    hi = np.clip(np.searchsorted(ALL_SCALES, t), 1, 255)
    lo = hi - 1
    dl, dh = t - ALL_SCALES[lo], ALL_SCALES[hi] - t
    byte = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    s = ALL_SCALES[byte].astype(np.float32)
    q = np.clip(np.rint(g / s[..., None]), -7, 7).astype(np.int64)      # binary32 quotient, half to even
    return q.reshape(x.shape), byte.astype(np.uint8)


def values(q, byte):
    g = q.reshape(*q.shape[:-1], q.shape[-1] // GROUP, GROUP)
    return (g * scale_of(byte)[..., None]).reshape(q.shape)


def parts(cache, D):
    """Views of the four fields: [pages, Hkv, 32, row bytes]."""
    P, H = cache.shape[:2]
    cut = [0, 16 * D, 32 * D, 33 * D, 34 * D]
    return [cache[:, :, a:b].reshape(P, H, BLOCK, (b - a) // BLOCK) for a, b in zip(cut, cut[1:])]


def pack(q):
    n = (q & 15).astype(np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def unpack(c):
    c = c.astype(np.int64)
    q = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], c.shape[-1] * 2)
    return q - 16 * (q >= 8)


def place(b, pos, NB, pages, table):
    """(page, slot) of a position, or None."""
    if pos < 0 or pos >= NB * BLOCK:
        return None
    page = b * NB + pos // BLOCK if table is None else int(table[b, pos // BLOCK])
    return (page, pos % BLOCK) if 0 <= page < pages else None


def write(cache, qkv, start, T, Hq, Hkv, D, NB, table=None, count=None):
    """The cache after qv_kv4_write, a copy."""
    cache = cache.copy()
    pages = cache.shape[0]
    for b in range(len(start)):
        n = T if count is None else min(T, int(count[b]))
        for j in range(max(n, 0)):
            at = place(b, int(start[b]) + j, NB, pages, table)
            if at is None:
                continue
            row = qkv[b * T + j]
            for f, o in ((0, Hq * D), (1, (Hq + Hkv) * D)):
                q, byte = quantize(row[o: o + Hkv * D].reshape(Hkv, D))
                c0, s0 = f * 16 * D + at[1] * (D // 2), (32 + f) * D + at[1] * (D // GROUP)
                cache[at[0], :, c0: c0 + D // 2] = pack(q)
                cache[at[0], :, s0: s0 + D // GROUP] = byte
    return cache


def read(cache, start, T, D, NB, k_out, v_out, table=None, count=None):
    """(k, v) [B, T, Hkv, D] float64 after qv_kv4_read into copies of k_out, v_out."""
    k, v = k_out.astype(np.float64), v_out.astype(np.float64)
    kc, vc, ks, vs = parts(cache, D)
    for b in range(len(start)):
        n = T if count is None else min(T, int(count[b]))
        for j in range(max(n, 0)):
            at = place(b, int(start[b]) + j, NB, cache.shape[0], table)
            if at is not None:
                p, s = at
                k[b, j] = values(unpack(kc[p, :, s]), ks[p, :, s])
                v[b, j] = values(unpack(vc[p, :, s]), vs[p, :, s])
    return k, v


def attend(qkv, cache, lens, T, Hq, Hkv, D, NB, scale, table=None):
    """Attention in 64 bits: (out [B*T, Hq*D], the largest |v| seen, the largest scale * sum |q||k| of a score)."""
    B, G = len(lens), Hq // Hkv
    x = np.asarray(qkv, dtype=np.float64).reshape(B, T, Hq + 2 * Hkv, D)
    kc, vc, ks, vs = parts(cache, D)
    out = np.zeros((B, T, Hq, D))
    vmax, smax = 0.0, 0.0
    for b in range(B):
        n = min(max(int(lens[b]), 0), NB * BLOCK)
        at = [place(b, p, NB, cache.shape[0], table) for p in range(n)]
        at = np.array([a for a in at if a is not None], dtype=np.int64).reshape(-1, 2)
        for h in range(Hkv):
            K = values(unpack(kc[at[:, 0], h, at[:, 1]]), ks[at[:, 0], h, at[:, 1]])
            V = values(unpack(vc[at[:, 0], h, at[:, 1]]), vs[at[:, 0], h, at[:, 1]])
            for j in range(T):
                Kj = np.concatenate([K, x[b, : j + 1, Hq + h]])
                Vj = np.concatenate([V, x[b, : j + 1, Hq + Hkv + h]])
                q = x[b, j, h * G:(h + 1) * G]
                with np.errstate(all="ignore"):
                    s = scale * (q @ Kj.T)
                    p = np.exp(s - s.max(1, keepdims=True))
                    out[b, j, h * G:(h + 1) * G] = (p / p.sum(1, keepdims=True)) @ Vj
                    vmax = max(vmax, float(np.nanmax(np.abs(np.where(np.isfinite(Vj), Vj, 0)))))
                    smax = max(smax, float(np.nanmax(np.where(np.isfinite(s), scale * (np.abs(q) @ np.abs(Kj.T)), 0))))
    return out.reshape(B * T, Hq * D), vmax, smax


def logprobs(x, tokens, K):
    """(logprob, entropy, top tokens, top logprobs) in 64 bits; rows with NaN or +inf are not handled here."""
    x = np.asarray(x, dtype=np.float64)
    M, V = x.shape
    lp, ent = np.zeros(M), np.zeros(M)
    tt, tl = np.zeros((M, K), dtype=np.int64), np.zeros((M, K))
    for r in range(M):
        m = x[r].max()
        with np.errstate(divide="ignore", invalid="ignore"):
            z = x[r] - m if np.isfinite(m) else x[r]
            lse = np.log(np.exp(z).sum()) if np.isfinite(m) else 0.0
            l = z - lse
            p = np.exp(l)
            ent[r] = -np.where(p > 0, p * np.where(p > 0, l, 0), 0).sum()
        lp[r] = l[tokens[r]] if 0 <= tokens[r] < V else 0.0
        order = np.lexsort((np.arange(V), -x[r]))[:K]          # by value, then by the lower index
        tt[r], tl[r] = order, l[order]
    return lp, ent, tt, tl
