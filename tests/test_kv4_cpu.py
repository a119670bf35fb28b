"""The 4-bit cache's reference pinned by hand-worked numbers and exact rational
arithmetic, and the refusals of its entry points: no GPU needed."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import kv4_ref as ref
from exact import round_to_f32


def test_scale_bytes():
    assert ref.scale_of(0) == 2.0 ** -15 and ref.scale_of(255) == 122880.0 and ref.scale_of(15 * 8) == 1.0
    assert ref.scale_of(15 * 8 + 3) == 1.375
    s = ref.ALL_SCALES
    assert np.all(s[1:] > s[:-1])
    # the kernels' decoding: the byte in place in a binary32 pattern, and doubled in a bf16 pair
    b = np.arange(256, dtype=np.uint32)
    assert np.array_equal(((b << 20) + (112 << 23)).astype(np.uint32).view(np.float32).astype(np.float64), s)
    assert np.array_equal((((b * 0x10 + 0x3800) << 16).astype(np.uint32)).view(np.float32).astype(np.float64), s)


def test_every_value_is_exact_in_16_bits():
    """q s has at most 8 significant bits (bf16), and q s 2^-6 is an f16 number, as are
    s 2^-6 and 24 s 2^-6; 24 s is a bf16 number."""
    def bf16(v):
        u = np.asarray(v, dtype=np.float32).view(np.uint32)
        return np.array_equal(np.asarray(v, dtype=np.float32).astype(np.float64), v) and not np.any(u & 0xFFFF)

    def f16(v):
        return np.array_equal(np.asarray(v).astype(np.float16).astype(np.float64), v)
    s = ref.ALL_SCALES
    for q in range(-8, 8):
        assert bf16(q * s) and f16(q * s / 64)
    assert bf16(24 * s) and f16(s / 64) and f16(24 * s / 64)


def test_worked_group():
    """max |x| = 3.5: t = 0.5, s = 0.5 (byte 112); 1.25 / 0.5 = 2.5 goes to the even 2, 1.75 / 0.5 = 3.5 to 4, -0.25 to -0."""
    x = np.zeros(32, np.float32)
    x[:5] = [3.5, 1.25, 1.75, -0.25, -3.0]
    q, b = ref.quantize(x)
    assert b.tolist() == [14 * 8] and q[:6].tolist() == [7, 2, 4, 0, -6, 0]
    assert ref.pack(q)[:3].tolist() == [0x27, 0x04, 0x0A]
    assert np.array_equal(ref.unpack(ref.pack(q)), q)


def test_scale_rounding_against_rationals():
    """The byte is the nearest scale to fl32(amax / 7); ties go to the even byte."""
    rng = np.random.default_rng(5)
    amax = np.concatenate([np.exp(rng.uniform(-14, 14, 300)), 7 * 17 / 16 * 2.0 ** np.arange(-5, 5),
                           7 * 19 / 16 * 2.0 ** np.arange(-5, 5), [0.0, 1e-30, 7 * 122880.0, 1e30, 3e38]]).astype(np.float32)
    for a in amax:
        x = np.zeros(32, np.float32)
        x[3] = -a
        q, b = ref.quantize(x)
        t = round_to_f32(Fraction(float(a)) / 7)
        dist = [abs(Fraction(float(t)) - Fraction(float(s))) for s in ref.ALL_SCALES]
        best = [i for i, d in enumerate(dist) if d == min(dist)]
        want = best[0] if len(best) == 1 else [i for i in best if i % 2 == 0][0]
        assert int(b[0]) == want
        s = float(ref.ALL_SCALES[want])
        assert abs(int(q[3])) == min(7, int(np.rint(np.float32(a) / np.float32(s))))


def test_non_finite_and_extremes():
    x = np.zeros(64, np.float32)
    x[0], x[1], x[2] = np.inf, -np.inf, 1.0
    x[32], x[33] = np.nan, 2.0
    q, b = ref.quantize(x)
    assert b[0] == 255 and q[:3].tolist() == [7, -7, 0] and q[32] == 0 and q[33] == 7


@pytest.fixture(scope="module")
def lib():
    from quantized_verification_gb300 import build, qv
    build.build()
    return qv.load()


def test_refusals_without_gpu(lib):
    from quantized_verification_gb300 import qv
    P, F = ctypes.c_void_p, ctypes.c_float
    f, bad = P(0x1000), P(0x1008)
    W = lambda **k: lib.qv_kv4_write(*[{**dict(qkv=f, dt=1, start=f, count=None, table=None, B=2, T=5, Hq=8, Hkv=2,
                                              D=64, NB=4, pages=8, cache=f, s=None), **k}[n]
                                      for n in ("qkv", "dt", "start", "count", "table", "B", "T", "Hq", "Hkv", "D", "NB",
                                                "pages", "cache", "s")])
    for k in (dict(qkv=None), dict(start=None), dict(cache=None), dict(dt=2), dict(B=0), dict(B=65536), dict(T=0),
              dict(T=1 << 24), dict(Hq=-1), dict(Hkv=0), dict(Hkv=1025), dict(D=96), dict(NB=0), dict(NB=-1),
              dict(NB=1 << 26), dict(pages=7), dict(pages=0, table=f), dict(pages=-1, table=f), dict(qkv=bad),
              dict(cache=bad), dict(start=P(0x1002)), dict(table=P(0x1002)), dict(count=P(0x1002))):
        assert W(**k) == qv.QV_ERR_INVALID_ARG, k
    assert W(pages=7) == qv.QV_ERR_INVALID_ARG and b"block table" in lib.qv_last_error()
    R = lambda **k: lib.qv_kv4_read(*[{**dict(cache=f, start=f, count=None, table=None, B=2, T=5, Hkv=2, D=64, NB=4,
                                             pages=8, k=f, v=f, dt=1, s=None), **k}[n]
                                     for n in ("cache", "start", "count", "table", "B", "T", "Hkv", "D", "NB", "pages",
                                               "k", "v", "dt", "s")])
    for k in (dict(cache=None), dict(start=None), dict(k=None), dict(v=None), dict(dt=7), dict(D=32), dict(T=0),
              dict(pages=7), dict(k=bad), dict(v=bad), dict(NB=0)):
        assert R(**k) == qv.QV_ERR_INVALID_ARG, k
    A = lambda **k: lib.qv_attention_verify_kv4(*[{**dict(qkv=f, cache=f, table=None, ln=f, B=2, T=5, Hq=8, Hkv=2, D=64,
                                                         NB=4, pages=8, scale=F(0.1), out=f, dt=0, ws=f, n=1 << 30,
                                                         s=None), **k}[n]
                                                 for n in ("qkv", "cache", "table", "ln", "B", "T", "Hq", "Hkv", "D",
                                                           "NB", "pages", "scale", "out", "dt", "ws", "n", "s")])
    for k in (dict(qkv=None), dict(cache=None), dict(ln=None), dict(out=None), dict(T=0), dict(T=257), dict(Hq=9),
              dict(Hq=1), dict(Hq=65538), dict(D=96), dict(pages=7), dict(scale=F(0.0)), dict(scale=F(-1.0)),
              dict(scale=F(float("nan"))), dict(scale=F(float("inf"))), dict(scale=F(2.5e38)), dict(out=bad), dict(qkv=bad), dict(cache=bad),
              dict(dt=3), dict(ln=P(0x1001)), dict(B=0)):
        assert A(**k) == qv.QV_ERR_INVALID_ARG, k
    T = lambda **k: lib.qv_token_logprobs(*[{**dict(x=f, dt=0, tok=f, M=2, V=10, K=3, lp=f, ent=None, tt=f, tl=f,
                                                   s=None), **k}[n]
                                           for n in ("x", "dt", "tok", "M", "V", "K", "lp", "ent", "tt", "tl", "s")])
    for k in (dict(x=None), dict(tok=None), dict(lp=None), dict(dt=2), dict(M=0), dict(M=65536), dict(V=0),
              dict(V=(1 << 24) + 1), dict(K=-1), dict(K=11), dict(K=33, V=100), dict(tt=None), dict(tl=None),
              dict(x=P(0x1002)), dict(x=P(0x1001), dt=1), dict(tok=P(0x1002)), dict(lp=P(0x1002)), dict(ent=P(0x1002))):
        assert T(**k) == qv.QV_ERR_INVALID_ARG, k


def test_binding_refusals_without_gpu():
    import torch
    from quantized_verification_gb300 import qv
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    cache = torch.zeros(8, 2, 34 * 64, dtype=torch.uint8)
    x = torch.zeros(10, 12 * 64)
    for call in (lambda: qv.qv_kv4_write(x, i32(2), cache, 5, 8, 4),                           # heads differ
                 lambda: qv.qv_kv4_write(x, i32(2), cache[:, :, :-1], 5, 8, 2),                # record size
                 lambda: qv.qv_kv4_write(x, i32(3), cache, 5, 8, 2),                           # pages not a multiple of B
                 lambda: qv.qv_kv4_write(x, torch.zeros(2), cache, 5, 8, 2),                   # dtype of start
                 lambda: qv.qv_kv4_write(x, i32(2), cache, 5, 8, 2, block_table=i32(3, 4)),    # rows of the table
                 lambda: qv.qv_kv4_write(x, i32(2), cache, 5, 8, 2, count=i32(3)),
                 lambda: qv.qv_kv4_write(x, i32(2), cache, 5, 8, 2),                           # host tensors
                 lambda: qv.qv_kv4_read(cache, i32(2), torch.zeros(2, 5, 2, 64), torch.zeros(2, 5, 2, 32)),
                 lambda: qv.qv_attention_verify_kv4(x, cache, i32(2), 5, 8, 2, 0.1, torch.zeros(10, 512), cache),
                 lambda: qv.qv_token_logprobs(torch.zeros(4, 9), i32(5), torch.zeros(4)),
                 lambda: qv.qv_token_logprobs(torch.zeros(4, 9), i32(4), torch.zeros(4), top_tokens=i32(4, 2))):
        with pytest.raises(ValueError):
            call()


def test_shortcuts_for_bf16_rows():
    """What the write kernel does for bf16 rows in place of two divisions gives the same bytes and codes: for every
    bf16 maximum, and for every significand of x, every one of s and reciprocals up to two units off."""
    f32 = np.float32
    am = (np.arange(0x7F80, dtype=np.uint32) << 16).view(f32)
    am = am[am <= 7 * 122880]

    def byte(u):
        return np.clip(((u + 0x7FFFF + ((u >> 20) & 1)) >> 20) - 896, 0, 255)
    bits = lambda t: t.view(np.uint32).astype(np.int64)  # noqa: E731
    assert np.array_equal(byte(bits(am / f32(7))), byte((bits(am * f32(1 / f32(7))) + 8) & ~15))
    for m in range(8):
        s = f32(1 + m / 8)
        for off in range(-2, 3):
            r = (np.array([f32(1) / s]).view(np.int32) + np.int32(off)).view(f32).astype(np.float64)
            for e in range(-24, 4):
                x = ((1 + np.arange(128) / 128) * 2.0 ** e).astype(f32)
                x = x[x <= 7.5 * s]
                x = np.concatenate([x, -x])
                t = (x.astype(np.float64) * r + 6144.0).astype(f32)
                q = (t.astype(np.float64) + (12582920.0 - 6144.0)).astype(f32)
                assert np.array_equal(bits(q) - 0x4B400000 - 8, np.rint(x / s).astype(np.int64)), (m, off, e)
