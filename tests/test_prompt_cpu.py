"""Host side of rotary positions, prompt attention and prefix attention: refusals before any device work, and the
frequency tables. No GPU."""
import ctypes
import math

import pytest
import torch

from quantized_verification_gb300 import build, qv

build.build()
P = ctypes.c_void_p
FAKE = 4096                                     # never dereferenced: every call here is refused


def status(name, *args):
    return getattr(qv.load(), name)(*args)


def prompt(B=1, M=4, Hq=4, Hkv=2, D=64, scale=0.1, out_dtype=0, qkv=FAKE, cu=FAKE, out=FAKE):
    return status("qv_attention_prompt", qkv, cu, B, M, Hq, Hkv, D, scale, out, out_dtype, None)


@pytest.mark.parametrize("kw", [dict(B=0), dict(M=0), dict(M=2 ** 24 + 1), dict(Hq=3), dict(Hq=0), dict(Hkv=0), dict(D=96),
                                dict(Hq=129, Hkv=1), dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf),
                                dict(out_dtype=2), dict(qkv=None), dict(cu=None), dict(out=None), dict(qkv=FAKE + 8),
                                dict(out=FAKE + 8), dict(cu=FAKE + 2), dict(out=FAKE + 64), dict(out=FAKE - 16)])
def test_prompt_refusals(kw):
    assert prompt(**kw) == qv.QV_ERR_INVALID_ARG
    assert qv.load().qv_last_error()


def test_prompt_too_many_blocks():
    assert prompt(M=2 ** 24, Hq=65535, Hkv=65535, out=2 ** 50) == qv.QV_ERR_UNSUPPORTED


def prefix(B=1, T=1, Hq=4, Hkv=2, D=64, Pm=10, Lmax=5, scale=0.1, out_dtype=0, n=FAKE, kc=FAKE, pk=FAKE, out=FAKE):
    return status("qv_attention_verify_prefix", FAKE, pk, FAKE, n, Pm, kc, FAKE, FAKE, B, T, Hq, Hkv, D, Lmax, scale, out,
                  out_dtype, FAKE, 1 << 30, None)


@pytest.mark.parametrize("kw", [dict(B=0), dict(T=0), dict(T=65), dict(Hq=3), dict(D=32), dict(Pm=0), dict(Pm=2 ** 24 + 1),
                                dict(Lmax=-1), dict(scale=0.0), dict(scale=math.nan), dict(out_dtype=3), dict(n=None),
                                dict(kc=None), dict(pk=None), dict(pk=FAKE + 2), dict(out=None), dict(out=FAKE + 4), dict(out=FAKE + 16)])
def test_prefix_refusals(kw):
    assert prefix(**kw) == qv.QV_ERR_INVALID_ARG


def rotary(M=2, Hq=2, Hkv=1, D=64, rot=64, mag=1.0, eps=1e-6, dtype=1, x=FAKE, out=FAKE, qg=None, kg=None, f=FAKE, pos=FAKE):
    return status("qv_rotary", x, dtype, pos, f, M, Hq, Hkv, D, rot, 0, mag, qg, kg, eps, out, None)


@pytest.mark.parametrize("kw", [dict(M=0), dict(M=2 ** 24 + 1), dict(Hq=0, Hkv=0), dict(Hq=-1), dict(D=4), dict(D=60),
                                dict(D=264), dict(rot=0), dict(rot=72), dict(rot=12), dict(mag=math.nan), dict(mag=math.inf),
                                dict(qg=FAKE), dict(qg=FAKE, kg=FAKE, eps=-1.0), dict(dtype=2), dict(x=None), dict(out=None),
                                dict(f=None), dict(pos=None), dict(x=FAKE + 8), dict(out=FAKE + 64), dict(f=FAKE + 1)])
def test_rotary_refusals(kw):
    assert rotary(**kw) == qv.QV_ERR_INVALID_ARG


def close(a, b):
    return all(abs(x - y) <= 2.0 ** -23 * abs(y) for x, y in zip(a.tolist(), b)) and len(a) == len(b)


def test_frequencies():
    rot, base = 64, 10000.0
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]
    f, m = qv.qv_rotary_frequencies(rot, base)
    assert f.dtype == torch.float32 and close(f, plain) and m == 1.0
    f, m = qv.qv_rotary_frequencies(rot, base, qv.QV_ROTARY_LINEAR, factor=8)
    assert close(f, [v / 8 for v in plain]) and m == 1.0
    f, m = qv.qv_rotary_frequencies(rot, base, qv.QV_ROTARY_BASE, factor=4)
    # the slowest pair is slowed by the whole factor, the fastest not at all
    assert f[0] == 1.0 and abs(float(f[-1]) * 4 / plain[-1] - 1) < 1e-6 and m == 1.0
    f, m = qv.qv_rotary_frequencies(rot, base, qv.QV_ROTARY_PARTS, factor=4, trained_length=4096, fast_turns=32, slow_turns=1)
    want = []
    for v in plain:
        turns = 4096 * v / (2 * math.pi)
        keep = 1.0 if turns >= 32 else 0.0 if turns <= 1 else (turns - 1) / 31
        want.append(v * keep + v / 4 * (1 - keep))
    assert close(f, want) and abs(m - (0.1 * math.log(4) + 1)) < 1e-6
    assert f[0] == 1.0 and abs(float(f[-1]) * 4 / plain[-1] - 1) < 1e-6
    assert close(qv.qv_rotary_frequencies(2, base)[0], [1.0])


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(rot=258), dict(base=1.0), dict(base=math.nan),
                                dict(scaling=4), dict(scaling=1, factor=0.5), dict(scaling=1, factor=math.nan),
                                dict(scaling=3, factor=2, trained_length=0), dict(scaling=3, factor=2, trained_length=10,
                                                                                  fast_turns=1, slow_turns=1)])
def test_frequency_refusals(kw):
    with pytest.raises(qv.QVError):
        qv.qv_rotary_frequencies(**{**dict(rot=64), **kw})
