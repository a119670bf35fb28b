"""qv_rotary against its definition in 64 bits."""
import pytest
import torch

import prompt_ref as ref
from gpu_util import require_gpu
from quantized_verification_gb300 import qv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    require_gpu()


def inputs(M, Hq, Hkv, D, rot, dtype, seed=0, norm=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(dtype)
    f, _ = qv.qv_rotary_frequencies(rot, 1e6)
    gammas = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) if norm else None for _ in range(2)]
    return x, f.cuda(), gammas


def check(got, x, pos, f, Hq, Hkv, **kw):
    want = ref.rotate(x, pos, f, Hq, Hkv, **kw)
    M, D = x.shape[0], x.shape[1] // (Hq + 2 * Hkv)
    d = (got.double() - want).abs().view(M, -1, D)
    heads = Hq + Hkv
    assert torch.equal(got.view(M, -1, D)[:, heads:], x.view(M, -1, D)[:, heads:]), "a value head changed"
    # one rounding of the result; before it a value of the pair is off by the angle (2e-7), the cosine's, the norm's
    # and three operations' roundings, all of the pair's size: 16 steps of 2^-24
    y = x.double()
    if kw.get("q_gamma") is not None:
        big = ref.rotate(x, torch.zeros_like(pos), f, Hq, Hkv, **{**kw, "magnitude": 1.0})
        y = big
    pair = y.view(M, -1, D)[:, :heads].abs().amax(-1, keepdim=True) * 1.5 * max(abs(kw.get("magnitude", 1.0)), 1.0)
    step = torch.finfo(x.dtype).eps / 2
    tol = step * want.view(M, -1, D)[:, :heads].abs() * 1.01 + 2.0 ** -20 * pair
    assert (d[:, :heads] <= tol).all(), float((d[:, :heads] - tol).max())


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (128, 64), (64, 24), (96, 32), (128, 8), (8, 8), (256, 256), (80, 80),
                                   (24, 16), (136, 136)])
def test_layouts(D, rot, norm, interleaved, dtype):
    M, Hq, Hkv = 7, 6, 2
    x, f, (qg, kg) = inputs(M, Hq, Hkv, D, rot, dtype, D + rot, norm)
    pos = torch.tensor([0, 1, 5, 77, 4095, 131071, 1000003], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 9.0)
    before = x.clone()
    kw = dict(interleaved=interleaved, magnitude=1.25, q_gamma=qg, k_gamma=kg)
    qv.qv_rotary(x, pos, f, Hq, Hkv, out=out, **kw)
    assert torch.equal(x, before)
    check(out, x, pos, f, Hq, Hkv, **kw)
    qv.qv_rotary(x, pos, f, Hq, Hkv, **kw)                      # in place: the same bits
    assert torch.equal(x, out)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [1, 2, 3, 5, 611, 1215, 1216, 2043])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (1, 1), (0, 3), (5, 0), (71, 1)])
def test_rows_and_heads(M, Hq, Hkv, dtype):
    x, f, (qg, kg) = inputs(M, Hq, Hkv, 64, 64, dtype, M, norm=True)
    pos = torch.arange(M, dtype=torch.int32, device="cuda") * 17 + 3
    out = torch.full_like(x, 9.0)
    qv.qv_rotary(x, pos, f, Hq, Hkv, out=out, q_gamma=qg, k_gamma=kg, eps=1e-5)
    check(out, x, pos, f, Hq, Hkv, q_gamma=qg, k_gamma=kg, eps=1e-5)


def test_far_and_negative_positions():
    Hq, Hkv, D = 2, 1, 64
    pos = torch.tensor([2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 12345, -1, -77777777, 0], dtype=torch.int32, device="cuda")
    x, f, _ = inputs(6, Hq, Hkv, D, D, torch.float32)
    y = x.clone()
    qv.qv_rotary(y, pos, f, Hq, Hkv)
    # the reference's angle in 64 bits: 2^31 * 2^-53 = 2.4e-7 of its own
    check(y, x, pos, f, Hq, Hkv)
    qv.qv_rotary(y, torch.where(pos == -(2 ** 31), pos, -pos), f, Hq, Hkv)
    back = (y - x).abs()[[0, 2, 3, 4, 5]]
    # turned forth and back: two rotations' errors
    assert float(back.max()) <= 2 * 2.0 ** -20 * 1.5 * float(x.abs().max())


@pytest.mark.parametrize("freq", [0.0, 1.0, 6.5, 1000.25, 2.0 ** -130, -0.75, 2.0 ** -60])
def test_any_frequency(freq):
    x, _, _ = inputs(4, 1, 1, 16, 16, torch.float32)
    f = torch.full((8,), freq, device="cuda")
    pos = torch.tensor([1, 3, 100, 65537], dtype=torch.int32, device="cuda")
    y = x.clone()
    qv.qv_rotary(y, pos, f, 1, 1)
    check(y, x, pos, f, 1, 1)


def test_norm_of_small_large_and_zero_heads():
    x, f, (qg, kg) = inputs(4, 2, 1, 64, 64, torch.float32, norm=True)
    x[0] *= 1e-12
    x[1] *= 1e12
    x[2] = 0
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    y = x.clone()
    qv.qv_rotary(y, pos, f, 2, 1, q_gamma=qg, k_gamma=kg)
    check(y, x, pos, f, 2, 1, q_gamma=qg, k_gamma=kg)
    assert (y[2] == 0).all()


def test_streams_and_graphs():
    Hq, Hkv, D, M = 8, 2, 128, 40
    x, f, _ = inputs(M, Hq, Hkv, D, D, torch.bfloat16)
    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qv.qv_rotary(x, pos, f, Hq, Hkv, out=out)
    torch.cuda.current_stream().wait_stream(side)
    check(out, x, pos, f, Hq, Hkv)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qv.qv_rotary(x, pos, f, Hq, Hkv, out=out)
    pos += 1000
    g.replay()
    check(out, x, pos, f, Hq, Hkv)


def test_refusals():
    x, f, (qg, kg) = inputs(4, 2, 1, 64, 64, torch.bfloat16, norm=True)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    before = x.clone()
    for bad in (dict(magnitude=float("nan")), dict(q_gamma=qg), dict(q_gamma=qg, k_gamma=kg, eps=-1.0),
                dict(inv_freq=torch.ones(36, device="cuda")), dict(inv_freq=torch.ones(6, device="cuda")),
                dict(inv_freq=torch.ones(0, device="cuda"))):
        with pytest.raises(qv.QVError):
            qv.qv_rotary(**{**dict(qkv=x, positions=pos, inv_freq=f, Hq=2, Hkv=1), **bad})
    for bad in (dict(positions=pos.long()), dict(positions=pos[:2]), dict(inv_freq=f.double()), dict(out=x.float()),
                dict(q_gamma=qg.float(), k_gamma=kg), dict(Hkv=2), dict(out=torch.empty(4, 256, device="cuda").t())):
        with pytest.raises((ValueError, TypeError)):
            qv.qv_rotary(**{**dict(qkv=x, positions=pos, inv_freq=f, Hq=2, Hkv=1), **bad})
    buf = torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(qv.QVError, match="overlap"):
        qv.qv_rotary(buf[:4], pos, f, 2, 1, out=buf[1:5])
    assert torch.equal(x, before)
