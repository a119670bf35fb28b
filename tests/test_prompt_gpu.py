"""qv_attention_prompt against its definition in 64 bits."""
import pytest
import torch

import prompt_ref as ref
from gpu_util import require_gpu
from quantized_verification_gb300 import qv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    require_gpu()


def rows(M, Hq, Hkv, D, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, (Hq + 2 * Hkv) * D, generator=g, device="cuda")
    x[:, Hq * D:(Hq + Hkv) * D:61] *= 4
    return x.to(torch.bfloat16)


def cumulated(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def run(x, cu, Hq, Hkv, D, scale, dtype, fill=7.0, **kw):
    out = torch.full((x.shape[0], Hq * D), fill, dtype=dtype, device="cuda")
    qv.qv_attention_prompt(x, torch.tensor(cu, dtype=torch.int32, device="cuda"), Hq, Hkv, scale, out, **kw)
    return out


def check(out, x, cu, Hq, Hkv, scale, fill=7.0):
    o, a = ref.prompt(x, cu, Hq, Hkv, scale)
    got = out.double().view(o.shape)
    inside = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    inside[cu[0]:cu[-1]] = True
    assert (got[~inside] == fill).all(), "a row of no sequence was written"
    d = (got - o).abs()[inside]
    assert (d <= ref.bound(o, a, out.dtype)[inside]).all(), f"off by {float(d.max())}"
    if inside.any():
        rel = float((got - o)[inside].norm() / o[inside].norm())
        assert rel <= ref.norm_bound(out.dtype), rel
    assert qv.qv_device_error() == 0


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 127, 128, 129, 300])
def test_one_short_prompt(n, dtype):
    x = rows(n, 8, 2, 128, n)
    check(run(x, [0, n], 8, 2, 128, 0.09, dtype), x, [0, n], 8, 2, 0.09)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (6, 2), (20, 4), (32, 4), (14, 2), (71, 1), (128, 1), (16, 16)])
def test_head_layouts(Hq, Hkv, D, dtype):
    lens = [70, 1, 200, 0, 37]
    cu = cumulated(lens)
    x = rows(cu[-1], Hq, Hkv, D, Hq)
    check(run(x, cu, Hq, Hkv, D, D ** -0.5, dtype), x, cu, Hq, Hkv, D ** -0.5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1000, 1300, 2100])
def test_many_rows_take_two_tiles(n, D, dtype):
    # above two tiles an SM a thread block takes two, several steps, sums flushed for fp32
    Hq, Hkv = 32, 8
    x = rows(n, Hq, Hkv, D, n)
    check(run(x, [0, n], Hq, Hkv, D, D ** -0.5, dtype), x, [0, n], Hq, Hkv, D ** -0.5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_prompt_one_head(dtype):
    n = 4500
    x = rows(n, 1, 1, 128, 3)
    check(run(x, [0, n], 1, 1, 128, 0.088, dtype), x, [0, n], 1, 1, 0.088)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (64, 16)])
@pytest.mark.parametrize("lens", [[5, 5, 5, 5, 900, 3, 3], [0, 0, 1, 0, 640, 0], [129] * 9, [1] * 300, [64, 64, 127, 1, 65, 500]])
def test_packed_prompts(lens, Hq, Hkv, dtype):
    cu = cumulated(lens)
    x = rows(cu[-1], Hq, Hkv, 128, len(lens))
    check(run(x, cu, Hq, Hkv, 128, 0.1, dtype), x, cu, Hq, Hkv, 0.1)


def test_thousands_of_sequences():
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 4, (3000,), generator=g).tolist()
    cu = cumulated(lens)
    x = rows(cu[-1], 2, 1, 64, 4)
    check(run(x, cu, 2, 1, 64, 0.125, torch.float32), x, cu, 2, 1, 0.125)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hq,Hkv,lens", [(8, 2, [100, 30]), (64, 16, [300, 333])])
def test_rows_of_no_sequence_may_hold_anything(Hq, Hkv, lens, dtype):
    cu = cumulated(lens, first=45)
    M = cu[-1] + 77
    x = rows(M, Hq, Hkv, 128, 5)
    x[:45], x[cu[-1]:] = float("nan"), float("inf")
    check(run(x, cu, Hq, Hkv, 128, 0.1, dtype), x, cu, Hq, Hkv, 0.1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hq,Hkv,lens", [(8, 2, [150, 60, 40]), (64, 16, [300, 333])])
@pytest.mark.parametrize("what", ["key", "value", "both"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_reaches_only_rows_that_see_it(Hq, Hkv, lens, what, bad, dtype):
    D, cu = 128, cumulated(lens)
    x = rows(cu[-1], Hq, Hkv, D, 6)
    clean = x.clone()
    at = cu[1] - 23                                             # in the first sequence, with rows behind it
    y = x.view(cu[-1], Hq + 2 * Hkv, D)
    if what != "value":
        y[at, Hq:Hq + Hkv] = bad
    if what != "key":
        y[at, Hq + Hkv:, 5] = bad
    out = run(x, cu, Hq, Hkv, D, 0.1, dtype)
    good = run(clean, cu, Hq, Hkv, D, 0.1, dtype)
    sees = torch.zeros(cu[-1], dtype=torch.bool, device="cuda")
    sees[at:cu[1]] = True
    check(out[~sees], clean[~sees], cumulated([at] + lens[1:]), Hq, Hkv, 0.1)
    if what != "key":
        assert not torch.isfinite(out[sees].view(-1, Hq, D)[:, :, 5]).any()
    assert torch.isfinite(good).all()


def test_scores_far_apart_and_masked_rows():
    # a running maximum that rises step by step by more than it may lag, then falls far below
    n, D = 700, 64
    x = rows(n, 1, 1, D, 8)
    y = x.view(n, 3, D)
    y[:, 0] = 0
    y[:, 0, 0] = 8
    y[:, 1] = 0
    y[:, 1, 0] = torch.cat([torch.linspace(-400, 400, 600), torch.full((100,), -2000.0)]).to("cuda")
    for dtype in DTYPES:
        out = run(x, [0, n], 1, 1, D, 0.125, dtype)
        o, a = ref.prompt(x, [0, n], 1, 1, 0.125)
        # scores up to 2000: binary32 holds them to 2^-24 of their size, and so the probabilities
        extra = 2000 * 2.0 ** -22 * a
        assert ((out.double().view(o.shape) - o).abs() <= ref.bound(o, a, dtype) + extra).all()


def test_sums_of_one_sign_do_not_drift():
    n, D = 6000, 64
    x = rows(n, 1, 1, D, 13)
    x[:, :2 * D] *= 0.25
    x[:, 2 * D:] = x[:, 2 * D:].abs()
    out = run(x, [0, n], 1, 1, D, 0.125, torch.float32)
    o, a = ref.prompt(x, [0, n], 1, 1, 0.125)
    # (without the rounded additions between them the sums would be off by 1e-5)
    assert float((out.double().view(o.shape) - o).norm() / o.norm()) <= ref.norm_bound(out.dtype)


def test_views_streams_graphs_and_repeats():
    Hq, Hkv, D, n = 8, 2, 128, 333
    big = rows(n + 40, Hq, Hkv, D, 9)
    x = big[17:17 + n]                                          # rows of a larger buffer
    cu = [0, 100, n]
    first = run(x, cu, Hq, Hkv, D, 0.1, torch.float32)
    check(first, x, cu, Hq, Hkv, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run(x, cu, Hq, Hkv, D, 0.1, torch.float32)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, second)
    # lengths are read on the device: one captured graph serves other lengths
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qv.qv_attention_prompt(x, c, Hq, Hkv, 0.1, out)
    graph.replay()
    assert torch.equal(out, first)
    c.copy_(torch.tensor([0, 7, 320], dtype=torch.int32))
    out.fill_(7.0)
    graph.replay()
    check(out, x, [0, 7, 320], Hq, Hkv, 0.1)


def test_two_calls_at_once_and_two_graphs():
    # no workspace: calls on two streams, and graphs replayed at once, do not touch each other
    Hq, Hkv, D = 16, 4, 128
    xs = [rows(n, Hq, Hkv, D, n) for n in (500, 777)]
    cus = [torch.tensor([0, 123, n], dtype=torch.int32, device="cuda") for n in (500, 777)]
    outs = [torch.zeros(x.shape[0], Hq * D, device="cuda") for x in xs]
    want = [run(x, c.tolist(), Hq, Hkv, D, 0.1, torch.float32) for x, c in zip(xs, cus)]
    streams = [torch.cuda.Stream() for _ in xs]
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                qv.qv_attention_prompt(xs[k], cus[k], Hq, Hkv, 0.1, outs[k])
        graphs.append(g)
    torch.cuda.synchronize()
    for k in range(2):
        with torch.cuda.stream(streams[k]):
            for _ in range(4):
                qv.qv_attention_prompt(xs[k], cus[k], Hq, Hkv, 0.1, outs[k], stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(outs[k], want[k])
        outs[k].zero_()
    torch.cuda.synchronize()
    for k in range(2):
        with torch.cuda.stream(streams[k]):
            graphs[k].replay()
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(outs[k], want[k])
    assert qv.qv_device_error() == 0


def test_results_are_the_same_from_call_to_call():
    Hq, Hkv, D, n = 32, 8, 128, 2500
    x = rows(n, Hq, Hkv, D, 14)
    for dtype in DTYPES:
        first = run(x, [0, 900, n], Hq, Hkv, D, 0.09, dtype)
        for _ in range(5):
            assert torch.equal(run(x, [0, 900, n], Hq, Hkv, D, 0.09, dtype), first)


def test_bounds_outside_the_buffer_are_clamped():
    Hq, Hkv, D, n = 4, 2, 64, 90
    x = rows(n, Hq, Hkv, D, 10)
    out = run(x, [-5, 40, 2000], Hq, Hkv, D, 0.1, torch.float32)
    check(out, x, [0, 40, n], Hq, Hkv, 0.1)


@pytest.mark.parametrize("cu", [[90, 40, 10, 0], [50, 10, 90, 3], [2 ** 31 - 1, -(2 ** 31), 5, 60]])
def test_bounds_that_fall_stay_in_the_buffers(cu):
    # unspecified outputs, but nothing outside the buffers is touched and the next call is right
    Hq, Hkv, D, n = 4, 2, 64, 90
    x = rows(n, Hq, Hkv, D, 11)
    guard = torch.full((3 * n, Hq * D), 7.0, device="cuda")
    qv.qv_attention_prompt(x, torch.tensor(cu, dtype=torch.int32, device="cuda"), Hq, Hkv, 0.1, guard[n:2 * n])
    assert (guard[:n] == 7.0).all() and (guard[2 * n:] == 7.0).all()
    check(run(x, [0, n], Hq, Hkv, D, 0.1, torch.float32), x, [0, n], Hq, Hkv, 0.1)


def test_refusals():
    Hq, Hkv, D, n = 4, 2, 64, 20
    x = rows(n, Hq, Hkv, D)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = torch.full((n, Hq * D), 7.0, device="cuda")
    ok = dict(qkv=x, cu_rows=cu, Hq=Hq, Hkv=Hkv, scale=0.1, out=out)
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.0)):
        with pytest.raises(qv.QVError):
            qv.qv_attention_prompt(**{**ok, **bad})
    for bad in (dict(qkv=x.float()), dict(cu_rows=cu.long()), dict(cu_rows=cu[:1]), dict(out=out[:5]), dict(qkv=x[:, :-1]),
                dict(out=out.t()), dict(cu_rows=cu.cpu())):
        with pytest.raises((ValueError, TypeError)):
            qv.qv_attention_prompt(**{**ok, **bad})
    with pytest.raises(TypeError):
        qv.qv_attention_prompt(**{**ok, "out": out.half()})
    flat = torch.zeros(x.numel() + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(qv.QVError, match="aligned"):
        qv.qv_attention_prompt(**{**ok, "qkv": flat[1:1 + x.numel()].view(x.shape)})
    with pytest.raises(qv.QVError, match="128"):
        y = torch.zeros(3, (129 + 2) * 64, dtype=torch.bfloat16, device="cuda")
        qv.qv_attention_prompt(y, cu, 129, 1, 0.1, torch.zeros(3, 129 * 64, device="cuda"))
    assert (out == 7.0).all()


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    Hq, Hkv, D = 64, 16, 128
    for n in (64, 700):
        x = rows(n, Hq, Hkv, D, 12)
        qv.qv_debug_set_slot_wait_ns(2_000_000)
        qv.qv_debug_hold_attention_loads(1)
        try:
            run(x, [0, n], Hq, Hkv, D, 0.1, torch.bfloat16)
            assert qv.qv_device_error() == qv.QV_DEVICE_ERR_FULL_WAIT
        finally:
            qv.qv_debug_hold_attention_loads(0)
            qv.qv_debug_set_slot_wait_ns(0)
        check(run(x, [0, n], Hq, Hkv, D, 0.1, torch.bfloat16), x, [0, n], Hq, Hkv, 0.1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1500], [700, 801], [2100, 3, 40]])
def test_values_that_are_not_finite_far_into_a_prompt(lens, D, dtype):
    # steps in which every row sees every key lie between those whose values are looked at; blocks of one and of two tiles
    for Hq, Hkv in ((8, 2), (32, 8)):
        cu = cumulated(lens)
        x = rows(cu[-1], Hq, Hkv, D, sum(lens))
        clean = run(x, cu, Hq, Hkv, D, 0.1, dtype)
        check(clean, x, cu, Hq, Hkv, 0.1)
        v = x.view(-1, Hq + 2 * Hkv, D)[:, Hq + Hkv:]
        for seq, n in enumerate(lens):
            for at in sorted({n - 1, n * 3 // 4, n // 2 + 1}):
                tok = cu[seq] + at
                kept = v[tok].clone()
                v[tok] = float("inf") if at % 2 else float("nan")
                out = run(x, cu, Hq, Hkv, D, 0.1, dtype)
                v[tok] = kept
                saw = torch.zeros(cu[-1], dtype=torch.bool, device="cuda")
                saw[tok:cu[seq + 1]] = True
                assert torch.equal(out[~saw], clean[~saw]) and not torch.isfinite(out[saw]).any()
    assert qv.qv_device_error() == 0
