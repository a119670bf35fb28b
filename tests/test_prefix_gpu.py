"""qv_attention_verify_prefix against its definition in 64 bits and against qv_attention_verify."""
import pytest
import torch

import prompt_ref as ref
from gpu_util import require_gpu
from quantized_verification_gb300 import qv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    require_gpu()


def case(B, T, Hq, Hkv, D, P, Lmax, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = r(B * T, (Hq + 2 * Hkv) * D)
    x[:, Hq * D:(Hq + Hkv) * D:61] *= 4
    return [t.to(torch.bfloat16) for t in (x, r(P, Hkv, D), r(P, Hkv, D), r(B, Lmax, Hkv, D), r(B, Lmax, Hkv, D))]


def workspace(B, T, Hq, Hkv, D, P):
    n = qv.qv_attention_prefix_workspace_bytes(B, T, Hq, Hkv, D, P)
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")       # NaN bits: it needs no initial value


def run(x, pk, pv, plen, kc, vc, lens, T, Hq, Hkv, scale, dtype, ws=None):
    P, _, D = pk.shape
    out = torch.full((x.shape[0], Hq * D), 7.0, dtype=dtype, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = workspace(len(lens), T, Hq, Hkv, D, P) if ws is None else ws
    qv.qv_attention_verify_prefix(x, pk, pv, i32([plen]), kc, vc, i32(lens), T, Hq, Hkv, scale, out, ws)
    return out


def check(out, x, pk, pv, plen, kc, vc, lens, T, Hq, Hkv, scale):
    o, a = ref.verify_prefix(x, pk, pv, plen, kc, vc, lens, T, Hq, Hkv, scale)
    got = out.double().view(o.shape)
    assert ((got - o).abs() <= ref.bound(o, a, out.dtype)).all(), float((got - o).abs().max())
    rel = float((got - o).norm() / o.norm())
    assert rel <= ref.norm_bound(out.dtype), rel
    assert qv.qv_device_error() == 0


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("plen", [0, 1, 2, 127, 128, 129, 500, 517])
def test_lengths_of_the_prefix(plen, dtype):
    P = 517
    x, pk, pv, kc, vc = case(2, 1, 8, 2, 128, P, 40, plen)
    pk[plen:], pv[plen:] = float("nan"), float("inf")            # behind the length: anything
    check(run(x, pk, pv, plen, kc, vc, [40, 3], 1, 8, 2, 0.09, dtype), x, pk, pv, plen, kc, vc, [40, 3], 1, 8, 2, 0.09)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (3, 5, 32, 8), (7, 3, 12, 4), (5, 1, 32, 1), (2, 32, 2, 2), (40, 4, 16, 2),
                                        (3, 2, 14, 2), (64, 1, 8, 1), (3, 33, 3, 1), (2, 128, 2, 2), (2, 1, 128, 1)])
def test_shapes(B, T, Hq, Hkv, D, dtype):
    P, Lmax = 700, 50
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, Lmax + 1, (B,), generator=g).tolist()
    x, pk, pv, kc, vc = case(B, T, Hq, Hkv, D, P, Lmax, B)
    for b, n in enumerate(lens):
        kc[b, n:], vc[b, n:] = float("nan"), float("nan")
    s = D ** -0.5
    check(run(x, pk, pv, 690, kc, vc, lens, T, Hq, Hkv, s, dtype), x, pk, pv, 690, kc, vc, lens, T, Hq, Hkv, s)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,Hq,Hkv,Lmax", [(1, 1, 4, 1, 3000), (3, 5, 32, 8, 1500), (24, 2, 16, 8, 1000)])
def test_long_caches(B, T, Hq, Hkv, Lmax, dtype):
    P = 150
    x, pk, pv, kc, vc = case(B, T, Hq, Hkv, 128, P, Lmax, 6)
    lens = [Lmax - 131 * b % Lmax for b in range(B)]
    for b, n in enumerate(lens):
        kc[b, n:], vc[b, n:] = float("inf"), float("nan")
    check(run(x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 0.09, dtype), x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 0.09)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,Hq,Hkv", [(2, 1, 4, 1), (30, 5, 32, 8)])
def test_long_prefix(B, T, Hq, Hkv, dtype):
    P = 20011
    x, pk, pv, kc, vc = case(B, T, Hq, Hkv, 128, P, 16, 5)
    lens = [b % 17 for b in range(B)]
    check(run(x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 0.09, dtype), x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 0.09)


def test_no_cache_behind_the_prefix():
    x, pk, pv, kc, vc = case(3, 2, 8, 2, 128, 300, 0)
    for dtype in DTYPES:
        check(run(x, pk, pv, 300, kc, vc, [0, 0, 0], 2, 8, 2, 0.09, dtype), x, pk, pv, 300, kc, vc, [0, 0, 0], 2, 8, 2, 0.09)


def test_the_prefix_in_every_cache_gives_the_same():
    B, T, Hq, Hkv, D, P = 3, 5, 32, 8, 128, 600
    x, pk, pv, kc, vc = case(B, T, Hq, Hkv, D, P, 30)
    lens = [30, 0, 11]
    whole_k, whole_v = torch.zeros(B, P + 30, Hkv, D, dtype=torch.bfloat16, device="cuda"), None
    whole_v = whole_k.clone()
    for t, p, c in ((whole_k, pk, kc), (whole_v, pv, vc)):
        t[:, :P] = p
        t[:, P:] = c
    out = torch.empty(B * T, Hq * D, device="cuda")
    qv.qv_attention_verify(x, whole_k, whole_v, torch.tensor([P + n for n in lens], dtype=torch.int32, device="cuda"), T, Hq,
                           Hkv, 0.09, out)
    got = run(x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 0.09, torch.float32)
    # both within about 5e-6 of the definition
    assert float((got - out).norm() / out.norm()) <= 1e-5


def test_one_side_far_above_the_other():
    # scores over the prefix 300 above the own ones, and the other way round
    for big in (0, 1):
        x, pk, pv, kc, vc = case(2, 2, 4, 1, 64, 200, 20)
        x[:, :4 * 64], x[:, 4 * 64:5 * 64] = 1.0, -1.0 if big == 0 else 3.0
        pk[:], kc[:] = (3.0 if big == 0 else -1.0), (-1.0 if big == 0 else 3.0)
        for dtype in DTYPES:
            check(run(x, pk, pv, 200, kc, vc, [20, 0], 2, 4, 1, 1.0, dtype), x, pk, pv, 200, kc, vc, [20, 0], 2, 4, 1, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_what_is_not_finite_in_the_prefix_reaches_every_row(dtype):
    x, pk, pv, kc, vc = case(2, 1, 4, 1, 64, 300, 20)
    for at in (10, 299):
        v = pv.clone()
        v[at, 0, 3] = float("inf")
        out = run(x, pk, v, 300, kc, vc, [20, 0], 1, 4, 1, 0.1, dtype)
        assert not torch.isfinite(out.view(2, 4, 64)[:, :, 3]).any()
        out = run(x, pk, v, at, kc, vc, [20, 0], 1, 4, 1, 0.1, dtype)
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [3, 100])                          # few rows and many: two merges
def test_what_is_not_finite_in_one_cache_or_token_stays_with_those_that_see_it(B, dtype):
    T, Hq, Hkv, D, P = 3, 8, 2, 128, 200
    x, pk, pv, kc, vc = case(B, T, Hq, Hkv, D, P, 30)
    lens = [30, 11, 0] + [5] * (B - 3)
    vc[1, 10, :, 7] = float("nan")
    x.view(B, T, Hq + 2 * Hkv, D)[2, 1, Hq:] = float("inf")        # the middle token of the last sequence
    out = run(x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 0.1, dtype).view(B, T, Hq, D)
    assert not torch.isfinite(out[1, :, :, 7]).any() and not torch.isfinite(out[2, 1:]).any()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2, 0]).all() and torch.isfinite(out[3:]).all()


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    for B, T, Hq, Hkv in ((2, 1, 8, 2), (20, 5, 32, 8)):
        x, pk, pv, kc, vc = case(B, T, Hq, Hkv, 128, 300, 20)
        args = (x, pk, pv, 300, kc, vc, [b % 21 for b in range(B)], T, Hq, Hkv, 0.1)
        qv.qv_debug_set_slot_wait_ns(2_000_000)
        qv.qv_debug_hold_attention_loads(1)
        try:
            run(*args, torch.float32)
            assert qv.qv_device_error() == qv.QV_DEVICE_ERR_FULL_WAIT
        finally:
            qv.qv_debug_hold_attention_loads(0)
            qv.qv_debug_set_slot_wait_ns(0)
        check(run(*args, torch.float32), *args)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [2, 150])
def test_scores_of_minus_infinity_on_one_side(B, dtype):
    # own keys that count for nothing beside a prefix, and a prefix that counts for nothing beside own keys
    T, Hq, Hkv, D, P = 1, 16, 4, 64, 300
    for own in (True, False):
        x, pk, pv, kc, vc = case(B, T, Hq, Hkv, D, P, 4)
        x[:, : Hq * D] = x[:, : Hq * D].abs() + 0.25             # positive queries
        if own:
            x[:, Hq * D: (Hq + Hkv) * D], kc[:] = float("-inf"), float("-inf")
        else:
            pk[:] = float("-inf")
        lens = [b % 5 for b in range(B)]
        check(run(x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 0.1, dtype), x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 0.1)


def test_lengths_outside_are_clamped_and_graphs_read_them():
    B, T, Hq, Hkv, D, P = 2, 1, 8, 2, 128, 200
    x, pk, pv, kc, vc = case(B, T, Hq, Hkv, D, P, 20)
    n, lens = torch.tensor([1000], dtype=torch.int32, device="cuda"), torch.tensor([5, 99], dtype=torch.int32, device="cuda")
    out, ws = torch.zeros(B * T, Hq * D, device="cuda"), workspace(B, T, Hq, Hkv, D, P)
    call = lambda: qv.qv_attention_verify_prefix(x, pk, pv, n, kc, vc, lens, T, Hq, Hkv, 0.1, out, ws)  # noqa: E731
    call()
    check(out, x, pk, pv, P, kc, vc, [5, 20], T, Hq, Hkv, 0.1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for plen in (-3, 0, 130):
        n.fill_(plen)
        g.replay()
        check(out, x, pk, pv, max(plen, 0), kc, vc, [5, 20], T, Hq, Hkv, 0.1)


def test_one_workspace_for_shapes_it_is_large_enough_for():
    ws = workspace(8, 4, 32, 8, 128, 3000)
    for B, T, Hq, Hkv, D, P in ((8, 4, 32, 8, 128, 3000), (2, 1, 8, 2, 64, 100), (5, 3, 8, 8, 128, 1000)):
        assert qv.qv_attention_prefix_workspace_bytes(B, T, Hq, Hkv, D, P) <= ws.numel()
        x, pk, pv, kc, vc = case(B, T, Hq, Hkv, D, P, 9)
        lens = [b % 10 for b in range(B)]
        check(run(x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 0.1, torch.float32, ws), x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, 0.1)


def test_refusals():
    B, T, Hq, Hkv, D, P = 2, 2, 8, 2, 64, 100
    x, pk, pv, kc, vc = case(B, T, Hq, Hkv, D, P, 9)
    n, lens = torch.tensor([50], dtype=torch.int32, device="cuda"), torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    out, ws = torch.full((B * T, Hq * D), 7.0, device="cuda"), workspace(B, T, Hq, Hkv, D, P)
    ok = dict(qkv=x, prefix_k=pk, prefix_v=pv, prefix_len=n, k_cache=kc, v_cache=vc, cache_len=lens, T=T, Hq=Hq, Hkv=Hkv,
              scale=0.1, out=out, workspace=ws)
    for bad in (dict(scale=0.0), dict(workspace=ws[:-16]), dict(workspace=ws[8:])):
        with pytest.raises(qv.QVError):
            qv.qv_attention_verify_prefix(**{**ok, **bad})
    for bad in (dict(prefix_v=pv[:50]), dict(prefix_k=pk.float()), dict(prefix_len=n.long()), dict(cache_len=lens[:1]),
                dict(v_cache=vc[:1]), dict(T=3), dict(out=out[:2]), dict(workspace=ws.view(torch.int8)),
                dict(prefix_len=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            qv.qv_attention_verify_prefix(**{**ok, **bad})
    assert qv.qv_attention_prefix_workspace_bytes(1, 129, 1, 1, 64, 10) == 0       # more than 128 rows a head group
    assert qv.qv_attention_prefix_workspace_bytes(1, 1, 1, 1, 64, 0) == 0
    assert qv.qv_attention_prefix_workspace_bytes(1, 1, 1, 1, 96, 10) == 0
    assert (out == 7.0).all()
