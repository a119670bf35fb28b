"""Attention over prompts and behind a prefix gives a row the same bits whatever else is in its tile: what an earlier kernel
left in shared memory (rows of a tile that 128 / G tokens do not fill), rows of no sequence, rows of other sequences."""
import pytest
import torch

from gpu_util import require_gpu
from quantized_verification_gb300 import qv

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    require_gpu()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows(M, Hq, Hkv, D, seed):
    """qkv rows whose scores rise along the rows, so that a row's maximum is not in its first 128 keys."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, (Hq + 2 * Hkv) * D, generator=g, device="cuda")
    x[:, Hq * D:(Hq + Hkv) * D] *= torch.linspace(0.5, 2.0, M, device="cuda")[:, None]
    return x.to(torch.bfloat16)


def leave_in_shared_memory(D, size, seed):
    """A call whose tiles are full (four query heads a key head, two tiles a block, every SM) with queries of this size."""
    Hq, Hkv, n = 32, 8, 2500
    x = rows(n, Hq, Hkv, D, seed)
    x[:, :Hq * D] *= size
    out = torch.empty(n, Hq * D, dtype=torch.bfloat16, device="cuda")
    qv.qv_attention_prompt(x, i32([0, n]), Hq, Hkv, 1e-3, out)


def prompt(x, cu, Hq, Hkv, D, dtype):
    out = torch.zeros(x.shape[0], Hq * D, dtype=dtype, device="cuda")
    qv.qv_attention_prompt(x, i32(cu), Hq, Hkv, D ** -0.5, out)
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", [(12, 4, 900), (20, 4, 700), (14, 2, 1100), (36, 12, 1500), (71, 1, 300)])
def test_prompts_do_not_depend_on_what_was_in_shared_memory(Hq, Hkv, n, D, dtype):
    x = rows(n, Hq, Hkv, D, n)
    got = []
    for size, seed in ((0.0, 1), (3e4, 2), (1e36, 3), (3e4, 4)):
        leave_in_shared_memory(D, size, seed)
        got.append(prompt(x, [0, n // 3, n], Hq, Hkv, D, dtype))
    assert torch.isfinite(got[0]).all()
    for other in got[1:]:
        assert torch.equal(got[0], other)
    assert qv.qv_device_error() == 0


def prefix_case(B, T, Hq, Hkv, D, P, Lmax, seed):
    x = rows(B * T, Hq, Hkv, D, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rising = lambda n, *s: (torch.randn(*s, generator=g, device="cuda")  # noqa: E731
                            * torch.linspace(0.5, 2.0, n, device="cuda")[:, None, None]).to(torch.bfloat16)
    return x, rising(P, P, Hkv, D), rising(P, P, Hkv, D), rising(Lmax, B, Lmax, Hkv, D), rising(Lmax, B, Lmax, Hkv, D)


def prefix(x, pk, pv, plen, kc, vc, lens, T, Hq, Hkv, dtype):
    P, _, D = pk.shape
    out = torch.zeros(x.shape[0], Hq * D, dtype=dtype, device="cuda")
    ws = torch.empty(qv.qv_attention_prefix_workspace_bytes(len(lens), T, Hq, Hkv, D, P), dtype=torch.uint8, device="cuda")
    qv.qv_attention_verify_prefix(x, pk, pv, i32([plen]), kc, vc, i32(lens), T, Hq, Hkv, D ** -0.5, out, ws)
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,Hq,Hkv", [(40, 2, 24, 8), (7, 3, 12, 4), (30, 5, 28, 4)])
def test_prefixes_do_not_depend_on_what_was_in_shared_memory(B, T, Hq, Hkv, D, dtype):
    P = 9000
    x, pk, pv, kc, vc = prefix_case(B, T, Hq, Hkv, D, P, 400, B)
    lens = [400 - 9 * b for b in range(B)]
    got = []
    for size, seed in ((0.0, 1), (3e4, 2), (1e36, 3), (3e4, 4)):
        leave_in_shared_memory(D, size, seed)
        got.append(prefix(x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, dtype))
    assert torch.isfinite(got[0]).all()
    for other in got[1:]:
        assert torch.equal(got[0], other)
    assert qv.qv_device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (32, 8), (12, 4)])
def test_rows_of_no_sequence_do_not_reach_the_bits_of_others(Hq, Hkv, dtype):
    D, first, n = 128, 45, 800
    x = rows(first + n + 77, Hq, Hkv, D, 5)
    cu = [first, first + n // 2 + 3, first + n]
    want = prompt(x, cu, Hq, Hkv, D, dtype)[first:first + n]
    for size in (0.0, 1e4, 1e36):
        y = x.clone()
        y[:first] *= size
        y[first + n:] *= size
        assert torch.equal(prompt(y, cu, Hq, Hkv, D, dtype)[first:first + n], want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_other_sequences_queries_do_not_reach_a_sequence_s_bits(dtype):
    # over the caches alone (the prefix is empty): the other sequences' rows lie in the same tile
    B, T, Hq, Hkv, D = 20, 2, 8, 2, 128
    x, pk, pv, kc, vc = prefix_case(B, T, Hq, Hkv, D, 130, 900, 6)
    lens = [900 - 11 * b for b in range(B)]
    want = prefix(x, pk, pv, 0, kc, vc, lens, T, Hq, Hkv, dtype)
    for size in (0.0, 1e4, 1e36):
        y = x.clone()
        y[:, :Hq * D] *= size
        y[3 * T:4 * T] = x[3 * T:4 * T]
        got = prefix(y, pk, pv, 0, kc, vc, lens, T, Hq, Hkv, dtype)
        assert torch.equal(got[3 * T:4 * T], want[3 * T:4 * T])


@pytest.mark.parametrize("dtype", DTYPES)
def test_prefix_results_are_the_same_from_call_to_call(dtype):
    B, T, Hq, Hkv, D, P = 24, 5, 32, 8, 128, 5000
    x, pk, pv, kc, vc = prefix_case(B, T, Hq, Hkv, D, P, 300, 7)
    lens = [300 - 12 * b for b in range(B)]
    first = prefix(x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, dtype)
    for _ in range(5):
        assert torch.equal(prefix(x, pk, pv, P, kc, vc, lens, T, Hq, Hkv, dtype), first)
