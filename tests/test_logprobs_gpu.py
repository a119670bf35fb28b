"""qv_token_logprobs against 64 bits. Tolerances: a logit's difference from the
maximum is exact to half an ulp of binary32 and its exponential within
2^-22 + 2^-24 |z|, |z| <= 150 only where the term is nothing; per-thread sums of
n terms add n 2^-24 at most, n <= V / 512 + 32 (V / 128 + 32 for many short rows); S and T are combined over at most
13 + 16 steps. So ln S is within (n + 40) 2^-23, a log probability within that and
2^-22 of its own and the logits' size, and the entropy within (n + 40) 2^-22 of
1 + its size (T's terms are at most 0.54 each)."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import np_, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qv():
    require_gpu()
    from quantized_verification_gb300 import qv as _qv
    _qv.load()
    return _qv


def call(qv, x, tok, K, entropy=True, stream=None):
    M = x.shape[0]
    lp = torch.full((M,), 5.0, device="cuda")
    ent = torch.full((M,), 5.0, device="cuda") if entropy else None
    tt = torch.full((M, K), -77, dtype=torch.int32, device="cuda") if K else None
    tl = torch.full((M, K), 5.0, device="cuda") if K else None
    qv.qv_token_logprobs(x, tok, lp, entropy=ent, top_tokens=tt, top_logprobs=tl, stream=stream)
    return lp, ent, tt, tl


def check(x, tok, K, got, threads=512):
    lp, ent, tt, tl = got
    M, V = x.shape
    xf = x.float().cpu().numpy()
    wlp, went, wtt, wtl = ref.logprobs(xf, tok.cpu().numpy(), K)
    fin = xf[np.isfinite(xf)]
    size = float(np.abs(fin).max()) if fin.size else 0.0
    n = V / threads + 32
    tol = (n + 40) * 2.0 ** -23 + 2.0 ** -22 * size

    def near(a, w, t):
        a = np_(a).astype(np.float64)
        inf = ~np.isfinite(w)
        assert np.array_equal(a[inf], w[inf])
        assert np.all(np.abs(a[~inf] - w[~inf]) <= t + 2.0 ** -22 * np.abs(w[~inf])), np.abs(a[~inf] - w[~inf]).max()
    near(lp, wlp, tol)
    if ent is not None:
        near(ent, went, 2 * tol * (1 + np.log(V)))
        assert float(ent.min()) >= 0
    if K:
        assert np.array_equal(np_(tt), wtt)
        near(tl, wtl, tol)


SHAPES = [  # M, V, K, dtype
    (1, 1, 1, torch.float32), (1, 1, 0, torch.bfloat16), (3, 2, 2, torch.float32), (5, 31, 31, torch.bfloat16),
    (2, 32, 32, torch.float32), (7, 1000, 5, torch.float32), (4, 1003, 32, torch.bfloat16),
    (5, 151936, 20, torch.float32), (1, 151936, 1, torch.bfloat16), (3, 100003, 7, torch.bfloat16),
    (2, 32003, 5, torch.float32), (160, 4099, 3, torch.bfloat16), (200, 9001, 20, torch.float32),
    (33, 65537, 32, torch.float32), (1, 600001, 32, torch.float32),
]


@pytest.mark.parametrize("M,V,K,dtype", SHAPES)
def test_logprobs(qv, M, V, K, dtype):
    g = torch.Generator().manual_seed(M * 31 + V)
    x = (torch.randn(M, V, generator=g) * 3).to(dtype).cuda()
    tok = torch.randint(0, V, (M,), generator=g, dtype=torch.int32).cuda()
    got = call(qv, x, tok, K)
    check(x, tok, K, got)
    again = call(qv, x, tok, K)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))
    lp, _, _, _ = call(qv, x, tok, 0, entropy=False)
    assert torch.equal(lp, got[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V", [(3, 5003), (2, 151936), (320, 3001)])
def test_masks_ties_and_padding(qv, dtype, M, V):
    """Rows where everything is equal, all masked, one token left, fewer left than asked for, masked by the type's lowest
    value, +-0 among the best, ascending (every entry a new maximum), one certain token; tokens outside the vocabulary."""
    K = 8
    g = torch.Generator().manual_seed(V)
    inf, low = float("inf"), float(torch.finfo(dtype).min)
    rows = [torch.full((V,), 2.5), torch.full((V,), -inf), torch.full((V,), low), torch.full((V,), -inf),
            torch.full((V,), -inf), torch.randn(V, generator=g), torch.full((V,), -5.0), torch.linspace(-30, 30, V),
            torch.randn(V, generator=g), torch.randn(V, generator=g)]
    rows[3][V // 2] = -4.0
    rows[4][[1, V // 3, V - 1]] = torch.tensor([0.5, 2.0, 0.5])
    rows[5][::2] = low
    rows[6][[7, 100, 300, V - 2]] = torch.tensor([0.0, -0.0, 0.0, -0.0])
    rows[8][V - 1] = 1000.0
    rows[9][: V - 3] = -inf
    x = torch.stack([rows[i % len(rows)] for i in range(M * 4)])[: max(M, len(rows))].to(dtype).cuda()
    n = x.shape[0]
    tok = torch.randint(0, V, (n,), generator=g, dtype=torch.int32)
    tok[0], tok[2 % n], tok[3 % n] = -1, V, V // 2
    check(x, tok.cuda(), K, call(qv, x, tok.cuda(), K))
    assert float(call(qv, x, tok.cuda(), 0)[0][0]) == 0.0


@pytest.mark.parametrize("V", [777, 151936])
def test_not_a_number_is_reported_and_stays_in_its_row(qv, V):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, V, generator=g)
    clean = x.clone()
    x[1, V // 2] = float("nan")
    x[2, 5] = float("inf")
    x, tok = x.cuda(), torch.zeros(4, dtype=torch.int32, device="cuda")
    lp, ent, tt, tl = call(qv, x, tok, 5)
    for r in (1, 2):
        assert bool(lp[r].isnan()) and bool(ent[r].isnan()) and bool(tl[r].isnan().all())
        assert int(tt[r].min()) >= -1 and int(tt[r].max()) < V
    keep = [0, 3]
    check(clean[keep].cuda(), tok[keep], 5, [t[keep] for t in (lp, ent, tt, tl)])


def test_graph_replay_on_other_logits(qv):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(5, 20011, generator=g).cuda()
    tok = torch.randint(0, 20011, (5,), generator=g, dtype=torch.int32).cuda()
    lp, tt, tl = torch.empty(5, device="cuda"), torch.empty(5, 4, dtype=torch.int32, device="cuda"), torch.empty(5, 4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    qv.qv_token_logprobs(x, tok, lp, top_tokens=tt, top_logprobs=tl)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        qv.qv_token_logprobs(x, tok, lp, top_tokens=tt, top_logprobs=tl, stream=torch.cuda.current_stream())
    x.copy_(torch.randn(5, 20011, generator=g) * 2)
    graph.replay()
    torch.cuda.synchronize()
    check(x, tok, 4, (lp, None, tt, tl))


def test_refusals_leave_outputs_untouched(qv):
    x = torch.zeros(2, 10, device="cuda")
    tok = torch.zeros(2, dtype=torch.int32, device="cuda")
    lp = torch.full((2,), 7.0, device="cuda")
    with pytest.raises(qv.QVError):
        qv.qv_token_logprobs(x, tok, lp, top_tokens=torch.zeros(2, 11, dtype=torch.int32, device="cuda"),
                             top_logprobs=torch.zeros(2, 11, device="cuda"))
    with pytest.raises(TypeError):
        qv.qv_token_logprobs(x.half(), tok, lp)
    with pytest.raises(ValueError):
        qv.qv_token_logprobs(x[:, ::2], tok, lp)
    torch.cuda.synchronize()
    assert bool((lp == 7.0).all())


@pytest.mark.parametrize("M,V,K,dtype", [
    (305, 3245, 20, torch.bfloat16), (700, 1, 1, torch.float32), (400, 33, 32, torch.bfloat16),
    (2000, 1000, 5, torch.float32), (611, 16384, 32, torch.bfloat16), (1300, 32003, 7, torch.float32),
    (900, 127, 0, torch.float32), (3859, 517, 20, torch.bfloat16),
])
def test_many_short_rows(qv, M, V, K, dtype):
    """A CTA of 128 threads a row: random rows, among them rows of equal logits, masked rows and ascending ones."""
    g = torch.Generator().manual_seed(M + V)
    x = torch.randn(M, V, generator=g) * 3
    x[::7] = 1.5
    x[1::7][torch.rand(x[1::7].shape, generator=g) < 0.9] = -float("inf")
    x[2::7] = -float("inf")
    x[3::7] = torch.linspace(-9, 9, V)
    x = x.to(dtype).cuda()
    tok = torch.randint(-1, V + 1, (M,), generator=g, dtype=torch.int32).cuda()
    got = call(qv, x, tok, K)
    check(x, tok, K, got, threads=128)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, call(qv, x, tok, K)))


def test_not_a_number_among_many_short_rows(qv):
    M, V = 400, 777
    g = torch.Generator().manual_seed(1)
    x = torch.randn(M, V, generator=g)
    clean = x.clone()
    x[1::9, V // 2], x[2::9, 5] = float("nan"), float("inf")
    bad = torch.zeros(M, dtype=torch.bool)
    bad[1::9] = bad[2::9] = True
    tok = torch.zeros(M, dtype=torch.int32, device="cuda")
    got = call(qv, x.cuda(), tok, 5)
    lp, ent, tt, tl = (t[bad.cuda()] for t in got)
    assert bool(lp.isnan().all()) and bool(ent.isnan().all()) and bool(tl.isnan().all())
    assert int(tt.min()) >= -1 and int(tt.max()) < V
    keep = ~bad
    check(clean[keep].cuda(), tok[keep.cuda()], 5, [t[keep.cuda()] for t in got], threads=128)
