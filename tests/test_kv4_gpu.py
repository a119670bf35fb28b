"""The 4-bit paged KV cache on the GPU: qv_kv4_write byte for byte, qv_kv4_read
value for value, and qv_attention_verify_kv4 against the binary64 definition
over the very values the cache holds.

Tolerances of attention, from the arithmetic. A score is a D-term sum of exact
products added in binary32, each addition off by at most 2^-23 of the sum of
magnitudes: D 2^-23 A with A the largest scale * sum |q||k| (computed from the
inputs); scaling, the exponential (2 ulp) and the subtraction of the running
maximum add at most 8 * 2^-23 A. An error d of the scores moves the output by at
most 2 d max |v|. The probabilities' parts add 2^-22 (fp32 outputs) or 2^-11
(bf16 outputs, one f16 part) of max |v|, sums over the keys and the merges less
than 2^-18 together. bf16 outputs are rounded once more: 2^-8 |o|."""
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


def gen(seed):
    return torch.Generator().manual_seed(seed)


def random_cache(pages, Hkv, D, seed):
    """Uniform codes in [-7, 7], scales of values up to about 4, as numpy."""
    g = gen(seed)
    q = torch.randint(-7, 8, (pages, Hkv, 64 * D), generator=g).numpy()
    s = torch.randint(11 * 8, 14 * 8, (pages, Hkv, 2 * D), generator=g).numpy().astype(np.uint8)
    return np.concatenate([ref.pack(q), s], axis=2)


def random_table(B, NB, pages, seed):
    return torch.randperm(pages, generator=gen(seed))[: B * NB].view(B, NB).to(torch.int32).numpy()


def cu(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


WRITES = [  # B, T, Hq, Hkv, D, NB, dtype, paged, start, count
    (1, 1, 4, 1, 64, 1, torch.bfloat16, False, [0], None),
    (1, 1, 4, 1, 64, 1, torch.float32, False, [31], None),
    (2, 5, 8, 2, 128, 3, torch.bfloat16, True, [30, 64], [5, 2]),
    (3, 7, 0, 3, 64, 2, torch.float32, True, [0, 60, 29], [7, 7, 0]),
    (2, 33, 16, 8, 128, 4, torch.bfloat16, True, [31, 95], None),
    (1, 200, 2, 1, 128, 7, torch.float32, False, [13], None),
    (2, 9, 10, 5, 64, 2, torch.bfloat16, True, [-3, 60], [9, -1]),
    (2, 40, 4, 4, 64, 2, torch.bfloat16, False, [50, 0], [100, 40]),      # past the table; count above T
    (1, 70, 30, 10, 128, 3, torch.bfloat16, True, [5], None),            # 320 items a row: two columns of blocks
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,NB,dtype,paged,start,count", WRITES)
def test_write_and_read_back(qv, B, T, Hq, Hkv, D, NB, dtype, paged, start, count):
    pages = B * NB + (3 if paged else 0)
    g = gen(7 * T + D)
    x = torch.randn(B * T, (Hq + 2 * Hkv) * D, generator=g)
    x[:, ::37] *= 20.0                                         # outlier channels
    x[0, Hq * D: Hq * D + 32] = 0.0                            # a group of zeros
    x[-1, Hq * D + 32: Hq * D + 64] *= 1e-6                    # one below the smallest scale
    x[-1, -32:] = torch.arange(32.0) / 4 - 3.5                 # many exact ties
    x = x.to(dtype)
    table = random_table(B, NB, pages, 3) if paged else None
    if paged and B > 1:
        table[1, 0] = pages                                    # no page
    before = np.random.default_rng(1).integers(0, 256, (pages, Hkv, 34 * D), dtype=np.uint8)
    cache = cu(before)
    st, cn = np.array(start, np.int32), None if count is None else np.array(count, np.int32)
    qv.qv_kv4_write(x.cuda(), cu(st), cache, T, Hq, Hkv, block_table=cu(table), count=cu(cn))
    want = ref.write(before, x.float().numpy(), st, T, Hq, Hkv, D, NB, table, cn)
    assert np.array_equal(np_(cache), want)                    # every byte, those not written among them
    for out in (torch.float32, torch.bfloat16):
        k = torch.full((B, T, Hkv, D), 7.0, dtype=out, device="cuda")
        v = torch.full((B, T, Hkv, D), -9.0, dtype=out, device="cuda")
        wk, wv = ref.read(want, st, T, D, NB, np_(k.float()), np_(v.float()), table, cn)
        qv.qv_kv4_read(cache, cu(st), k, v, block_table=cu(table), count=cu(cn))
        assert np.array_equal(np_(k.double()), wk) and np.array_equal(np_(v.double()), wv)


def test_write_takes_non_finite_rows(qv):
    D = 64
    x = torch.randn(2, 2 * D, generator=gen(1))
    x[0, 3], x[0, 40], x[0, 41] = float("nan"), float("inf"), -float("inf")
    x[1, 64:96] = float("nan")
    for dtype in (torch.float32, torch.bfloat16):
        before = np.zeros((1, 1, 34 * D), np.uint8)
        cache = cu(before)
        qv.qv_kv4_write(x.to(dtype).cuda(), cu(np.zeros(1, np.int32)), cache, 2, 0, 1)
        assert np.array_equal(np_(cache), ref.write(before, x.to(dtype).float().numpy(), [0], 2, 0, 1, D, 1))


def test_codes_of_every_scale(qv):
    """Groups whose maxima run over 40 octaves and every 8 bits of mantissa, in fp32: the bytes of all scales."""
    D, T = 128, 2560
    g = gen(9)
    amax = torch.exp2(torch.linspace(-20, 20, T * 8).reshape(T, 8))
    x = (torch.rand(T, 8, 32, generator=g) * 2 - 1) * amax[:, :, None]
    x[:, :, 5] = amax
    x = x.reshape(T, 2 * D)
    before = np.zeros((T // 32, 1, 34 * D), np.uint8)
    cache = cu(before)
    qv.qv_kv4_write(x.cuda(), cu(np.zeros(1, np.int32)), cache, T, 0, 1)
    assert np.array_equal(np_(cache), ref.write(before, x.numpy(), [0], T, 0, 1, D, T // 32))
    assert len(np.unique(np_(cache)[:, :, 32 * D:])) == 256


ATTENDS = [  # B, T, Hq, Hkv, D, NB, lens, paged
    (1, 1, 4, 4, 64, 1, [1], False),
    (1, 1, 8, 1, 128, 0, [0], False),                          # no cache at all
    (2, 1, 8, 2, 128, 2, [0, 64], True),
    (1, 1, 32, 8, 128, 17, [517], False),
    (1, 5, 32, 8, 128, 64, [2043], False),
    (3, 5, 32, 8, 128, 12, [384, 1, 255], True),
    (2, 5, 8, 1, 128, 40, [1279, 33], True),                   # 40 query rows: two row tiles
    (2, 16, 8, 4, 128, 9, [288, 257], True),                   # 32 rows, all four n8 tiles
    (1, 40, 4, 2, 64, 5, [131], False),                        # more own rows than a unit, 80 query rows
    (4, 3, 8, 2, 64, 33, [1056, 31, 32, 700], True),
    (2, 8, 16, 4, 64, 20, [639, 5], True),
    (2, 6, 8, 2, 64, 20, [640, 17], False),                    # 24 rows
    (1, 4, 16, 4, 128, 70, [2240], True),                      # 16 rows
    (40, 2, 4, 2, 64, 3, None, True),
    (300, 1, 2, 1, 128, 2, None, True),                        # more sequences than threads
    (2, 1, 8, 8, 128, 300, [9600, 9000], False),               # ranges of many records: the ring refilled
    (1, 256, 2, 1, 64, 2, [50], False),                        # the longest step
    (2, 2, 4, 2, 128, 4, [-5, 400], False),                    # lengths outside [0, 32 NB] are clamped
]


def attend_inputs(B, T, Hq, Hkv, D, NB, lens, paged, seed=0):
    pages = B * NB + (5 if paged else 0)
    g = gen(seed + 31 * T + NB)
    qkv = torch.randn(B * T, (Hq + 2 * Hkv) * D, generator=g)
    qkv[:, Hq * D: (Hq + Hkv) * D: 29] *= 4.0
    qkv = qkv.to(torch.bfloat16)
    if lens is None:
        lens = torch.randint(0, 32 * NB + 1, (B,), generator=g).tolist()
    cache = random_cache(max(pages, 1), Hkv, D, seed + 5)[:pages]
    table = random_table(B, NB, pages, seed + 2) if paged else None
    return qkv, cache, np.array(lens, np.int32), table


def close(out, want, vmax, smax, D):
    """Inside the bound of this file's head, element for element."""
    d = (D + 8) * 2.0 ** -23 * smax
    tol = vmax * (2 * d + 2.0 ** -22 + 2.0 ** -18)
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -11 * vmax + 2.0 ** -8 * np.abs(want)
    err = np.abs(np_(out.double()) - want)
    assert np.all(err <= tol), (float(err.max()), float(np.max(tol)))
    if out.dtype == torch.float32:
        assert np.linalg.norm(err) <= (2.0 ** -18 + 2 * d) * np.linalg.norm(want)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,NB,lens,paged", ATTENDS)
def test_attention(qv, B, T, Hq, Hkv, D, NB, lens, paged, out_dtype):
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, lens, paged)
    scale = float(np.float32(D ** -0.5))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    args = (qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale)
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, table)
    first = None
    for _ in range(2):                                         # the second call on the workspace the first left
        out = torch.full((B * T, Hq * D), float("nan"), dtype=out_dtype, device="cuda")
        qv.qv_attention_verify_kv4(*args, out, ws, block_table=cu(table))
        close(out, want, vmax, smax, D)
        assert first is None or torch.equal(first, out)        # the same bits
        first = out
    assert int(ws[:4096].max()) == 0
    assert qv.qv_device_error() == 0


def test_attention_ignores_what_is_not_there(qv):
    """Positions past a length, pages past it, and block table entries that are no page: any bytes and any page number."""
    B, T, Hq, Hkv, D, NB = 3, 5, 8, 2, 128, 10
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, [100, 320, 0], True)
    scale = float(np.float32(D ** -0.5))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    out = torch.empty(B * T, Hq * D, device="cuda")
    qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out, ws, block_table=cu(table))
    other = np.full_like(cache, 0xFF)                          # the largest scales and codes of -1 everywhere ...
    for b in range(B):
        for p in range(int(ln[b])):                            # ... but where a position is cached
            page, s = int(table[b, p // 32]), p % 32
            for a, w in ((0, D // 2), (16, D // 2), (32, D // 32), (33, D // 32)):
                at = slice(a * D + s * w, a * D + (s + 1) * w)
                other[page, :, at] = cache[page, :, at]
    t2 = table.copy()
    t2[0, 4:] = [-1, 2 ** 31 - 1, -2 ** 31, 35, 10 ** 9, -7]
    t2[2] = -1
    out2 = torch.empty_like(out)
    qv.qv_attention_verify_kv4(qkv.cuda(), cu(other), cu(ln), T, Hq, Hkv, scale, out2, ws, block_table=cu(t2))
    assert torch.equal(out, out2)
    # pages taken out of the middle: their positions are absent, not zero
    t3 = table.copy()
    t3[1, [0, 3, 9]] = [-1, 35, 2 ** 30]
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, t3)
    qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out2, ws, block_table=cu(t3))
    close(out2, want, vmax, smax, D)
    # no cached position left at all
    t3[:] = -1
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, t3)
    qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out2, ws, block_table=cu(t3))
    close(out2, want, vmax, smax, D)


@pytest.mark.parametrize("D,T,Hq,Hkv", [(128, 5, 8, 2), (64, 40, 4, 2)])
def test_attention_keeps_later_rows_out(qv, D, T, Hq, Hkv):
    """NaN and infinities in a row of the step reach the rows that see it and no others."""
    B, NB = 2, 6
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, [150, 40], True)
    scale = float(np.float32(D ** -0.5))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, table)
    j0 = T - 2
    bad = qkv.clone()
    for j in (j0, T - 1):
        bad[j, (Hq) * D:] = float("nan")                       # keys and values of sequence 0's last rows
    bad[T + j0, (Hq + Hkv) * D + 3] = float("inf")             # one value of sequence 1
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(B * T, Hq * D, dtype=dt, device="cuda")
        qv.qv_attention_verify_kv4(bad.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out, ws, block_table=cu(table))
        o = out.view(B, T, Hq, D)
        keep = torch.ones(B, T, dtype=torch.bool)
        keep[:, j0:] = False
        k = keep.view(-1)
        close(out[k.cuda()], want[k.numpy()], vmax, smax, D)
        assert bool(o[0, j0:].isnan().all())
        G = Hq // Hkv
        assert bool((o[1, j0:, :G, 3] == float("inf")).all())
        rest = o[1, j0:].clone()
        rest[:, :G, 3] = 0
        assert bool(rest.isfinite().all())
    # a query row that is not finite spoils its own output only
    bad = qkv.clone()
    bad[1, :D] = float("nan")
    out = torch.empty(B * T, Hq * D, device="cuda")
    qv.qv_attention_verify_kv4(bad.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out, ws, block_table=cu(table))
    o = np_(out.double()).reshape(B, T, Hq, D)
    assert np.isnan(o[0, 1, 0]).all()
    o[0, 1, 0] = want.reshape(B, T, Hq, D)[0, 1, 0]
    close(torch.from_numpy(o.reshape(B * T, -1)), want, vmax, smax, D)


def test_attention_extreme_scores(qv):
    """Scores that rise by hundreds from record to record (every unit moves the running maximum), and scales at the
    format's ends: the largest (values of 860160) and the smallest (2^-15)."""
    T, Hq, Hkv, D, NB = 2, 4, 1, 128, 9
    qkv, cache, ln, table = attend_inputs(1, T, Hq, Hkv, D, NB, [288], False, seed=4)
    for i in range(NB):                                        # key scales grow with the position
        cache[i, :, 32 * D: 33 * D] = 8 * (8 + i)
    cache[:, :, 33 * D:] = np.where(np.arange(D) % 2 == 0, 255, 0)
    scale = float(np.float32(D ** -0.5))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(1, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, table)
    out = torch.empty(T, Hq * D, device="cuda")
    qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out, ws)
    close(out, want, vmax, smax, D)


def test_attention_equals_the_bf16_kernel_on_the_read_back_cache(qv):
    """qv_kv4_read into a bf16 cache, then qv_attention_verify: the same values, so the same result but for rounding."""
    B, T, Hq, Hkv, D, NB = 2, 5, 32, 8, 128, 20
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, [640, 201], True)
    scale = float(np.float32(D ** -0.5))
    kc = torch.empty(B, 32 * NB, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    qv.qv_kv4_read(cu(cache), cu(np.zeros(B, np.int32)), kc, vc, block_table=cu(table))
    a, b = torch.empty(B * T, Hq * D, device="cuda"), torch.empty(B * T, Hq * D, device="cuda")
    qv.qv_attention_verify(qkv.cuda(), kc, vc, cu(ln), T, Hq, Hkv, scale, a)
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, b, ws, block_table=cu(table))
    _, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, table)
    tol = vmax * (4 * (D + 8) * 2.0 ** -23 * smax + 2.0 ** -16)         # both sides' bounds
    assert float((a - b).abs().max()) <= tol


def test_one_workspace_for_several_shapes_and_graph_replay(qv):
    """One workspace through calls of different shapes, on a stream of its own, eagerly and as a captured graph whose
    inputs change between replays."""
    shapes = [(1, 1, 8, 1, 128, 60, [1900], False), (3, 5, 32, 8, 128, 6, [192, 3, 70], True),
              (2, 4, 8, 2, 64, 30, [960, 500], True)]
    data = [attend_inputs(*s) for s in shapes]
    ws = torch.zeros(max(qv.qv_attention_kv4_workspace_bytes(s[0], s[1], s[2], s[3], s[4], s[5]) for s in shapes),
                     dtype=torch.uint8, device="cuda")
    dev = [(d[0].cuda(), cu(d[1]), cu(d[2]), cu(d[3])) for d in data]
    outs = [torch.empty(s[0] * s[1], s[2] * s[4], device="cuda") for s in shapes]

    def go(stream):
        for s, d, o in zip(shapes, dev, outs):
            qv.qv_attention_verify_kv4(d[0], d[1], d[2], s[1], s[2], s[3], s[4] ** -0.5, o, ws, block_table=d[3],
                                       stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    go(side)
    torch.cuda.synchronize()
    eager = [o.clone() for o in outs]
    for s, d, o in zip(shapes, data, eager):
        want, vmax, smax = ref.attend(d[0].float().numpy(), d[1], d[2], s[1], s[2], s[3], s[4], s[5], s[4] ** -0.5, d[3])
        close(o, want, vmax, smax, s[4])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(torch.cuda.current_stream())
    for o in outs:
        o.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, eager))
    dev[0][2].fill_(7)                                         # another length, read on the device
    g.replay()
    torch.cuda.synchronize()
    s, d = shapes[0], data[0]
    want, vmax, smax = ref.attend(d[0].float().numpy(), d[1], [7], s[1], s[2], s[3], s[4], s[5], s[4] ** -0.5, d[3])
    close(outs[0], want, vmax, smax, s[4])
    assert torch.equal(outs[1], eager[1])


def test_refusals_leave_outputs_untouched(qv):
    B, T, Hq, Hkv, D, NB = 1, 1, 4, 2, 64, 2
    qkv, cache, ln, _ = attend_inputs(B, T, Hq, Hkv, D, NB, [40], False)
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    assert qv.qv_attention_kv4_workspace_bytes(1, 257, 4, 2, 64, 2) == 0
    assert qv.qv_attention_kv4_workspace_bytes(1, 1, 4, 3, 64, 2) == 0
    out = torch.full((T, Hq * D), 7.0, device="cuda")
    for call in (lambda: qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, 0.0, out, ws),
                 lambda: qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, 0.1, out, ws[:-16])):
        with pytest.raises(qv.QVError):
            call()
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())


def test_a_wait_that_runs_out_is_reported(qv):
    """The test hook leaves every record unrequested: the call returns, the error word says why, and the next call on
    the same workspace is right."""
    B, T, Hq, Hkv, D, NB = 2, 2, 8, 2, 128, 40
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, [1280, 700], True)
    scale = D ** -0.5
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    out = torch.empty(B * T, Hq * D, device="cuda")
    args = (qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out, ws)
    assert qv.qv_device_error() == 0
    try:
        qv.qv_debug_set_slot_wait_ns(2_000_000)
        qv.qv_debug_hold_attention_loads(1)
        qv.qv_attention_verify_kv4(*args, block_table=cu(table))
        assert qv.qv_device_error() == qv.QV_DEVICE_ERR_FULL_WAIT
    finally:
        qv.qv_debug_set_slot_wait_ns(0)
        qv.qv_debug_hold_attention_loads(0)
    assert int(ws[:4096].max()) == 0
    qv.qv_attention_verify_kv4(*args, block_table=cu(table))
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, table)
    close(out, want, vmax, smax, D)
    assert qv.qv_device_error() == 0


# Contexts that may be long, or more tiles than the GPU holds CTAs: the units of all tiles cut into equal ranges,
# parts of tiles joined through the workspace.
LINES = [  # B, T, Hq, Hkv, D, NB, lens, paged
    (1, 1, 4, 1, 128, 420, [13440], False),
    (2, 3, 8, 2, 128, 400, [12800, 77], True),                 # 12 rows a tile
    (2, 5, 8, 2, 128, 400, [12345, 4097], True),               # 20 rows
    (3, 5, 8, 2, 128, 390, [0, 31, 9000], False),
    (1, 8, 8, 2, 128, 390, [12480], True),                     # 32 rows
    (1, 9, 8, 2, 128, 400, [12001], False),                    # 36 rows: two tiles of 18
    (2, 256, 2, 1, 128, 400, [50, 6000], True),                # the longest step, 16 tiles of 32 rows
    (1, 2, 4, 1, 64, 400, [12799], True),
    (2, 4, 8, 2, 64, 400, [1, 12001], False),                  # 16 rows
    (3, 6, 8, 2, 64, 400, [12800, 1, 5000], True),             # 24 rows
    (1, 8, 8, 2, 64, 400, [12333], False),                     # 32 rows
    (200, 2, 4, 4, 128, 3, None, True),                        # 800 tiles of 2 rows
    (160, 5, 8, 2, 128, 5, None, True),                        # 320 tiles of 20 rows
    (31, 20, 40, 20, 128, 2, None, False),                     # 40 rows a head group
    (700, 1, 4, 1, 128, 2, None, True),
    (200, 7, 6, 2, 64, 3, None, True),                         # 21 rows
    (80, 1, 8, 4, 64, 42, None, True),
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,NB,lens,paged", LINES)
def test_attention_on_one_line(qv, B, T, Hq, Hkv, D, NB, lens, paged, out_dtype):
    if NB > 40 or (D == 128 and T * Hq // Hkv > 16):           # (else the many tiles have a thread block each)
        assert qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB) > 4096  # parts of tiles have room there
    test_attention(qv, B, T, Hq, Hkv, D, NB, lens, paged, out_dtype)


@pytest.mark.parametrize("T,Hq", [(1, 8), (5, 8), (8, 8)])
def test_long_attention_ignores_what_is_not_there(qv, T, Hq):
    """Blocks without a page inside a long context, whole runs of them, and a sequence with nothing else."""
    B, Hkv, D, NB = 3, 2, 128, 400
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, [6000, 12800, 900], True)
    scale = float(np.float32(D ** -0.5))
    table[0, ::3] = -1
    table[1, 8:200] = 2 ** 30
    table[2] = -5
    args = (qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale)
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, table)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(B * T, Hq * D, dtype=dt, device="cuda")
        qv.qv_attention_verify_kv4(*args, out, ws, block_table=cu(table))
        close(out, want, vmax, smax, D)


@pytest.mark.parametrize("D,T,Hq,Hkv", [(128, 5, 8, 2), (128, 3, 4, 2), (128, 40, 4, 2), (64, 40, 4, 2)])
def test_long_attention_keeps_later_rows_out(qv, D, T, Hq, Hkv):
    """As test_attention_keeps_later_rows_out, where tiles are cut anywhere."""
    B, NB, j0 = 2, 400, T - 2
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, [1500, 40], True)
    scale = float(np.float32(D ** -0.5))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, table)
    bad = qkv.clone()
    for j in (j0, T - 1):
        bad[j, Hq * D:] = float("nan")
    bad[T + j0, (Hq + Hkv) * D + 3] = float("inf")
    G = Hq // Hkv
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(B * T, Hq * D, dtype=dt, device="cuda")
        qv.qv_attention_verify_kv4(bad.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out, ws, block_table=cu(table))
        o = out.view(B, T, Hq, D)
        keep = torch.ones(B, T, dtype=torch.bool)
        keep[:, j0:] = False
        k = keep.view(-1)
        close(out[k.cuda()], want[k.numpy()], vmax, smax, D)
        assert bool(o[0, j0:].isnan().all())
        assert bool((o[1, j0:, :G, 3] == float("inf")).all())
        rest = o[1, j0:].clone()
        rest[:, :G, 3] = 0
        assert bool(rest.isfinite().all())


@pytest.mark.parametrize("D,T,Hq", [(128, 1, 4), (128, 5, 4), (128, 8, 4), (64, 6, 4)])
def test_long_attention_extreme_scores(qv, D, T, Hq):
    """Scores whose size grows 4000-fold along the cache, so that maxima move all the time, and the format's end
    scales among the values."""
    NB = 400
    qkv, cache, ln, table = attend_inputs(1, T, Hq, 1, D, NB, [32 * NB], False, seed=4)
    for i in range(NB):
        cache[i, :, 32 * D: 33 * D] = 60 + i // 4
    cache[:, :, 33 * D:] = np.where(np.arange(D) % 2 == 0, 255, 0)
    scale = float(np.float32(D ** -0.5))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(1, T, Hq, 1, D, NB), dtype=torch.uint8, device="cuda")
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, 1, D, NB, scale, table)
    out = torch.empty(T, Hq * D, device="cuda")
    qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, 1, scale, out, ws)
    close(out, want, vmax, smax, D)


@pytest.mark.parametrize("T,D", [(1, 128), (5, 128), (5, 64)])
def test_a_wait_that_runs_out_on_one_line(qv, T, D):
    B, Hq, Hkv, NB = 2, 8, 2, 400
    qkv, cache, ln, table = attend_inputs(B, T, Hq, Hkv, D, NB, [1280, 700], True)
    scale = D ** -0.5
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    out = torch.empty(B * T, Hq * D, device="cuda")
    args = (qkv.cuda(), cu(cache), cu(ln), T, Hq, Hkv, scale, out, ws)
    assert qv.qv_device_error() == 0
    try:
        qv.qv_debug_set_slot_wait_ns(2_000_000)
        qv.qv_debug_hold_attention_loads(1)
        qv.qv_attention_verify_kv4(*args, block_table=cu(table))
        assert qv.qv_device_error() == qv.QV_DEVICE_ERR_FULL_WAIT
    finally:
        qv.qv_debug_set_slot_wait_ns(0)
        qv.qv_debug_hold_attention_loads(0)
    assert int(ws[:4096].max()) == 0
    qv.qv_attention_verify_kv4(*args, block_table=cu(table))
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, Hkv, D, NB, scale, table)
    close(out, want, vmax, smax, D)
    assert qv.qv_device_error() == 0


def test_a_pool_of_more_than_4_gib(qv):
    """Records whose byte offsets pass 32 bits are written, read and attended to like others."""
    B, T, Hq, Hkv, D, NB = 2, 5, 16, 8, 128, 3
    pages = 2 ** 32 // (Hkv * 34 * D) + 40
    far = torch.zeros(pages, Hkv, 34 * D, dtype=torch.uint8, device="cuda")
    near = torch.zeros(B * NB, Hkv, 34 * D, dtype=torch.uint8, device="cuda")
    t_near = torch.arange(B * NB, dtype=torch.int32, device="cuda").view(B, NB)
    t_far = pages - 1 - t_near
    rows = torch.randn(B * 90, (Hq + 2 * Hkv) * D, generator=gen(1)).to(torch.bfloat16).cuda()
    step = rows[: B * T].contiguous()
    zero, ln = cu(np.zeros(B, np.int32)), cu(np.full(B, 90, np.int32))
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    got = []
    for cache, table in ((near, t_near), (far, t_far)):
        qv.qv_kv4_write(rows, zero, cache, 90, Hq, Hkv, block_table=table)
        k = torch.empty(B, 90, Hkv, D, dtype=torch.bfloat16, device="cuda")
        v, out = torch.empty_like(k), torch.empty(B * T, Hq * D, device="cuda")
        qv.qv_kv4_read(cache, zero, k, v, block_table=table)
        qv.qv_attention_verify_kv4(step, cache, ln, T, Hq, Hkv, 0.1, out, ws, block_table=table)
        got.append((k, v, out))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(far[t_far.long()], near[t_near.long()]) and bool((got[0][0] != 0).any())
    assert int(far[: pages - B * NB].max()) == 0


@pytest.mark.parametrize("D,T,Hq", [(128, 1, 64), (128, 4, 32), (128, 5, 32), (128, 8, 32), (64, 1, 8), (64, 8, 32)])
def test_long_sums_do_not_drift(qv, D, T, Hq):
    """Queries of zero: every output is the mean of the values it sees, all of them positive here, over ranges of
    thousands of positions per thread block. A product of the tensor cores may cut its sum off below the last bit
    (2^-23 of it at most, half of that on average), so a run of n products from zero loses n 2^-25 on average, its sums
    being half of its result on average: 2^-20 for 32 products. Rounded additions err both ways: over at most 1100 of
    them 2^-24 sqrt(1100 / 9) at one standard deviation, 2^-18.5 at four. Without an end to the runs the loss would be
    above 2^-16 (500 products or more)."""
    B, Hkv, NB, L = 38, 8, 250, 8000
    g = gen(3)
    codes = torch.randint(1, 8, (NB, Hkv, 16 * D), generator=g) | (torch.randint(1, 8, (NB, Hkv, 16 * D), generator=g) << 4)
    scales = torch.randint(11 * 8, 13 * 8, (NB, Hkv, D), generator=g)
    cache = torch.cat([torch.zeros(NB, Hkv, 16 * D), codes, torch.zeros(NB, Hkv, D), scales], 2).to(torch.uint8).cuda()
    table = torch.stack([torch.randperm(NB, generator=g) for _ in range(B)]).to(torch.int32).cuda()
    qkv = torch.zeros(B, T, Hq + 2 * Hkv, D, dtype=torch.bfloat16)
    qkv[:, :, Hq + Hkv:] = torch.rand(B, T, Hkv, D, generator=g).to(torch.bfloat16)
    qkv = qkv.cuda()
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(B, T, Hq, Hkv, D, NB), dtype=torch.uint8, device="cuda")
    out = torch.empty(B * T, Hq * D, device="cuda")
    qv.qv_attention_verify_kv4(qkv.view(B * T, -1), cache, cu(np.full(B, L, np.int32)), T, Hq, Hkv, 1.0, out, ws,
                               block_table=table)
    k = torch.empty(1, L, Hkv, D, device="cuda")
    v = torch.empty_like(k)
    qv.qv_kv4_read(cache, cu(np.zeros(1, np.int32)), k, v, block_table=table[:1].contiguous())
    own = qkv[:, :, Hq + Hkv:].double().cumsum(1)
    n = L + 1 + torch.arange(T, device="cuda").view(1, T, 1, 1)
    want = ((v[0].double().sum(0) + own) / n).repeat_interleave(Hq // Hkv, 2).reshape(B * T, Hq * D)
    err = (out.double() / want - 1).abs().max()
    assert float(err) <= 2.0 ** -20 + 2.0 ** -18.5, float(err)


@pytest.mark.parametrize("NB", [9, 400])
@pytest.mark.parametrize("D,T,Hq", [(128, 1, 2), (128, 5, 4), (128, 8, 4), (64, 3, 4)])
def test_scores_of_millions(qv, NB, D, T, Hq):
    """Keys at the format's largest scale and queries that fit them: the best score is far above the others and lies at
    1e5 to 9e7, where binary32 has few bits or none behind the point. The output is the best key's value: every other
    probability is 2^-10000 or less, and the weight of the best is one f16 number or two over their own sum (2^-11 of
    it for bf16 outputs, which are rounded by 2^-9 more). Beyond 2^27 ln 2 it is NaN."""
    n = 32 * NB
    g = gen(8)
    codes = torch.randint(-2, 3, (NB, 1, 64 * D), generator=g).numpy()
    steps = np.linspace(3, n - 2, 5).astype(int)               # ever better keys along the cache
    for i, p in enumerate(steps):
        codes[p // 32, 0, (p % 32) * D:(p % 32 + 1) * D] = 3 + i
    cache = np.concatenate([ref.pack(codes), np.full((NB, 1, D), 255, np.uint8),
                            np.random.default_rng(1).integers(80, 130, (NB, 1, D)).astype(np.uint8)], axis=2)
    _, vc, _, vs = ref.parts(cache, D)
    p = steps[-1]
    best = ref.values(ref.unpack(vc[p // 32, 0, p % 32]), vs[p // 32, 0, p % 32])
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(1, T, Hq, 1, D, NB), dtype=torch.uint8, device="cuda")
    scale = 1.0 / D
    for want_max in (1e5, 6.9e5, 7.6e5, 3e6, 1.4e7, 5e7, 9e7, 1e8, 1e12):
        qkv = torch.randn(T, (Hq + 2) * D, generator=g)
        qkv[:, : Hq * D] = want_max / (7 * 122880)
        qkv = qkv.to(torch.bfloat16)
        top = float(qkv[0, 0]) * 7 * 122880
        for dt in (torch.float32, torch.bfloat16):
            out = torch.empty(T, Hq * D, dtype=dt, device="cuda")
            qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(np.array([n], np.int32)), T, Hq, 1, scale, out, ws)
            o = np_(out.double()).reshape(T * Hq, D)
            if top >= 2 ** 27 * np.log(2):
                assert np.isnan(o).all()
            else:
                tol = 2.0 ** -20 if dt == torch.float32 else 2.0 ** -11 + 2.0 ** -8
                assert np.all(np.abs(o - best) <= tol * np.abs(best) + 1e-30), (want_max, np.abs(o - best).max())


@pytest.mark.parametrize("NB", [9, 400])
@pytest.mark.parametrize("D,T,Hq", [(128, 1, 2), (128, 5, 4), (128, 8, 4), (64, 5, 4)])
def test_own_scores_of_minus_infinity(qv, NB, D, T, Hq):
    """Own keys with an infinity that makes every own score -inf, over cached scores far below 0 (about -300): the own
    rows have no part in the output, which is the mean of the cached values (all cached keys are equal, and so are the
    probabilities). Sums round by 2^-24 each, 300 of them a range at most. A probability is 2^(7 + f), f a score's part
    behind the point, so that its f16 parts are off by 2^-22 of it, or 2^-11 where bf16 outputs keep one part (the sum of
    the probabilities is not rounded along with them); bf16 outputs are rounded by 2^-8 once more."""
    n = 32 * NB - 5
    g = gen(12)
    codes = np.concatenate([np.full((NB, 1, 32 * D), -7), torch.randint(-7, 8, (NB, 1, 32 * D), generator=g).numpy()], axis=2)
    scales = np.concatenate([np.full((NB, 1, D), 17 * 8), np.full((NB, 1, D), 15 * 8)], axis=2).astype(np.uint8)
    cache = np.concatenate([ref.pack(codes), scales], axis=2)
    qkv = torch.randn(T, (Hq + 2) * D, generator=g)
    qkv[:, : Hq * D] = 1.0
    qkv[:, Hq * D + 3] = -float("inf")
    qkv = qkv.to(torch.bfloat16)
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(1, T, Hq, 1, D, NB), dtype=torch.uint8, device="cuda")
    want = codes[:, 0, 32 * D:].reshape(NB * 32, D)[:n].mean(0)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(T, Hq * D, dtype=dt, device="cuda")
        qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(np.array([n], np.int32)), T, Hq, 1, 12.0 / D, out, ws)
        err = np.abs(np_(out.double()).reshape(T * Hq, D) - want)
        rounding = 2.0 ** -8 + 2.0 ** -11 if dt == torch.bfloat16 else 2.0 ** -22
        assert np.all(err <= 7 * 300 * 2.0 ** -24 + rounding * np.abs(want)), err.max()


@pytest.mark.parametrize("NB", [9, 400])
@pytest.mark.parametrize("D,T,Hq", [(128, 1, 2), (128, 5, 4), (128, 8, 4), (64, 5, 4)])
def test_keys_of_no_weight_at_all(qv, NB, D, T, Hq):
    """Every other block's scores are about -1e8, beyond what the running maxima hold: the result is that of the other
    blocks alone, within their bound."""
    n, g, odd = 32 * NB - 5, gen(13), np.arange(NB) % 2
    codes = torch.randint(-7, 8, (NB, 1, 64 * D), generator=g).numpy()
    codes[odd == 0, :, : 32 * D] = -7
    scales = np.full((NB, 1, 2 * D), 15 * 8, np.uint8)
    scales[:, :, :D] = np.where(odd == 0, 255, 8 * 5)[:, None, None]
    cache = np.concatenate([ref.pack(codes), scales], axis=2)
    qkv = torch.randn(T, (Hq + 2) * D, generator=g)
    qkv[:, : Hq * D] = 16.0
    qkv = qkv.to(torch.bfloat16)
    table = np.arange(NB, dtype=np.int32)[None]
    alone = np.where(odd == 0, -1, table).astype(np.int32)
    scale, ln = 12.0 / D, np.array([n], np.int32)
    ws = torch.zeros(qv.qv_attention_kv4_workspace_bytes(1, T, Hq, 1, D, NB), dtype=torch.uint8, device="cuda")
    want, vmax, smax = ref.attend(qkv.float().numpy(), cache, ln, T, Hq, 1, D, NB, scale, alone)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(T, Hq * D, dtype=dt, device="cuda")
        qv.qv_attention_verify_kv4(qkv.cuda(), cu(cache), cu(ln), T, Hq, 1, scale, out, ws, block_table=cu(table))
        close(out, want, vmax, smax, D)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,NB,lens", [
    (1, 1, 4, 1, 128, 2000, [63990]), (1, 5, 4, 1, 128, 2000, [63990]), (1, 8, 4, 1, 128, 1400, [44800]),
    (1, 6, 4, 1, 64, 2000, [64000]), (2, 1, 8, 1, 64, 1500, [48000, 33]), (3, 5, 4, 1, 128, 1500, [47000, 200, 48000]),
    (2, 2, 8, 2, 128, 1100, [1, 35200]),
])
def test_attention_over_hundreds_of_parts(qv, B, T, Hq, Hkv, D, NB, lens, out_dtype):
    """Few heads over long contexts: so many thread blocks share a tile that their results are joined in groups."""
    test_attention(qv, B, T, Hq, Hkv, D, NB, lens, True, out_dtype)
