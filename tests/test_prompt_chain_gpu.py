"""Rotary positions, attention over a prompt and behind a shared prefix, as the chained layers use them: a prompt becomes
the prefix of a batch, verify steps follow behind it. Tolerances are prompt_ref's; linears and norms are the chain's."""
import pytest
import torch

import prompt_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

MODEL = {"hidden": 256, "kv": 128, "ffn": 512, "layers": 2, "vocab": 1000}
B, GAMMA, D, L, P = 3, 3, 64, 50, 300
T, HQ, HKV = GAMMA + 1, 256 // D, 128 // D


@pytest.fixture(scope="module")
def qv():
    require_gpu()
    from quantized_verification_gb300 import qv as _qv
    _qv.load()
    return _qv


def make(**kw):
    from quantized_verification_gb300.stack import VerifyStack
    st = VerifyStack(model=MODEL, B=B, gamma=GAMMA, seed=9)
    st.prepare_chain(head_dim=D, **{**dict(cache_len=L, prefix_len=P, rope_base=1e4), **kw})
    if st.kv_bits == 16:
        st.cache_lens.copy_(torch.tensor([L, L - 17, 0], dtype=torch.int32))
    return st


def rotated_is_right(st, before, after, positions, l):
    qg, kg = st.head_norms[l]
    want = ref.rotate(before, positions, st.rope, HQ, HKV, q_gamma=qg, k_gamma=kg, eps=st.eps)
    # half a step of bf16, and roundings in binary32
    assert ((after.double() - want).abs() <= 2.0 ** -8 * want.abs() * 1.01 + 2.0 ** -18 * want.abs().amax()).all()


def step_is_right(st, prefix):
    """The last layer's attention, from the rotated rows still there."""
    lens = st.cache_lens.tolist()
    o, a = ref.verify_prefix(st.y_qkv, st.prefix_k[-1], st.prefix_v[-1], prefix, st.k_cache[-1], st.v_cache[-1], lens, T,
                             HQ, HKV, D ** -0.5)
    got = st.attn_out[-1].double().view(o.shape)
    assert ((got - o).abs() <= ref.bound(o, a, torch.float32)).all()


def test_steps_behind_a_seeded_prefix(qv):
    st = make()
    st.enqueue_chain()
    torch.cuda.synchronize()
    step_is_right(st, P)
    want = (P + st.cache_lens.view(-1, 1) + torch.arange(T, device="cuda")).to(torch.int32)
    assert torch.equal(st.positions, want)
    eager = [t.clone() for t in (st.tokens, st.max_logit, st.accept_len, st.attn_out[-1])]
    g = st.capture_chain()
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(eager, (st.tokens, st.max_logit, st.accept_len, st.attn_out[-1])):
        assert torch.equal(x, y)
    assert qv.qv_device_error() == 0


@pytest.mark.parametrize("n", [1, 130, 300])
def test_a_prompt_becomes_the_prefix(qv, n):
    from quantized_verification_gb300 import synth
    st = make()
    seeded = st.prefix_k[0].clone()
    h = synth.activations(n, MODEL["hidden"], 77, device="cuda")
    calls = []
    rotary, prompt = qv.qv_rotary, qv.qv_attention_prompt

    def spy_rotary(rows, positions, *a, **kw):
        before = rows.clone()
        rotary(rows, positions, *a, **kw)
        calls.append((before, rows.clone(), positions))

    def spy_prompt(qkv, cu, hq, hkv, scale, out, **kw):
        prompt(qkv, cu, hq, hkv, scale, out, **kw)
        calls[-1] += (out.clone(),)

    qv.qv_rotary, qv.qv_attention_prompt = spy_rotary, spy_prompt
    try:
        out = st.fill_prefix(h)
    finally:
        qv.qv_rotary, qv.qv_attention_prompt = rotary, prompt
    assert out.shape == h.shape and torch.isfinite(out.float()).all() and st.prefix_lens.item() == n
    assert len(calls) == MODEL["layers"]
    for l, (before, after, positions, attn) in enumerate(calls):
        assert torch.equal(positions, torch.arange(n, dtype=torch.int32, device="cuda"))
        rotated_is_right(st, before, after, positions, l)
        heads = after.view(n, HQ + 2 * HKV, D)
        assert torch.equal(st.prefix_k[l][:n], heads[:, HQ:HQ + HKV])
        assert torch.equal(st.prefix_v[l][:n], heads[:, HQ + HKV:])
        o, a = ref.prompt(after, [0, n], HQ, HKV, D ** -0.5)
        assert ((attn.double().view(o.shape) - o).abs() <= ref.bound(o, a, torch.bfloat16)).all()
    assert torch.equal(st.prefix_k[0][n:], seeded[n:])
    # layer 0's rows before rotation are the quantized linear of the normed prompt, whatever slices it ran in
    xq = torch.empty(n, MODEL["hidden"], dtype=torch.int8, device="cuda")
    sx, y = torch.empty(n, device="cuda"), torch.empty(n, (HQ + 2 * HKV) * D, dtype=torch.bfloat16, device="cuda")
    qv.qv_rmsnorm_quant(h.clone(), st.norm_w[0][0], xq, sx, eps=st.eps)
    wq, sw = st.weights[0][0]
    for r in range(0, n, 100):
        m = min(100, n - r)
        qv.qv_w8a8_linear(xq[r:r + m], sx[r:r + m], wq, sw, y[r:r + m],
                          qv.workspace(qv.QV_OP_LINEAR, m, xq.shape[1], wq.shape[0]))
    assert torch.equal(y, calls[0][0])
    # and verify steps follow behind it
    st.enqueue_chain()
    torch.cuda.synchronize()
    step_is_right(st, n)
    want = (n + st.cache_lens.view(-1, 1) + torch.arange(T, device="cuda")).to(torch.int32)
    assert torch.equal(st.positions, want)
    assert qv.qv_device_error() == 0


def test_rotary_positions_without_a_prefix(qv):
    for kw in (dict(prefix_len=None), dict(prefix_len=None, kv_bits=4)):
        st = make(**kw)
        st.enqueue_chain()
        torch.cuda.synchronize()
        want = (st.cache_lens.view(-1, 1) + torch.arange(T, device="cuda")).to(torch.int32)
        assert torch.equal(st.positions, want)
        plain = make(**kw, rope_base=None)
        plain.enqueue_chain()
        torch.cuda.synchronize()
        assert not torch.equal(st.attn_out[0], plain.attn_out[0])
        assert qv.qv_device_error() == 0


def test_refusals(qv):
    from quantized_verification_gb300.stack import VerifyStack
    st = VerifyStack(model=MODEL, B=B, gamma=GAMMA, seed=9)
    for kw in (dict(prefix_len=10), dict(cache_len=4, prefix_len=0), dict(cache_len=4, prefix_len=5, kv_bits=4),
               dict(rope_base=1e4)):
        with pytest.raises(ValueError):
            st.prepare_chain(head_dim=D, **kw)
    st.prepare_chain(cache_len=0, head_dim=D)
    with pytest.raises(ValueError):
        st.fill_prefix(torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"))
    st.prepare_chain(cache_len=0, prefix_len=8, head_dim=D)
    for bad in (torch.zeros(9, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 256, device="cuda"),
                torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(ValueError):
            st.fill_prefix(bad)
