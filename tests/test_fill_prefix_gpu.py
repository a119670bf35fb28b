"""VerifyStack.fill_prefix with prompts longer than the row-wise calls take at once, and its roundings."""
import pytest
import torch

import prompt_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
MODEL = {"hidden": 256, "kv": 128, "ffn": 512, "layers": 2, "vocab": 1000}
GAMMA, D = 3, 64
HQ, HKV = 256 // D, 128 // D


@pytest.fixture(scope="module")
def qv():
    require_gpu()
    from quantized_verification_gb300 import qv as _qv
    _qv.load()
    return _qv


def make(prefix_len, **kw):
    from quantized_verification_gb300.stack import VerifyStack
    st = VerifyStack(model=MODEL, B=2, gamma=GAMMA, seed=9)
    st.prepare_chain(head_dim=D, cache_len=20, prefix_len=prefix_len, rope_base=1e4, **kw)
    return st


def test_more_rows_than_one_call_takes(qv):
    from quantized_verification_gb300 import synth
    n, short = 66001, 300
    h = synth.activations(n, MODEL["hidden"], 77, device="cuda")
    st, few = make(n), make(short)
    out, first = st.fill_prefix(h), few.fill_prefix(h[:short])
    # causal: the first rows do not know what follows them, and the integer products are exact
    assert torch.equal(out[:short], first)
    for l in range(MODEL["layers"]):
        assert torch.equal(st.prefix_k[l][:short], few.prefix_k[l])
        assert torch.equal(st.prefix_v[l][:short], few.prefix_v[l])
    # the last rows' keys and values of layer 0, from the calls themselves
    m = 200
    xq, sx = torch.empty(m, MODEL["hidden"], dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    y = torch.empty(m, (HQ + 2 * HKV) * D, dtype=torch.bfloat16, device="cuda")
    qv.qv_rmsnorm_quant(h[-m:].clone(), st.norm_w[0][0], xq, sx, eps=st.eps)
    wq, sw = st.weights[0][0]
    qv.qv_w8a8_linear(xq, sx, wq, sw, y, qv.workspace(qv.QV_OP_LINEAR, m, xq.shape[1], wq.shape[0]))
    qg, kg = st.head_norms[0]
    qv.qv_rotary(y, torch.arange(n - m, n, dtype=torch.int32, device="cuda"), st.rope, HQ, HKV, q_gamma=qg, k_gamma=kg,
                 eps=st.eps)
    heads = y.view(m, HQ + 2 * HKV, D)
    assert torch.equal(st.prefix_k[0][-m:], heads[:, HQ:HQ + HKV])
    assert torch.equal(st.prefix_v[0][-m:], heads[:, HQ + HKV:])
    assert torch.isfinite(out.float()).all() and st.prefix_lens.item() == n
    st.enqueue_chain()
    torch.cuda.synchronize()
    assert qv.qv_device_error() == 0


def test_attention_outputs_are_quantized_from_fp32_as_a_step_s_are(qv):
    from quantized_verification_gb300 import synth
    n = 300
    st = make(n)
    prompt, quantize, seen = qv.qv_attention_prompt, qv.qv_quantize_act, []

    def spy_prompt(qkv, cu, hq, hkv, scale, out, **kw):
        prompt(qkv, cu, hq, hkv, scale, out, **kw)
        seen.append([qkv.clone(), out.clone()])

    def spy_quantize(x, xq, sx, **kw):
        quantize(x, xq, sx, **kw)
        if x.shape[1] == HQ * D:
            seen[-1].append(x.clone())

    qv.qv_attention_prompt, qv.qv_quantize_act = spy_prompt, spy_quantize
    try:
        st.fill_prefix(synth.activations(n, MODEL["hidden"], 78, device="cuda"))
    finally:
        qv.qv_attention_prompt, qv.qv_quantize_act = prompt, quantize
    assert len(seen) == MODEL["layers"]
    for qkv, out, quantized in seen:
        assert out.dtype == st.attn_out[0].dtype == torch.float32 and torch.equal(out, quantized)
        o, a = ref.prompt(qkv, [0, n], HQ, HKV, D ** -0.5)
        assert ((out.double().view(o.shape) - o).abs() <= ref.bound(o, a, torch.float32)).all()


def test_a_chain_prepared_again_without_a_prefix_has_none(qv):
    h = torch.zeros(4, MODEL["hidden"], dtype=torch.bfloat16, device="cuda")
    for kw in (dict(), dict(cache_len=20), dict(cache_len=20, kv_bits=4)):
        st = make(8)
        st.fill_prefix(h)
        st.prepare_chain(head_dim=D, **kw)
        with pytest.raises(ValueError, match="prefix_len"):
            st.fill_prefix(h)
        st.enqueue_chain()
    torch.cuda.synchronize()
    assert qv.qv_device_error() == 0
