"""The 4-bit cache, its attention and the log probabilities in the chained verify step: steps that follow one another,
each attending to what the ones before it wrote, eagerly and as a captured graph. Tolerances are those of
test_kv4_gpu.py and test_logprobs_gpu.py; the cache is compared byte for byte."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import np_, require_gpu
from test_kv4_gpu import close
from test_logprobs_gpu import check

pytestmark = pytest.mark.gpu

MODEL = {"hidden": 256, "kv": 128, "ffn": 512, "layers": 2, "vocab": 1000}
B, GAMMA, D, L = 3, 3, 64, 50
T, HQ, HKV = GAMMA + 1, 256 // D, 128 // D


@pytest.fixture(scope="module")
def qv():
    require_gpu()
    from quantized_verification_gb300 import qv as _qv
    _qv.load()
    return _qv


def make(room, **sampling):
    from quantized_verification_gb300.stack import VerifyStack
    st = VerifyStack(model=MODEL, B=B, gamma=GAMMA, seed=9)
    st.prepare_chain(cache_len=L, head_dim=D, kv_bits=4, room=room)
    if sampling:
        st.prepare_sampling(**sampling)
    st.cache_lens.copy_(torch.tensor([L, L - 17, 0], dtype=torch.int32))
    return st


def step_is_right(st, before, lens):
    """The last layer's attention and the cache it left, from the qkv rows still there."""
    nb = st.block_table.shape[1]
    table, scale = np_(st.block_table), float(np.float32(D ** -0.5))
    x = np_(st.y_qkv.float())
    want, vmax, smax = ref.attend(x, before, lens, T, HQ, HKV, D, nb, scale, table)
    close(st.attn_out[-1], want, vmax, smax, D)
    assert np.array_equal(np_(st.kv4_cache[-1]), ref.write(before, x, lens, T, HQ, HKV, D, nb, table))


def test_seeded_positions(qv):
    """The cache holds the bf16 cache's positions, rounded to the format, and cached() gives them back."""
    from quantized_verification_gb300.stack import VerifyStack
    st = make(room=9)
    sb = VerifyStack(model=MODEL, B=B, gamma=GAMMA, seed=9, share_weights=st)
    sb.prepare_chain(cache_len=L, head_dim=D)
    for l in range(MODEL["layers"]):
        k, v = st.cached(l)
        kb, vb = sb.cached(l)
        assert k.shape == (B, 64, HKV, D) and kb.shape == (B, L, HKV, D)
        for a, b in ((k, kb), (v, vb)):
            q, byte = ref.quantize(np_(b.float()).reshape(-1, D))
            assert np.array_equal(np_(a[:, :L].double()).reshape(-1, D), ref.values(q, byte))


def test_greedy_steps(qv):
    """Three steps over growing caches; the third has no room for all of its rows."""
    st = make(room=9)
    cap = st.block_table.shape[1] * 32
    lens = np.array([L, L - 17, 0])
    for n in range(3):
        if n == 2:
            lens = np.array([cap - 2, lens[1], cap])
            st.cache_lens.copy_(torch.from_numpy(lens.astype(np.int32)))
        before = np_(st.kv4_cache[-1]).copy()
        st.drafts.random_(0, MODEL["vocab"])
        st.enqueue_chain()
        step_is_right(st, before, lens)
        st.advance_chain()
        lens = np.minimum(lens + np_(st.accept_len), cap)
        assert np.array_equal(np_(st.cache_lens), lens)
    assert qv.qv_device_error() == 0


def test_sampled_steps_with_logprobs(qv):
    st = make(room=20, temperature=0.9, seed=5, top_logprobs=4)
    lens = np.array([L, L - 17, 0])
    for n in range(3):
        before = np_(st.kv4_cache[-1]).copy()
        st.enqueue_chain_sampled()
        step_is_right(st, before, lens)
        assert int(st.accept_len.min()) >= 1 and int(st.accept_len.max()) <= T
        check(st.logits, st.out_tokens.view(-1), 4,
              (st.logprob.view(-1), st.entropy.view(-1), st.top_tokens.view(-1, 4), st.top_logprobs.view(-1, 4)))
        assert bool((st.logprob[st.out_tokens < 0] == 0).all()) and bool((st.logprob[st.out_tokens >= 0] < 0).all())
        st.advance_chain()
        lens = lens + np_(st.accept_len)
        assert np.array_equal(np_(st.cache_lens), lens)
        st.h0.copy_(st.h0.roll(1, 0))                          # other rows in the next step
    assert qv.qv_device_error() == 0


def test_captured_steps_equal_eager_ones(qv):
    """Step and advance in one graph, replayed: the same caches, tokens and log probabilities as eager steps."""
    runs = []
    for graph in (False, True):
        st = make(room=20, temperature=0.9, seed=5, top_logprobs=0)
        for c in st.kv4_cache:                                 # the bytes never written are the same in both runs
            c.view(-1, 34 * D)[st.block_table[:, -1].long().repeat_interleave(HKV) * HKV
                               + torch.arange(HKV, device="cuda").repeat(B)] = 0x5A
        st.cache_lens.clamp_(max=64)
        start = [c.clone() for c in st.kv4_cache], st.cache_lens.clone()

        def step(stream=None):
            st.enqueue_chain_sampled(stream)
            st.advance_chain(stream)
        g = st._capture(step, st.device) if graph else None    # (one eager step before the capture: undone here)
        for c, s in zip(st.kv4_cache, start[0]):
            c.copy_(s)
        st.cache_lens.copy_(start[1])
        seen = []
        for _ in range(3):
            g.replay() if graph else step()
            torch.cuda.synchronize()
            seen.append([t.clone() for t in (st.cache_lens, st.out_tokens, st.accept_len, st.logprob, st.entropy,
                                             *st.kv4_cache, *st.attn_out)])
        runs.append(seen)
    for a, b in zip(*runs):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_logprobs_are_asked_for(qv):
    st = make(room=4, temperature=0.8, seed=1)
    st.enqueue_chain_sampled()
    assert not hasattr(st, "logprob")


def test_refusals(qv):
    from quantized_verification_gb300.stack import VerifyStack
    st = VerifyStack(model=MODEL, B=1, gamma=1, seed=2)
    for kw in (dict(kv_bits=8, cache_len=4, head_dim=D), dict(kv_bits=4), dict(room=3),
               dict(cache_len=4, room=3, head_dim=D), dict(cache_len=-1, head_dim=D),
               dict(cache_len=4, room=-2, kv_bits=4, head_dim=D), dict(cache_len=0, room=0, kv_bits=4, head_dim=D)):
        with pytest.raises(ValueError):
            st.prepare_chain(**kw)
    with pytest.raises(ValueError):
        st.advance_chain()
    with pytest.raises(ValueError):
        st.cached(0)
    st.prepare_chain(cache_len=0, head_dim=D, kv_bits=4)               # nothing cached yet, space for one step's rows
    st.enqueue_chain()
    st.advance_chain()
    assert np.array_equal(np_(st.cache_lens), np_(st.accept_len)) and st.cached(0)[0].shape[1] == 32
    assert bool(st.attn_out[-1].isfinite().all()) and qv.qv_device_error() == 0
