"""Buffers side by side are taken, a workspace over what a call reads is refused and nothing is written."""
import pytest
import torch

import prompt_ref as ref
from gpu_util import require_gpu
from quantized_verification_gb300 import qv

pytestmark = pytest.mark.gpu
B, T, HQ, HKV, D, P, L = 3, 2, 8, 2, 64, 100, 40


@pytest.fixture(scope="module", autouse=True)
def _built():
    require_gpu()


def arena(order, sizes):
    """Views of one buffer, one right behind the other in this order (each a multiple of 16 bytes)."""
    buf = torch.zeros(sum(sizes.values()), dtype=torch.uint8, device="cuda")
    at, views = 0, {}
    for name in order:
        views[name] = buf[at:at + sizes[name]]
        at += sizes[name]
    return buf, views


def make(order):
    need = qv.qv_attention_prefix_workspace_bytes(B, T, HQ, HKV, D, P)
    sizes = {"qkv": B * T * (HQ + 2 * HKV) * D * 2, "pk": P * HKV * D * 2, "pv": P * HKV * D * 2, "n": 16,
             "kc": B * L * HKV * D * 2, "vc": B * L * HKV * D * 2, "lens": 16, "out": B * T * HQ * D * 4, "ws": need}
    buf, v = arena(order, sizes)
    g = torch.Generator(device="cuda").manual_seed(3)
    t = {"qkv": v["qkv"].view(torch.bfloat16).view(B * T, -1), "ws": v["ws"], "n": v["n"].view(torch.int32)[:1],
         "lens": v["lens"].view(torch.int32)[:B], "out": v["out"].view(torch.float32).view(B * T, -1)}
    for name in ("pk", "pv"):
        t[name] = v[name].view(torch.bfloat16).view(P, HKV, D)
    for name in ("kc", "vc"):
        t[name] = v[name].view(torch.bfloat16).view(B, L, HKV, D)
    for name in ("qkv", "pk", "pv", "kc", "vc"):
        t[name].copy_(torch.randn(t[name].shape, generator=g, device="cuda"))
    t["n"].fill_(P)
    t["lens"].copy_(torch.tensor([40, 0, 7], dtype=torch.int32))
    t["out"].fill_(7.0)
    return buf, t


def call(t, **kw):
    t = {**t, **kw}
    qv.qv_attention_verify_prefix(t["qkv"], t["pk"], t["pv"], t["n"], t["kc"], t["vc"], t["lens"], T, HQ, HKV, 0.1, t["out"], t["ws"])


@pytest.mark.parametrize("order", ["qkv pk pv n kc vc lens out ws", "ws lens out n qkv vc kc pv pk", "out qkv ws pk kc lens pv vc n"])
def test_side_by_side(order):
    _, t = make(order.split())
    call(t)
    o, a = ref.verify_prefix(t["qkv"], t["pk"], t["pv"], P, t["kc"], t["vc"], [40, 0, 7], T, HQ, HKV, 0.1)
    assert ((t["out"].double().view(o.shape) - o).abs() <= ref.bound(o, a, torch.float32)).all()


@pytest.mark.parametrize("name", ["qkv", "pk", "pv", "n", "kc", "vc", "lens", "out"])
def test_a_workspace_over_what_is_read_is_refused(name):
    order = "qkv pk pv n kc vc lens out ws".split()
    buf, t = make([o for o in order if o not in (name, "ws")] + [name, "ws"])
    before = buf.clone()
    n = t["ws"].numel()
    with pytest.raises(qv.QVError, match="overlap"):
        call(t, ws=buf[buf.numel() - n - 16:buf.numel() - 16])     # 16 bytes into what lies before it
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    # a buffer that is longer than needed may hold something else behind what is needed
    buf, t = make(["ws", name] + [o for o in order if o not in (name, "ws")])
    call(t, ws=buf)
    torch.cuda.synchronize()
    assert not (t["out"] == 7.0).any()
