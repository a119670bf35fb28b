"""Outputs and workspaces over what a call reads are refused on the host, before any device work. No GPU."""
import pytest

from quantized_verification_gb300 import build, qv

build.build()
# never dereferenced: every call here is refused
AT = {name: (i + 1) << 40 for i, name in enumerate(("qkv", "pk", "pv", "n", "kc", "vc", "lens", "out", "ws", "cu", "pos", "freq",
                                                    "qg", "kg"))}
B, T, HQ, HKV, D, P, L, M = 3, 2, 8, 2, 64, 100, 40, 50
SIZE = {"qkv": B * T * (HQ + 2 * HKV) * D * 2, "pk": P * HKV * D * 2, "kc": B * L * HKV * D * 2, "n": 4, "lens": B * 4}
SIZE.update(pv=SIZE["pk"], vc=SIZE["kc"])


def prefix(out_dtype=0, **at):
    p = {**AT, **at}
    return qv.load().qv_attention_verify_prefix(p["qkv"], p["pk"], p["pv"], p["n"], P, p["kc"], p["vc"], p["lens"], B, T, HQ, HKV,
                                                D, L, 0.1, p["out"], out_dtype, p["ws"], 1 << 30, None)


@pytest.mark.parametrize("name", ["qkv", "pk", "pv", "n", "kc", "vc", "lens"])
def test_prefix_outputs_over_what_is_read(name):
    for dtype, size in ((0, 4), (1, 2)):
        for at in (AT[name], AT[name] + (SIZE[name] - 4) // 16 * 16, AT[name] + 16 - B * T * HQ * D * size):
            assert prefix(dtype, out=at) == qv.QV_ERR_INVALID_ARG
            assert b"overlap" in qv.load().qv_last_error()


def test_prompt_outputs_over_the_sequences_bounds():
    def call(out, dtype):
        return qv.load().qv_attention_prompt(AT["qkv"], AT["cu"], 5, M, HQ, HKV, D, 0.1, out, dtype, None)
    for dtype, size in ((0, 4), (1, 2)):
        for at in (AT["cu"], AT["cu"] + 16, AT["cu"] + 16 - M * HQ * D * size):
            assert call(at, dtype) == qv.QV_ERR_INVALID_ARG
            assert b"overlap" in qv.load().qv_last_error()


@pytest.mark.parametrize("name,size", [("pos", 4 * M), ("freq", 4 * 32), ("qg", 2 * D), ("kg", 2 * D)])
def test_rotary_outputs_over_what_is_read(name, size):
    def call(out, dtype):
        return qv.load().qv_rotary(AT["qkv"], dtype, AT["pos"], AT["freq"], M, HQ, HKV, D, 64, 0, 1.0, AT["qg"], AT["kg"], 1e-6, out,
                                   None)
    for dtype, width in ((0, 4), (1, 2)):
        rows = M * (HQ + 2 * HKV) * D * width
        for at in (AT[name], AT[name] + (size - 4) // 16 * 16, AT[name] + 16 - rows):
            assert call(at, dtype) == qv.QV_ERR_INVALID_ARG
            assert b"overlap" in qv.load().qv_last_error()
