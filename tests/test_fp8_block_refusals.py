"""Host refusals of the block-scaled 8-bit entry points: bad sizes, types, pointers and buffers are
answered before any device work (these run without a GPU)."""
import ctypes

import pytest
import torch

from fine_grained_mixture_moe_b200 import binding as B, build

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = 4096          # an aligned address that is never read: every call below is refused or empty


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def test_quantize_block(lib):
    f = lib.moe_quantize_fp8_block
    assert f(P, 1, -1, 32, None, P, P, None) == INVALID
    assert f(P, 1, 4, 0, None, P, P, None) == INVALID
    assert f(P, 1, 4, 24, None, P, P, None) == UNSUPPORTED
    assert f(P, 1, 4, (1 << 20) + 16, None, P, P, None) == UNSUPPORTED
    assert f(P, 2, 4, 32, None, P, P, None) == UNSUPPORTED        # codes are not an input here
    assert f(P, 1, 1 << 31, 32, None, P, P, None) == UNSUPPORTED
    assert f(None, 1, 0, 32, None, None, None, None) == OK
    for args in ((None, P, P), (P + 8, P, P), (P, None, P), (P, P + 4, P), (P, P, None)):
        assert f(args[0], 1, 4, 32, None, args[1], args[2], None) == INVALID
    assert f(P, 1, 4, 32, P + 2, P, P, None) == INVALID           # misaligned row counter


def test_quantize_weight(lib):
    f = lib.moe_quantize_fp8_weight
    assert f(P, 1, 0, 32, 32, P, P, None, None, None) == INVALID
    assert f(P, 1, 1025, 32, 32, P, P, None, None, None) == UNSUPPORTED
    assert f(P, 1, 2, 24, 32, P, P, None, None, None) == UNSUPPORTED
    assert f(P, 1, 2, 32, 40, P, P, None, None, None) == UNSUPPORTED
    assert f(P, 2, 2, 32, 32, P, P, None, None, None) == UNSUPPORTED
    assert f(P, 1, 2, 32, 32, P, P, P, None, None) == INVALID     # transposed codes without scales
    assert f(P, 1, 2, 32, 32, P, P, None, P, None) == INVALID
    assert f(None, 1, 2, 32, 32, P, P, None, None, None) == INVALID


def test_quantize_tokens(lib):
    f = lib.moe_quantize_fp8_tokens
    assert f(P, 1, None, 4, 24, P, 2, P, P, None) == UNSUPPORTED
    assert f(P, 5, None, 4, 32, P, 2, P, P, None) == UNSUPPORTED
    assert f(P, 1, None, 4, 32, None, 2, P, P, None) == INVALID
    assert f(P, 1, P, 4, 32, P, 2, P, P, None) == INVALID         # bf16 rows carry no scales
    assert f(P, 2, None, 4, 32, P, 2, P, P, None) == INVALID      # codes need theirs
    assert f(P, 1, None, 4, 32, P, 2048, P, P, None) == UNSUPPORTED
    assert f(P, 1, None, 0, 32, P, 2, None, None, None) == OK
    assert lib.moe_fp8_token_blocks(-1, 2) == -1
    assert lib.moe_fp8_token_blocks(4, 0) == -1
    assert lib.moe_fp8_token_blocks(4, 1025) == -1
    with pytest.raises(B.MoEError):
        B.moe_fp8_token_blocks(4, 0)


def test_gemm(lib):
    f = lib.moe_gemm_fp8_block
    ok = dict(a=P, s=P, rows=4, off=P, E=2, n=32, k=32, w=P, ws=P, out=P, dt=1)

    def call(**kw):
        v = dict(ok, **kw)
        return f(v["a"], v["s"], v["rows"], v["off"], v["E"], v["n"], v["k"], v["w"], v["ws"],
                 v["out"], v["dt"], None)
    assert call(rows=-1) == INVALID and call(rows=0) == OK
    assert call(n=8) == UNSUPPORTED and call(k=40) == UNSUPPORTED and call(n=0) == INVALID
    assert call(E=0) == INVALID and call(E=1025) == UNSUPPORTED
    assert call(dt=2) == UNSUPPORTED
    assert call(off=None) == INVALID                              # only one expert needs none
    assert call(E=1024, n=1 << 20, k=16, rows=1 << 30) == UNSUPPORTED
    for bad in (dict(a=None), dict(a=P + 8), dict(s=None), dict(w=None), dict(ws=None),
                dict(out=P + 8), dict(out=P + 16), dict(off=P + 2)):
        assert call(**bad) == INVALID
    # more tiles than a 32-bit tile number holds
    assert call(rows=(1 << 31) - 4096, n=1 << 20, E=1, off=None) == UNSUPPORTED


def test_wgrad(lib):
    f = lib.moe_wgrad_fp8_block
    ok = dict(a=P, s=P, b=P, bs=P, rows=4, off=P, E=2, n=32, k=32, dw=P)

    def call(**kw):
        v = dict(ok, **kw)
        return f(v["a"], v["s"], v["b"], v["bs"], v["rows"], v["off"], v["E"], v["n"], v["k"],
                 v["dw"], None)
    assert call(rows=-4) == INVALID and call(n=24) == UNSUPPORTED and call(E=-1) == INVALID
    for bad in (dict(a=None), dict(s=None), dict(b=P + 4), dict(bs=None), dict(off=None),
                dict(dw=None), dict(dw=P + 8), dict(dw=P + 16)):
        assert call(**bad) == INVALID


def test_swiglu(lib):
    f, g = lib.moe_swiglu_fp8_forward, lib.moe_swiglu_fp8_backward
    assert f(P, 1, 4, 64, None, P, None, None, None, None, None) == UNSUPPORTED  # ffn % 128
    assert f(P, 2, 4, 128, None, P, None, None, None, None, None) == UNSUPPORTED
    assert f(P, 1, 4, 128, None, None, None, None, None, None, None) == INVALID  # no output
    assert f(P, 1, 4, 128, None, None, P, None, None, None, None) == INVALID     # codes, no scales
    assert f(P, 1, 4, 128, None, P, None, None, None, P, None) == INVALID
    assert f(P + 8, 1, 4, 128, None, P, None, None, None, None, None) == INVALID
    assert f(None, 1, 0, 128, None, None, None, None, None, None, None) == OK
    assert g(P, P, P, 1, 4, 192, None, P, None, None, None, None) == UNSUPPORTED
    assert g(P, P, P, 1, 4, 128, None, None, None, None, None, None) == INVALID
    assert g(P, None, P, 1, 4, 128, None, P, None, None, None, None) == INVALID
    assert g(P, P, P, 1, 4, 128, None, None, P, None, None, None) == INVALID
    assert g(P, P, P, 7, 4, 128, None, P, None, None, None, None) == UNSUPPORTED


def test_buffers_are_checked(lib):
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.uint8)
    with pytest.raises(ValueError, match="current CUDA device"):
        B.moe_quantize_fp8_block(x, 4, 32, q, s, stream=0)
    with pytest.raises(TypeError, match="x has dtype"):
        B.moe_quantize_fp8_block(x.half(), 4, 32, q, s, stream=0)
    with pytest.raises(ValueError, match="needs 160"):
        B.moe_quantize_fp8_block(x, 5, 32, q, s, stream=0)
    with pytest.raises(ValueError, match="not contiguous"):
        B.moe_quantize_fp8_block(torch.zeros((32, 4), dtype=torch.bfloat16).t(), 4, 32, q, s, stream=0)
    with pytest.raises(TypeError, match="bf16, fp32 or E4M3"):
        B.moe_swiglu_fp8_forward(P, 4, 128, h=P, stream=0)
