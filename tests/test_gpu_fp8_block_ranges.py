"""The block-scaled 8-bit operators at the ends of their ranges, against the fp64 oracle.

Tolerances, from the arithmetic alone:
* token quantiser: exact, as every value code * 2^(byte - 127) has four significant bits.
"""
import numpy as np
import pytest
import torch

from fine_grained_mixture_moe_b200 import binding as B
from oracle import moe_fp8_block as FB
from tests.test_gpu_fp8_block import DEV, check_device, np8, splits, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fine_grained_mixture_moe_b200 import build
    build.build()
    B.load()


def dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for a in arrays]


def signed_codes(rng, shape, most=0x7E):
    """Codes of magnitudes 0 .. most (0x7E: 448), both signs."""
    return (rng.integers(0, most + 1, shape) | rng.integers(0, 2, shape) << 7).astype(np.uint8)


# ------------------------------------------------------------------ token quantiser
def check_tokens(q0, s0, offs):
    R, C = q0.shape
    E = len(offs) - 1
    nb = B.moe_fp8_token_blocks(R, E)
    q, s = u8(C, 128 * nb), u8(nb, C)
    x, xs, o = dev(q0, s0, offs)
    B.moe_quantize_fp8_tokens(x, xs, R, C, o, E, q, s)
    check_device()
    rq, rs = FB.quantize_tokens(FB.values_rows(q0, s0), offs)
    n = rs.shape[0]
    assert np.array_equal(np8(s)[:n], rs)
    assert np.array_equal(np8(q)[:, :128 * n], rq)


@pytest.mark.parametrize("lo,hi", [(1, 1), (1, 9), (118, 136), (238, 254), (246, 247), (247, 254),
                                   (254, 254), (1, 254)])
@pytest.mark.parametrize("most", [0x7E, 0x08])
@pytest.mark.parametrize("R,E", [(128, 1), (300, 3)])
def test_quantize_tokens_of_any_scale_byte(lo, hi, most, R, E):
    """Rows of any valid scale byte; with bytes of both ends in one block, also columns where the
    loud rows hold zeros, so that a column's own scale lies at the other end."""
    rng = np.random.default_rng(lo + 300 * hi + most + R)
    C = 144
    q0 = signed_codes(rng, (R, C), most)
    s0 = rng.integers(lo, hi + 1, (R, 2)).astype(np.uint8)
    s0[0], s0[R - 1] = lo, hi
    q0[5] = 0
    for c in range(0, C, 3):                             # only the rows up to a limit, another per column
        limit = lo + (hi - lo) * c // C
        q0[s0[:, c // 128] > limit, c] &= 0x80           # (a zero keeps its sign)
    check_tokens(q0, s0, splits("skew" if E > 1 else "even", R, E, rng))


def test_quantize_tokens_of_one_loud_row():
    """One row of byte 254 among rows of byte 1, in one block: its zeros leave the other rows' columns
    as they are without it."""
    R, C = 128, 32
    rng = np.random.default_rng(9)
    q0, s0 = signed_codes(rng, (R, C)), np.ones((R, 1), np.uint8)
    s0[77] = 254
    q0[77, ::2] = 0
    check_tokens(q0, s0, np.array([0, R], np.int32))


def test_quantize_tokens_of_the_largest_bf16_rows():
    """The largest bf16 value rounds up to 2^128 as a code; the checkpoint is read all the same."""
    R, C = 200, 128
    M = np.random.default_rng(3).standard_normal((R, C)).astype(np.float32) * 2.0 ** 100
    big = torch.finfo(torch.bfloat16).max
    M[::7] = big
    M[1::7, ::2] = -big
    x = torch.from_numpy(M).to(torch.bfloat16).to(DEV)
    q, s = u8(R, C), u8(R, 1)
    B.moe_quantize_fp8_block(x, R, C, q, s)
    check_device()
    rq, rs = FB.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(np8(q), rq) and np.array_equal(np8(s), rs) and rs.max() == 247
    check_tokens(rq, rs, np.array([0, 90, R], np.int32))
