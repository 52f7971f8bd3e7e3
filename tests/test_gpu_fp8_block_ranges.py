"""The block-scaled 8-bit operators at the ends of their ranges, against the fp64 oracle: scale bytes
from 1 to 254, the least codes, and sums and tile lists longer than the ordinary ones.

Tolerances, from the arithmetic alone:
* token quantiser: exact, as every value code * 2^(byte - 127) has four significant bits.
* SwiGLU backward: for |g| below 128 the bounds of the ordinary cases; from there on the sigmoid is
  0 or 1 in fp32 (e^-128 < 2^-184), so an output errs by a few fp32 roundings (2^-22 of it); a
  sigmoid below 2^-126 counts as 0.
* products: fp32 sums, see :func:`sum_tol`.
"""
import numpy as np
import pytest
import torch

from fine_grained_mixture_moe_b200 import binding as B
from oracle import moe_fp8_block as FB
from tests.test_gpu_fp8_block import (DEV, check_codes, check_device, np8, product_tol, row_blocks,
                                      splits, u8)

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


# ------------------------------------------------------------------ SwiGLU backward
def backward_errors(gu, dh):
    """Reference (a sigmoid below 2^-126 counts as 0), and how far fp32 arithmetic may be off."""
    f = dh.shape[1]
    ref, rh = FB.swiglu_backward(gu, dh)
    g, u, d = np.abs(gu[:, :f]), np.abs(gu[:, f:]), np.abs(dh)
    s = 1.0 / (1.0 + np.exp(np.clip(-gu[:, :f], -700, 700)))
    zero = s < 2.0 ** -126
    ref, rh = np.where(np.tile(zero, 2), 0.0, ref), np.where(zero, 0.0, rh)
    e1 = (8 + 1.2 * np.minimum(g, 128)) * 2.0 ** -23
    near = g < 128
    gn = np.where(near, g, 0.0)
    e_slope = np.where(near, s * (1 + gn) * (e1 + 2.0 ** -22) + s * gn * (s * e1 + 2.0 ** -24), 0.0)
    e_gs = np.where(near, gn * s * (e1 + 2.0 ** -22), 0.0)
    border = np.where((s > 2.0 ** -127) & (s < 2.0 ** -125), s * (1 + g), 0.0)   # counts as 0 or not
    e_dg = d * u * (e_slope + border) + 2.0 ** -22 * np.abs(ref[:, :f])
    e_du = d * (e_gs + border) + 2.0 ** -22 * np.abs(ref[:, f:])
    e_h = u * (e_gs + border) + 2.0 ** -22 * np.abs(rh)
    # a first product below the normals of fp32 is kept to its last bit, 2^-149
    gs, slope = g * s, s * (1 + gn * (1 - s))
    e_dg += np.where(slope * u < 2.0 ** -126, d * 2.0 ** -149, 0.0)
    e_du += np.where(gs < 2.0 ** -126, d * 2.0 ** -149, 0.0)
    e_h += np.where(gs < 2.0 ** -126, u * 2.0 ** -149, 0.0)
    return ref, np.concatenate([e_dg, e_du], 1) + 2.0 ** -148, rh, e_h + 2.0 ** -148


def check_backward(gq, gs, dh, f, with_h):
    R = gq.shape[0]
    gu = FB.values_rows(gq, gs)
    ref, err, rh, eh = backward_errors(gu, dh.astype(np.float64))
    assert np.abs(ref).max() < 2.0 ** 127 and (not with_h or np.abs(rh).max() < 2.0 ** 127)
    dgu = torch.full((R, 2 * f), -7.0, dtype=torch.bfloat16, device=DEV)
    h = torch.full((R, f), -7.0, dtype=torch.bfloat16, device=DEV) if with_h else None
    dq, ds = u8(R, 2 * f), u8(R, 2 * f // 128)
    a = dev(gq, gs, dh)
    B.moe_swiglu_fp8_backward(*a, R, f, dgu, dq, ds, h)
    check_device()
    # bf16 has fp32's exponents: half a step, or half the last bit of its subnormals
    half = np.maximum(2.0 ** -8 * np.abs(ref), 2.0 ** -134)
    assert np.all(np.abs(dgu.float().cpu().numpy() - ref) <= half + 2 * err)
    if with_h:
        assert np.all(np.abs(h.float().cpu().numpy() - rh) <= np.maximum(2.0 ** -8 * np.abs(rh), 2.0 ** -134) + 2 * eh)
    check_codes(np8(dq), np8(ds), ref, err)


@pytest.mark.parametrize("gate,up,dh_power,with_h", [
    ((246, 254), (120, 130), -40, False),    # gates past the largest fp32 value
    ((120, 124), (246, 254), -40, False),    # the other factor
    ((120, 128), (246, 254), -40, False),    # beside slopes down to 2^-126
    ((246, 254), (246, 254), -60, False),
    ((40, 70), (246, 254), -40, True),
    ((246, 254), (60, 80), -60, True),
    ((236, 244), (100, 110), -40, True),     # around the byte from which the scales are split
    ((100, 110), (236, 244), -40, False),
    ((1, 9), (1, 9), 0, True),
    ((1, 9), (120, 130), 20, True),
    ((30, 254), (60, 80), -20, True),
])
def test_swiglu_backward_of_any_scale_byte(gate, up, dh_power, with_h):
    rng = np.random.default_rng(sum(gate) + 7 * sum(up))
    R, f = 70, 256
    gq = signed_codes(rng, (R, 2 * f))
    gs = np.concatenate([rng.integers(gate[0], gate[1] + 1, (R, 2)),
                         rng.integers(up[0], up[1] + 1, (R, 2))], 1).astype(np.uint8)
    gs[0], gs[1] = [gate[0], gate[1], up[0], up[1]], [gate[1], gate[0], up[1], up[0]]
    dh = (rng.uniform(1.0, 2.0, (R, f)) * 2.0 ** dh_power * rng.choice([-1, 1], (R, f))).astype(np.float32)
    gq[2, :f] = 0
    gq[3, f:] = 0x80
    dh[4] = 0
    check_backward(gq, gs, dh, f, with_h)


def test_swiglu_backward_of_the_largest_gradient():
    """A slope above 1 (at most 1.1, near g = 2.4) beside the largest dh, and an up that makes up for it."""
    R, f = 2, 128
    gu = np.full((R, 2 * f), 2.5, np.float32)
    gu[:, f:] = [[2.0 ** -10], [-2.0 ** -3]]
    gq, gs = FB.quantize_rows(gu)
    dh = np.full((R, f), torch.finfo(torch.bfloat16).max / 8, np.float32)
    dh[0] = 0.0
    dh[1] *= 1.5
    check_backward(gq, gs, dh, f, True)
    # d_up alone leaves the range here, d_gate does not
    dh = np.full((R, f), torch.finfo(torch.float32).max, np.float32)
    dgu = torch.empty((R, 2 * f), dtype=torch.bfloat16, device=DEV)
    B.moe_swiglu_fp8_backward(*dev(gq, gs, dh), R, f, dgu)
    check_device()
    ref, _ = FB.swiglu_backward(FB.values_rows(gq, gs), dh.astype(np.float64))
    assert np.all(np.abs(dgu[:, :f].float().cpu().numpy() - ref[:, :f]) <=
                  (2.0 ** -8 + 2.0 ** -20) * np.abs(ref[:, :f]))


def test_swiglu_of_the_largest_bf16_values_and_back():
    """gate and up at the ends of bf16, through the forward's own checkpoint: no NaN, the formula's
    derivative at the values that the checkpoint holds."""
    R, f = 6, 128
    big = torch.finfo(torch.bfloat16).max
    gu = np.ones((R, 2 * f), np.float32)
    gu[0, :f], gu[1, :f] = big, -big
    gu[2, f:], gu[3, f:] = big, -big
    gu[4, :f:2], gu[5, 1:f:2] = big, -big
    t = torch.from_numpy(gu).to(torch.bfloat16).to(DEV)
    gq, gs = u8(R, 2 * f), u8(R, 2 * f // 128)
    B.moe_swiglu_fp8_forward(t, R, f, gu_q=gq, gu_scale=gs)
    check_device()
    rq, rs = FB.quantize_rows(gu)
    assert np.array_equal(np8(gq), rq) and np.array_equal(np8(gs), rs)
    dh = np.random.default_rng(4).uniform(-1e-3, 1e-3, (R, f)).astype(np.float32)
    check_backward(rq, rs, dh, f, False)


# ------------------------------------------------------------------ products
@pytest.mark.parametrize("R,n", [(3, 64), (16, 64), (600, 256)])
@pytest.mark.parametrize("pair", [(1, 254), (254, 1), (1, 127), (10, 240), (240, 10), (14, 240), (1, 1)])
@pytest.mark.parametrize("most", [0x07, 0x10, 0x38])
def test_gemm_of_the_least_codes_at_both_ends(R, n, pair, most):
    """Small codes under a small scale that a large one makes up for. A sum of products of codes is a
    multiple of 2^-18 and the least scale 2^-126, so that even below fp32's normals, whose last bit
    is 2^-149, applying the smaller scale first rounds nothing."""
    rng = np.random.default_rng(R + sum(pair) + most)
    k = 272
    q, w = signed_codes(rng, (R, k), most), signed_codes(rng, (1, n, k), most)
    q[:, ::5] = 0
    s, ws = np.full((R, 3), pair[0], np.uint8), np.full((1, -(-n // 128), 3), pair[1], np.uint8)
    out = torch.empty(R, n, device=DEV)
    a, as_, b, bs = dev(q, s, w, ws)
    B.moe_gemm_fp8_block(a, as_, R, None, 1, n, k, b, bs, out)
    check_device()
    offs = np.array([0, R])
    A, W = FB.values_rows(q, s), FB.values_weight(w, ws)
    ref, mag = FB.gemm(A, W, offs), FB.gemm(A, W, offs, absolute=True)
    # an output below the normals is kept to fp32's last bit, in each of the sum's three blocks
    tol = product_tol(ref, mag, k, "f32") + (3 * 2.0 ** -149 if sum(pair) < 127 else 0.0)
    assert np.all(np.abs(out.cpu().numpy() - ref) <= tol)


def sum_tol(ref, mag, K):
    """A tile's sum stays in the tensor core's fp32 accumulator over all of K: one addition per 32 of K,
    each off by at most one last bit (2^-23, a sum that is cut off, not rounded) of the sum of
    magnitudes S, and 32 more for the additions within a step. The stored value is that fp32 sum."""
    return (K / 32 + 32) * 2.0 ** -23 * mag


def token_operand(vals, offs, nb):
    """The tokens layout of `vals`, and the values its codes stand for, in row order."""
    q, s = FB.quantize_tokens(vals, offs)
    qf = np.full((vals.shape[1], 128 * nb), 0x7F, np.uint8)
    sf = np.full((nb, vals.shape[1]), 250, np.uint8)
    qf[:, :q.shape[1]], sf[:s.shape[0]] = q, s
    v = FB.values_tokens(q, s).T
    return qf, sf, np.concatenate([v[128 * b:128 * b + m] for b, m in row_blocks(offs)])


@pytest.mark.parametrize("R,E,n,k", [(30000, 40, 640, 512), (30000, 40, 512, 640), (20000, 24, 1040, 448),
                                     (60000, 300, 256, 240)])
def test_wgrad_several_long_tiles_per_pair(R, E, n, k):
    """More tiles than twice the CTA pairs, each of several blocks of K, an odd number of them among
    them: the rounds' alternating direction, the ring of scale buffers and both accumulators over
    long tiles, with either side as the rows, and with more experts than are put in order."""
    rng = np.random.default_rng(R + E + n)
    c = rng.multinomial(R, rng.dirichlet(np.full(E, 4.0)))
    offs = np.concatenate([[0], np.cumsum(c)]).astype(np.int32)
    nb = FB.token_blocks(R, E)
    aq, as_, A = token_operand(rng.standard_normal((R, n)), offs, nb)
    bq, bs, V = token_operand(rng.standard_normal((R, k)), offs, nb)
    d = dev(aq, as_, bq, bs, offs)
    dw = torch.full((E, n, k), -7.0, device=DEV)
    B.moe_wgrad_fp8_block(*d[:4], R, d[4], E, n, k, dw)
    check_device()
    ref, mag = FB.wgrad(A, V, offs), FB.wgrad(A, V, offs, absolute=True)
    longest = int(c.max())
    assert np.all(np.abs(dw.cpu().numpy() - ref) <= sum_tol(ref, mag, longest))


@pytest.mark.parametrize("R", [65536, 131072 + 40])
def test_wgrad_of_one_sign(R):
    """The longest sums, where nothing cancels: every product is positive."""
    rng = np.random.default_rng(R)
    n, k = 256, 48
    offs = np.array([0, R], np.int32)
    nb = FB.token_blocks(R, 1)
    aq, as_, A = token_operand(np.abs(rng.standard_normal((R, n))) + 0.1, offs, nb)
    bq, bs, V = token_operand(np.abs(rng.standard_normal((R, k))) + 0.1, offs, nb)
    d = dev(aq, as_, bq, bs, offs)
    dw = torch.full((1, n, k), -7.0, device=DEV)
    B.moe_wgrad_fp8_block(*d[:4], R, d[4], 1, n, k, dw)
    check_device()
    ref = FB.wgrad(A, V, offs)
    assert np.all(np.abs(dw.cpu().numpy() - ref) <= sum_tol(ref, ref, R))


@pytest.mark.parametrize("R", [3, 600])
def test_gemm_of_one_sign(R):
    rng = np.random.default_rng(R)
    n, k = 256, 65536 + 144
    q, s = FB.quantize_rows(np.abs(rng.standard_normal((R, k))) + 0.1)
    w, ws = FB.quantize_weight(np.abs(rng.standard_normal((1, n, k))) + 0.1)
    out = torch.empty(R, n, device=DEV)
    a, as_, b, bs = dev(q, s, w, ws)
    B.moe_gemm_fp8_block(a, as_, R, None, 1, n, k, b, bs, out)
    check_device()
    ref = FB.gemm(FB.values_rows(q, s), FB.values_weight(w, ws), [0, R])
    assert np.all(np.abs(out.cpu().numpy() - ref) <= sum_tol(ref, ref, k))


def test_wgrad_tile_longer_than_a_wait():
    """One tile whose sum takes longer than the bound on a single wait: each step comes in time, so no wait
    may run out, the one for the finished tile among them."""
    R, n = 1 << 22, 16
    offs = torch.tensor([0, R], dtype=torch.int32, device=DEV)
    nb = B.moe_fp8_token_blocks(R, 1)
    x = torch.randn((R, n), device=DEV).to(torch.bfloat16)
    q, s = u8(n, 128 * nb), u8(nb, n)
    B.moe_quantize_fp8_tokens(x, None, R, n, offs, 1, q, s)
    outs = [torch.full((1, n, n), -7.0, device=DEV) for _ in range(2)]
    B.moe_wgrad_fp8_block(q, s, q, s, R, offs, 1, n, n, outs[0])
    check_device()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    B.moe_debug_set(B.DEBUG_WAIT_LIMIT_NS, 1_000_000)
    try:
        start.record()
        B.moe_wgrad_fp8_block(q, s, q, s, R, offs, 1, n, n, outs[1])
        end.record()
        check_device()
    finally:
        B.moe_debug_set(B.DEBUG_WAIT_LIMIT_NS, 2_000_000_000)
    assert start.elapsed_time(end) > 1.0                     # (the case is what it says)
    assert torch.equal(outs[0], outs[1])
