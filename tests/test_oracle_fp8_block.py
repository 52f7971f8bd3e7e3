"""Pins of the block-scaled E4M3 oracle: the scale against its definition in exact rationals, codes
against a brute-force nearest search, layouts against each other, and gradients against central
differences."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import moe_fp8 as F8
from oracle import moe_fp8_block as FB


def test_scale_is_the_least_power_of_two_that_fits():
    rng = np.random.default_rng(3)
    amax = np.concatenate([rng.standard_normal(200) * np.exp(rng.uniform(-60, 60, 200)),
                           [448.0, 449.0, 447.0, 1.75, 1.7500001, 1e-45, 1e-38, 3.4e38, 896.0]])
    amax = np.abs(amax).astype(np.float32)
    for a, b in zip(amax, FB.scale_bytes(amax)):
        j = int(b) - 127
        fits = Fraction(float(a)) <= 448 * Fraction(2) ** j
        assert fits
        assert j == -126 or Fraction(float(a)) > 448 * Fraction(2) ** (j - 1)
    assert FB.scale_bytes(0.0) == 127


def test_codes_are_nearest_values():
    rng = np.random.default_rng(4)
    M = (rng.standard_normal((6, 272)) * np.exp(rng.uniform(-20, 20, (6, 1)))).astype(np.float32)
    M[2, :130] = 0.0
    q, b = FB.quantize_rows(M)
    table = F8.e4m3_decode_table()
    finite = [Fraction(float(v)) for v in table[:0x7F]]
    for r, c in [(i, j) for i in range(6) for j in (0, 1, 127, 128, 129, 255, 256, 271)]:
        v = abs(Fraction(float(M[r, c]))) / Fraction(2) ** (int(b[r, c // 128]) - 127)
        best = min(abs(v - f) for f in finite)
        assert abs(v - abs(Fraction(float(table[q[r, c]])))) == best


def test_layouts_agree():
    rng = np.random.default_rng(5)
    W = rng.standard_normal((2, 200, 144)).astype(np.float32)
    q, b = FB.quantize_weight(W)
    qt, bt = FB.quantize_weight(W.transpose(0, 2, 1))
    assert np.array_equal(qt, q.transpose(0, 2, 1)) and np.array_equal(bt, b.transpose(0, 2, 1))
    # one expert whose rows start at a block: the transposed matrix in the rows layout
    M = rng.standard_normal((200, 48)).astype(np.float32)
    qt, bt = FB.quantize_tokens(M, [0, 200])
    q, b = FB.quantize_rows(M.T)
    assert np.array_equal(qt[:, :200], q) and not qt[:, 200:].any() and np.array_equal(bt, b.T)
    # error of a code: half a step (2^-4 of the value, or 2^-10 of the scale below the normals)
    err = np.abs(FB.values_rows(q, b) - M.T)
    bound = np.maximum(np.abs(M.T) * 2.0 ** -4, FB._spread(FB.scale_values(b), 200, 1) * 2.0 ** -10)
    assert np.all(err <= bound)


@pytest.mark.parametrize("rows,E", [(0, 4), (1, 4), (5, 2), (128, 1), (129, 1), (1000, 7), (3, 1000)])
def test_token_blocks_hold_any_split(rows, E):
    from fine_grained_mixture_moe_b200 import binding as B, build
    build.build()
    n = FB.token_blocks(rows, E)
    assert B.moe_fp8_token_blocks(rows, E) == n
    rng = np.random.default_rng(rows + E)
    worst = 0
    for _ in range(200):
        p = rng.dirichlet(np.full(E, rng.choice([0.05, 1.0, 20.0])))
        worst = max(worst, int(sum(-(-c // 128) for c in rng.multinomial(rows, p))))
    spread = np.zeros(E, int)                    # the worst split: one row to all but one expert
    spread[:min(rows, E)] = 1
    if rows:
        spread[0] += rows - spread.sum()
    worst = max(worst, int(sum(-(-c // 128) for c in spread)))
    assert worst <= n


def test_gradients_match_differences():
    rng = np.random.default_rng(6)
    gu, dh = rng.standard_normal((3, 2 * 8)), rng.standard_normal((3, 8))
    got, h = FB.swiglu_backward(gu, dh)
    assert np.allclose(h, FB.swiglu(gu), rtol=1e-13)
    for i in np.ndindex(*gu.shape):
        d = np.zeros_like(gu)
        d[i] = 1e-5
        num = np.sum(dh * (FB.swiglu(gu + d) - FB.swiglu(gu - d))) / 2e-5
        assert abs(num - got[i]) <= 1e-8 * (1 + abs(num))
    # product: J = sum(dy * gemm(A, W)) is bilinear, so differences are exact up to fp64
    A, W = rng.standard_normal((5, 4)), rng.standard_normal((2, 3, 4))
    offs, dy = [0, 2, 5], rng.standard_normal((5, 3))
    dW = FB.wgrad(dy, A, offs)
    dA = FB.gemm(dy, W.transpose(0, 2, 1), offs)
    for i in np.ndindex(*W.shape):
        d = np.zeros_like(W)
        d[i] = 0.5
        assert abs(np.sum(dy * (FB.gemm(A, W + d, offs) - FB.gemm(A, W - d, offs))) - dW[i]) < 1e-12
    for i in np.ndindex(*A.shape):
        d = np.zeros_like(A)
        d[i] = 0.5
        assert abs(np.sum(dy * (FB.gemm(A + d, W, offs) - FB.gemm(A - d, W, offs))) - dA[i]) < 1e-12
