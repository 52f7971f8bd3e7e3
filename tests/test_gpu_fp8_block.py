"""GPU parity of the block-scaled 8-bit operators against the fp64 oracle, each on its own inputs.

Tolerances, from the arithmetic alone:
* quantisers: exact (powers of two divide exactly; one rounding to E4M3): codes and bytes equal.
* products: the values of the codes multiply exactly; sums are fp32. A sum of K products in any
  order errs by at most about K 2^-24 of the sum of magnitudes S; the tensor cores' sum within a
  block of 128 may truncate rather than round (one more bit), so 2 (128 + K / 128) 2^-24 S, plus
  half a step of the stored value: 2^-8 |ref| in bf16 (its type's eps / 2), 2^-24 |ref| in fp32.
* SwiGLU: e^-g by the fast exponential has 2 + 1.2 |g| ulps and the fast quotient 2, so sigmoid's
  relative error is e1 = (8 + 1.2 |g|) 2^-23 at most; the outputs follow by their formulas.
"""
import numpy as np
import pytest
import torch

from fine_grained_mixture_moe_b200 import binding as B
from oracle import moe_fp8 as F8
from oracle import moe_fp8_block as FB

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fine_grained_mixture_moe_b200 import build
    build.build()
    B.load()


def u8(*shape, fill=0xAA):
    return torch.full(shape, fill, dtype=torch.uint8, device=DEV)


def np8(t):
    return t.cpu().numpy()


def check_device():
    torch.cuda.synchronize()
    st, info = B.moe_get_device_error()
    assert st == 0, (B.status_str(st), info)


def values(rng, R, C):
    """Rows over many binades with a loud column, zeros, subnormals and block-limit values."""
    M = rng.standard_normal((R, C)) * np.exp(rng.uniform(-8, 8, (R, 1)))
    if C > 3:
        M[:, 3] *= 50
    if R > 4:
        M[1] = 0.0
        M[2, :min(C, 128)] = 448.0 * 2.0 ** -5 * np.sign(M[2, :min(C, 128)])
        M[3] *= 1e-37
        M[4, 0] = 450.0
    return M.astype(np.float32)


def torch_in(M, dtype):
    t = torch.from_numpy(M).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t.to(DEV), t.float().numpy()


def splits(kind, R, E, rng):
    """Offsets of E experts over at most R rows."""
    if kind == "even":
        c = np.full(E, R // E)
    elif kind == "empty":                    # most experts empty, the first and last among them
        c = np.zeros(E, int)
        live = rng.permutation(np.arange(1, max(E - 1, 2)))[:max(1, E // 4)] % E
        c[live] = R // len(live)
    elif kind == "none":
        c = np.zeros(E, int)
    elif kind == "drop":                     # rows behind the last kept pair
        c = rng.multinomial(R * 3 // 4, np.full(E, 1 / E))
    else:                                    # skewed, all rows
        c = rng.multinomial(R, rng.dirichlet(np.full(E, 0.5)))
    return np.concatenate([[0], np.cumsum(c)]).astype(np.int32)


# ------------------------------------------------------------------ quantisers
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", [(1, 16), (1, 1024), (7, 128), (6, 144), (33, 640), (300, 272),
                                 (5, 2064), (1000, 112)])
def test_quantize_rows(dtype, R, C):
    t, M = torch_in(values(np.random.default_rng(R * C), R, C), dtype)
    q, s = u8(R, C), u8(R, -(-C // 128))
    B.moe_quantize_fp8_block(t, R, C, q, s)
    check_device()
    rq, rs = FB.quantize_rows(M)
    assert np.array_equal(np8(s), rs)
    assert np.array_equal(np8(q), rq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [-5, 0, 1, 17, 40, 99])
def test_rows_behind_the_counter_are_left(dtype, n):
    R, C = 40, 384
    M = values(np.random.default_rng(1), R, C)
    k = min(max(n, 0), R)
    M[k:] = np.nan
    t, M = torch_in(M, dtype)
    q, s = u8(R, C), u8(R, 3)
    cnt = torch.tensor([n], dtype=torch.int32, device=DEV)
    B.moe_quantize_fp8_block(t, R, C, q, s, n_rows=cnt)
    check_device()
    rq, rs = FB.quantize_rows(M[:k])
    assert np.array_equal(np8(s)[:k], rs) and np.array_equal(np8(q)[:k], rq)
    assert (np8(q)[k:] == 0xAA).all() and (np8(s)[k:] == 0xAA).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,R,C", [(1, 16, 16), (3, 128, 128), (2, 144, 272), (5, 640, 320), (1, 48, 1040)])
@pytest.mark.parametrize("both", [True, False])
def test_quantize_weight(dtype, E, R, C, both):
    t, M = torch_in(values(np.random.default_rng(E + R), E * R, C), dtype)
    M = M.reshape(E, R, C)
    nr, nc = -(-R // 128), -(-C // 128)
    q, s = u8(E, R, C), u8(E, nr, nc)
    q_t, s_t = (u8(E, C, R), u8(E, nc, nr)) if both else (None, None)
    B.moe_quantize_fp8_weight(t, E, R, C, q, s, q_t, s_t)
    check_device()
    rq, rs = FB.quantize_weight(M)
    assert np.array_equal(np8(s), rs) and np.array_equal(np8(q), rq)
    if both:
        assert np.array_equal(np8(s_t), rs.transpose(0, 2, 1))
        assert np.array_equal(np8(q_t), rq.transpose(0, 2, 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("R,E,C,kind", [(1, 1, 16, "even"), (128, 1, 128, "even"), (129, 1, 144, "even"),
                                        (500, 7, 272, "skew"), (500, 7, 272, "drop"),
                                        (640, 12, 128, "empty"), (96, 40, 80, "skew"),
                                        (64, 5, 32, "none"), (200, 1024, 48, "skew")])
def test_quantize_tokens(dtype, R, E, C, kind):
    rng = np.random.default_rng(R + E + C)
    M = values(rng, R, C)
    offs = splits(kind, R, E, rng)
    N = int(offs[-1])
    if dtype == "e4m3":
        q0, s0 = FB.quantize_rows(M)
        q0[N:] = 0x7F                                    # NaN codes behind the last row
        x, xs = torch.from_numpy(q0).to(DEV), torch.from_numpy(s0).to(DEV)
        M = FB.values_rows(q0, s0)
    else:
        M[N:] = np.nan
        x, M = torch_in(M, dtype)
        xs = None
    nb = B.moe_fp8_token_blocks(R, E)
    q, s = u8(C, 128 * nb), u8(nb, C)
    B.moe_quantize_fp8_tokens(x, xs, R, C, torch.from_numpy(offs).to(DEV), E, q, s)
    check_device()
    rq, rs = FB.quantize_tokens(M, offs)
    n = rs.shape[0]
    assert np.array_equal(np8(s)[:n], rs)
    assert np.array_equal(np8(q)[:, :128 * n], rq)
    assert (np8(s)[n:] == 0xAA).all() and (np8(q)[:, 128 * n:] == 0xAA).all()


@pytest.mark.parametrize("span", [0, 3, 15, 16, 40])
@pytest.mark.parametrize("R,E", [(128, 1), (300, 3)])
def test_quantize_tokens_from_codes_of_any_size(span, R, E):
    """Every code magnitude, from columns of the least subnormal to columns of 448, under row scales
    that span 2^span (up to 2^15 the kernel works in fp16), with zero rows and zero columns."""
    rng = np.random.default_rng(span + R)
    C = 144
    top = np.minimum(np.arange(C) % 128, 126)            # column c holds codes up to `top`
    q0 = (rng.integers(0, 1 << 30, (R, C)) % (top + 1)).astype(np.uint8)
    q0 |= (rng.integers(0, 2, (R, C)) << 7).astype(np.uint8)
    q0[5] = 0
    s0 = (120 - rng.integers(0, span + 1, (R, 2))).astype(np.uint8)
    s0[0], s0[1] = 120, 120 - span
    offs = splits("skew" if E > 1 else "even", R, E, rng)
    nb = B.moe_fp8_token_blocks(R, E)
    q, s = u8(C, 128 * nb), u8(nb, C)
    B.moe_quantize_fp8_tokens(torch.from_numpy(q0).to(DEV), torch.from_numpy(s0).to(DEV), R, C,
                              torch.from_numpy(offs).to(DEV), E, q, s)
    check_device()
    rq, rs = FB.quantize_tokens(FB.values_rows(q0, s0), offs)
    n = rs.shape[0]
    assert np.array_equal(np8(s)[:n], rs)
    assert np.array_equal(np8(q)[:, :128 * n], rq)


# ------------------------------------------------------------------ products
def product_tol(ref, mag, K, dtype):
    return (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(ref) \
        + 2 * (128 + K / 128) * 2.0 ** -24 * mag


PRODUCTS = [  # R, E, n, k, split
    (1, 1, 16, 16, "even"), (1, 1, 1280, 1024, "even"), (6, 24, 1280, 1024, "skew"),
    (8, 3, 256, 128, "skew"), (9, 2, 144, 272, "even"), (33, 1, 128, 640, "even"),
    (40, 1, 272, 144, "even"), (300, 5, 640, 384, "skew"), (300, 5, 400, 208, "drop"),
    (700, 3, 512, 2048, "skew"), (512, 2, 256, 256, "even"), (513, 16, 896, 128, "empty"),
    (64, 8, 64, 64, "none"), (257, 1, 1040, 1168, "even"), (2000, 7, 336, 1536, "skew"),
    (2048, 1024, 128, 256, "skew"), (97, 97, 112, 48, "skew"), (4096, 4, 256, 112, "skew"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,E,n,k,kind", PRODUCTS)
def test_gemm(dtype, R, E, n, k, kind):
    rng = np.random.default_rng(R + n + k)
    offs = splits(kind, R, E, rng)
    N = int(offs[-1])
    q, s = FB.quantize_rows(rng.standard_normal((R, k)) * np.exp(rng.uniform(-4, 4, (R, 1))))
    q[N:] = 0x7F
    wq, ws = FB.quantize_weight(rng.standard_normal((E, n, k)) * np.exp(rng.uniform(-3, 3, (E, n, 1))))
    d = [torch.from_numpy(a).to(DEV) for a in (q, s, offs, wq, ws)]
    out = torch.full((R, n), -7.0, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device=DEV)
    B.moe_gemm_fp8_block(d[0], d[1], R, d[2], E, n, k, d[3], d[4], out)
    check_device()
    A, W = FB.values_rows(q[:N], s[:N]), FB.values_weight(wq, ws)
    ref, mag = FB.gemm(A, W, offs), FB.gemm(A, W, offs, absolute=True)
    got = out.float().cpu().numpy().astype(np.float64)
    err = np.abs(got[:N] - ref)
    assert np.all(err <= product_tol(ref, mag, k, dtype)), float(np.nanmax(err / np.maximum(mag, 1e-300)))
    assert (got[N:] == -7.0).all()


@pytest.mark.parametrize("R,E,n,k", [(5000, 1, 16, 16), (4200, 3, 48, 144), (6000, 1024, 32, 80),
                                     (300, 4, 640, 512)])
def test_rows_before_the_first_expert(R, E, n, k):
    """Offsets that start behind row 0 (and, from 4,097 rows, the tile form at its smallest widths):
    the product, the token quantiser and the weight gradient agree on which rows an expert has."""
    rng = np.random.default_rng(R)
    offs = splits("skew", R - 40, E, rng) + 23
    q, s = FB.quantize_rows(rng.standard_normal((R, k)))
    q[:23] = 0x7F
    q[R - 17:] = 0x7F
    wq, ws = FB.quantize_weight(rng.standard_normal((E, n, k)))
    d = [torch.from_numpy(a).to(DEV) for a in (q, s, offs.astype(np.int32), wq, ws)]
    out = torch.full((R, n), -7.0, device=DEV)
    B.moe_gemm_fp8_block(d[0], d[1], R, d[2], E, n, k, d[3], d[4], out)
    check_device()
    q[:23] = q[R - 17:] = 0
    A, W = FB.values_rows(q, s), FB.values_weight(wq, ws)
    ref, mag = FB.gemm(A, W, offs), FB.gemm(A, W, offs, absolute=True)
    live = slice(23, R - 17)
    got = out.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - ref)[live] <= product_tol(ref, mag, k, "f32")[live])
    assert (got[:23] == -7.0).all() and (got[R - 17:] == -7.0).all()
    nb = B.moe_fp8_token_blocks(R, E)
    xq, xs = u8(k, 128 * nb), u8(nb, k)
    B.moe_quantize_fp8_tokens(d[0], d[1], R, k, d[2], E, xq, xs)
    dw = torch.full((E, k, k), -7.0, device=DEV)
    if E <= 8:
        B.moe_wgrad_fp8_block(xq, xs, xq, xs, R, d[2], E, k, k, dw)
    check_device()
    rq, rs = FB.quantize_tokens(A, offs)
    m = rs.shape[0]
    assert np.array_equal(np8(xs)[:m], rs) and np.array_equal(np8(xq)[:, :128 * m], rq)
    if E <= 8:
        vals = FB.values_tokens(rq, rs).T
        V = np.zeros((R, k))
        V[live] = np.concatenate([vals[128 * b:128 * b + c] for b, c in row_blocks(offs)])
        ref, mag = FB.wgrad(V, V, offs), FB.wgrad(V, V, offs, absolute=True)
        assert np.all(np.abs(dw.cpu().numpy() - ref) <= product_tol(ref, mag, R, "f32"))


@pytest.mark.parametrize("R,n", [(3, 64), (16, 64), (600, 256)])
@pytest.mark.parametrize("idle", [(254, 254), (1, 1), (254, 1), (200, 200)])
@pytest.mark.parametrize("pair", [(240, 14), (14, 240), (254, 1), (1, 254), (127, 127), (20, 220)])
def test_gemm_scale_bytes_at_both_ends(R, n, idle, pair):
    """Two scales whose product leaves the range of fp32 on a block whose sum is zero, and ones that
    make up for each other: the result is the sum, in the form for few rows and in the other."""
    rng = np.random.default_rng(R + sum(idle) + sum(pair))
    k = 256
    q, w = (rng.integers(0, 0x7F, (m, k)).astype(np.uint8) for m in (R, n))
    q[:, 0:128:2] = 0                                    # block 0: no code meets a code
    w[:, 1:128:2] = 0
    w = w[None]
    s = np.tile(np.array([idle[0], pair[0]], np.uint8), (R, 1))
    ws = np.tile(np.array([idle[1], pair[1]], np.uint8), (1, -(-n // 128), 1))
    out = torch.empty(R, n, device=DEV)
    d = [torch.from_numpy(a).to(DEV) for a in (q, s, w, ws)]
    B.moe_gemm_fp8_block(d[0], d[1], R, None, 1, n, k, d[2], d[3], out)
    check_device()
    offs = np.array([0, R])
    A, W = FB.values_rows(q, s)[:, 128:], FB.values_weight(w, ws)[:, :, 128:]
    ref, mag = FB.gemm(A, W, offs), FB.gemm(A, W, offs, absolute=True)
    assert np.all(np.abs(out.cpu().numpy() - ref) <= product_tol(ref, mag, k, "f32"))


@pytest.mark.parametrize("R,n,k", [(1, 64, 128), (5, 256, 272), (500, 256, 384)])
def test_gemm_without_offsets(R, n, k):
    rng = np.random.default_rng(R)
    q, s = FB.quantize_rows(rng.standard_normal((R, k)))
    wq, ws = FB.quantize_weight(rng.standard_normal((1, n, k)))
    d = [torch.from_numpy(a).to(DEV) for a in (q, s, wq, ws)]
    outs = []
    for offs in (None, torch.tensor([0, R], dtype=torch.int32, device=DEV)):
        out = torch.full((R, n), -7.0, dtype=torch.float32, device=DEV)
        B.moe_gemm_fp8_block(d[0], d[1], R, offs, 1, n, k, d[2], d[3], out)
        outs.append(out)
    check_device()
    assert torch.equal(outs[0], outs[1])
    ref = FB.gemm(FB.values_rows(q, s), FB.values_weight(wq, ws), [0, R])
    mag = FB.gemm(FB.values_rows(q, s), FB.values_weight(wq, ws), [0, R], absolute=True)
    assert np.all(np.abs(outs[0].cpu().numpy() - ref) <= product_tol(ref, mag, k, "f32"))


@pytest.mark.parametrize("R,E,n,k,kind", [
    (1, 1, 16, 16, "even"), (128, 1, 256, 256, "even"), (129, 1, 144, 272, "even"),
    (700, 5, 640, 384, "skew"), (700, 5, 272, 400, "drop"), (640, 12, 128, 128, "empty"),
    (64, 8, 64, 80, "none"), (3000, 3, 1280, 256, "skew"), (300, 1024, 32, 48, "skew"),
    (5000, 2, 512, 528, "even")])
def test_wgrad(R, E, n, k, kind):
    rng = np.random.default_rng(R + n + k)
    offs = splits(kind, R, E, rng)
    M1 = rng.standard_normal((R, n)) * np.exp(rng.uniform(-4, 4, (1, n)))
    M2 = rng.standard_normal((R, k)) * np.exp(rng.uniform(-4, 4, (R, 1)))
    nb = FB.token_blocks(R, E)

    def operand(M):
        q, s = FB.quantize_tokens(M, offs)
        # what no expert's block covers holds NaN codes and wild scales
        qf = np.full((M.shape[1], 128 * nb), 0x7F, np.uint8)
        sf = np.full((nb, M.shape[1]), 250, np.uint8)
        qf[:, :q.shape[1]], sf[:s.shape[0]] = q, s
        vals = FB.values_tokens(q, s).T                  # block order -> row order
        rows = [vals[128 * b:128 * b + m] for b, m in row_blocks(offs)]
        return qf, sf, np.concatenate(rows) if rows else np.zeros((0, M.shape[1]))
    aq, as_, A = operand(M1)
    bq, bs, Bv = operand(M2)
    d = [torch.from_numpy(x).to(DEV) for x in (aq, as_, bq, bs, offs)]
    dw = torch.full((E, n, k), -7.0, dtype=torch.float32, device=DEV)
    B.moe_wgrad_fp8_block(d[0], d[1], d[2], d[3], R, d[4], E, n, k, dw)
    check_device()
    ref, mag = FB.wgrad(A, Bv, offs), FB.wgrad(A, Bv, offs, absolute=True)
    err = np.abs(dw.cpu().numpy() - ref)
    assert np.all(err <= product_tol(ref, mag, R, "f32")), float(np.max(err / np.maximum(mag, 1e-300)))


def row_blocks(offs):
    out, b = [], 0
    for a, z in FB.experts_of(offs):
        for r in range(a, z, 128):
            out.append((b, min(128, z - r)))
            b += 1
    return out


def test_no_rows():
    E, n, k = 3, 64, 128
    offs = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    w, ws = u8(E, n, k), u8(E, 1, 1)
    B.moe_gemm_fp8_block(u8(1, k), u8(1, 1), 0, offs, E, n, k, w, ws, torch.empty((1, n), device=DEV))
    dw = torch.full((E, n, k), 3.0, device=DEV)
    B.moe_wgrad_fp8_block(u8(1), u8(4), u8(1), u8(4), 0, offs, E, n, k, dw)
    check_device()
    assert not dw.any()


@pytest.mark.parametrize("bad", [[0, 50, 20, 60], [0, 1000, 1000, 1000], [-5, 10, 2 ** 31 - 1, -1],
                                 [60, 40, 20, 0], [0, 60, 0, 60]])
@pytest.mark.parametrize("R", [60, 5000])
def test_offsets_out_of_range_stay_in_bounds(bad, R):
    """Offsets that moe_permute never writes: clamped, or refused by the device where they decrease, so
    nothing outside the buffers is touched (each buffer is the middle of a larger one whose ends must
    keep their fill)."""
    E, n, k, pad = 3, 64, 128, 1 << 16
    offs = torch.tensor(bad, dtype=torch.int32, device=DEV)
    nb = B.moe_fp8_token_blocks(R, E)

    def inner(numel, dtype):
        t = torch.full((numel + 2 * pad,), 77, dtype=dtype, device=DEV)
        return t, t[pad:pad + numel]
    q, s = FB.quantize_rows(np.random.default_rng(0).standard_normal((R, k)))
    q, s = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    w, ws = u8(E, n, k, fill=0x38), u8(E, 1, 1, fill=127)
    outer = []

    def out(numel, dtype):
        o, i = inner(numel, dtype)
        outer.append((o, numel))
        return i
    B.moe_gemm_fp8_block(q, s, R, offs, E, n, k, w, ws, out(R * n, torch.float32))
    qt, st = out(k * 128 * nb, torch.uint8), out(nb * k, torch.uint8)
    B.moe_quantize_fp8_tokens(q, s, R, k, offs, E, qt, st)
    B.moe_wgrad_fp8_block(qt, st, qt, st, R, offs, E, k, k, out(E * k * k, torch.float32))
    torch.cuda.synchronize()
    clamped = np.clip(bad, 0, R)
    assert B.moe_get_device_error() == ((6, 4) if (np.diff(clamped) < 0).any() else (0, 0))
    for o, numel in outer:
        assert (o[:pad] == 77).all() and (o[pad + numel:] == 77).all()


def test_offsets_that_decrease_behind_the_last_block():
    """One row for each of the first experts, so that every block and group of rows is found among them,
    and offsets that decrease much later."""
    R, E, n, k = 64, 1024, 16, 128
    offs = np.minimum(np.arange(E + 1), R).astype(np.int32)
    nb = B.moe_fp8_token_blocks(R, E)
    assert nb == R
    q, s, w, ws = u8(R, k, fill=0x38), u8(R, 1, fill=127), u8(E, n, k, fill=0x38), u8(E, 1, 1, fill=127)
    qt, st = u8(k, 128 * nb), u8(nb, k)
    out = torch.empty(R, n, device=DEV)
    for at in (None, 40, 129, 700, 1023):
        o = offs.copy()
        if at is not None:
            o[at] = 7
        o = torch.from_numpy(o).to(DEV)
        for call in (lambda: B.moe_gemm_fp8_block(q, s, R, o, E, n, k, w, ws, out),
                     lambda: B.moe_quantize_fp8_tokens(q, s, R, k, o, E, qt, st)):
            call()
            torch.cuda.synchronize()
            assert B.moe_get_device_error() == ((0, 0) if at is None else (6, 4))
    assert B.moe_get_device_error() == (0, 0)


# ------------------------------------------------------------------ SwiGLU
def check_codes(q, s, ref, err):
    """Codes and bytes of values known to within `err` of `ref`: the byte is the scale of an amax
    within the error, each code within half a step of its value (plus the error)."""
    R, C = ref.shape
    for i in range(0, C, 128):
        a = np.abs(ref[:, i:i + 128])
        lo = FB.scale_bytes((a - err[:, i:i + 128]).max(1).clip(0))
        hi = FB.scale_bytes((a + err[:, i:i + 128]).max(1))
        b = s[:, i // 128]
        assert np.all(((b >= lo) & (b <= hi)) | (b == 127) & (a.max(1) == 0))
    scale = FB._spread(FB.scale_values(s), C, 1)
    got = F8.e4m3_decode(q) * scale
    half = np.maximum(np.abs(ref) * 2.0 ** -4, scale * 2.0 ** -10)
    assert np.all(np.abs(got - ref) <= half + 2 * err)


def gate_up(rng, R, f):
    gu = rng.standard_normal((R, 2 * f)) * np.exp(rng.uniform(-3, 3, (R, 1)))
    gu[0, :4] = [0.0, 60.0, -60.0, -100.0]               # both ends of the sigmoid
    if R > 2:
        gu[1] = 0.0
        gu[2, :f] = -1.2784645                           # where silu's slope vanishes
    return gu.astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,f", [(1, 128), (1, 640), (7, 256), (130, 384), (1001, 128)])
def test_swiglu_forward(dtype, R, f):
    t, gu = torch_in(gate_up(np.random.default_rng(R + f), R, f), dtype)
    h = torch.full((R, f), -7.0, dtype=torch.bfloat16, device=DEV)
    hq, hs, gq, gs = u8(R, f), u8(R, f // 128), u8(R, 2 * f), u8(R, 2 * f // 128)
    B.moe_swiglu_fp8_forward(t, R, f, h, hq, hs, gq, gs)
    check_device()
    rq, rs = FB.quantize_rows(gu)
    assert np.array_equal(np8(gs), rs) and np.array_equal(np8(gq), rq)
    ref = FB.swiglu(gu)
    err = (10 + 1.2 * np.abs(gu[:, :f])) * 2.0 ** -23 * np.abs(ref) + 1e-37
    assert np.all(np.abs(h.float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * err)
    check_codes(np8(hq), np8(hs), ref, err)
    # each output alone is the same
    h1, hq1, hs1, gq1, gs1 = torch.empty_like(h), u8(R, f), u8(R, f // 128), u8(R, 2 * f), u8(R, 2 * f // 128)
    B.moe_swiglu_fp8_forward(t, R, f, h=h1)
    B.moe_swiglu_fp8_forward(t, R, f, h_q=hq1, h_scale=hs1)
    B.moe_swiglu_fp8_forward(t, R, f, gu_q=gq1, gu_scale=gs1)
    check_device()
    assert all(torch.equal(a, b) for a, b in ((h, h1), (hq, hq1), (hs, hs1), (gq, gq1), (gs, gs1)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,f", [(1, 128), (1, 640), (7, 256), (130, 384), (1001, 128)])
def test_swiglu_backward(dtype, R, f):
    rng = np.random.default_rng(R + f)
    gq, gs = FB.quantize_rows(gate_up(rng, R, f))
    gu = FB.values_rows(gq, gs)
    t, dh = torch_in((rng.standard_normal((R, f)) * 1e-3).astype(np.float32), dtype)
    dgu = torch.full((R, 2 * f), -7.0, dtype=torch.bfloat16, device=DEV)
    h = torch.full((R, f), -7.0, dtype=torch.bfloat16, device=DEV)
    dq, ds = u8(R, 2 * f), u8(R, 2 * f // 128)
    d = [torch.from_numpy(a).to(DEV) for a in (gq, gs)]
    B.moe_swiglu_fp8_backward(d[0], d[1], t, R, f, dgu, dq, ds, h)
    check_device()
    ref, rh = FB.swiglu_backward(gu, dh)
    g, u = np.abs(gu[:, :f]), np.abs(gu[:, f:])
    s = 1.0 / (1.0 + np.exp(-gu[:, :f]))
    e1 = (8 + 1.2 * g) * 2.0 ** -23
    # s (1 + g (1 - s)): e1 on s, and s e1 + 2^-24 on 1 - s times g, and two fp32 roundings
    e_dg = np.abs(dh) * u * (s * (1 + g) * (e1 + 2.0 ** -22) + s * g * (s * e1 + 2.0 ** -24))
    e_du = np.abs(dh) * g * s * (e1 + 2.0 ** -22)
    err = np.concatenate([e_dg, e_du], 1) + 1e-37
    assert np.all(np.abs(dgu.float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * err)
    assert np.all(np.abs(h.float().cpu().numpy() - rh) <=
                  2.0 ** -8 * np.abs(rh) + 2 * g * s * u * (e1 + 2.0 ** -22) + 1e-37)
    check_codes(np8(dq), np8(ds), ref, err)


def test_swiglu_backward_of_large_factors():
    """dh and up whose product leaves the range of fp32 beside a slope that is zero."""
    f = 128
    gu = np.zeros((2, 2 * f), np.float32)
    gu[:, :f] = [[-2.0 ** 13], [-2.0 ** 20]]
    gu[:, f:] = 2.0 ** 100
    gq, gs = FB.quantize_rows(gu)
    d = [torch.from_numpy(a).to(DEV) for a in (gq, gs)]
    dh = torch.full((2, f), 2.0 ** 60, device=DEV)
    dgu = torch.full((2, 2 * f), -7.0, dtype=torch.bfloat16, device=DEV)
    dq, ds = u8(2, 2 * f), u8(2, 2)
    B.moe_swiglu_fp8_backward(d[0], d[1], dh, 2, f, dgu, dq, ds)
    check_device()
    assert (dgu == 0).all() and (np8(dq) & 0x7F == 0).all() and (np8(ds) == 127).all()


@pytest.mark.parametrize("n", [0, 3, 29, 50])
def test_swiglu_rows_behind_the_counter_are_left(n):
    R, f = 29, 256
    rng = np.random.default_rng(n)
    gu = gate_up(rng, R, f)
    k = min(n, R)
    gu[k:] = np.nan
    t, _ = torch_in(gu, "bf16")
    cnt = torch.tensor([n], dtype=torch.int32, device=DEV)
    h = torch.full((R, f), -7.0, dtype=torch.bfloat16, device=DEV)
    hq, hs, gq, gs = u8(R, f), u8(R, 2), u8(R, 2 * f), u8(R, 4)
    B.moe_swiglu_fp8_forward(t, R, f, h, hq, hs, gq, gs, n_rows=cnt)
    dgu = torch.full((R, 2 * f), -7.0, dtype=torch.bfloat16, device=DEV)
    h2 = h.clone()
    dq, ds = u8(R, 2 * f), u8(R, 4)
    B.moe_swiglu_fp8_backward(gq, gs, t[:, :f].contiguous(), R, f, dgu, dq, ds, h2, n_rows=cnt)
    check_device()
    for x in (h, h2, dgu):
        assert (x[k:] == -7.0).all() and torch.isfinite(x[:k]).all()
    for x in (hq, hs, gq, gs, dq, ds):
        assert (x[k:] == 0xAA).all()


# ------------------------------------------------------------------ together
class Experts8:
    """The routed SwiGLU experts in 8 bits, as a training step uses the operators."""

    def __init__(self, wg, wu, wd):
        self.E, self.f, self.d = wg.shape
        self.w1 = self._weights(torch.cat([wg, wu], 1))
        self.w2 = self._weights(wd)

    @staticmethod
    def _weights(w):
        E, r, c = w.shape
        out = u8(E, r, c), u8(E, -(-r // 128), -(-c // 128)), u8(E, c, r), u8(E, -(-c // 128), -(-r // 128))
        B.moe_quantize_fp8_weight(w.contiguous(), E, r, c, *out)
        return out

    def rows(self, x, R, C):
        q, s = u8(R, C), u8(R, -(-C // 128))
        B.moe_quantize_fp8_block(x, R, C, q, s, n_rows=self.n)
        return q, s

    def forward(self, x, offs):
        R, f, d = x.shape[0], self.f, self.d
        self.offs, self.n, self.R = offs, offs[self.E:], R
        self.x8 = self.rows(x, R, d)
        gu = torch.zeros((R, 2 * f), dtype=torch.bfloat16, device=DEV)
        B.moe_gemm_fp8_block(*self.x8, R, offs, self.E, 2 * f, d, *self.w1[:2], gu)
        h8 = u8(R, f), u8(R, f // 128)
        self.gu8 = u8(R, 2 * f), u8(R, 2 * f // 128)
        B.moe_swiglu_fp8_forward(gu, R, f, None, *h8, *self.gu8, n_rows=self.n)
        y = torch.zeros((R, d), dtype=torch.bfloat16, device=DEV)
        B.moe_gemm_fp8_block(*h8, R, offs, self.E, d, f, *self.w2[:2], y)
        return y

    def tokens(self, x, scale, C):
        nb = B.moe_fp8_token_blocks(self.R, self.E)
        q, s = u8(C, 128 * nb), u8(nb, C)
        B.moe_quantize_fp8_tokens(x, scale, self.R, C, self.offs, self.E, q, s)
        return q, s

    def backward(self, dy):
        R, f, d, E = self.R, self.f, self.d, self.E
        dy8 = self.rows(dy, R, d)
        dh = torch.zeros((R, f), dtype=torch.bfloat16, device=DEV)
        B.moe_gemm_fp8_block(*dy8, R, self.offs, E, f, d, *self.w2[2:], dh)
        dgu = torch.zeros((R, 2 * f), dtype=torch.bfloat16, device=DEV)
        h = torch.zeros((R, f), dtype=torch.bfloat16, device=DEV)
        dgu8 = u8(R, 2 * f), u8(R, 2 * f // 128)
        B.moe_swiglu_fp8_backward(*self.gu8, dh, R, f, dgu, *dgu8, h, n_rows=self.n)
        dx = torch.zeros((R, d), dtype=torch.bfloat16, device=DEV)
        B.moe_gemm_fp8_block(*dgu8, R, self.offs, E, d, 2 * f, *self.w1[2:], dx)
        dw1 = torch.full((E, 2 * f, d), -7.0, device=DEV)
        dw2 = torch.full((E, d, f), -7.0, device=DEV)
        B.moe_wgrad_fp8_block(*self.tokens(dgu, None, 2 * f), *self.tokens(*self.x8, d), R, self.offs,
                              E, 2 * f, d, dw1)
        B.moe_wgrad_fp8_block(*self.tokens(dy, None, d), *self.tokens(h, None, f), R, self.offs, E, d,
                              f, dw2)
        return dx, dw1, dw2


def permuted_layer():
    """A Quartz-shaped layer's routing and permuted rows, from the layer's own entry points."""
    from moe_synth import get_config, make_inputs
    from tests.gpu_helpers import LayerOnGpu
    c = get_config("quartz", T=200, n_shared=0, capacity_factor=1.1)
    run = LayerOnGpu(c, make_inputs(c))
    return c, run, run.steps()


def cosine(a, b):
    a, b = a.double().flatten(), b.double().flatten()
    return float(a @ b / (a.norm() * b.norm()))


def test_experts_forward_and_backward_together():
    """A training step of the experts on the rows the layer permuted, a capacity's dropped rows
    behind them, against fp64 on the unquantised weights and rows.

    An E4M3 code is off by at most 2^-4 of its value, spread about evenly over +-step / 2: relative
    rms error 2^-4 / sqrt(3) * about 0.7 (where the value lies in its binade) = 0.026 per operand.
    A product of two quantised operands whose errors are independent: 0.036 of its rms. The down
    product adds its own (h's code, W_d): sqrt(2 * 0.036^2 + 2 * 0.026^2) = 0.063; the gradients go
    through at most three products, 0.08. Twice that, 0.16, bounds each tensor's relative error, i.e.
    cosine >= 1 - 0.16^2 / 2."""
    c, run, o = permuted_layer()
    E, f, d, offs, N = c.E, c.ffn, c.d, o["offsets"], int(o["offsets"][-1])
    R = o["x_perm"].shape[0]
    assert N < R
    o["x_perm"][N:] = float("nan")
    ex = Experts8(run.w["w_gate"], run.w["w_up"], run.w["w_down"])
    y = ex.forward(o["x_perm"], offs)
    dy = (torch.randn((R, d), generator=torch.Generator().manual_seed(3)) * 1e-2).to(torch.bfloat16).to(DEV)
    dy[N:] = float("nan")
    dx, dw1, dw2 = ex.backward(dy)
    check_device()
    assert not y[N:].any() and not dx[N:].any()
    x64, dy64 = o["x_perm"].double(), dy.double()
    W1 = torch.cat([run.w["w_gate"], run.w["w_up"]], 1).double()
    W2 = run.w["w_down"].double()
    off = offs.tolist()
    for e in range(E):
        a, z = off[e], off[e + 1]
        if a == z:
            assert not dw1[e].any() and not dw2[e].any()
            continue
        x = x64[a:z].requires_grad_()
        w1, w2 = W1[e].clone().requires_grad_(), W2[e].clone().requires_grad_()
        g, u = (x @ w1.T).split(f, 1)
        yr = (torch.nn.functional.silu(g) * u) @ w2.T
        yr.backward(dy64[a:z])
        for got, ref in ((y[a:z], yr), (dx[a:z], x.grad), (dw1[e], w1.grad), (dw2[e], w2.grad)):
            ref = ref.detach()
            rel = float((got.double() - ref).norm() / ref.norm())
            assert rel <= 0.16, (e, rel)
            assert cosine(got, ref) >= 1 - 0.16 ** 2 / 2
    # the layer's own combine takes the rows
    out = torch.empty((c.T, d), dtype=torch.float32, device=DEV)
    B.moe_combine(run.cfg, y, None, o["slot_pos"], o["w"], out)
    check_device()
    assert float((out - o["y"]).norm() / o["y"].norm()) <= 0.16


def test_reproducible_streams_and_graphs():
    """The same bits from a second call, from another stream beside a busy one, and from a captured
    graph replayed on new inputs."""
    c, run, o = permuted_layer()
    N = int(o["offsets"][-1])
    ex = Experts8(run.w["w_gate"], run.w["w_up"], run.w["w_down"])
    x = o["x_perm"].clone()
    dy = torch.randn((x.shape[0], c.d), device=DEV).to(torch.bfloat16)

    def step():
        y = ex.forward(x, o["offsets"])
        return (y,) + ex.backward(dy)
    first = [t.clone() for t in step()]
    for a, b in zip(first, step()):
        assert torch.equal(a, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    res = []
    for s in (s1, s2):
        with torch.cuda.stream(s):
            res.append(step())
    torch.cuda.synchronize()
    for r in res:
        for a, b in zip(first, r):
            assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    x[:N] = x[:N].flip(0)                # (rows past N were never written by the permutation)
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in captured]
    for a, b in zip(got, step()):
        assert torch.equal(a, b)
    check_device()
    assert not torch.equal(got[0], first[0])


@pytest.mark.parametrize("call", ["gemm", "wgrad"])
def test_first_call_of_a_thread(call):
    """A thread whose first use of the GPU is a product (the driver's context is not yet bound to it)."""
    import threading
    R, n, k = 8192, 128, 256
    rng = np.random.default_rng(5)
    offs = np.array([0, R], np.int32)
    q, s = FB.quantize_rows(rng.standard_normal((R, k)))
    w, ws = FB.quantize_weight(rng.standard_normal((1, n, k)))
    xq, xs = FB.quantize_tokens(rng.standard_normal((R, k)), offs)
    d = [torch.from_numpy(a).to(DEV) for a in (q, s, offs, w, ws, xq, xs)]
    outs = [torch.empty((R, n) if call == "gemm" else (k, k), device=DEV) for _ in range(2)]
    st = torch.cuda.current_stream().cuda_stream
    status = []

    def run(out):
        p = [t.data_ptr() for t in d]
        if call == "gemm":
            status.append(B.load().moe_gemm_fp8_block(p[0], p[1], R, p[2], 1, n, k, p[3], p[4],
                                                      out.data_ptr(), 0, st))
        else:
            status.append(B.load().moe_wgrad_fp8_block(p[5], p[6], p[5], p[6], R, p[2], 1, k, k,
                                                       out.data_ptr(), st))
    run(outs[0])
    t = threading.Thread(target=run, args=(outs[1],))
    t.start()
    t.join()
    check_device()
    assert status == [0, 0]
    assert torch.equal(outs[0], outs[1])


def test_several_threads():
    """Calls of one kernel with different numbers of experts (and so different shared memory) from
    several threads at once, each on its own stream."""
    from concurrent.futures import ThreadPoolExecutor
    n = k = 128
    calls = 400

    def case(E):
        rng = np.random.default_rng(E)
        R = 8192
        offs = splits("even", R, E, rng)
        q, s = FB.quantize_rows(rng.standard_normal((R, k)))
        w, ws = FB.quantize_weight(rng.standard_normal((E, n, k)))
        d = [torch.from_numpy(a).to(DEV) for a in (q, s, offs, w, ws)]
        return R, E, d, torch.empty(R, n, device=DEV), torch.empty(R, n, device=DEV)

    def run(c):
        R, E, d, first, out = c
        st = torch.cuda.Stream()
        for i in range(calls):
            B.moe_gemm_fp8_block(d[0], d[1], R, d[2], E, n, k, d[3], d[4], out, stream=st)
        st.synchronize()
    cases = [case(E) for E in (1, 1024, 64, 512)]
    for R, E, d, first, _ in cases:
        B.moe_gemm_fp8_block(d[0], d[1], R, d[2], E, n, k, d[3], d[4], first)
    torch.cuda.synchronize()
    with ThreadPoolExecutor(len(cases)) as pool:
        for f in [pool.submit(run, c) for c in cases]:
            f.result()
    check_device()
    for R, E, d, first, out in cases:
        assert torch.equal(first, out)


def test_large_addresses():
    """Codes of more than 2^31 bytes: the last rows are quantised and multiplied like the first."""
    R, k, n = (1 << 20) + 40, 2064, 48
    need = R * k * 3 + R * n * 4
    if torch.cuda.mem_get_info()[0] < 2 * need:
        pytest.skip("not enough device memory")
    x = torch.zeros((R, k), dtype=torch.bfloat16, device=DEV)
    x[-300:] = torch.randn((300, k), device=DEV).to(torch.bfloat16)
    q, s = torch.zeros((R, k), dtype=torch.uint8, device=DEV), u8(R, 17)
    B.moe_quantize_fp8_block(x, R, k, q, s)
    rq, rs = FB.quantize_rows(x[-300:].float().cpu().numpy())
    assert np.array_equal(np8(q[-300:]), rq) and np.array_equal(np8(s[-300:]), rs)
    assert not q[:-300].any() and (s[:-300] == 127).all()
    wq, ws = FB.quantize_weight(np.random.default_rng(0).standard_normal((2, n, k)))
    out = torch.full((R, n), -7.0, device=DEV)
    offs = torch.tensor([0, R - 170, R], dtype=torch.int32, device=DEV)
    B.moe_gemm_fp8_block(q, s, R, offs, 2, n, k, torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV), out)
    check_device()
    A, W = FB.values_rows(rq, rs), FB.values_weight(wq, ws)
    ref, mag = FB.gemm(A, W, [0, 130, 300]), FB.gemm(A, W, [0, 130, 300], absolute=True)
    assert np.all(np.abs(out[-300:].cpu().numpy() - ref) <= product_tol(ref, mag, k, "f32"))
    assert not out[:-300].any()


def _room(nbytes):
    if torch.cuda.mem_get_info()[0] < 2 * nbytes:
        pytest.skip("not enough device memory")


def test_large_addresses_tokens_and_weight_gradient():
    """Transposed codes of more than 2^31 bytes: only the last rows are not zero, so the last blocks and
    the weight gradient are those of the last rows alone."""
    R, k, n, tail = (1 << 20) + 40, 2064, 48, 168          # the last block holds 40 rows
    _room(R * (3 * k + 4 * n))
    x = torch.zeros((R, k), dtype=torch.bfloat16, device=DEV)
    x[-tail:] = torch.randn((tail, k), device=DEV).to(torch.bfloat16)
    dy = torch.zeros((R, n), device=DEV)
    dy[-tail:] = torch.randn((tail, n), device=DEV)
    offs = torch.tensor([0, R], dtype=torch.int32, device=DEV)
    nb = B.moe_fp8_token_blocks(R, 1)
    out = []
    for t, C in ((dy, n), (x, k)):
        q, s = u8(C, 128 * nb), u8(nb, C)
        B.moe_quantize_fp8_tokens(t, None, R, C, offs, 1, q, s)
        out += [q, s]
    dw = torch.full((1, n, k), -7.0, device=DEV)
    B.moe_wgrad_fp8_block(*out, R, offs, 1, n, k, dw)
    check_device()
    vals = []
    for t, q, s in ((dy, out[0], out[1]), (x, out[2], out[3])):
        rq, rs = FB.quantize_tokens(t[-tail:].float().cpu().numpy(), [0, tail])
        assert np.array_equal(np8(q[:, -256:]), rq) and np.array_equal(np8(s[-2:]), rs)
        assert not q[:, :-256].any() and (s[:-2] == 127).all()
        vals.append(FB.values_tokens(rq, rs).T)
    ref, mag = vals[0].T @ vals[1], np.abs(vals[0]).T @ np.abs(vals[1])
    assert np.all(np.abs(dw[0].cpu().numpy() - ref) <= product_tol(ref, mag, tail, "f32"))


def test_large_addresses_swiglu():
    """More than 2^31 values: the last rows are what a call on them alone gives."""
    R, f, tail = (1 << 20) + 24, 1024, 64
    _room(R * f * 20)
    gu = torch.randn((R, 2 * f), device=DEV, dtype=torch.bfloat16)
    dh = torch.randn((R, f), device=DEV, dtype=torch.bfloat16)

    def both(gu, dh):
        R = gu.shape[0]
        o = [torch.empty((R, f), dtype=torch.bfloat16, device=DEV), u8(R, f), u8(R, f // 128),
             u8(R, 2 * f), u8(R, f // 64), torch.empty((R, 2 * f), dtype=torch.bfloat16, device=DEV),
             u8(R, 2 * f), u8(R, f // 64)]
        B.moe_swiglu_fp8_forward(gu, R, f, *o[:5])
        B.moe_swiglu_fp8_backward(o[3], o[4], dh, R, f, *o[5:])
        check_device()
        return o
    large = [t[-tail:].clone() for t in both(gu, dh)]
    for a, b in zip(large, both(gu[-tail:].clone(), dh[-tail:].clone())):
        assert torch.equal(a, b)
