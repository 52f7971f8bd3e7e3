"""The 8-bit training and serving operators of the experts: their cases and plain forms.

The format everywhere is block-scaled E4M3: 8-bit codes, and for every block of 128 values one
E8M0 byte b, which stands for 2^(b - 127), the least power of two with amax / scale <= 448 (1 for
an all-zero block). Blocks run along a row (1 x 128: activations, checkpoints), are square
(128 x 128: weights), or run along the rows of one expert (128 x 1: the operands of a weight
gradient).

  rows     quantise activation rows in 1 x 128 blocks
  weight   quantise stacked expert weights in 128 x 128 blocks, with the transposed copy
  tokens   quantise along an expert's rows, transposed, from bf16 rows or from 8-bit ones
  product  grouped product of quantised rows and quantised expert weights
  wgrad    weight gradient of every expert from the two transposed operands
  swiglu   h = silu(g) u in 8 bits, g and u kept as an 8-bit checkpoint
  swiglu_backward   dg, du and h from that checkpoint and dh
"""
import math

import torch

own = False

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
BLK = 128


def listed():
    return [
        # one token of a served Quartz-shaped layer: its top-6 rows before the gate/up product
        dict(name="rows_token", op="rows", rows=6, cols=1024, dtype="bf16"),
        # the permuted rows of a full training batch of the sigmoid configuration
        dict(name="rows_batch", op="rows", rows=131072, cols=1536, dtype="bf16"),
        # all gate|up weights of the Quartz configuration after an optimiser step
        dict(name="weights_gate_up", op="weight", E=24, rows=1280, cols=1024, dtype="bf16"),
        # the layer input, kept in 8 bits since the forward pass, made the weight gradient's operand
        dict(name="tokens_from_checkpoint", op="tokens", T=4096, top_k=6, E=24, cap=0.0, cols=1024,
             dtype="fp8"),
        # one token through the gate|up weights of its six experts
        dict(name="product_token", op="product", T=1, top_k=6, E=24, cap=0.0, n=1280, k=1024,
             out="bf16"),
        # a small serving batch through the down weights; few rows per expert, odd counts
        dict(name="product_serve", op="product", T=61, top_k=6, E=24, cap=0.0, n=1024, k=640,
             out="bf16"),
        # the gate|up product of the Quartz training step
        dict(name="product_train", op="product", T=4096, top_k=6, E=24, cap=0.0, n=1280, k=1024,
             out="bf16"),
        # the input gradient of the sigmoid configuration: d(gate|up) through the transposed weights
        dict(name="product_dgrad", op="product", T=32768, top_k=4, E=48, cap=0.0, n=1536, k=1536,
             out="bf16"),
        # the gate|up weight gradient of the Quartz training step
        dict(name="wgrad_gate_up", op="wgrad", T=4096, top_k=6, E=24, cap=0.0, n=1280, k=1024),
        # the down weight gradient of the capacity configuration: dropped rows, ragged experts
        dict(name="wgrad_down_capacity", op="wgrad", T=16384, top_k=3, E=32, cap=1.25, n=896,
             k=1024),
        # the SwiGLU of the Quartz training step, keeping its checkpoint
        dict(name="swiglu_train", op="swiglu", T=4096, top_k=6, ffn=640, dtype="bf16"),
        # its backward pass on a full batch of the sigmoid configuration
        dict(name="swiglu_backward", op="swiglu_backward", T=32768, top_k=4, ffn=768,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _one(rng):
    op = rng.choice(["rows", "weight", "tokens", "product", "product", "product", "wgrad", "wgrad",
                     "swiglu", "swiglu_backward"])
    wide = lambda lo, hi: 16 * _log(rng, lo // 16, hi // 16)
    E = rng.choice([8, 16, 24, 32, 48, 97, 256])
    top_k = rng.randint(1, 6)
    T = _log(rng, 1, 32768)
    cap = rng.choice([0.0, 0.0, 1.25])
    if op == "rows":
        return dict(op=op, rows=_log(rng, 1, 131072), cols=wide(64, 2048),
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "weight":
        return dict(op=op, E=rng.randint(1, 32), rows=wide(64, 2048), cols=wide(64, 2048),
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "tokens":
        return dict(op=op, T=T, top_k=top_k, E=E, cap=cap, cols=wide(64, 2048),
                    dtype=rng.choice(["bf16", "f32", "fp8"]))
    if op == "product":
        return dict(op=op, T=T, top_k=top_k, E=E, cap=cap, n=wide(64, 2048), k=wide(64, 2048),
                    out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "wgrad":
        return dict(op=op, T=T, top_k=top_k, E=E, cap=cap, n=wide(64, 1536), k=wide(64, 1536))
    return dict(op=op, T=T, top_k=top_k, ffn=128 * rng.randint(1, 12),
                dtype=rng.choice(["bf16", "bf16", "f32"]))


def draw(rng):
    most = {m: max(work(c)[m] for c in listed()) for m in ("bytes", "flops")}
    while True:
        case = _one(rng)
        w = work(case)
        if all(w[m] <= most[m] for m in most):
            return case


# ------------------------------------------------------------------ sizes

def _cdiv(a, b):
    return -(-a // b)


def _rows(case):
    return case["rows"] if "rows" in case else case["T"] * case["top_k"]


def _blocks(rows, E):
    """128-row blocks that hold any split of `rows` rows among E experts."""
    return (rows + 127 * min(rows, E)) // BLK


def _itemsize(dtype):
    return {"bf16": 2, "f32": 4, "fp8": 1}[dtype]


def work(case):
    op = case["op"]
    if op == "rows":
        R, C, b = case["rows"], case["cols"], _itemsize(case["dtype"])
        return dict(bytes=R * C * (b + 1) + R * _cdiv(C, BLK), flops=2 * R * C)
    if op == "weight":
        E, R, C, b = case["E"], case["rows"], case["cols"], _itemsize(case["dtype"])
        return dict(bytes=E * (R * C * (b + 2) + 2 * _cdiv(R, BLK) * _cdiv(C, BLK)),
                    flops=2 * E * R * C)
    R = _rows(case)
    if op == "tokens":
        C, b = case["cols"], _itemsize(case["dtype"])
        own_scale = R * _cdiv(C, BLK) if case["dtype"] == "fp8" else 0
        return dict(bytes=R * C * (b + 1) + own_scale + _cdiv(R, BLK) * C, flops=2 * R * C)
    if op == "product":
        n, k, E = case["n"], case["k"], min(case["E"], R)
        b = _itemsize(case["out"])
        return dict(bytes=R * (k + _cdiv(k, BLK)) + E * (n * k + _cdiv(n, BLK) * _cdiv(k, BLK))
                    + R * n * b, flops=2 * R * n * k)
    if op == "wgrad":
        n, k, E = case["n"], case["k"], case["E"]
        return dict(bytes=(R + _cdiv(R, BLK)) * (n + k) + 4 * E * n * k, flops=2 * R * n * k)
    f, b = case["ffn"], _itemsize(case["dtype"])
    if op == "swiglu":
        return dict(bytes=R * f * (2 * b + 3) + 3 * R * (f // BLK), flops=12 * R * f)
    return dict(bytes=R * f * (2 + b + 8) + 4 * R * (f // BLK), flops=20 * R * f)


# ------------------------------------------------------------------ the format, plain

def _scale_exponent(amax):
    """j with 2^j the least power of two such that amax / 2^j <= 448 (0 for amax = 0)."""
    m, e = torch.frexp(amax)                    # amax = m 2^e, 0.5 <= m < 1;  448 = 0.875 * 2^9
    j = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126)
    return torch.where(amax > 0, j, torch.zeros_like(j))


def _power(j):
    return ((j + 127) << 23).to(torch.int32).view(torch.float32)


def _byte(j):
    return (j + 127).to(torch.uint8)


def _quantise(v, dim):
    """Codes of fp32 `v` with one block along `dim` (or dims), and the blocks' exponents."""
    j = _scale_exponent(v.abs().amax(dim, keepdim=True))
    return (v * _power(-j)).to(E4M3), j


def _pad(v, dim, to):
    if v.shape[dim] % to == 0:
        return v
    shape = list(v.shape)
    shape[dim] = _cdiv(shape[dim], to) * to
    out = torch.zeros(shape, dtype=v.dtype, device=v.device)
    out.narrow(dim, 0, v.shape[dim]).copy_(v)
    return out


def _quantise_rows(v):
    """Codes [R, C] uint8 and scale bytes [R, ceil(C / 128)] of fp32 rows."""
    R, C = v.shape
    w = _pad(v, 1, BLK).view(R, -1, BLK)
    q, j = _quantise(w, 2)
    return (q.view(torch.uint8).reshape(R, -1)[:, :C].contiguous(),
            _byte(j).reshape(R, -1))


def _quantise_weight(v):
    """Codes [E, R, C] uint8 and scale bytes [E, ceil(R / 128), ceil(C / 128)]."""
    E, R, C = v.shape
    w = _pad(_pad(v, 1, BLK), 2, BLK)
    w = w.view(E, w.shape[1] // BLK, BLK, w.shape[2] // BLK, BLK)
    q, j = _quantise(w, (2, 4))
    q = q.view(torch.uint8).reshape(E, w.shape[1] * BLK, w.shape[3] * BLK)[:, :R, :C].contiguous()
    return q, _byte(j).reshape(E, w.shape[1], w.shape[3])


def _quantise_tokens(v, counts, blocks):
    """Codes [C, 128 blocks] uint8 and scale bytes [blocks, C], blocks along the experts' rows."""
    C = v.shape[1]
    q_t = torch.zeros((C, BLK * blocks), dtype=torch.uint8, device=v.device)
    s_t = torch.zeros((blocks, C), dtype=torch.uint8, device=v.device)
    row = at = 0
    for n in counts:
        if n:
            w = _pad(v[row:row + n], 0, BLK).view(-1, BLK, C)
            q, j = _quantise(w, 1)
            q_t[:, BLK * at:BLK * (at + w.shape[0])] = q.view(torch.uint8).reshape(-1, C).t()
            s_t[at:at + w.shape[0]] = _byte(j).reshape(-1, C)
            row, at = row + n, at + w.shape[0]
    return q_t, s_t


def _values_rows(q, s):
    """fp32 values of quantised rows."""
    C = q.shape[1]
    w = _power(s.to(torch.int32) - 127).repeat_interleave(BLK, 1)[:, :C]
    return q.view(E4M3).to(torch.float32) * w


def _values_weight(q, s):
    E, R, C = q.shape
    w = _power(s.to(torch.int32) - 127).repeat_interleave(BLK, 1)[:, :R]
    w = w.repeat_interleave(BLK, 2)[:, :, :C]
    return q.view(E4M3).to(torch.float32) * w


def _values_tokens(q_t, s_t):
    w = _power(s_t.t().to(torch.int32) - 127).repeat_interleave(BLK, 1)
    return q_t.view(E4M3).to(torch.float32) * w


# ------------------------------------------------------------------ inputs

def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _activations(gen, R, C, sigma=1.0):
    """Rows of different loudness with a few loud columns, as a normalised residual stream has."""
    v = torch.randn((R, C), generator=gen, device="cuda")
    loud = 1.0 + 15.0 * (torch.rand((1, C), generator=gen, device="cuda") < 0.01)
    row = torch.exp(0.5 * torch.randn((R, 1), generator=gen, device="cuda"))
    return v.mul_(loud).mul_(row).mul_(sigma)


def _counts(gen, case):
    """Kept rows of each expert: top-k distinct experts per token, clipped to the capacity."""
    T, k, E = case["T"], min(case["top_k"], case["E"]), case["E"]
    pull = 0.5 * torch.randn((1, E), generator=gen, device="cuda")
    noise = torch.rand((T, E), generator=gen, device="cuda").clamp_(min=1e-30)
    idx = (pull - torch.log(-torch.log(noise).clamp_(min=1e-30))).topk(k, dim=1).indices
    n = torch.bincount(idx.reshape(-1), minlength=E)
    if case["cap"] > 0:
        n = n.clamp(max=math.ceil(case["cap"] * T * k / E))
    counts = n.tolist()
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(n, 0)
    return counts, offsets


def _weights(gen, E, n, k):
    return torch.randn((E, n, k), generator=gen, device="cuda").mul_(k ** -0.5).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device="cuda")
    op = case["op"]
    st = dict(case=case)
    if op == "rows":
        R, C = case["rows"], case["cols"]
        st["x"] = _activations(gen, R, C).to(_dtype(case["dtype"]))
        st["q"], st["s"] = u8(R, C), u8(R, _cdiv(C, BLK))
    elif op == "weight":
        E, R, C = case["E"], case["rows"], case["cols"]
        st["w"] = _weights(gen, E, R, C).to(_dtype(case["dtype"]))
        st["q"], st["s"] = u8(E, R, C), u8(E, _cdiv(R, BLK), _cdiv(C, BLK))
        st["q_t"], st["s_t"] = u8(E, C, R), u8(E, _cdiv(C, BLK), _cdiv(R, BLK))
    elif op == "tokens":
        R, C, E = _rows(case), case["cols"], case["E"]
        st["counts"], st["offsets"] = _counts(gen, case)
        x = _activations(gen, R, C)
        if case["dtype"] == "fp8":
            st["x"], st["x_scale"] = _quantise_rows(x)
        else:
            st["x"], st["x_scale"] = x.to(_dtype(case["dtype"])), None
        nb = _blocks(R, E)
        st["q_t"], st["s_t"] = u8(C, BLK * nb), u8(nb, C)
    elif op == "product":
        R, n, k = _rows(case), case["n"], case["k"]
        st["counts"], st["offsets"] = _counts(gen, case)
        st["a"], st["a_scale"] = _quantise_rows(_activations(gen, R, k))
        st["w"], st["w_scale"] = _quantise_weight(_weights(gen, case["E"], n, k).float())
        st["out"] = torch.zeros((R, n), dtype=_dtype(case["out"]), device="cuda")
    elif op == "wgrad":
        R, n, k, E = _rows(case), case["n"], case["k"], case["E"]
        st["counts"], st["offsets"] = _counts(gen, case)
        nb = _blocks(R, E)
        st["a"], st["a_scale"] = _quantise_tokens(_activations(gen, R, n, 1e-3), st["counts"], nb)
        st["b"], st["b_scale"] = _quantise_tokens(_activations(gen, R, k), st["counts"], nb)
        st["dw"] = torch.zeros((E, n, k), dtype=torch.float32, device="cuda")
    else:
        R, f = _rows(case), case["ffn"]
        gu = _activations(gen, R, 2 * f)
        if op == "swiglu":
            st["gu"] = gu.to(_dtype(case["dtype"]))
            st["h_q"], st["h_s"] = u8(R, f), u8(R, f // BLK)
            st["gu_q"], st["gu_s"] = u8(R, 2 * f), u8(R, 2 * f // BLK)
        else:
            st["gu_q"], st["gu_s"] = _quantise_rows(gu)
            st["dh"] = _activations(gen, R, f, 1e-3).to(_dtype(case["dtype"]))
            st["dgu"] = torch.zeros((R, 2 * f), dtype=torch.bfloat16, device="cuda")
            st["h"] = torch.zeros((R, f), dtype=torch.bfloat16, device="cuda")
            st["dgu_q"], st["dgu_s"] = u8(R, 2 * f), u8(R, 2 * f // BLK)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    return (_run_own if own else _run_plain)(case["op"], case, st)


def _run_own(op, case, st):
    import fine_grained_mixture_moe_b200 as moe
    if op == "rows":
        moe.moe_quantize_fp8_block(st["x"], case["rows"], case["cols"], st["q"], st["s"])
        return dict(q=st["q"].view(E4M3), scale=st["s"].view(E8M0))
    if op == "weight":
        moe.moe_quantize_fp8_weight(st["w"], case["E"], case["rows"], case["cols"], st["q"],
                                    st["s"], st["q_t"], st["s_t"])
        return dict(q=st["q"].view(E4M3), scale=st["s"].view(E8M0), q_t=st["q_t"].view(E4M3),
                    scale_t=st["s_t"].view(E8M0))
    R = _rows(case)
    if op == "tokens":
        moe.moe_quantize_fp8_tokens(st["x"], st["x_scale"], R, case["cols"], st["offsets"],
                                    case["E"], st["q_t"], st["s_t"])
        return dict(q_t=st["q_t"].view(E4M3), scale_t=st["s_t"].view(E8M0))
    if op == "product":
        moe.moe_gemm_fp8_block(st["a"], st["a_scale"], R, st["offsets"], case["E"], case["n"],
                               case["k"], st["w"], st["w_scale"], st["out"])
        return st["out"]
    if op == "wgrad":
        moe.moe_wgrad_fp8_block(st["a"], st["a_scale"], st["b"], st["b_scale"], R, st["offsets"],
                                case["E"], case["n"], case["k"], st["dw"])
        return st["dw"]
    if op == "swiglu":
        moe.moe_swiglu_fp8_forward(st["gu"], R, case["ffn"], None, st["h_q"], st["h_s"],
                                   st["gu_q"], st["gu_s"])
        return dict(h=st["h_q"].view(E4M3), h_scale=st["h_s"].view(E8M0),
                    gu=st["gu_q"].view(E4M3), gu_scale=st["gu_s"].view(E8M0))
    moe.moe_swiglu_fp8_backward(st["gu_q"], st["gu_s"], st["dh"], R, case["ffn"], st["dgu"],
                                st["dgu_q"], st["dgu_s"], st["h"])
    return dict(dgu=st["dgu"], dgu_q=st["dgu_q"].view(E4M3), dgu_scale=st["dgu_s"].view(E8M0),
                h=st["h"])


def _run_plain(op, case, st):
    if op == "rows":
        q, s = _quantise_rows(st["x"].float())
        return dict(q=q.view(E4M3), scale=s.view(E8M0))
    if op == "weight":
        q, s = _quantise_weight(st["w"].float())
        return dict(q=q.view(E4M3), scale=s.view(E8M0),
                    q_t=q.transpose(1, 2).contiguous().view(E4M3),
                    scale_t=s.transpose(1, 2).contiguous().view(E8M0))
    if op == "tokens":
        x = st["x"].float() if st["x_scale"] is None else _values_rows(st["x"], st["x_scale"])
        q, s = _quantise_tokens(x, st["counts"], st["s_t"].shape[0])
        return dict(q_t=q.view(E4M3), scale_t=s.view(E8M0))
    if op == "product":
        a, w = _values_rows(st["a"], st["a_scale"]), _values_weight(st["w"], st["w_scale"])
        out, row = st["out"], 0
        for e, n in enumerate(st["counts"]):
            if n:
                out[row:row + n] = (a[row:row + n] @ w[e].t()).to(out.dtype)
                row += n
        return out
    if op == "wgrad":
        a, b = _values_tokens(st["a"], st["a_scale"]), _values_tokens(st["b"], st["b_scale"])
        dw, at = st["dw"], 0
        for e, n in enumerate(st["counts"]):
            to = at + _cdiv(n, BLK) * BLK
            dw[e] = a[:, at:to] @ b[:, at:to].t()
            at = to
        return dw
    f = case["ffn"]
    if op == "swiglu":
        gu = st["gu"].float()
        g, u = gu[:, :f], gu[:, f:]
        h = g / (1.0 + torch.exp(-g)) * u
        h_q, h_s = _quantise_rows(h)
        gu_q, gu_s = _quantise_rows(gu)
        return dict(h=h_q.view(E4M3), h_scale=h_s.view(E8M0), gu=gu_q.view(E4M3),
                    gu_scale=gu_s.view(E8M0))
    gu = _values_rows(st["gu_q"], st["gu_s"])
    g, u, dh = gu[:, :f], gu[:, f:], st["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    dgu = torch.cat([dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig], 1)
    q, s = _quantise_rows(dgu)
    return dict(dgu=dgu.to(torch.bfloat16), dgu_q=q.view(E4M3), dgu_scale=s.view(E8M0),
                h=(g * sig * u).to(torch.bfloat16))


# ------------------------------------------------------------------ the definition, in 64 bits

def _powers(lo, hi, times=1.0):
    """times * 2^i for lo <= i <= hi, exactly."""
    return torch.tensor([math.ldexp(times, i) for i in range(lo, hi + 1)], dtype=torch.float64,
                        device="cuda")


def _e4m3_64(v):
    """Nearest E4M3 value, ties to even, of |v| <= 448: spacing 2^-3 of the value's power of two,
    which is 2^-6 at least."""
    power = _powers(-6, 8)
    at = (torch.bucketize(v.abs().contiguous(), power, right=True) - 1).clamp(min=0)
    step = power[at] / 8.0
    return torch.round(v / step) * step


def _blocks_64(v, dim):
    amax = v.abs().amax(dim, keepdim=True)
    at = torch.bucketize(amax, _powers(-126, 127, 448.0))     # first 448 2^j >= amax
    scale = torch.where(amax > 0, _powers(-126, 128)[at], torch.ones_like(amax))
    return _e4m3_64(v / scale), scale


def _rows_64(v):
    parts = [_blocks_64(c, 1) for c in v.split(BLK, dim=1)]
    return torch.cat([q for q, _ in parts], 1), torch.cat([s for _, s in parts], 1)


def _e8m0_64(b):
    return _powers(-127, 128)[b.long()]


def _read_rows_64(q, s):
    return torch.cat([c * s[:, i:i + 1] for i, c in enumerate(q.double().split(BLK, dim=1))], 1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rows":
        q, s = _rows_64(st["x"].double())
        return dict(q=q, scale=s)
    if op == "weight":
        q = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        s = torch.zeros(st["s"].shape, dtype=torch.float64, device="cuda")
        for i in range(s.shape[1]):
            for j in range(s.shape[2]):
                at = (slice(None), slice(BLK * i, BLK * i + BLK), slice(BLK * j, BLK * j + BLK))
                c, sc = _blocks_64(st["w"][at].double(), (1, 2))
                q[at], s[:, i, j] = c, sc.reshape(-1)
        return dict(q=q, scale=s, q_t=q.transpose(1, 2), scale_t=s.transpose(1, 2))
    first = 0
    if op == "tokens":
        x = st["x"].double() if st["x_scale"] is None else \
            _read_rows_64(st["x"].view(E4M3), _e8m0_64(st["x_scale"]))
        q = torch.zeros(st["q_t"].shape, dtype=torch.float64, device="cuda")
        s = torch.full(st["s_t"].shape, 2.0 ** -127, dtype=torch.float64, device="cuda")
        block = 0
        for n in st["counts"]:
            for r in range(0, n, BLK):
                rows = x[first + r:first + min(r + BLK, n)]
                c, sc = _blocks_64(rows, 0)
                q[:, BLK * block:BLK * block + rows.shape[0]] = c.t()
                s[block] = sc[0]
                block += 1
            first += n
        return dict(q_t=q, scale_t=s)
    if op == "product":
        a = _read_rows_64(st["a"].view(E4M3), _e8m0_64(st["a_scale"]))
        w, ws = st["w"].view(E4M3).double(), _e8m0_64(st["w_scale"])
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        for e, n in enumerate(st["counts"]):
            for c in range(0, case["n"], BLK):
                if n:
                    we = _read_rows_64(w[e, c:c + BLK], ws[e, c // BLK:c // BLK + 1])
                    out[first:first + n, c:c + BLK] = a[first:first + n] @ we.t()
            first += n
        return out
    if op == "wgrad":
        a, b = st["a"].view(E4M3).double(), st["b"].view(E4M3).double()
        sa, sb = _e8m0_64(st["a_scale"]), _e8m0_64(st["b_scale"])
        dw = torch.zeros(st["dw"].shape, dtype=torch.float64, device="cuda")
        block = 0
        for e, n in enumerate(st["counts"]):
            for _ in range(0, n, BLK):
                cols = slice(BLK * block, BLK * block + BLK)
                dw[e] += (a[:, cols] * sa[block][:, None]) @ (b[:, cols] * sb[block][:, None]).t()
                block += 1
        return dw
    f = case["ffn"]
    if op == "swiglu":
        g, u = st["gu"].double().split(f, dim=1)
        h_q, h_s = _rows_64(g * torch.sigmoid(g) * u)
        gu_q, gu_s = _rows_64(st["gu"].double())
        return dict(h=h_q, h_scale=h_s, gu=gu_q, gu_scale=gu_s)
    g, u = _read_rows_64(st["gu_q"].view(E4M3), _e8m0_64(st["gu_s"])).split(f, dim=1)
    dh = st["dh"].double()
    s = torch.sigmoid(g)
    dgu = torch.cat([dh * u * (s + g * s * (1.0 - s)), dh * g * s], 1)
    q, sc = _rows_64(dgu)
    return dict(dgu=dgu, dgu_q=q, dgu_scale=sc, h=g * s * u)
