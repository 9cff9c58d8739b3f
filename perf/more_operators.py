"""The 8-bit operators with block scales as a measuring tool sees them: the cases, their inputs, a plain form in
elementary torch operations, the library's calls, the work a pass cannot do without, and the exact results.

Three kinds of pass:
  quantize  x [rows, cols] -> e4m3 codes and one fp32 scale per block, and the values read back from them
  gemm      D = alpha * A B^T + bias of two 8-bit operands: activations A (a scale per 128 columns of a row) and
            weights B (a scale per block of 128 x 128)
  rms       total = x + residual, the RMS norm of it (* gamma + beta, SiLU) written as an 8-bit operand; the total
            and the values read back

A block's scale is the fp32 quotient max|x| / 448, at least 2^-126; its codes round the fp32 quotients x / scale to e4m3
(nearest, ties to even).  codes [rows, cols rounded up to 16], zeros behind the last column; scales [column blocks, row
blocks], a row block being one row (activations) or 128 (weights).
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 128


def ceil_to(n, m):
    return -(-n // m) * m


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token's activations before a projection: latency
        {"name": "quantize_token", "op": "quantize", "rows": 1, "cols": 4096, "dtype": "bf16", "block_rows": 1},
        # activations of one 81-frame clip at the mid block (21 x 44 x 80 tokens, 1024 channels)
        {"name": "quantize_clip", "op": "quantize", "rows": 73920, "cols": 1024, "dtype": "bf16", "block_rows": 1},
        # packing a projection's fp32 weights at create time
        {"name": "quantize_weight", "op": "quantize", "rows": 4096, "cols": 4096, "dtype": "fp32", "block_rows": 128},
        # rows and columns that fill no block, rows that start off a vector boundary
        {"name": "quantize_ragged", "op": "quantize", "rows": 5003, "cols": 1001, "dtype": "fp32", "block_rows": 1},
        # one token through a projection: the weights' bytes
        {"name": "gemm_token", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "out": "bf16", "bias": False},
        # a small batch of tokens served together
        {"name": "gemm_batch", "op": "gemm", "m": 48, "n": 8192, "k": 2048, "out": "bf16", "bias": True},
        # one latent frame's tokens (44 x 80) through a 1024-channel projection
        {"name": "gemm_frame", "op": "gemm", "m": 3520, "n": 1024, "k": 1024, "out": "bf16", "bias": True},
        # a wide product whose time is the multiplications'
        {"name": "gemm_wide", "op": "gemm", "m": 16384, "n": 4096, "k": 4096, "out": "bf16", "bias": False},
        # odd everything: output columns that fit no vector, a K that ends inside a block; fp32 result
        {"name": "gemm_ragged", "op": "gemm", "m": 777, "n": 333, "k": 1000, "out": "fp32", "bias": True},
        # one token's norm between two blocks
        {"name": "rms_token", "op": "rms", "rows": 1, "cols": 4096, "dtype": "bf16", "res": "bf16", "silu": False},
        # a clip's tokens, fp32 residual stream
        {"name": "rms_clip", "op": "rms", "rows": 73920, "cols": 1024, "dtype": "bf16", "res": "fp32", "silu": False},
        # a narrow stage's pixels, odd width, with SiLU
        {"name": "rms_ragged", "op": "rms", "rows": 40013, "cols": 333, "dtype": "bf16", "res": "bf16", "silu": True},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("quantize", "gemm", "gemm", "rms"))
    if op == "gemm":
        n, k = spread(16, 8192), spread(32, 8192)
        if rng.random() < 0.6:  # projections between channel counts
            n, k = ceil_to(n, 64), ceil_to(k, 64)
        m = spread(1, min(100000, 60_000_000 // max(n, k)))
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(("bf16", "bf16", "fp32")), "bias": rng.random() < 0.5}
    cols = spread(16, 8192)
    if rng.random() < 0.6:
        cols = ceil_to(cols, 32)
    rows = spread(1, min(150000, 70_000_000 // cols))
    case = {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(("bf16", "fp32"))}
    if op == "quantize":
        return {**case, "block_rows": rng.choice((1, 1, 128))}
    return {**case, "res": rng.choice(("bf16", "fp32")), "silu": rng.random() < 0.4}


# ------------------------------------------------------------------------------------------------ inputs
def activations(shape, gen):
    """Activations: normal, a gain per channel, a few channels that run hot."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return x * torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device="cuda"))


def buffers(rows, cols, block_rows):
    return (torch.empty((rows, ceil_to(cols, 16)), dtype=torch.float8_e4m3fn, device="cuda"),
            torch.empty((-(-cols // BLOCK), -(-rows // block_rows)), dtype=torch.float32, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = quantize_plain(activations((m, k), gen), 1)
        s["b"] = quantize_plain(torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k), BLOCK)
        s["bias"] = 0.1 * torch.randn(n, generator=gen, device="cuda") if case["bias"] else None
        s["d"] = torch.empty((m, n), dtype=DTYPE[case["out"]], device="cuda")
        return s
    shape = (case["rows"], case["cols"])
    s["x"] = activations(shape, gen).to(DTYPE[case["dtype"]])
    if case["op"] == "quantize":
        s["codes"], s["scales"] = buffers(*shape, case["block_rows"])
        s["y"] = torch.empty_like(s["x"])
        return s
    s["residual"] = (2.0 * activations(shape, gen)).to(DTYPE[case["res"]])
    s["gamma"] = 1.0 + 0.2 * torch.randn(shape[1], generator=gen, device="cuda")
    s["beta"] = 0.1 * torch.randn(shape[1], generator=gen, device="cuda")
    s["total"] = torch.empty_like(s["residual"])
    s["codes"], s["scales"] = buffers(*shape, 1)
    s["y"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ a pass
def run(s):
    if own:
        return run_own(s)
    if s["op"] == "quantize":
        return values_plain(*quantize_plain(s["x"].float(), s["block_rows"]), s["cols"], s["block_rows"]).to(s["x"].dtype)
    if s["op"] == "gemm":
        d = values_plain(*s["a"], s["k"], 1) @ values_plain(*s["b"], s["k"], BLOCK).t()
        return (d + s["bias"] if s["bias"] is not None else d).to(s["d"].dtype)
    h = s["x"].float() + s["residual"].float()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["gamma"] + s["beta"]
    if s["silu"]:
        y = y / (1.0 + torch.exp(-y))
    return h.to(s["residual"].dtype), values_plain(*quantize_plain(y, 1), s["cols"], 1).to(s["y"].dtype)


def run_own(s):
    from patch_tiled_causal_gb300 import vaedec as vd
    if s["op"] == "quantize":
        vd.quantize_fp8(s["x"], s["codes"], s["scales"], block_rows=s["block_rows"])
        return vd.dequantize_fp8(s["codes"], s["scales"], s["y"], block_rows=s["block_rows"])
    if s["op"] == "gemm":
        return vd.gemm_fp8(*s["a"], *s["b"], s["d"], s["k"], bias=s["bias"])
    vd.residual_rmsnorm_silu_fp8(s["x"], s["residual"], s["gamma"], s["beta"], s["total"], s["codes"], s["scales"],
                                 eps=1e-6, silu=s["silu"])
    return s["total"], vd.dequantize_fp8(s["codes"], s["scales"], s["y"])


# ------------------------------------------------------------------------------------------------ the plain form
def quantize_plain(x, block_rows):
    """fp32 x [rows, cols] -> e4m3 codes [rows, pitch], fp32 scales [column blocks, row blocks]."""
    rows, cols = x.shape
    nr, nc = -(-rows // block_rows), -(-cols // BLOCK)
    x = torch.nn.functional.pad(x, (0, nc * BLOCK - cols, 0, nr * block_rows - rows))
    x = x.reshape(nr, block_rows, nc, BLOCK)
    amax = x.abs().amax((1, 3))
    scale = (amax / torch.full_like(amax, 448.0)).clamp(min=2.0 ** -126)
    codes = (x / scale[:, None, :, None]).to(torch.float8_e4m3fn).reshape(nr * block_rows, nc * BLOCK)
    return codes[:rows, :ceil_to(cols, 16)].contiguous(), scale.t().contiguous()


def values_plain(codes, scales, cols, block_rows):
    """Codes and scales -> fp32 [rows, cols]."""
    rows = codes.shape[0]
    scale = scales.t().repeat_interleave(block_rows, dim=0)[:rows].repeat_interleave(BLOCK, dim=1)[:, :cols]
    return codes[:, :cols].float() * scale


# ------------------------------------------------------------------------------------------------ work
def operand_bytes(rows, cols, block_rows):
    return rows * cols + 4 * -(-rows // block_rows) * -(-cols // BLOCK)


def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": operand_bytes(m, k, 1) + operand_bytes(n, k, BLOCK) + m * n * size[case["out"]] + 4 * n * case["bias"],
                "flops": 2 * m * n * k}
    n = case["rows"] * case["cols"]
    if case["op"] == "quantize":  # x in; codes and scales out and in again; values out
        return {"bytes": 2 * n * size[case["dtype"]] + 2 * operand_bytes(case["rows"], case["cols"], case["block_rows"]),
                "flops": 4 * n}
    # x and the residual in, the total out; gamma and beta in; the operand out and in again; values out
    return {"bytes": n * (size[case["dtype"]] + 2 * size[case["res"]] + 2) + 8 * case["cols"]
            + 2 * operand_bytes(case["rows"], case["cols"], 1), "flops": 12 * n}


# ------------------------------------------------------------------------------------------------ exact results
def exact(case, seed):
    """The pass's result from the definitions, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return exact_values(s["x"].double(), case["block_rows"])
    if case["op"] == "gemm":
        a, b = exact_read(*s["a"], case["k"], 1), exact_read(*s["b"], case["k"], BLOCK)
        d = torch.einsum("mk,nk->mn", a, b)
        return d if s["bias"] is None else torch.add(d, s["bias"].double())
    h = torch.add(s["x"].double(), s["residual"].double())
    rms = torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / h.shape[1] + 1e-6)
    y = torch.addcmul(s["beta"].double(), h / rms[:, None], s["gamma"].double())
    if case["silu"]:
        y = y * torch.sigmoid(y)
    return h, exact_values(y, 1)


def exact_values(x, block_rows):
    """code * scale of every element: the e4m3 value nearest to x / scale, block by block of columns."""
    rows, cols = x.shape
    out = torch.empty_like(x)
    for c0 in range(0, cols, BLOCK):
        piece = x[:, c0:c0 + BLOCK]
        top = piece.abs().max(dim=1).values
        if block_rows > 1:
            top = torch.cat([t.max().expand(t.numel()) for t in top.split(block_rows)])
        scale = (top / 448.0).float().double().clamp(min=2.0 ** -126)[:, None]
        v = (piece / scale).float().double()  # the definition's fp32 quotient
        # e4m3: 3 mantissa bits from 2^-6 on, steps of 2^-9 below
        _, ex = torch.frexp(v)
        step = torch.exp2((ex - 4).clamp(min=-9).double())
        out[:, c0:c0 + BLOCK] = (torch.round(v / step) * step).clamp(-448.0, 448.0) * scale
    return out


def exact_read(codes, scales, cols, block_rows):
    """Values of an operand, each bit field by its meaning."""
    byte = codes.view(torch.uint8)[:, :cols].int()
    ex, man = (byte >> 3) & 15, (byte & 7).double()
    mag = torch.where(ex > 0, (1 + man / 8) * torch.exp2(ex.double() - 7), man * 2.0 ** -9)
    r = torch.arange(byte.shape[0], device=codes.device)[:, None] // block_rows
    c = torch.arange(cols, device=codes.device)[None] // BLOCK
    return torch.where(byte >= 128, -mag, mag) * scales[c, r].double()
