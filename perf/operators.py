"""The microscaled 4-bit operators as a measuring tool sees them: the cases, their inputs, a plain form in
elementary torch operations, the library's calls, the work a pass cannot do without, and the exact results.

Three kinds of pass:
  quantize  x [rows, cols] -> 4-bit codes and block scales, and the values read back from them
  gemm      D = alpha * A B^T + bias of two 4-bit operands (packed codes and scales in, bf16 / fp32 out)
  gn, rms   a norm (group norm over patches, or channel RMS norm) + SiLU of channels-last activations written
            as 4-bit operands, and the product that reads them: a 1x1 projection of the normed activations

Formats: "mx" (blocks of 32, power-of-two scale) and "nv" (blocks of 16, e4m3 scale times one fp32 tensor
scale t).  Codes are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two to a byte, low nibble first, rows padded to
32 elements; scale bytes lie in tiles of 128 rows x 4 blocks, byte (row % 32) * 16 + (row % 128) // 32 * 4 + block % 4.
An nv block's scale byte is the e4m3 value nearest the fp32 quotient max|x| / (6 t), s its value; its codes round the
fp32 quotients x / (s t), with 6 t and s t in fp32.
"""
import math

import torch

own = False

BLOCK = {"mx": 32, "nv": 16}
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def ceil_to(n, m):
    return -(-n // m) * m


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # packing one attention projection's fp32 weights (1024 channels, the Wan-shaped mid block) at create time
        {"name": "quantize_weight_mx", "op": "quantize", "rows": 1024, "cols": 1024, "dtype": "fp32", "format": "mx"},
        # activations of one 81-frame clip at the mid block (21 x 44 x 80 tokens), bf16
        {"name": "quantize_clip_nv", "op": "quantize", "rows": 73920, "cols": 1024, "dtype": "bf16", "format": "nv"},
        # rows and columns that fill neither a block nor a scale tile, and rows that start off a vector boundary
        {"name": "quantize_ragged_nv", "op": "quantize", "rows": 5003, "cols": 1001, "dtype": "fp32", "format": "nv"},
        # one token: latency
        {"name": "gemm_one_row_nv", "op": "gemm", "m": 1, "n": 1024, "k": 1024, "format": "nv", "out": "bf16",
         "bias": True},
        # one latent frame's tokens (44 x 80) through a 1024-channel projection
        {"name": "gemm_frame_mx", "op": "gemm", "m": 3520, "n": 1024, "k": 1024, "format": "mx", "out": "bf16",
         "bias": True},
        # a whole clip's tokens through the same projection
        {"name": "gemm_clip_nv", "op": "gemm", "m": 73920, "n": 1024, "k": 1024, "format": "nv", "out": "bf16",
         "bias": True},
        # a wide product whose time is the multiplications'
        {"name": "gemm_wide_mx", "op": "gemm", "m": 16384, "n": 4096, "k": 4096, "format": "mx", "out": "bf16",
         "bias": False},
        # odd everything: output columns that fit no vector, a K that ends inside a block; fp32 result
        {"name": "gemm_ragged_nv", "op": "gemm", "m": 777, "n": 333, "k": 1000, "format": "nv", "out": "fp32",
         "bias": True},
        # the small decoder's group norm, in patches, into a narrow projection
        {"name": "gn_small_nv", "op": "gn", "b": 1, "t": 3, "h": 18, "w": 26, "c": 128, "groups": 32, "silu": True,
         "nph": 2, "npw": 2, "n": 64, "dtype": "bf16", "format": "nv"},
        # group norm + SiLU of a 512-channel stage in 4 width patches, into a 512-channel pointwise product
        {"name": "gn_stage_mx", "op": "gn", "b": 1, "t": 21, "h": 88, "w": 160, "c": 512, "groups": 32, "silu": True,
         "nph": 1, "npw": 4, "n": 512, "dtype": "bf16", "format": "mx"},
        # channel RMS norm of one small frame
        {"name": "rms_small_mx", "op": "rms", "b": 1, "t": 1, "h": 9, "w": 13, "c": 256, "silu": True, "n": 256,
         "dtype": "bf16", "format": "mx"},
        # channel RMS norm (no SiLU) of the fp32 residual stream before the attention's projections
        {"name": "rms_clip_nv", "op": "rms", "b": 1, "t": 21, "h": 44, "w": 80, "c": 1024, "silu": False, "n": 1024,
         "dtype": "fp32", "format": "nv"},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("quantize", "gemm", "gemm", "gn", "rms"))
    case = {"op": op, "format": rng.choice(("mx", "nv"))}
    if op == "quantize":
        cols = spread(16, 4096)
        case.update(rows=spread(1, min(100000, 75_000_000 // cols)), cols=cols, dtype=rng.choice(("bf16", "fp32")))
    elif op == "gemm":
        n, k = spread(16, 4096), spread(32, 4096)
        if rng.random() < 0.5:  # projections between channel counts
            n, k = ceil_to(n, 32), ceil_to(k, 32)
        m = spread(1, min(100000, 60_000_000 // max(n, k)))
        case.update(m=m, n=n, k=k, out=rng.choice(("bf16", "bf16", "fp32")), bias=rng.random() < 0.5)
    else:
        c = rng.choice((32, 64, 128, 256, 512, 768, 1024) if op == "rms" else (32, 64, 128, 256, 512, 1024))
        px = spread(1, 140_000_000 // c // 4)
        t = rng.randint(1, max(1, min(21, px)))
        w = spread(1, min(200, max(1, px // t)))
        h = max(1, min(200, px // t // w))
        case.update(b=rng.choice((1, 1, 2)), t=t, h=h, w=w, c=c, silu=rng.random() < 0.7,
                    n=rng.choice((48, 64, 100, 128, 256, 512, 1024)), dtype=rng.choice(("bf16", "fp32")))
        if op == "gn":
            case.update(groups=rng.choice((8, 32)), nph=rng.randint(1, min(3, h)), npw=rng.randint(1, min(4, w)))
    return case


def edges(length, n):
    """Band edges: the first length % n bands get one more."""
    return [i * (length // n) + min(i, length % n) for i in range(n + 1)]


# ------------------------------------------------------------------------------------------------ inputs
def activations(shape, gen):
    """Post-norm values of a decoder: normal, a gain per channel, and a few channels that run hot."""
    x = torch.randn(shape, generator=gen, device="cuda")
    gain = torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device="cuda"))
    return x * gain


def tensor_scale(case, amax):
    """The calibrated constant of an nv tensor: its largest value uses the whole range of the block scales."""
    return float(torch.tensor(amax / (6.0 * 448.0))) if case["format"] == "nv" else 1.0  # an fp32 number


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    fmt, op, s = case["format"], case["op"], dict(case)
    if op == "quantize":
        x = activations((case["rows"], case["cols"]), gen)
        s["ts"] = tensor_scale(case, float(x.abs().max()))
        s["x"] = x.to(DTYPE[case["dtype"]])
        s["codes"], s["scales"] = buffers(case["rows"], case["cols"], fmt)
        s["y"] = torch.empty_like(s["x"])
        return s
    n = case["n"]
    k = case["k"] if op == "gemm" else case["c"]
    w = torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)
    ts_b = tensor_scale(case, float(w.abs().max()))
    s["b"] = quantize_plain(w, fmt, ts_b)
    s["bias"] = 0.1 * torch.randn(n, generator=gen, device="cuda") if op != "gemm" or case["bias"] else None
    if op == "gemm":
        a = activations((case["m"], k), gen)
        ts_a = tensor_scale(case, float(a.abs().max()))
        s["a"] = quantize_plain(a, fmt, ts_a)
        s["alpha"] = ts_a * ts_b
        s["d"] = torch.empty((case["m"], n), dtype=DTYPE[case["out"]], device="cuda")
        return s
    shape = (case["b"], case["t"], case["h"], case["w"], k)
    s["x"] = (activations(shape, gen) + 0.3 * torch.randn(k, generator=gen, device="cuda")).to(DTYPE[case["dtype"]])
    s["gamma"] = 1.0 + 0.2 * torch.randn(k, generator=gen, device="cuda")
    s["beta"] = 0.1 * torch.randn(k, generator=gen, device="cuda")
    s["ts"] = tensor_scale(case, 12.0)
    s["alpha"] = s["ts"] * ts_b
    rows = shape[0] * shape[1] * shape[2] * shape[3]
    s["codes"], s["scales"] = buffers(rows, k, fmt)
    s["d"] = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    if op == "gn":
        s["ph"], s["pw"] = edges(case["h"], case["nph"]), edges(case["w"], case["npw"])
        # a user's program keeps the norm's scratch: 32 bytes per (patch, frame, group), 8 per (frame, channel)
        frames = case["b"] * case["t"]
        parts = ceil_to(case["nph"] * case["npw"] * frames * case["groups"] * 32, 256)
        s["ws"] = torch.empty(parts + frames * k * 8, dtype=torch.uint8, device="cuda")
    return s


def buffers(rows, cols, fmt):
    blocks = -(-cols // BLOCK[fmt])
    return (torch.empty((rows, ceil_to(cols, 32) // 2), dtype=torch.uint8, device="cuda"),
            torch.empty(ceil_to(rows, 128) * ceil_to(blocks, 4), dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------------------------------------ a pass
def run(s):
    if own:
        return run_own(s)
    fmt, op = s["format"], s["op"]
    if op == "quantize":
        codes, scales = quantize_plain(s["x"].float(), fmt, s["ts"])
        return (values_plain(codes, scales, s["rows"], s["cols"], fmt) * s["ts"]).to(s["x"].dtype)
    if op == "gemm":
        a, m, k = s["a"], s["m"], s["k"]
    else:
        y = gn_plain(s) if op == "gn" else rms_plain(s)
        y = y / (1.0 + torch.exp(-y)) if s["silu"] else y
        k = s["c"]
        m = y.numel() // k
        a = quantize_plain(y.reshape(m, k), fmt, s["ts"])
    d = values_plain(*a, m, k, fmt) @ values_plain(*s["b"], s["n"], k, fmt).t() * s["alpha"]
    return (d + s["bias"] if s["bias"] is not None else d).to(s["d"].dtype)


def run_own(s):
    from patch_tiled_causal_gb300 import vaedec as vd
    fmt = vd.VAE_MXFP4 if s["format"] == "mx" else vd.VAE_NVFP4
    op = s["op"]
    if op == "quantize":
        vd.quantize_fp4(s["x"], s["codes"], s["scales"], fmt, tensor_scale=s["ts"])
        return vd.dequantize_fp4(s["codes"], s["scales"], s["y"], fmt, tensor_scale=s["ts"])
    if op == "gemm":
        return vd.gemm_fp4(*s["a"], *s["b"], s["d"], s["k"], fmt, bias=s["bias"], alpha=s["alpha"])
    b, t, h, w, c = s["x"].shape
    if op == "gn":
        desc = vd.gn_desc(b, t, h, w, c, s["groups"], s["ph"], s["pw"], silu=s["silu"],
                          in_dtype=vd.VAE_FP32 if s["dtype"] == "fp32" else vd.VAE_BF16)
        vd.patch_groupnorm_silu_fp4(s["x"], s["gamma"], s["beta"], s["codes"], s["scales"], s["ws"], desc, fmt,
                                    tensor_scale=s["ts"])
    else:
        vd.channel_rmsnorm_silu_fp4(s["x"], s["gamma"], s["beta"], s["codes"], s["scales"], b, t, h, w, c, fmt,
                                    tensor_scale=s["ts"], silu=s["silu"])
    return vd.gemm_fp4(s["codes"], s["scales"], *s["b"], s["d"], c, fmt, bias=s["bias"], alpha=s["alpha"])


# ------------------------------------------------------------------------------------------------ the plain form
def quantize_plain(x, fmt, ts):
    """fp32 x [rows, cols] -> packed codes [rows, pitch] and tiled scale bytes."""
    rows, cols = x.shape
    blk = BLOCK[fmt]
    wide = ceil_to(cols, 32)
    x = torch.nn.functional.pad(x, (0, wide - cols)).reshape(rows, wide // blk, blk)
    amax = x.abs().amax(-1)
    if fmt == "mx":
        # the power of two that puts the block's largest value below 7, which rounds to 6: 2^(floor(log2 amax) - 2),
        # one more where the mantissa is 1.75 or above
        e = (((amax.view(torch.int32) + 0x200000) >> 23) - 2).clamp(min=0)
        byte, scale = e.to(torch.uint8), torch.ldexp(torch.ones_like(amax), e - 127)
        v = x / scale[..., None]
    else:
        q = amax / torch.full_like(amax, 6.0 * ts)
        byte = q.clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = byte.view(torch.float8_e4m3fn).float() * torch.full_like(amax, ts)
        v = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    a = v.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    code += (a > 0.25)
    code += (a >= 0.75)
    code += (a > 1.25)
    code += (a >= 1.75)
    code += (a > 2.5)
    code += (a >= 3.5)
    code += (a > 5.0)
    code += torch.signbit(x) * 8
    code = code.reshape(rows, wide // 2, 2)
    blocks = -(-cols // blk)
    r, g = ceil_to(rows, 128), ceil_to(blocks, 4)
    tiles = torch.nn.functional.pad(byte[:, :blocks], (0, g - blocks, 0, r - rows))
    tiles = tiles.reshape(r // 128, 4, 32, g // 4, 4).permute(0, 3, 2, 1, 4)
    return code[..., 0] | (code[..., 1] << 4), tiles.reshape(-1).contiguous()


def values_plain(codes, scales, rows, cols, fmt):
    """Packed codes and tiled scale bytes -> fp32 [rows, cols] (without the tensor scale)."""
    blk = BLOCK[fmt]
    blocks = -(-cols // blk)
    g = ceil_to(blocks, 4)
    byte = scales.reshape(-1, g // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, g)[:rows, :blocks]
    if fmt == "mx":
        scale = torch.ldexp(torch.ones(byte.shape, device=byte.device), byte.int() - 127)
    else:
        scale = byte.contiguous().view(torch.float8_e4m3fn).float()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).reshape(rows, -1)[:, :cols].int()]
    return v * scale.repeat_interleave(blk, dim=1)[:, :cols]


def gn_plain(s):
    x, groups = s["x"].float(), s["groups"]
    b, t, h, w, c = x.shape
    g = x.reshape(b * t, h * w, groups, c // groups)
    mean = g.double().mean((1, 3), keepdim=True)
    var = (g.double() - mean).square().mean((1, 3), keepdim=True)
    y = (g - mean.float()) * torch.rsqrt(var + 1e-6).float()
    return y.reshape(x.shape) * s["gamma"] + s["beta"]


def rms_plain(s):
    x = s["x"].float()
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["gamma"] + s["beta"]


# ------------------------------------------------------------------------------------------------ work
def operand_bytes(rows, cols, fmt):
    return rows * cols / 2 + rows * -(-cols // BLOCK[fmt])


def work(case):
    op, fmt = case["op"], case["format"]
    if op == "quantize":  # x in; codes and scales out and in again; values out
        n, e = case["rows"] * case["cols"], 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * n * e + 2 * operand_bytes(case["rows"], case["cols"], fmt), "flops": 4 * n}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": operand_bytes(m, k, fmt) + operand_bytes(n, k, fmt) + m * n * out + 4 * n * case["bias"],
                "flops": 2 * m * n * k}
    m, n, k = case["b"] * case["t"] * case["h"] * case["w"], case["n"], case["c"]
    # x in; the operand out and in again; the weights and the bias in; the product out
    size = m * k * (4 if case["dtype"] == "fp32" else 2)
    return {"bytes": size + 2 * operand_bytes(m, k, fmt) + operand_bytes(n, k, fmt) + 4 * n + 2 * m * n,
            "flops": 2 * m * n * k + 10 * m * k}


# ------------------------------------------------------------------------------------------------ exact results
def exact(case, seed):
    """The pass's result from the definitions, in 64 bits."""
    s = prepare(case, seed)
    fmt, op = case["format"], case["op"]
    if op == "quantize":
        return exact_values(s["x"].double(), fmt, s["ts"]) * s["ts"]
    if op == "gemm":
        a = exact_unpack(s["a"], case["m"], case["k"], fmt)
        k = case["k"]
    else:
        x = s["x"].double()
        if op == "gn":
            b, t, h, w, c = x.shape
            g = x.reshape(b, t, h, w, case["groups"], -1)
            var, mean = torch.var_mean(g, dim=(2, 3, 5), correction=0, keepdim=True)
            y = ((g - mean) / torch.sqrt(var + 1e-6)).reshape(x.shape)
        else:
            y = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + 1e-6)
        y = y * s["gamma"].double() + s["beta"].double()
        y = y * torch.sigmoid(y) if case["silu"] else y
        k = case["c"]
        a = exact_values(y.reshape(-1, k), fmt, s["ts"])
    d = a @ exact_unpack(s["b"], case["n"], k, fmt).t() * s["alpha"]
    return d if s["bias"] is None else d + s["bias"].double()


def exact_values(x, fmt, ts):
    """code * scale of every element (without the tensor scale): the nearest e2m1 value to x / scale."""
    rows, cols = x.shape
    blk = BLOCK[fmt]
    out = torch.empty_like(x)
    for c0 in range(0, cols, blk):
        piece = x[:, c0:c0 + blk]
        top = piece.abs().max(dim=1, keepdim=True).values
        if fmt == "mx":
            mant, ex = torch.frexp(top)  # top = mant 2^ex, mant in [0.5, 1)
            scale = torch.exp2((ex - 3 + (mant >= 0.875)).double().clamp(min=-127))
            real = scale
        else:
            # e4m3: 3 mantissa bits above 2^-6, steps of 2^-9 below
            q = (top / float(torch.tensor(6.0 * ts))).float().double().clamp(max=448.0)  # fp32, as the definition says
            step = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -6))) - 3)
            scale = torch.round(q / step) * step
            real = (scale * ts).float().double()  # likewise s t ...
        v = (piece / torch.where(real > 0, real, torch.inf)).float().double()  # ... and the quotient
        mag = v.abs().clamp(max=6.0)
        step = torch.exp2(torch.floor(torch.log2(mag.clamp(min=1.0))) - 1)
        out[:, c0:c0 + blk] = torch.round(mag / step) * step * torch.sign(v) * scale
    return out


def exact_unpack(packed, rows, cols, fmt):
    """The same from packed codes and tiled scale bytes, each bit field by its meaning."""
    codes, scales = packed
    blk = BLOCK[fmt]
    col = torch.arange(cols, device=codes.device)
    nib = (codes[:, col // 2].int() >> (4 * (col % 2)).int()) & 15
    ex, man = (nib >> 1) & 3, nib & 1
    mag = torch.where(ex > 0, (1 + 0.5 * man.double()) * torch.exp2(ex.double() - 1), 0.5 * man.double())
    groups = -(-(-(-cols // blk)) // 4)
    r, b = torch.arange(rows, device=codes.device)[:, None], torch.arange(-(-cols // blk), device=codes.device)[None]
    byte = scales[(r // 128 * groups + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4].int()
    if fmt == "mx":
        scale = torch.exp2(byte.double() - 127)
    else:
        ex, man = byte >> 3, byte & 7
        scale = torch.where(ex > 0, (1 + man.double() / 8) * torch.exp2(ex.double() - 7), man.double() * 2.0 ** -9)
    return torch.where(nib >= 8, -mag, mag) * scale[:, col // blk]
