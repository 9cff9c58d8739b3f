"""4-bit operands at their largest sizes, beyond 32-bit offsets in the norms, and from several host threads at once."""
import threading

import numpy as np
import pytest
import torch

from oracle import fp4

pytestmark = pytest.mark.gpu

KMAX = 262144


@pytest.fixture(scope="module")
def vd():
    from patch_tiled_causal_gb300 import build, vaedec
    build.build()
    vaedec.load()
    vaedec.last_error()
    return vaedec


def operand(rows, cols, fmt, seed, per_row=False):
    """Codes of 0, +-0.5 and +-1 (or one of 0.5 and 1 per row) and scales of 1: a product is a multiple of 1/4, and sums of
    2^18 of them lie below 2^18, so that every partial sum is an fp32 number."""
    rng = np.random.default_rng(seed)
    codes = np.repeat(rng.integers(1, 3, (rows, 1)), cols, axis=1) if per_row else rng.choice([0, 1, 2, 9, 10], (rows, cols))
    codes = codes.astype(np.uint8)
    byte = np.full((rows, -(-cols // fp4.BLOCK[fmt])), 127 if fmt == "mx" else 56, np.uint8)
    return codes, byte


def upload(codes, byte):
    return torch.from_numpy(fp4.pack_codes(codes)).cuda(), torch.from_numpy(fp4.pack_scales(byte)).cuda()


def fid(vd, fmt):
    return vd.VAE_MXFP4 if fmt == "mx" else vd.VAE_NVFP4


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(5, 9, KMAX), (130, 40, KMAX - 17)])
def test_longest_sums(vd, fmt, M, N, K):
    (ac, ab), (bc, bb) = operand(M, K, fmt, 1), operand(N, K, fmt, 2)
    want = fp4.gemm(fp4.values(ac, ab, fmt), fp4.values(bc, bb, fmt))
    D = torch.empty((M, N), device="cuda")
    vd.gemm_fp4(*upload(ac, ab), *upload(bc, bb), D, K, fid(vd, fmt))
    np.testing.assert_array_equal(D.cpu().numpy(), want)
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_longest_sums_on_many_tiles(vd, fmt):
    # one value per row: D[m, n] = K a[m] b[n] (more than 152 tiles of 128 x 128: the CTA pairs)
    M, N, blk = 2600, 1030, fp4.BLOCK[fmt]
    (ac, ab), (bc, bb) = operand(M, 32, fmt, 3, True), operand(N, 32, fmt, 4, True)

    def whole(codes, byte):
        rows = codes.shape[0]
        c = torch.from_numpy(fp4.pack_codes(codes)).cuda().repeat(1, KMAX // 32)
        s = torch.full((-(-rows // 128) * (KMAX // blk // 4) * 512,), int(byte[0, 0]), dtype=torch.uint8, device="cuda")
        return c, s

    D = torch.empty((M, N), device="cuda")
    vd.gemm_fp4(*whole(ac, ab), *whole(bc, bb), D, KMAX, fid(vd, fmt))
    want = KMAX * np.outer(fp4.values(ac, ab, fmt)[:, 0], fp4.values(bc, bb, fmt)[:, 0])
    np.testing.assert_array_equal(D.cpu().numpy(), want)
    assert vd.last_error()[0] == vd.VAE_OK


def scale_bytes(scales, first, n):
    """The bytes of block 0 of rows first .. first + n - 1 of an operand of up to 4 blocks."""
    r = torch.arange(first, first + n, device="cuda")
    return scales[r // 128 * 512 + r % 32 * 16 + r % 128 // 32 * 4]


def test_norm_offsets_beyond_32_bits(vd):
    """4.5e9 values of 32 channels: rows (frames) that repeat must come out alike, first, last and in between."""
    C, f = 32, vd.VAE_MXFP4
    gen = torch.Generator(device="cuda").manual_seed(5)
    g, b = 1 + 0.2 * torch.randn(C, generator=gen, device="cuda"), 0.1 * torch.randn(C, generator=gen, device="cuda")
    T, H, W = 70, 1000, 2000
    rows = T * H * W
    assert rows * C > 1 << 32
    frame = torch.randn((H * W, C), generator=gen, device="cuda").to(torch.bfloat16)
    x = frame.repeat(T, 1)
    op, one = vd.fp4_empty(rows, C, f), vd.fp4_empty(H * W, C, f)

    def check():
        for t in (0, 33, 34, 67, T - 1):
            assert torch.equal(op[0][t * H * W:(t + 1) * H * W], one[0]), t
            assert torch.equal(scale_bytes(op[1], t * H * W, H * W), scale_bytes(one[1], 0, H * W)), t
        assert vd.last_error()[0] == vd.VAE_OK

    vd.channel_rmsnorm_silu_fp4(frame, g, b, *one, 1, 1, H, W, C, f)
    vd.channel_rmsnorm_silu_fp4(x, g, b, *op, 1, T, H, W, C, f)
    check()
    for t in op + one:
        t.fill_(0xA5)
    for o, n, xx in ((one, 1, frame), (op, T, x)):
        d = vd.gn_desc(1, n, H, W, C, 32, [0, 300, H], [0, W])
        vd.patch_groupnorm_silu_fp4(xx, g, b, *o, vd.gn_workspace(d, "cuda"), d, f)
    check()


def test_several_host_threads(vd):
    """8 threads on streams of their own, every operator from each of them many times: the results of one thread alone."""
    f, errors = vd.VAE_NVFP4, []
    jobs = []
    for i in range(8):
        gen = torch.Generator(device="cuda").manual_seed(20 + i)
        H, W, C = (9, 13, 256) if i % 2 else (70, 61, 128)
        T, N = (3, 70) if i % 4 < 2 else (41, 300)
        x = torch.randn((1, T, H, W, C), generator=gen, device="cuda").to(torch.bfloat16)
        d = vd.gn_desc(1, T, H, W, C, 32, [0, H], [0, W // 2, W])
        w = vd.quantize_fp4(torch.randn((N, C), generator=gen, device="cuda"), *vd.fp4_empty(N, C, f), f, tensor_scale=2.0 ** -8)
        jobs.append({"x": x, "d": d, "w": w, "dims": (1, T, H, W, C), "rows": T * H * W, "N": N, "ws": vd.gn_workspace(d, "cuda"),
                     "g": torch.ones(C, device="cuda"), "b": torch.zeros(C, device="cuda"), "s": torch.cuda.Stream()})

    def run(j):
        C, out = j["dims"][-1], []
        for k in range(2):
            op = vd.fp4_empty(j["rows"], C, f)
            if k:
                vd.channel_rmsnorm_silu_fp4(j["x"], j["g"], j["b"], *op, *j["dims"], f, tensor_scale=2.0 ** -7)
            else:
                vd.patch_groupnorm_silu_fp4(j["x"], j["g"], j["b"], *op, j["ws"], j["d"], f, tensor_scale=2.0 ** -7)
            D = torch.empty((j["rows"], j["N"]), device="cuda")
            vd.gemm_fp4(*op, *j["w"], D, C, f, alpha=2.0 ** -15)
            out += [*op, D]
        return out

    want = [run(j) for j in jobs]
    torch.cuda.synchronize()

    def work(j, ref):
        try:
            with torch.cuda.stream(j["s"]):
                for _ in range(10):
                    got = run(j)
                    j["s"].synchronize()
                    for i in (0, 2, 3, 5):  # (the scale tiles' bytes are all written: compared, too)
                        assert torch.equal(got[i], ref[i]) and torch.equal(got[1], ref[1]) and torch.equal(got[4], ref[4])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j, r)) for j, r in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]
    assert vd.last_error()[0] == vd.VAE_OK
