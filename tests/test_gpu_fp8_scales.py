"""Products of 8-bit operands whose scales multiply past either end of fp32's range, through the C ABI.

The result of a k block is sum * a b with fp32 scales a, b; a b alone may leave fp32 where the result does not (sums lie
between 2^-18 and 448^2 * 128).  Against float64, with tolerances fixed before the first run: per k block of 128 columns the
sum's 128 roundings, then one each for a b, for the sum times its first factor, for the addition and for the exchange
between parts of K, so (K + 4 blocks + 4) 2^-23 sum |a b| as for ordinary scales, plus 2^-23 of the result for alpha; below
2^-126 each of the (blocks + parts of K + 2) roundings of a partial sum is off by 2^-149 at most instead.  A scale of 2^-126,
the least that quantisation writes, times one below 1 is rounded to a multiple of 2^-149: 2^-150 * 448^2 * 128 < 2^-125 for
each k block.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

# rows of A as the MMA's columns (16, 32, 64), 128 x 128 tiles, 256 x 256 tiles (one and several per pair)
SIZES = [(2, 130), (20, 130), (40, 300), (100, 130), (3000, 1100), (6000, 2050)]


@pytest.fixture(scope="module")
def vd():
    from patch_tiled_causal_gb300 import build, vaedec
    build.build()
    vaedec.load()
    vaedec.last_error()
    return vaedec


def generator(*seed):
    return torch.Generator(device="cuda").manual_seed(sum(s * 1009 ** i for i, s in enumerate(seed)) % (1 << 31))


def codes(rows, K, lo, hi, gen):
    """Bytes of magnitudes lo .. hi - 1 with random signs."""
    shape = (rows, (K + 15) // 16 * 16)
    byte = torch.randint(lo, hi, shape, generator=gen, device="cuda") + 128 * torch.randint(0, 2, shape, generator=gen, device="cuda")
    return byte.to(torch.uint8).view(torch.float8_e4m3fn)


def powers(blocks, n, lo, hi, gen):
    """Scales [blocks, n]: a power of two for each of n (exponents lo .. hi - 1), another factor of 1 .. 4 for each block."""
    e = torch.randint(lo, hi, (1, n), generator=gen, device="cuda").double()
    return (torch.exp2(e) * (1 + 3 * torch.rand((blocks, n), generator=gen, device="cuda").double())).float()


def values(c, scales, K, block_rows):
    s = scales.double().t().repeat_interleave(block_rows, 0)[:c.shape[0]].repeat_interleave(128, 1)[:, :K]
    return c[:, :K].double() * s


def check(D, a, b, K, alpha=1.0, least=False):
    av, bv = values(*a, K, 1), values(*b, K, 128)
    want, size = alpha * (av @ bv.t()), abs(alpha) * (av.abs() @ bv.abs().t())
    blocks = (K + 127) // 128
    tol = (K + 4 * blocks + 4) * 2.0 ** -23 * size + 2.0 ** -23 * want.abs() + (blocks + 10) * 2.0 ** -149 * max(1.0, abs(alpha))
    tol = tol + blocks * 2.0 ** -125 if least else tol
    assert bool((size < 2.0 ** 128).all())  # (no partial sum overflows)
    over = (D.double() - want).abs() - tol
    assert bool((over <= 0).all()), (float((over / tol).max()), int((over > 0).sum()))


@pytest.mark.parametrize("M,N", SIZES)
def test_scales_that_multiply_past_the_top(vd, M, N):
    K, gen = 700, generator(M, N)
    a = codes(M, K, 0, 8, gen), powers(6, M, 58, 63, gen)  # codes up to 7 * 2^-9
    b = codes(N, K, 0, 8, gen), powers(6, (N + 127) // 128, 62, 64, gen)
    a[1][0, 0], b[1][0, 0] = 2.0 ** 63.5, 2.0 ** 64.75  # past the end
    a[1][5, M - 1], b[1][5, -1] = 2.0 ** 58, 2.0 ** 62  # below it
    a[1][1, M // 2].neg_()
    b[1][2, 0].neg_()
    D = torch.full((M, N), float("nan"), device="cuda")
    vd.gemm_fp8(*a, *b, D, K)
    check(D, a, b, K)
    vd.gemm_fp8(*a, *b, D, K, alpha=-2.0 ** -130)
    check(D, a, b, K, alpha=-2.0 ** -130)
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("M,N", SIZES)
def test_scales_that_multiply_past_the_bottom(vd, M, N):
    K, gen = 700, generator(M, N, 1)
    a = codes(M, K, 0, 127, gen), powers(6, M, -90, -55, gen)
    b = codes(N, K, 0, 127, gen), powers(6, (N + 127) // 128, -72, -50, gen)
    a[0][M // 2] = 0.0  # a row of zeros, as quantisation writes it
    a[1][:, M // 2] = 2.0 ** -126
    a[1][1, 0].neg_()
    D = torch.full((M, N), float("nan"), device="cuda")
    vd.gemm_fp8(*a, *b, D, K)
    check(D, a, b, K)
    assert not bool(D[M // 2].any())
    vd.gemm_fp8(*a, *b, D, K, alpha=2.0 ** 20)
    check(D, a, b, K, alpha=2.0 ** 20)
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("M,N", SIZES)
def test_operands_quantised_from_tiny_values(vd, M, N):
    K, gen = 700, generator(M, N, 2)
    ops = []
    for rows, e, br in ((M, -60, 1), (N, -58, 128)):
        x = torch.randn((rows, K), generator=gen, device="cuda") * 2.0 ** e
        ops.append(vd.quantize_fp8(x, *vd.fp8_empty(rows, K, br), block_rows=br))
    D = torch.empty((M, N), device="cuda")
    vd.gemm_fp8(*ops[0], *ops[1], D, K)
    check(D, *ops, K)


@pytest.mark.parametrize("M,N", SIZES)
def test_powers_of_two_around_both_ends_are_exact(vd, M, N):
    # every sum a small multiple of one power of two: exact in fp32 at each step, on both sides of each end
    K, gen = 700, generator(M, N, 3)
    for lo, hi, ea, eb in ((0, 4, (65, 63, 64, 62), 64), (0x38, 0x39, (-70, -63, -64, -62, -50, -80), -63)):
        a = codes(M, K, lo, hi, gen), torch.exp2(torch.tensor(ea, device="cuda").float()).repeat(M)[:M].repeat(6, 1).contiguous()
        b = codes(N, K, lo, hi, gen), torch.full((6, (N + 127) // 128), 2.0 ** eb, device="cuda")
        for sign in (1.0, -1.0):  # (-2^127 and -2^-126 among the products)
            a[1].mul_(sign)
            D = torch.full((M, N), float("nan"), device="cuda")
            vd.gemm_fp8(*a, *b, D, K)
            assert torch.equal(D, (values(*a, K, 1) @ values(*b, K, 128).t()).float())


@pytest.mark.parametrize("M,N", SIZES)
def test_results_beyond_the_range(vd, M, N):
    K, gen = 100, generator(M, N, 4)
    a, b = (codes(M, K, 0, 4, gen), torch.full((1, M), 3e38, device="cuda")), \
        (codes(N, K, 0, 4, gen), torch.full((1, (N + 127) // 128), 3e38, device="cuda"))
    D = torch.empty((M, N), device="cuda")
    vd.gemm_fp8(*a, *b, D, K)
    want = a[0][:, :K].double() @ b[0][:, :K].double().t()
    assert torch.equal(D, torch.where(want == 0, 0.0, torch.sign(want) * float("inf")).float())
    for v in (2.0 ** -100, 1e-45):
        a[1].fill_(v)
        b[1].fill_(v)
        vd.gemm_fp8(*a, *b, D, K)
        assert not bool(D.any())


@pytest.mark.parametrize("M,N", SIZES)
def test_the_least_scale(vd, M, N):
    # 2^-126, which blocks of zeros and of values below 448 * 2^-126 have: off by at most 2^-125 for each k block
    K, gen = 700, generator(M, N, 5)
    a = codes(M, K, 0, 127, gen), powers(6, M, -20, 20, gen)
    b = codes(N, K, 0, 127, gen), powers(6, (N + 127) // 128, -8, 8, gen)
    a[1][:, 1] = 2.0 ** -126
    if M > 16:
        a[1][3], b[1][4] = 2.0 ** -126, 2.0 ** -126
    D = torch.empty((M, N), device="cuda")
    vd.gemm_fp8(*a, *b, D, K)
    check(D, a, b, K, least=True)


@pytest.mark.parametrize("M,N,K", [(300, 30000, 1300), (10, 300, 1300), (60, 300, 1300), (120, 300, 1300)])
@pytest.mark.parametrize("e", [64, -80])
def test_single_wide_scales(vd, M, N, K, e):
    # one row's scale of one k block at a time meets one block of B's rows: each half of the columns, each place in a group
    blocks, nb = (K + 127) // 128, (N + 127) // 128
    lo, hi = (0, 4) if e > 0 else (0x38, 0x40)
    a = codes(M, K, lo, hi, generator(1)), torch.ones((blocks, M), device="cuda")
    b = codes(N, K, lo, hi, generator(2)), torch.ones((blocks, nb), device="cuda")
    a[0].view(torch.uint8)[:, :] &= 0x7f
    b[0].view(torch.uint8)[:, :] &= 0x7f
    for k in range(blocks):
        a[1].fill_(0.0)
        b[1].fill_(1.0)
        r, n = (37 * k + 5) % M, (3 * k + 1) % nb
        a[1][k, r], b[1][k, n] = 2.0 ** e, 2.0 ** e
        D = torch.full((M, N), float("nan"), device="cuda")
        vd.gemm_fp8(*a, *b, D, K)
        want = (values(*a, K, 1)[r] @ values(*b, K, 128).t()).float()
        assert torch.equal(D[r], want)
        D[r] = 0.0
        assert not bool(D.any())


@pytest.mark.parametrize("M,N,K", [(300, 30000, 1300), (10, 300, 1300), (60, 300, 1300), (120, 300, 1300)])
def test_wide_scales_beside_infinities_nan_and_zeros(vd, M, N, K):
    # scales of which some are no ordinary numbers, in the same k blocks and rows of 64 as wide ones
    blocks, nb = (K + 127) // 128, (N + 127) // 128
    a = codes(M, K, 1, 4, generator(1)), torch.ones((blocks, M), device="cuda")
    b = codes(N, K, 1, 4, generator(2)), torch.full((blocks, nb), 2.0 ** 64, device="cuda")
    for c in (a[0], b[0]):
        c.view(torch.uint8)[:, :] &= 0x7f  # (sums above zero)
    a[1][2:, 0] = 2.0 ** 65
    a[1][1, 1], a[1][5, 2], a[1][3, 3] = float("inf"), float("nan"), float("-inf")
    a[1][:, 4], a[1][::2, 5] = 0.0, 2.0 ** -126
    a[1][:, 6] = 2.0 ** 64
    D = torch.empty((M, N), device="cuda")
    vd.gemm_fp8(*a, *b, D, K)
    inf = float("inf")
    assert bool((D[1] == inf).all()) and bool(torch.isnan(D[2]).all()) and bool((D[3] == -inf).all()) and not bool(D[4].any())
    rows = [r for r in range(M) if r not in (1, 2, 3)]
    want = values(*a, K, 1)[rows] @ values(*b, K, 128).t()
    tol = (K + 4 * blocks + 4) * 2.0 ** -23 * want  # (all terms are positive)
    assert bool(((D[rows].double() - want).abs() <= tol).all())
