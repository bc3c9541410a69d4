"""harp_matmul_quant with scales whose fp32 product leaves the normal range although the terms do not: the
quantizers write scales from 2^-109 to 2^119, and a block's sum is anything from 2^-18 to 2^25, or zero.
Against 64 bits, on every kernel.

Bound: that of test_matmul_gpu ((132 + kb) 2^-23 of sum |sx sw x w|) with one more rounding per block where
the sum meets the scales one after the other, and, for results below the normal range, half of the smallest
denormal number 2^-149 for every addition, every product and the result: (2 kb + 1) 2^-150, rounded up."""
import pytest

torch = pytest.importorskip("torch")

import structured_rotations_b200 as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
K = 400                       # four blocks of k, the last one short
KB = 4
# (rows, n): the kernel for few rows at 16, 32, 64 and 128 rows per tile, the one for many rows with narrow
# and wide tiles
SIZES = [(1, 300), (20, 257), (64, 130), (100, 260), (150, 270), (2560, 1536)]


def _codes(rows, k, value, shift):
    """A matrix of codes of `value` (a tensor that fits), rows a multiple of 16 bytes apart; shift 3: unaligned."""
    ld = -(-(k + shift) // 16) * 16
    q = torch.zeros(rows, ld, dtype=torch.uint8, device=DEV)[:, shift:shift + k]
    q.copy_(value.to(torch.float8_e4m3fn).view(torch.uint8))
    return q.view(torch.float8_e4m3fn)


def _full(q, s, rows):
    return q.double() * s.double().repeat_interleave(rows, 0)[: q.shape[0]].repeat_interleave(128, 1)[:, :K]


def _run(xq, xs, wq, ws, kernel=None):
    x, w = _full(xq, xs, 1), _full(wq, ws, 128)
    want, mag = x @ w.t(), x.abs() @ w.abs().t()
    got = H.matmul_quant(xq, xs, wq, ws, dtype=torch.float32)
    if kernel:
        assert H.last_kernel() == kernel
    bound = (133 + KB) * 2.0 ** -23 * mag + (2 * KB + 1) * 2.0 ** -150
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"{int((~(off <= bound)).sum())} of {off.numel()} off"   # NaN fails too
    assert torch.equal(H.matmul_quant(xq, xs, wq, ws), got.bfloat16())
    return got


def _operands(m, n, seed, shift=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(m, K, generator=g, device=DEV) * 100
    w = torch.randn(n, K, generator=g, device=DEV) * 100
    u = [1 + torch.rand(r, KB, generator=g, device=DEV) for r in (m, -(-n // 128))]
    return x.clamp_(-448, 448), w.clamp_(-448, 448), *u


KERNEL = {0: None, 3: "matmul_simple_kernel"}


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("ex,ew", [(-100, -40), (-40, -100), (-70, -69), (-105, -60), (0, -130), (-20, -109)])
def test_products_below_the_normal_range(m, n, ex, ew, shift):
    x, w, us, uw = _operands(m, n, m + n)
    _run(_codes(m, K, x, shift), us * 2.0 ** ex, _codes(n, K, w, shift), uw * 2.0 ** ew, KERNEL[shift])


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("ex,ew", [(100, 60), (119, 119), (40, 100)])
def test_blocks_of_zeros_with_large_scales(m, n, ex, ew, shift):
    """A block's sum of zero stays zero whatever the scales; the other blocks count."""
    x, w, us, uw = _operands(m, n, m + 2 * n)
    x[:, 128:256] = 0
    us[:, 1] *= 2.0 ** ex
    uw[:, 1] *= 2.0 ** ew
    got = _run(_codes(m, K, x, shift), us, _codes(n, K, w, shift), uw, KERNEL[shift])
    assert bool((got != 0).any())


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("ex,ew", [(80, 50), (49, 81), (119, 11)])
def test_products_above_the_largest_number(m, n, ex, ew, shift):
    """One product of the smallest codes per block: 2^-18 2^130 is finite although the scales' product is not."""
    x, w = torch.zeros(m, K, device=DEV), torch.zeros(n, K, device=DEV)
    x[:, ::128] = 2.0 ** -9
    w[:, ::128] = 2.0 ** -9
    _, _, us, uw = _operands(m, n, 3 * m + n)
    got = _run(_codes(m, K, x, shift), us * 2.0 ** ex, _codes(n, K, w, shift), uw * 2.0 ** ew, KERNEL[shift])
    assert bool(got.isfinite().all())


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("m,n", SIZES)
def test_ordinary_rows_beside_extreme_ones(m, n, shift):
    """Rows of every kind in one tile: the ordinary ones keep the bits that they have among their like."""
    x, w, us, uw = _operands(m, n, m + 5 * n)
    xq, wq = _codes(m, K, x, shift), _codes(n, K, w, shift)
    plain = H.matmul_quant(xq, us, wq, uw, dtype=torch.float32)
    kind = torch.arange(m, device=DEV) % 5
    es = torch.tensor([0.0, -135.0, 0.0, -140.0, 0.0], device=DEV)[kind]
    s = (us.double() * torch.exp2(es.double())[:, None]).float()
    s[kind == 4, 2] = 0
    got = _run(xq, s, wq, uw, KERNEL[shift])
    keep = (kind == 0) | (kind == 2)
    assert torch.equal(got[keep], plain[keep])


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("m,n", SIZES)
def test_scales_that_are_not_finite_stay_in_their_rows(m, n, shift):
    x, w, us, uw = _operands(m, n, m + 7 * n)
    xq, wq = _codes(m, K, x, shift), _codes(n, K, w, shift)
    plain = H.matmul_quant(xq, us, wq, uw, dtype=torch.float32)
    s = us.clone()
    s[m - 1, 3] = float("nan")
    s[m // 2, 0] = float("inf")
    got = H.matmul_quant(xq, s, wq, uw, dtype=torch.float32)
    assert bool(got[m - 1].isnan().all()) and not bool(got[m // 2].isfinite().any())
    keep = [r for r in range(m) if r not in (m - 1, m // 2)]
    assert torch.equal(got[keep], plain[keep])
