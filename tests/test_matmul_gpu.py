"""harp_matmul_quant.  Two kinds of operands:

* exact ones: small integer codes and power-of-two scales chosen so that every partial sum is an
  integer multiple of one power of two below 2^24 of it: any order of fp32 additions gives the same
  bits, so the result must equal the 64-bit one.  These go over the sizes, edges and strides.
* random codes and scales, against 64 bits.  Bound: a product of two e4m3 values is exact in fp32;
  each of a block's 128 additions errs by at most one fp32 ulp (2^-23, whether it rounds or
  truncates) of a partial sum that is at most S_b = sum |x w| of the block; scaling and adding up the
  kb blocks adds (kb + 4) 2^-23 of the sum of all |terms|.  Together (132 + kb) 2^-23 sum |sx sw x w|,
  and half an ulp of the result's type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import structured_rotations_b200 as H
from structured_rotations_b200 import harp as HB
from tests import _codes as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _f8(a):
    return a.to(torch.float8_e4m3fn)


def _pad16(q):
    out = torch.zeros(q.shape[0], -(-q.shape[1] // 16) * 16, dtype=torch.uint8, device=DEV)[:, : q.shape[1]]
    out.copy_(q.view(torch.uint8))
    return out.view(torch.float8_e4m3fn)


def _spread(s, brows, rows, k):
    return s.double().repeat_interleave(brows, 0)[:rows].repeat_interleave(128, 1)[:, :k]


def _want(xq, xs, wq, ws, absolute=False):
    x, w = xq.double() * _spread(xs, 1, *xq.shape), wq.double() * _spread(ws, 128, *wq.shape)
    return x.abs() @ w.abs().t() if absolute else x @ w.t()


def _exact_operands(m, n, k, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kb, nb = -(-k // 128), -(-n // 128)
    # |codes| <= 2: a block's sum is at most 512; scales 1, 2 (rows) and 1/2, 1 (weight): terms are
    # multiples of 1/2, and the sum over k <= 8192 stays below 2 * 4 * 8192 = 2^16
    xq = _pad16(_f8(torch.randint(-2, 3, (m, k), generator=g, device=DEV).float()))
    wq = _pad16(_f8(torch.randint(-2, 3, (n, k), generator=g, device=DEV).float()))
    xs = torch.randint(0, 2, (m, kb), generator=g, device=DEV).float() + 1
    ws = (torch.randint(0, 2, (nb, kb), generator=g, device=DEV).float() + 1) / 2
    return xq, xs, wq, ws


def _random_operands(m, n, k, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    xq, xs = H.quantize(torch.randn(m, k, generator=g, device=DEV) * torch.exp(torch.randn(m, 1, generator=g, device=DEV)))
    wq, ws = H.quantize(torch.randn(n, k, generator=g, device=DEV), (128, 128))
    return xq, xs, wq, ws


SIZES = [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 130, 100), (3, 33, 129), (8, 257, 384), (15, 1000, 272), (16, 512, 8192),
         (17, 144, 640), (31, 128, 1000), (33, 300, 511), (64, 4100, 512), (65, 129, 257), (100, 5120, 5120), (127, 255, 128),
         (128, 128, 4096), (129, 384, 2048), (200, 28672, 256), (255, 264, 1024), (256, 256, 256), (300, 513, 1152),
         (513, 1030, 2050), (1000, 64, 136), (1111, 3333, 1000), (4097, 200, 384)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_exact_sums(m, n, k):
    xq, xs, wq, ws = _exact_operands(m, n, k, m + n + k)
    want = _want(xq, xs, wq, ws)
    assert torch.equal(H.matmul_quant(xq, xs, wq, ws, dtype=torch.float32), want.float())
    assert torch.equal(H.matmul_quant(xq, xs, wq, ws), want.float().bfloat16())
    H.device_status()


@pytest.mark.parametrize("m,n,k", SIZES[::2] + [(7, 28672, 8192), (700, 4096, 8192)])
def test_random_codes(m, n, k):
    xq, xs, wq, ws = _random_operands(m, n, k, 7 * m + n + k)
    want, mag = _want(xq, xs, wq, ws), _want(xq, xs, wq, ws, True)
    bound = (132 + xs.shape[1]) * 2.0 ** -23 * mag
    got = H.matmul_quant(xq, xs, wq, ws, dtype=torch.float32)
    assert torch.all((got.double() - want).abs() <= bound + 2.0 ** -24 * want.abs())
    half = H.matmul_quant(xq, xs, wq, ws)
    assert torch.equal(half, got.bfloat16())            # the same sums, rounded once
    assert torch.equal(got, H.matmul_quant(xq, xs, wq, ws, dtype=torch.float32))   # equal calls, equal bits


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [(1, 200, 300), (20, 129, 257), (150, 270, 500), (300, 515, 700)])
def test_strides_and_untouched_surroundings(m, n, k, out):
    """Operands inside of wider buffers (aligned, then at odd offsets), results into odd strides, and
    scales with padded rows: the same bits, and nothing written beside the result."""
    xq, xs, wq, ws = _exact_operands(m, n, k, 5)
    want = _want(xq, xs, wq, ws).float().to(out)
    for shift, pad in ((16, 48), (0, 32), (3, 21)):
        def wide(q):
            b = torch.full((q.shape[0] + 1, q.shape[1] + shift + pad), 0x7F, dtype=torch.uint8, device=DEV)   # NaN codes around
            if shift != 3:
                ld = -(-b.shape[1] // 16) * 16
                b = torch.full((q.shape[0] + 1, ld), 0x7F, dtype=torch.uint8, device=DEV)
            v = b[: q.shape[0], shift:shift + q.shape[1]]
            v.copy_(q.view(torch.uint8))
            return v.view(torch.float8_e4m3fn)
        xsw = torch.full((m + 1, xs.shape[1] + 3), float("nan"), device=DEV)
        xsw[:m, : xs.shape[1]] = xs
        wsw = torch.full((ws.shape[0] + 1, ws.shape[1] + 1), float("nan"), device=DEV)
        wsw[: ws.shape[0], : ws.shape[1]] = ws
        for ld in (n, n + 1, n + 16):
            buf = torch.full((m + 2, ld), 7.0, dtype=out, device=DEV)
            y = buf[1:m + 1, :n]
            H.matmul_quant(wide(xq), xsw[:m, : xs.shape[1]], wide(wq), wsw[: ws.shape[0], : ws.shape[1]], out=y)
            assert torch.equal(y, want)
            y.fill_(7.0)
            assert torch.all(buf == 7.0)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_nonfinite_scales_and_codes_stay_in_their_rows(m):
    n, k = 300, 400
    xq, xs, wq, ws = _exact_operands(m, n, k, 11)
    want = _want(xq, xs, wq, ws).float()
    xs = xs.clone()
    xs[m - 1, 1] = float("nan")
    wq = wq.view(torch.uint8).clone()
    wq[5, 3] = 0x7F                                     # a NaN code
    wp = _pad16(wq)
    got = H.matmul_quant(xq, xs, wp, ws, dtype=torch.float32)
    assert torch.all(got[m - 1].isnan()) and torch.all(got[:, 5].isnan())
    keep = [j for j in range(n) if j != 5]
    assert torch.equal(got[: m - 1, keep], want[: m - 1, keep])


def test_zero_scales_and_tiny_values():
    """Zero blocks (scale 0) contribute nothing; the smallest codes are not flushed."""
    xq, xs, wq, ws = _exact_operands(130, 140, 256, 3)
    xs[:, 1] = 0
    assert torch.equal(H.matmul_quant(xq, xs, wq, ws, dtype=torch.float32), _want(xq, xs, wq, ws).float())
    tiny = torch.full((130, 256), 2.0 ** -9, device=DEV)     # e4m3's smallest value
    got = H.matmul_quant(_f8(tiny), torch.ones(130, 2, device=DEV), _f8(tiny), torch.ones(2, 2, device=DEV), dtype=torch.float32)
    assert torch.all(got == 256 * 2.0 ** -18)


def test_empty_and_refusals():
    xq, xs, wq, ws = _exact_operands(4, 130, 256, 1)
    assert H.matmul_quant(xq[:0], xs[:0], wq, ws).shape == (0, 130)
    assert H.matmul_quant(xq, xs, wq[:0], ws[:0]).shape == (4, 0)
    with pytest.raises(ValueError):
        H.matmul_quant(xq, xs[:, :1], wq, ws)
    with pytest.raises(ValueError):
        H.matmul_quant(xq, xs, wq, ws[:1])
    with pytest.raises(ValueError):
        H.matmul_quant(xq, xs, wq[:, :128], ws)
    with pytest.raises(TypeError):
        H.matmul_quant(xq.view(torch.int8), xs, wq, ws)
    with pytest.raises(TypeError):
        H.matmul_quant(xq, xs, wq, ws, dtype=torch.float16)
    with pytest.raises(TypeError):
        H.matmul_quant(xq, xs, wq, ws, out=torch.empty(4, 130, device=DEV), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        H.matmul_quant(xq.cpu(), xs, wq, ws)
    with pytest.raises(ValueError):
        H.matmul_quant(xq, xs, wq, ws, out=torch.empty(4, 260, device=DEV)[:, ::2])
    buf = torch.zeros(4, 512, device=DEV)
    with pytest.raises(HB.HarpError) as e:              # the result over the scales
        H.matmul_quant(xq, buf[:, 130:132], wq, ws, out=buf[:, :130])
    assert e.value.status == HB.HARP_ERR_INVALID_ARG


def test_capture_streams_and_threads():
    """Captured products replay on new operands; two streams and two host threads at once."""
    import threading
    sets = [_exact_operands(m, n, k, m) for m, n, k in ((1, 700, 512), (33, 640, 512), (300, 640, 1024))]
    outs = [H.matmul_quant(*o, dtype=torch.float32) for o in sets]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for o, y in zip(sets, outs):
            H.matmul_quant(*o, out=y)
    for xq, xs, wq, ws in sets:
        xs.mul_(2)
        wq.view(torch.uint8).bitwise_xor_(0x80)         # -w
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for o, y in zip(sets, outs):
        assert torch.equal(y, _want(*o).float())
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None] * len(sets)

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                got[i] = H.matmul_quant(*sets[i], dtype=torch.float32)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for o, y in zip(sets, got):
        assert torch.equal(y, _want(*o).float())


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(1111, 3333), (333, 4101), (1000, 2500)])
def test_unaligned_results_of_many_rows(m, n, out):
    """Results whose rows lie at odd distances, of 256- and 128-column tiles: exact, nothing beside them written."""
    xq, xs, wq, ws = _exact_operands(m, n, 130, 17)
    want = _want(xq, xs, wq, ws).float().to(out)
    for ld in (n, n + 1, n + 7):
        buf = torch.full((m + 2, ld), 7.0, dtype=out, device=DEV)
        y = buf[1:m + 1, :n]
        H.matmul_quant(xq, xs, wq, ws, out=y)
        assert torch.equal(y, want)
        y.fill_(7.0)
        assert torch.all(buf == 7.0)
