"""harp_quantize / harp_dequantize against the plain definition: bit for bit in codes and scales (the
definition's fp32 operations repeated in NumPy), within half a step of the values, over block
shapes, types, ragged edges, odd and padded strides, blocks that are zero, tiny or not finite."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import structured_rotations_b200 as H
from structured_rotations_b200 import harp as HB
from tests import _codes as C

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCKS = [(1, 32), (1, 64), (1, 128), (1, 256), (128, 128)]


def _values(rows, cols, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    return x.to(dtype)


def _check(x, q, s, block, code):
    qr, sr = C.quantize(x.float().cpu().numpy(), *block, code)
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(C.to_numpy(q), qr)
    C.check_error(x.double().cpu().numpy(), C.to_numpy(q), s.cpu().numpy(), *block, code)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 7), (129, 130), (128, 128), (5, 1000), (300, 264), (257, 2047)])
def test_codes_and_values(rows, cols, block, dtype, code):
    x = _values(rows, cols, dtype, rows + cols).to(DEV)
    q, s = H.quantize(x, block, code)
    for out in (torch.bfloat16, torch.float32):
        y = H.dequantize(q, s, block, dtype=out)
        want = C.decode(C.to_numpy(q), s.cpu().numpy(), *block, code).astype(np.float32)   # one fp32 rounding
        assert torch.equal(y.cpu(), torch.from_numpy(want).to(out))
    _check(x, q, s, block, code)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("shift", [0, 1])
def test_strided_and_unaligned(block, shift):
    """Padded rows, rows that start off every alignment, and nothing written outside of the outputs."""
    rows, cols = 131, 391
    wide = _values(rows, 420, torch.bfloat16).to(DEV)
    x = wide[:, shift:shift + cols]
    qw = torch.full((rows, 409), 77, dtype=torch.uint8, device=DEV)
    nr, nc = -(-rows // block[0]), -(-cols // block[1])
    sw = torch.full((nr + 1, nc + 3), -5.0, device=DEV)
    q, s = qw[:, shift:shift + cols].view(torch.float8_e4m3fn), sw[:nr, :nc]
    H.quantize(x, block, "e4m3", q=q, scales=s)
    _check(x, q, s, block, "e4m3")
    rest = qw.clone()
    rest[:, shift:shift + cols] = 77
    assert torch.all(rest == 77)
    assert torch.all(sw[nr:] == -5) and torch.all(sw[:, nc:] == -5)
    yw = torch.full((rows, 400), 3.0, dtype=torch.float32, device=DEV)
    H.dequantize(q, s, block, out=yw[:, shift:shift + cols])
    want = C.decode(C.to_numpy(q), s.cpu().numpy(), *block, "e4m3").astype(np.float32)
    assert np.array_equal(yw[:, shift:shift + cols].cpu().numpy(), want)
    yw[:, shift:shift + cols] = 3.0
    assert torch.all(yw == 3.0)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("block", BLOCKS)
def test_zero_tiny_and_nonfinite_blocks(block, code):
    """Zero blocks, blocks below and at 2^-100, fp32's largest values, ties, and blocks with a NaN or an
    infinity, which decode to NaN throughout while their neighbours stay as they are."""
    br, bc = block
    x = torch.zeros(9 * br, 2 * bc)
    v = _values(9 * br, 2 * bc, torch.float32, 3)
    rows = [slice(i * br, (i + 1) * br) for i in range(9)]
    x[rows[1]] = v[rows[1]]
    x[rows[1].start, 3] = float("nan")
    x[rows[2]] = v[rows[2]]
    x[rows[2].start, 5] = float("-inf")
    x[rows[3]] = v[rows[3]] * 1e-32
    x[rows[4]] = 2.0 ** -100
    x[rows[5]] = v[rows[5]].sign() * 3.0e38
    x[rows[6]] = (torch.arange(2 * bc) % 255 - 127).float() / 2      # ties of the int8 grid where a = 127 / 2
    x[rows[7]] = v[rows[7]] * 2.0 ** -99
    x[rows[8], 0] = -1.0                                            # one-hot
    q, s = H.quantize(x.to(DEV), block, code)
    qr, sr = C.quantize(x.numpy(), *block, code)
    assert np.array_equal(s.cpu().numpy(), sr, equal_nan=True)
    y = H.dequantize(q, s, block, dtype=torch.float32).cpu().numpy()
    with np.errstate(all="ignore"):
        want = C.decode(qr, sr, *block, code).astype(np.float32)
    assert np.array_equal(y, want, equal_nan=True)
    assert np.all(np.isnan(y[rows[1], :bc])) and np.all(np.isnan(y[rows[2], :bc]))
    assert np.all(np.isfinite(y[rows[1], bc:])) and np.all(np.isfinite(y[rows[2], bc:]))
    assert np.all(y[rows[0]] == 0)
    small = np.abs(x.numpy()).reshape(9, br, 2, bc).max(axis=(1, 3)) < 2.0 ** -100    # blocks that count as zero
    assert np.all(y.reshape(9, br, 2, bc)[small.nonzero()[0], :, small.nonzero()[1]] == 0)


def test_empty_and_refusals():
    x = torch.zeros(4, 256, device=DEV)
    q, s = H.quantize(torch.zeros(0, 256, device=DEV))
    assert q.shape == (0, 256) and s.shape == (0, 2)
    assert H.dequantize(q, s).shape == (0, 256)
    assert H.quantize(torch.zeros(3, 0, device=DEV))[0].shape == (3, 0)
    for block in [(1, 16), (1, 512), (128, 64), (64, 128), (2, 128)]:
        with pytest.raises(HB.HarpError) as e:
            H.quantize(x, block)
        assert e.value.status == HB.HARP_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        H.quantize(x, (0, 128))
    with pytest.raises(ValueError):
        H.quantize(x, code="e5m2")
    with pytest.raises(ValueError):
        H.quantize(x.t())                                   # columns are not contiguous
    with pytest.raises(TypeError):
        H.quantize(x.double())
    with pytest.raises(ValueError):
        H.quantize(x.cpu())
    with pytest.raises(ValueError):
        H.quantize(x, scales=torch.empty(4, 3, device=DEV))
    with pytest.raises(TypeError):
        H.quantize(x, code="int8", q=torch.empty(4, 256, dtype=torch.float8_e4m3fn, device=DEV))
    with pytest.raises(HB.HarpError) as e:                  # codes over the values
        H.quantize(x, code="int8", q=x.view(torch.int8)[:, :256])
    assert e.value.status == HB.HARP_ERR_INVALID_ARG


def test_capture_and_side_stream():
    """A captured call replays on new values; a call on a side stream is ordered by that stream alone."""
    x = _values(200, 1000, torch.bfloat16).to(DEV)
    q, s = H.quantize(x)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        H.quantize(x, q=q, scales=s)
    x.copy_(_values(200, 1000, torch.bfloat16, 9).to(DEV))
    g.replay()
    torch.cuda.synchronize()
    _check(x, q, s, (1, 128), "e4m3")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x2 = x * 2
        q2, s2 = H.quantize(x2, (128, 128))
    side.synchronize()
    _check(x2, q2, s2, (128, 128), "e4m3")
