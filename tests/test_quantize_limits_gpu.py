"""The block quantizer and its inverse at the ends of the value range: masks of the type's lowest value, its
largest one, and what a block of such values decodes to.  Half a step of the block is the bound of
_codes.check_error; fp32 decoding rounds once more (2^-24 of the value)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import structured_rotations_b200 as H
from tests import _codes as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("block", [(1, 64), (128, 128)])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [256, 1280, 203])
def test_largest_values_stay_finite(cols, dtype, code, block):
    """1280 columns take the units of four groups when there are many rows, 203 the loads one by one."""
    rows = 3000
    top = torch.finfo(dtype).max
    x = torch.randn(rows, cols, generator=torch.Generator(device=DEV).manual_seed(cols), device=DEV).to(dtype)
    x[1] = -top                                   # a masked row
    x[4, ::3] = top
    x[5, cols - 1] = -top
    x[700:900] *= top / 8
    q, s = H.quantize(x, block, code)
    qr, sr = C.quantize(x.float().cpu().numpy(), *block, code)
    assert np.array_equal(C.to_numpy(q), qr) and np.array_equal(s.cpu().numpy(), sr)
    y = H.dequantize(q, s, block, dtype=dtype)
    assert bool(y.isfinite().all())
    v = x.double().cpu().numpy()
    sp = C._spread(s.double().cpu().numpy(), *block, v.shape)
    half = sp / 2 if code == "int8" else np.maximum(np.abs(v) * 2.0 ** -4, sp * 2.0 ** -10)
    # the codes' roundings (check_error) and the result's own
    got = y.double().cpu().numpy()
    bound = half * (1 + 2.0 ** -20) + 4 * 2.0 ** -24 * np.abs(v) + 2.0 ** -100 + torch.finfo(dtype).eps / 2 * np.abs(got)
    assert not (np.abs(got - v) > bound).any()


def test_infinite_scales_still_decode_to_nothing_finite():
    """A scale that is infinite or NaN is not brought back into the range."""
    q = torch.tensor([[3, -127, 127, 0] * 16] * 2, dtype=torch.int8, device=DEV)
    s = torch.tensor([[float("inf")], [float("nan")]], device=DEV)
    y = H.dequantize(q, s, (1, 64), dtype=torch.float32)
    assert not bool(y.isfinite().any())
    assert bool(y[0, 0] == float("inf")) and bool(y[0, 1] == -float("inf"))
