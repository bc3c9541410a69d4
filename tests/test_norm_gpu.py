"""harp_rms_norm_quant against its definition.  The row factor is rn32 of a double, and the rest are
single fp32 operations, so codes, scales, the sum and the normalized rows are compared bit for bit
with a NumPy restatement (the double sums differ by about 1e-16, which moves the fp32 factor with
a probability of about 1e-8 per row), and the codes within half a step of the norm in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import structured_rotations_b200 as H
from structured_rotations_b200 import harp as HB
from tests import _codes as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(rows, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, d, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(dtype)
    r = (3 * torch.randn(rows, d, generator=g)).to(dtype)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    return x, r, w


def _reference(x, r, w, eps, qblock, code):
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    h32 = h.float().numpy()
    f = (1.0 / np.sqrt((h32.astype(np.float64) ** 2).sum(1) / h32.shape[1] + eps)).astype(np.float32)
    u = h32 * f[:, None]
    if w is not None:
        u = u * w.float().numpy()[None, :]
    assert u.dtype == np.float32
    q, s = C.quantize(u, 1, qblock, code)
    return h, torch.from_numpy(u).to(x.dtype), q, s


def _check64(x, r, w, eps, q, s, qblock, code):
    h = (x if r is None else (x.float() + r.float()).to(x.dtype)).double().numpy()
    u = h / np.sqrt((h ** 2).mean(1, keepdims=True) + eps)
    if w is not None:
        u = u * w.double().numpy()
    # on top of half a step: the factor and two products, 3 roundings of fp32 (in check_error's slack of
    # 4 x 2^-24 together with the quantizer's own they make 7; the step is at least 2^-8 of the block)
    got = C.decode(q, s, 1, qblock, code)
    sp = C._spread(s.astype(np.float64), 1, qblock, u.shape)
    half = sp / 2 if code == "int8" else np.maximum(np.abs(u) * 2.0 ** -4, sp * 2.0 ** -10)
    assert np.all(np.abs(got - u) <= half * (1 + 2.0 ** -20) + 8 * 2.0 ** -24 * np.abs(u) + 2.0 ** -100)


@pytest.mark.parametrize("code,qblock", [("int8", 32), ("int8", 256), ("e4m3", 64), ("e4m3", 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 8192), (3, 31), (2, 257), (67, 512), (5, 4100), (9, 5120), (2, 32768), (3, 20001)])
def test_vs_definition(rows, d, dtype, code, qblock):
    x, r, w = _inputs(rows, d, dtype, rows * d)
    for res, wt in ((r, w), (None, w), (r, None), (None, None)):
        y = torch.empty(rows, d, dtype=dtype, device=DEV)
        q, s, h = H.rms_norm_quant(x.to(DEV), None if wt is None else wt.to(DEV), None if res is None else res.to(DEV),
                                   eps=1e-5, qblock=qblock, code=code, y=y)
        assert H.last_kernel() == "rms_norm_quant_kernel"
        hr, ur, qr, sr = _reference(x, res, wt, 1e-5, qblock, code)
        assert torch.equal(h.cpu(), hr)
        assert torch.equal(y.cpu(), ur)
        assert np.array_equal(s.cpu().numpy(), sr)
        assert np.array_equal(C.to_numpy(q), qr)
        _check64(x, res, wt, 1e-5, C.to_numpy(q), s.cpu().numpy(), qblock, code)


def test_in_place_strided_and_many_rows():
    """h over the residual and over x, padded and unaligned rows, outputs that stay inside of their rows."""
    rows, d = 5000, 264
    x, r, w = _inputs(rows, d, torch.bfloat16, 1)
    hr, _, qr, sr = _reference(x, r, w, 1e-6, 128, "e4m3")
    for over in ("residual", "x"):
        for shift in (0, 1):
            xw = torch.zeros(rows, 300, dtype=torch.bfloat16, device=DEV)
            rw = torch.full((rows, 289), 2.0, dtype=torch.bfloat16, device=DEV)
            xd, rd = xw[:, shift:shift + d], rw[:, shift:shift + d]
            xd.copy_(x)
            rd.copy_(r)
            qw = torch.full((rows, 280), 9, dtype=torch.uint8, device=DEV)
            sw = torch.full((rows, 4), -1.0, device=DEV)
            q = qw[:, shift:shift + d].view(torch.float8_e4m3fn)
            _, _, h = H.rms_norm_quant(xd, w.to(DEV), rd, h=rd if over == "residual" else xd, q=q, scales=sw[:, :3])
            assert torch.equal(h.cpu(), hr)
            assert torch.equal(xd.cpu(), hr if over == "x" else x)
            assert np.array_equal(C.to_numpy(q), qr) and np.array_equal(sw[:, :3].cpu().numpy(), sr)
            qw[:, shift:shift + d] = 9
            rw[:, shift:shift + d] = 2.0
            assert torch.all(qw == 9) and torch.all(rw == 2.0) and torch.all(sw[:, 3] == -1.0)


def test_zero_and_nonfinite_rows():
    x = torch.randn(6, 300, generator=torch.Generator().manual_seed(2))
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 250] = float("inf")
    x[4] *= 1e30
    x[5] *= 1e-30
    q, s, _ = H.rms_norm_quant(x.to(DEV), eps=1e-12, code="int8", qblock=128)
    y = C.decode(C.to_numpy(q), s.cpu().numpy(), 1, 128, "int8")
    assert np.all(y[1] == 0)
    assert np.all(np.isnan(y[2]))                       # the sum is NaN, so the row is
    # an infinity has factor 0: its own block is NaN (0 times infinity), the others zeros
    assert np.all(np.isnan(y[3, 128:256])) and np.all(y[3, :128] == 0) and np.all(y[3, 256:] == 0)
    for i in (0, 4, 5):
        _, _, qr, sr = _reference(x[i:i + 1], None, None, 1e-12, 128, "int8")
        assert np.array_equal(C.to_numpy(q)[i:i + 1], qr) and np.array_equal(s.cpu().numpy()[i:i + 1], sr)


def test_empty_refusals_and_capture():
    x = torch.randn(4, 256, device=DEV)
    q, s, h = H.rms_norm_quant(x[:0])
    assert q.shape == (0, 256) and s.shape == (0, 2) and h.shape == (0, 256)
    for kw, status in (({"eps": 0.0}, HB.HARP_ERR_INVALID_ARG), ({"eps": float("nan")}, HB.HARP_ERR_INVALID_ARG)):
        with pytest.raises(HB.HarpError) as e:
            H.rms_norm_quant(x, **kw)
        assert e.value.status == status
    with pytest.raises(HB.HarpError) as e:
        H.rms_norm_quant(torch.zeros(1, 32769, device=DEV))
    assert e.value.status == HB.HARP_ERR_INVALID_ARG
    with pytest.raises(HB.HarpError) as e:              # y over x
        H.rms_norm_quant(x, y=x)
    assert e.value.status == HB.HARP_ERR_INVALID_ARG
    wide = torch.zeros(8, 256, device=DEV)
    with pytest.raises(HB.HarpError) as e:              # h shifted against the residual
        H.rms_norm_quant(x, residual=wide[:4], h=wide[1:5])
    assert e.value.status == HB.HARP_ERR_INVALID_ARG
    for bad in (dict(qblock=100), dict(code="fp8")):
        with pytest.raises(ValueError):
            H.rms_norm_quant(x, **bad)
    with pytest.raises(TypeError):
        H.rms_norm_quant(x, residual=x.bfloat16())
    with pytest.raises(ValueError):
        H.rms_norm_quant(x, weight=torch.ones(255, device=DEV))
    with pytest.raises(ValueError):
        H.rms_norm_quant(x, weight=torch.ones(512, device=DEV)[::2])
    g = torch.cuda.CUDAGraph()
    res, q, s = torch.zeros_like(x), torch.empty(4, 256, dtype=torch.int8, device=DEV), torch.empty(4, 2, device=DEV)
    H.rms_norm_quant(x, residual=res, h=res, code="int8", q=q, scales=s)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        H.rms_norm_quant(x, residual=res, h=res, code="int8", q=q, scales=s)
    res.zero_()
    g.replay()
    g.replay()                                          # the residual accumulates: x, then 2 x
    torch.cuda.synchronize()
    hr, _, qr, sr = _reference(x.cpu(), x.cpu(), None, 1e-6, 128, "int8")
    assert torch.equal(res.cpu(), hr) and np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)
