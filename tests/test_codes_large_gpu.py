"""The 8-bit operators past 2^31 elements, called first inside of a capture, and in long chains without a
wait in between."""
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import structured_rotations_b200 as H
from tests import _codes as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _free():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_offsets_past_32_bits():
    """70,000 rows of 32,768 (2.3e9 elements): sampled rows, the last ones among them, bit for bit."""
    rows, d = 70000, 32768
    x = torch.empty(rows, d, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    for r in range(0, rows, 10000):
        x[r:r + 10000] = torch.randn(10000, d, generator=g, device=DEV)
    idx = torch.tensor([0, 1, 32768, 65535, 65536, 65537, rows - 2, rows - 1], device=DEV)
    q, s = H.quantize(x, (1, 128), "int8")
    qr, sr = C.quantize(x[idx].float().cpu().numpy(), 1, 128, "int8")
    assert np.array_equal(q[idx].cpu().numpy(), qr) and np.array_equal(s[idx].cpu().numpy(), sr)
    y = H.dequantize(q, s, (1, 128))
    want = torch.from_numpy(C.decode(qr, sr, 1, 128, "int8").astype(np.float32)).bfloat16()
    assert torch.equal(y[idx].cpu(), want)
    # in place over the restored rows: h = y + x
    q2, s2, h = H.rms_norm_quant(x, None, y, h=y, qblock=256)
    hr = (x[idx].float() + want.to(DEV).float()).bfloat16()
    assert torch.equal(h[idx], hr)
    h32 = hr.float().cpu().numpy()
    f = (1 / np.sqrt((h32.astype(np.float64) ** 2).mean(1) + 1e-6)).astype(np.float32)
    qn, sn = C.quantize(h32 * f[:, None], 1, 256, "e4m3")
    assert np.array_equal(C.to_numpy(q2[idx]), qn) and np.array_equal(s2[idx].cpu().numpy(), sn)
    qt, st = H.quantize(x, (128, 128), "e4m3")
    last = (rows - 1) // 128 * 128
    qr, sr = C.quantize(x[last:].float().cpu().numpy(), 128, 128, "e4m3")
    assert np.array_equal(C.to_numpy(qt[last:]), qr) and np.array_equal(st[-1:].cpu().numpy(), sr)
    del x, y, h, q, q2
    _free()
    # the product's result past 2^31 elements, its weight the tiles above: the last rows and columns
    xq, xs = H.quantize(torch.randn(40000, 256, generator=g, device=DEV))
    wq, ws = qt[:, :256], st[:, :2]                       # 70,000 rows, 32,768 apart
    y = H.matmul_quant(xq, xs, wq, ws)
    for r in (0, 39999):
        for j in (0, 69999 // 128 * 128):
            xd = xq[r].double() * xs[r].double().repeat_interleave(128)
            wd = wq[j:j + 112].double() * ws[j // 128].double().repeat_interleave(128)
            want = wd @ xd
            # (132 + 2) additions' ulps of the terms, and bf16's rounding
            assert torch.all((y[r, j:j + 112].double() - want).abs() <= 134 * 2.0 ** -23 * (wd.abs() @ xd.abs()) + 2.0 ** -8 * want.abs())
    H.device_status()
    del y
    _free()


FIRST = """
import torch, structured_rotations_b200 as H
x = torch.randn(40, 512, device="cuda").bfloat16()
w = torch.randn(384, 512, device="cuda")
z = torch.empty(40, 384, device="cuda"); big = torch.empty(200, 384, device="cuda")
q, s = torch.empty(40, 512, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(40, 4, device="cuda")
qb, sb = torch.empty(200, 512, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(200, 4, device="cuda")
wq, ws = torch.empty(384, 512, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(3, 4, device="cuda")
xb = x.repeat(5, 1)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    H.quantize(w, (128, 128), q=wq, scales=ws)
    H.rms_norm_quant(x, q=q, scales=s)
    H.matmul_quant(q, s, wq, ws, out=z)
    H.quantize(xb, q=qb, scales=sb)
    H.matmul_quant(qb, sb, wq, ws, out=big)
g.replay()
torch.cuda.synchronize()
wd = wq.double() * ws.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
for a, sa, y in ((q, s, z), (qb, sb, big)):
    ad = a.double() * sa.double().repeat_interleave(128, 1)
    assert torch.all((y.double() - ad @ wd.t()).abs() <= 136 * 2.0 ** -23 * (ad.abs() @ wd.abs().t()))
H.device_status()
print("captured first")
"""


def test_first_calls_inside_a_capture():
    """A process whose first call of every operator is captured."""
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_chain_without_waits(rows):
    """Sixty dependent norms, quantizers and products in a row (each prologue may overlap the end of the one
    before): the bits of the same calls with a synchronization after each."""
    d = 640
    g = torch.Generator(device=DEV).manual_seed(rows)
    ws = [H.quantize(torch.randn(d, d, generator=g, device=DEV) / d ** 0.5, (128, 128)) for _ in range(3)]
    x0 = torch.randn(rows, d, generator=g, device=DEV).bfloat16()

    def run(wait):
        x, res = x0.clone(), torch.zeros_like(x0)
        q, s = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(rows, d // 128, device=DEV)
        for i in range(60):
            H.rms_norm_quant(x, None, res, h=res, q=q, scales=s)
            if wait:
                torch.cuda.synchronize()
            H.matmul_quant(q, s, *ws[i % 3], out=x)
            if wait:
                torch.cuda.synchronize()
            if i % 5 == 4:
                H.quantize(x, q=q, scales=s)
                H.dequantize(q, s, out=x)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return x, res

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    H.device_status()
