"""The rotation with a fused e4m3 quantizer (harp_apply_quant_ex, HARP_CODE_E4M3).  The epilogue is
checked bit for bit on the tiled kernel against the kernel's own fp32 rows; every kernel is checked
against the float64 oracle: a scale is off by at most what the fp32 row transform may move the block's
maximum (2e-6 |x|, the row transform's parity bound) over 448 and three fp32 roundings, and a
decoded value by half an e4m3 step (2^-4 of the value, s 2^-10 below the normal range) of the moved
value."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import workloads as W
import structured_rotations_b200 as H
from structured_rotations_b200 import harp as HB
from tests import _codes as C
from tests.test_parity_gpu import DEV, plans, to_dev, decode

pytestmark = pytest.mark.gpu


def _check(q, s, y64, x64, qblock, what):
    q, s = C.to_numpy(q), s.cpu().numpy()
    tau = 2e-6 * np.linalg.norm(x64, axis=1)[:, None]
    a = np.abs(y64).reshape(y64.shape[0], -1, qblock).max(2)
    assert np.all(np.abs(s - a / 448) <= tau / 448 + 3 * 2.0 ** -24 * a / 448), f"{what}: scales"
    got = C.decode(q, s, 1, qblock, "e4m3")
    sp = np.repeat(s.astype(np.float64), qblock, 1)
    half = np.maximum((np.abs(y64) + tau) * 2.0 ** -4, sp * 2.0 ** -10)
    bad = np.abs(got - y64) > half * (1 + 2.0 ** -20) + tau + 4 * 2.0 ** -24 * np.abs(y64)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off"


@pytest.mark.parametrize("name", ["d4096", "d5120", "d8192_int8"])
@pytest.mark.parametrize("direction", ["forward", "inverse"])
@pytest.mark.parametrize("rows,qblock", [(1, 128), (16, 64), (37, 32), (37, 256), (70, 128), (700, 128)])
def test_vs_oracle(name, direction, rows, qblock):
    gp, tr = plans(name)
    xe = W.draw_encoded(W.get(name), 0, rows)
    q, s = gp.apply_quant(to_dev(xe), qblock, direction, code="e4m3")
    assert q.dtype == torch.float8_e4m3fn and q.shape == (rows, gp.d) and s.shape == (rows, gp.d // qblock)
    x64 = decode(xe)
    _check(q, s, tr.apply(x64, direction), x64, qblock, f"{name} {direction} {rows}")
    gp.device_status()


@pytest.mark.parametrize("qblock", [32, 64, 128, 256])
@pytest.mark.parametrize("rows", [32, 45, 1000])
def test_fast_kernel(monkeypatch, rows, qblock):
    monkeypatch.setenv("HARP_KERNEL", "fast")
    gp, tr = plans("d4096")
    xe = W.draw_encoded(W.get("d4096"), 0, rows)
    xe[3] = 0
    xe[7] = 0
    xe[7, 1234] = W.encode_bf16(np.array([5.0]))[0]
    qp = torch.full((rows, 4096 + 48), 5, dtype=torch.uint8, device=DEV)
    sp = torch.full((rows, 4096 // qblock + 3), -1.0, device=DEV)
    q, s = qp[:, :4096].view(torch.float8_e4m3fn), sp[:, : 4096 // qblock]
    gp.apply_quant(to_dev(xe), qblock, q=q, scales=s, code="e4m3")
    assert H.last_kernel() == "harp_fast_d4096_fwd_kernel"
    x64 = decode(xe)
    _check(q, s, tr.forward(x64), x64, qblock, f"fast rows={rows} qblock={qblock}")
    assert torch.all(s[3] == 0) and torch.all(q[3].float() == 0)
    assert torch.all(qp[:, 4096:] == 5) and torch.all(sp[:, 4096 // qblock:] == -1.0)
    gp.device_status()


@pytest.mark.parametrize("rows", [5, 700])
@pytest.mark.parametrize("qblock", [32, 64, 128, 256])
def test_epilogue_bit_for_bit(monkeypatch, rows, qblock):
    monkeypatch.setenv("HARP_KERNEL", "tiled")
    gp, _ = plans("d5120")
    x = to_dev(W.draw_encoded(W.get("d5120"), 0, rows))
    y32 = torch.empty(rows, gp.d, dtype=torch.float32, device=DEV)
    gp.apply_ex(x, y32)
    q, s = gp.apply_quant(x, qblock, code="e4m3")
    qr, sr = C.quantize(y32.cpu().numpy(), 1, qblock, "e4m3")
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(C.to_numpy(q), qr)


@pytest.mark.parametrize("rows", [4, 64])
@pytest.mark.parametrize("direction", ["forward", "inverse"])
def test_nonfinite_rows(rows, direction):
    """A rotation mixes every coordinate into every other: a NaN or an infinity reaches the whole row, all
    of which decodes to NaN; the other rows keep their codes."""
    gp, _ = plans("d4096")
    x = to_dev(W.draw_encoded(W.get("d4096"), 0, rows))
    q0, s0 = gp.apply_quant(x, 128, direction, code="e4m3")
    x = x.clone()
    x[1, 17] = float("nan")
    x[2, 4000] = float("inf")
    q, s = gp.apply_quant(x, 128, direction, code="e4m3")
    y = q.float() * s.repeat_interleave(128, 1)
    assert torch.all(y[1].isnan()) and torch.all(y[2].isnan())
    keep = [r for r in range(rows) if r not in (1, 2)]
    assert torch.equal(q[keep].view(torch.uint8), q0[keep].view(torch.uint8)) and torch.equal(s[keep], s0[keep])


def test_refusals_and_empty():
    gp, _ = plans("d4096")
    x = torch.zeros(4, 4096, dtype=torch.bfloat16, device=DEV)
    assert gp.apply_quant(x[:0], code="e4m3")[0].shape == (0, 4096)
    for bad in (48, 512):
        with pytest.raises(HB.HarpError) as e:
            gp.apply_quant(x, bad, code="e4m3")
        assert e.value.status == HB.HARP_ERR_INVALID_ARG
    with pytest.raises(HB.HarpError) as e:                      # fp32 rows
        gp.apply_quant(x.float(), code="e4m3")
    assert e.value.status == HB.HARP_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        gp.apply_quant(x, code="fp8")
    with pytest.raises(TypeError):
        gp.apply_quant(x, code="e4m3", q=torch.empty(4, 4096, dtype=torch.int8, device=DEV))
    with pytest.raises(ValueError):
        gp.apply_quant(x, code="e4m3", scales=torch.empty(4, 31, device=DEV))
    with pytest.raises(HB.HarpError) as e:                      # code rows not 16-byte aligned
        gp.apply_quant(x, code="e4m3", q=torch.empty(4, 4104, dtype=torch.float8_e4m3fn, device=DEV)[:, :4096])
    assert e.value.status == HB.HARP_ERR_UNSUPPORTED


@pytest.mark.parametrize("rows,qblock", [(1, 32), (4, 128), (16, 256), (33, 64), (64, 128)])
def test_cluster_kernel_equals_the_tiled_one(monkeypatch, rows, qblock):
    """Small batches of the inverse split each row over a cluster; the stage arithmetic is the tiled kernel's,
    so codes and scales are the same bits, also in padded outputs, which stay as they were beside them."""
    gp, _ = plans("d8192_int8")
    x = to_dev(W.draw_encoded(W.get("d8192_int8"), 0, rows))
    x[rows - 1, 100:] = 0
    monkeypatch.setenv("HARP_KERNEL", "tiled")
    q0, s0 = gp.apply_quant(x, qblock, "inverse", code="e4m3")
    monkeypatch.delenv("HARP_KERNEL")
    qp = torch.full((rows, 8192 + 16), 5, dtype=torch.uint8, device=DEV)
    sp = torch.full((rows, 8192 // qblock + 1), -1.0, device=DEV)
    gp.apply_quant(x, qblock, "inverse", q=qp[:, :8192].view(torch.float8_e4m3fn), scales=sp[:, : 8192 // qblock], code="e4m3")
    assert H.last_kernel() == "harp_cluster_kernel"
    assert torch.equal(qp[:, :8192], q0.view(torch.uint8)) and torch.equal(sp[:, : 8192 // qblock], s0)
    assert torch.all(qp[:, 8192:] == 5) and torch.all(sp[:, 8192 // qblock:] == -1.0)
    gp.device_status()
