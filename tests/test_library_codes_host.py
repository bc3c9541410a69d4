"""Argument checks of the 8-bit operators' C entries, which return before any device work, so they
run without a GPU on addresses that are never read; and the codes' reference against torch's e4m3."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from structured_rotations_b200 import harp as HB
from tests import _codes as C

OK, INVALID, UNSUPPORTED = HB.HARP_OK, HB.HARP_ERR_INVALID_ARG, HB.HARP_ERR_UNSUPPORTED
P = 1 << 40                # addresses 2^30 bytes apart
A, B, D, E, F = (P + (i << 30) for i in range(5))


def test_reference_e4m3():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(codes.astype(np.float64), C.E4M3, equal_nan=True)
    g = np.random.default_rng(0)
    t = np.concatenate([g.uniform(-448, 448, 20000), g.uniform(-0.1, 0.1, 20000), C.E4M3[:126],
                        (C.E4M3[:126] + C.E4M3[1:127]) / 2, [-0.0, 448.0, -448.0]]).astype(np.float32)
    want = torch.from_numpy(t).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(C.round_e4m3(t), want)
    assert np.array_equal(C.round_e4m3(np.array([1e9, -449.0, np.inf])), [0x7E, 0xFE, 0x7E])


def _quantize(L, **kw):
    a = dict(x=A, rows=4, cols=256, ld=256, dtype=1, code=1, br=1, bc=128, q=B, ld_q=256, s=D, ld_s=2) | kw
    return L.harp_quantize(a["x"], a["rows"], a["cols"], a["ld"], a["dtype"], a["code"], a["br"], a["bc"], a["q"], a["ld_q"],
                           a["s"], a["ld_s"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), OK), (dict(cols=0), OK), (dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(ld=255), INVALID),
    (dict(ld_q=255), INVALID), (dict(ld_s=1), INVALID), (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(code=2), UNSUPPORTED), (dict(bc=48), INVALID),
    (dict(br=2), INVALID), (dict(br=128, bc=64), INVALID), (dict(br=0), INVALID), (dict(q=A), INVALID), (dict(q=A + 2047), INVALID),
    (dict(s=B + 512), INVALID), (dict(x=A + 1), INVALID), (dict(s=D + 2), INVALID),
])
def test_quantize_arguments(kw, status):
    assert _quantize(HB.lib(), **kw) == status


def test_dequantize_arguments():
    L = HB.lib()
    assert L.harp_dequantize(A, 256, B, 2, 0, 1, 128, 0, 256, D, 256, 1, None) == OK
    assert L.harp_dequantize(A, 256, B, 2, 0, 1, 100, 4, 256, D, 256, 1, None) == INVALID
    assert L.harp_dequantize(A, 256, B, 2, 0, 1, 128, 4, 256, A + 64, 256, 1, None) == INVALID
    assert L.harp_dequantize(A, 256, B, 2, 0, 1, 128, 4, 256, None, 256, 1, None) == INVALID
    assert L.harp_dequantize(A, 256, B, 2, 3, 1, 128, 4, 256, D, 256, 1, None) == UNSUPPORTED


def _norm(L, **kw):
    a = dict(x=A, ld_x=256, r=B, ld_r=256, w=None, rows=4, d=256, dtype=1, eps=1e-6, h=None, ld_h=256, y=None, ld_y=256, code=1,
             qb=128, q=D, ld_q=256, s=E, ld_s=2) | kw
    return L.harp_rms_norm_quant(a["x"], a["ld_x"], a["r"], a["ld_r"], a["w"], a["rows"], a["d"], a["dtype"], a["eps"], a["h"],
                                 a["ld_h"], a["y"], a["ld_y"], a["code"], a["qb"], a["q"], a["ld_q"], a["s"], a["ld_s"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), OK), (dict(rows=-1), INVALID), (dict(d=0), INVALID), (dict(d=32769, ld_x=40000, ld_r=40000, ld_q=40000, ld_s=999), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(qb=16), INVALID), (dict(s=None), INVALID), (dict(q=None), INVALID), (dict(q=None, s=None), INVALID), (dict(x=None), INVALID),
    (dict(ld_x=255), INVALID), (dict(ld_r=255), INVALID), (dict(ld_q=255), INVALID), (dict(ld_s=1), INVALID),
    (dict(h=F, ld_h=200), INVALID), (dict(y=F, ld_y=200), INVALID), (dict(h=B, ld_h=300), INVALID), (dict(h=A + 512), INVALID),
    (dict(y=A), INVALID), (dict(y=B), INVALID), (dict(h=F, y=F), INVALID), (dict(q=A), INVALID), (dict(q=E - 1000), INVALID),
    (dict(w=D), INVALID), (dict(x=A + 1), INVALID), (dict(w=F + 1), INVALID), (dict(dtype=5), UNSUPPORTED), (dict(code=9), UNSUPPORTED),
])
def test_norm_arguments(kw, status):
    assert _norm(HB.lib(), **kw) == status


def _matmul(L, **kw):
    a = dict(x=A, ld_x=256, sx=B, ld_sx=2, w=D, ld_w=256, sw=E, ld_sw=2, rows=4, n=300, k=256, y=F, ld_y=300, dtype=1) | kw
    return L.harp_matmul_quant(a["x"], a["ld_x"], a["sx"], a["ld_sx"], a["w"], a["ld_w"], a["sw"], a["ld_sw"], a["rows"], a["n"],
                               a["k"], a["y"], a["ld_y"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), OK), (dict(n=0), OK), (dict(rows=-1), INVALID), (dict(n=-1), INVALID), (dict(k=0), INVALID), (dict(k=257), INVALID),
    (dict(ld_x=255), INVALID), (dict(ld_w=255), INVALID), (dict(ld_sx=1), INVALID), (dict(ld_sw=1), INVALID), (dict(ld_y=299), INVALID),
    (dict(x=None), INVALID), (dict(sx=None), INVALID), (dict(w=None), INVALID), (dict(sw=None), INVALID), (dict(y=None), INVALID),
    (dict(dtype=4), UNSUPPORTED), (dict(y=A), INVALID), (dict(y=B), INVALID), (dict(y=D + 64), INVALID), (dict(y=E), INVALID),
    (dict(y=F + 1), INVALID), (dict(sx=B + 1), INVALID), (dict(sw=E + 2), INVALID), (dict(rows=1 << 31), INVALID),
    (dict(n=1 << 31, ld_y=1 << 31), INVALID),
])
def test_matmul_arguments(kw, status):
    assert _matmul(HB.lib(), **kw) == status


def test_plan_entries():
    L = HB.lib()
    plan = HB.Plan(64, (8, 8))

    def quant(p, code=1, qb=64, x=A, dtype=1):
        return L.harp_apply_quant_ex(p, x, 4, 64, dtype, code, B, 64, D, 1, qb, 0, None)

    assert quant(None) == INVALID and quant(plan.handle, code=2) == UNSUPPORTED and quant(plan.handle, qb=48) == INVALID
    assert quant(plan.handle, dtype=0) == UNSUPPORTED and quant(plan.handle, x=None) == INVALID
    assert quant(plan.handle) == HB.HARP_ERR_NOT_MATERIALIZED

    def grad(p, code=0, qb=64, ld_s=1, s=B, g=D):
        return L.harp_grad_theta_quant(p, A, 64, code, s, ld_s, qb, g, 64, 1, 4, E, F, 1 << 20, None)

    assert grad(None) == INVALID and grad(plan.handle, code=7) == UNSUPPORTED and grad(plan.handle, qb=8) == INVALID
    assert grad(plan.handle, ld_s=0) == INVALID and grad(plan.handle, s=B + 1) == INVALID and grad(plan.handle, g=D + 1) == INVALID
    assert grad(plan.handle) == HB.HARP_ERR_NOT_MATERIALIZED


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError):
        HB.quantize(x)
    with pytest.raises(ValueError):
        HB.rms_norm_quant(x)
    with pytest.raises(ValueError):
        HB.dequantize(torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        HB.matmul_quant(x.to(torch.float8_e4m3fn), torch.zeros(4, 2), x.to(torch.float8_e4m3fn), torch.zeros(1, 2))
