"""The calibration backward from 8-bit checkpoints (harp_grad_theta_quant) against the float64 oracle
on the decoded rows x^ = rn32(code * scale), with the element-wise and the l2 bound of the gradient
from plain rows (test_grad_gpu: decoding adds no error, x^ being the operand of both sides);
against harp_grad_theta on the same decoded rows; and against differences of the loss in theta."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import harp_oracle as O
import workloads as W
import structured_rotations_b200 as H
from structured_rotations_b200 import harp as HB
from tests import _codes as C
from tests.test_grad_gpu import _check, _tile_rows
from tests.test_parity_gpu import DEV, plans, to_dev, decode

pytestmark = pytest.mark.gpu


def _decoded(q, s, qblock, code):
    return C.decode(C.to_numpy(q), s.cpu().numpy(), 1, qblock, code).astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("code,qblock,f32", [("int8", 32, False), ("e4m3", 64, True), ("int8", 64, True), ("e4m3", 32, False)])
@pytest.mark.parametrize("name,rows", [("d64", 37), ("d64_hadamard", 53), ("d4096", 23), ("d5120", 19), ("d8192_int8", 11), ("d4096", 1)])
def test_vs_oracle(name, rows, code, qblock, f32):
    gp, tr = plans(name)
    w = W.get(name)
    x = to_dev(W.draw_encoded(w, 0, rows))
    g = to_dev(W.draw_upstream(w, 0, rows))
    g = g.float() if f32 else g.bfloat16()
    q, s = H.quantize(x, (1, qblock), code)
    dth = gp.grad_theta_quant(q, s, g)
    _check(dth.cpu().numpy(), _decoded(q, s, qblock, code), g.double().cpu().numpy(), tr.plan, f"{name} {rows} {code}",
           -(-rows // _tile_rows(w.d)))


@pytest.mark.parametrize("schedule", [(5, 2, 8), (7, 8), (3, 4, 2), (6, 6), (2, 2, 2, 2, 2, 2, 2), (3,), (8, 7, 6, 5, 4)])
def test_other_radices_and_short_blocks(schedule):
    """Dimensions that qblock does not divide (a short last block), odd strides, many tiles."""
    d = int(np.prod(schedule))
    theta = W.draw_theta(O.theta_count(schedule), 0.3, 23)
    gp = H.Plan(d, schedule, theta=theta, sign_seed=9).materialize()
    op = O.make_plan(d, schedule, theta.astype(np.float32).astype(np.float64), sign_seed=9)
    rows = 3 * _tile_rows(d) + 5
    gen = torch.Generator().manual_seed(d)
    x, g = torch.randn(rows, d, generator=gen).to(DEV), torch.randn(rows, d + 3, generator=gen).to(DEV)[:, 1:d + 1]
    for code, qblock in (("int8", 64), ("e4m3", 32)):
        qw = torch.zeros(rows, d + 5, dtype=torch.uint8, device=DEV)[:, 2:d + 2]
        q = qw.view(torch.int8 if code == "int8" else torch.float8_e4m3fn)
        q, s = H.quantize(x, (1, qblock), code, q=q)
        dth = gp.grad_theta_quant(q, s, g, qblock=qblock)
        _check(dth.cpu().numpy(), _decoded(q, s, qblock, code), g.double().cpu().numpy(), op, f"{schedule} {code}", 4)


@pytest.mark.parametrize("name,rows", [("d4096", 2000), ("d5120", 700)])
def test_equals_the_gradient_of_the_restored_rows(name, rows):
    """The same kernel chain on the same fp32 rows; only the order of the atomic additions may differ:
    (tiles of a sum) ulps, 2e-5 in l2 as in the oracle's bound."""
    gp, _ = plans(name)
    x = to_dev(W.draw_encoded(W.get(name), 0, rows))
    g = torch.randn(rows, gp.d, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    q, s = H.quantize(x, (1, 128), "int8")
    a = gp.grad_theta_quant(q, s, g).double()
    b = gp.grad_theta(H.dequantize(q, s, (1, 128), dtype=torch.float32), g).double()
    assert ((a - b).norm() / b.norm()).item() <= 2e-5


def test_against_differences():
    """d64: the loss sum g . T(theta) x^ in float64 at theta +- 1e-5 along each of some parameters.  The
    central difference errs by h^2 / 6 |L'''| (about 1e-10 of the terms) and 1e-16 |L| / h (1e-11); the
    kernel by the bound of `_check`, here 1e-5 of the gradient's largest entry."""
    w = W.get("d64")
    gp, tr = plans("d64")
    x, g = to_dev(W.draw_encoded(w, 0, 40)), to_dev(W.draw_upstream(w, 0, 40)).float()
    q, s = H.quantize(x, (1, 64), "int8")
    got = gp.grad_theta_quant(q, s, g).double().cpu().numpy()
    xh, g64 = _decoded(q, s, 64, "int8"), g.double().cpu().numpy()
    th = tr.plan.theta

    def loss(t):
        return float((O.Transform(O.make_plan(64, w.schedule, t, sign_seed=w.sign_seed)).forward(xh) * g64).sum())

    top = np.abs(got).max()
    for i in range(0, th.size, 37):
        e = np.zeros_like(th)
        e[i] = 1e-5
        diff = (loss(th + e) - loss(th - e)) / 2e-5
        assert abs(diff - got[i]) <= 1e-5 * top, i


def test_workspace_capture_and_refusals():
    gp, tr = plans("d64")
    w = W.get("d64")
    x, g = to_dev(W.draw_encoded(w, 0, 40)), to_dev(W.draw_upstream(w, 0, 40))
    q, s = H.quantize(x, (1, 32), "int8")
    ws = gp.grad_workspace()
    out = torch.full((H.theta_count(w.schedule),), 7.0, device=DEV)
    gp.grad_theta_quant(q[:0], s[:0], g[:0], dtheta=out, workspace=ws)
    assert torch.count_nonzero(out).item() == 0
    gp.grad_theta_quant(q, s, g, dtheta=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        H.quantize(x, (1, 32), "int8", q=q, scales=s)
        gp.grad_theta_quant(q, s, g, dtheta=out, workspace=ws)
    xe = W.draw_encoded(w, 40, 40)
    x.copy_(to_dev(xe))
    graph.replay()
    torch.cuda.synchronize()
    _check(out.cpu().numpy(), _decoded(q, s, 32, "int8"), decode(W.draw_upstream(w, 0, 40)), tr.plan, "captured", 3)
    with pytest.raises(ValueError):
        gp.grad_theta_quant(q, s[:, :1], g)                     # one scale for 64: taken as qblock 64,
        gp.grad_theta_quant(q, s[:, :0], g)                     # none: refused
    with pytest.raises(ValueError):
        gp.grad_theta_quant(q, s, g, qblock=48)
    with pytest.raises(ValueError):
        gp.grad_theta_quant(q, s, g[:39])
    with pytest.raises(TypeError):
        gp.grad_theta_quant(q.view(torch.uint8), s, g)
    with pytest.raises(TypeError):
        gp.grad_theta_quant(q, s, g.half())
    with pytest.raises(HB.HarpError) as e:
        gp.grad_theta_quant(q, s, g, workspace=ws[:-16])
    assert e.value.status == HB.HARP_ERR_INVALID_ARG
    big = H.Plan(32, (16, 2), sign_seed=1).materialize()        # radix above 8
    with pytest.raises(HB.HarpError) as e:
        big.grad_theta_quant(torch.zeros(2, 32, dtype=torch.int8, device=DEV), torch.zeros(2, 1, device=DEV),
                             torch.zeros(2, 32, device=DEV))
    assert e.value.status == HB.HARP_ERR_UNSUPPORTED
    both = H.Plan.compose([gp, gp])
    with pytest.raises(HB.HarpError) as e:
        both.grad_theta_quant(q, s, g)
    assert e.value.status == HB.HARP_ERR_UNSUPPORTED
