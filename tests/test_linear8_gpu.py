"""The operators together, as a layer uses them: the residual norm, the rotation into e4m3, the product
with the rotated and quantized weight, the rotation back; and its calibration from the norm's codes.

W' = T_U^T W T_V is what the weight holds, so y = W u = T_U (W' (T_V^T u))."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import harp_oracle as O
import workloads as W
import structured_rotations_b200 as H
from tests import _codes as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rotation(d, schedule, seed):
    theta = W.draw_theta(O.theta_count(schedule), 0.2, seed).astype(np.float32)
    return (H.Plan(d, schedule, theta=theta, sign_seed=seed).materialize(),
            O.Transform(O.make_plan(d, schedule, theta.astype(np.float64), sign_seed=seed)))


@pytest.mark.parametrize("rows", [1, 7, 200])
def test_layer(rows):
    n_in, n_out = 512, 1280
    pv, tv = _rotation(n_in, (8, 8, 8), 4)
    pu, tu = _rotation(n_out, (8, 8, 5, 4), 5)
    gen = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, n_in, generator=gen).bfloat16()
    res = torch.randn(rows, n_in, generator=gen).bfloat16()
    gain = (1 + 0.1 * torch.randn(n_in, generator=gen)).bfloat16()
    w = (0.05 * torch.randn(n_out, n_in, generator=gen)).bfloat16()

    # once per weight
    w_rot = H.apply_two_sided(pu, pv, w.to(DEV).float())
    wq, ws = H.quantize(w_rot, (128, 128))
    # per step
    u = torch.empty(rows, n_in, dtype=torch.bfloat16, device=DEV)
    nq, ns, h = H.rms_norm_quant(x.to(DEV), gain.to(DEV), res.to(DEV), code="int8", y=u)
    xq, xs = pv.apply_quant(u, 128, "inverse", code="e4m3")
    z = H.matmul_quant(xq, xs, wq, ws, dtype=torch.float32)
    y = pu.apply(z)

    # step by step in 64 bits, each from the operands that the step was given
    h64 = h.double().cpu().numpy()
    u64 = h64 / np.sqrt((h64 ** 2).mean(1, keepdims=True) + 1e-6) * gain.double().numpy()
    # three fp32 roundings, one to bf16
    assert np.all(np.abs(u.double().cpu().numpy() - u64) <= (2.0 ** -8 + 4 * 2.0 ** -24) * np.abs(u64))
    xh = C.decode(C.to_numpy(xq), xs.cpu().numpy(), 1, 128, "e4m3")
    wh = C.decode(C.to_numpy(wq), ws.cpu().numpy(), 128, 128, "e4m3")
    z64 = xh @ wh.T
    assert np.all(np.abs(z.double().cpu().numpy() - z64) <= (132 + 4) * 2.0 ** -23 * (np.abs(xh) @ np.abs(wh).T))
    y64 = tu.forward(z.double().cpu().numpy())
    assert np.all(np.abs(y.double().cpu().numpy() - y64).max(1) <= 2e-6 * np.linalg.norm(z.double().cpu().numpy(), axis=1))

    # and the layer as a whole against W u: every decoded factor is off by at most half an e4m3 step, 2^-4 of
    # it (or 2^-10 of its scale, below 2^-4 / 64 of a normal value), the rotated rows by one more bf16
    # rounding of u, which the rotation keeps in l2: |y - W u| <= 2^-3 (1 + 2^-3) sum |x'| |w'| in l2
    xr, wr = tv.inverse(u64), O.two_sided(tu.plan, tv.plan, w.double().numpy())
    worst = np.abs(xr) @ np.abs(wr).T
    err = np.linalg.norm(y.double().cpu().numpy() - u64 @ w.double().numpy().T, axis=1)
    assert np.all(err <= 2.0 ** -3 * (1 + 2.0 ** -3) * np.linalg.norm(worst, axis=1))

    # calibration from the codes that the norm left: g = y of the rotation, so the gradient has the scale of
    # the terms; against the oracle on the decoded rows
    g = torch.randn(rows, n_in, generator=gen).to(DEV)
    d_theta = pv.grad_theta_quant(nq, ns, g).double().cpu().numpy()
    want = O.theta_grad(tv.plan, C.decode(C.to_numpy(nq), ns.cpu().numpy(), 1, 128, "int8"), g.double().cpu().numpy())
    assert np.linalg.norm(d_theta - want) <= 2e-5 * np.linalg.norm(want)


def test_layer_captured():
    """The whole step in one graph, replayed on new rows: the same bits as the calls one by one."""
    n_in, n_out, rows = 512, 512, 33
    pv, _ = _rotation(n_in, (8, 8, 8), 4)
    w = torch.randn(n_out, n_in, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    wq, ws = H.quantize(H.apply_two_sided(pv, pv, w), (128, 128))
    x, res = torch.randn(rows, n_in, device=DEV).bfloat16(), torch.randn(rows, n_in, device=DEV).bfloat16()
    h, u = torch.empty_like(x), torch.empty_like(x)

    def step():
        nq, ns, _ = H.rms_norm_quant(x, None, res, h=h, y=u)
        xq, xs = pv.apply_quant(u, 128, "inverse", code="e4m3")
        return nq, ns, xq, xs, H.matmul_quant(xq, xs, wq, ws), H.matmul_quant(nq, ns, wq, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    x.copy_(torch.randn(rows, n_in, device=DEV).bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(kept, step()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
