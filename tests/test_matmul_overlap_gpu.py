"""Products whose prologue overlaps the kernels before them (programmatic dependent launch): a decode step's
chain of the rotation's cluster kernel and the product's rows kernel, each of which lets the next one start
early, on scales of which one 128-byte line holds a row that is read now and a row that is written next.
Every result must be the one that the same calls give one after the other."""
import pytest

torch = pytest.importorskip("torch")

import workloads as W
import structured_rotations_b200 as H

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name,ld", [("d4096", 33), ("d5120", 41), ("d8192_int8", 65)])
def test_rotation_and_product_in_turn(name, ld, captured):
    w = W.get(name)
    d, kb, steps = w.d, w.d // 128, 24
    plan = H.Plan(d, w.schedule, theta=W.draw_theta(H.theta_count(w.schedule), 0.2, 3), sign_seed=5).materialize()
    gen = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn(steps, d, generator=gen, device=DEV).bfloat16()
    wq, ws = H.quantize(torch.randn(384, d, generator=gen, device=DEV), (128, 128))
    q = torch.zeros(steps, d, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.zeros(steps, ld, device=DEV)[:, :kb]
    y = torch.zeros(steps, 384, device=DEV)

    def step(i):
        plan.apply_quant(x[i:i + 1], 128, "inverse", q=q[i:i + 1], scales=s[i:i + 1], code="e4m3")
        assert H.last_kernel() == "harp_cluster_kernel"
        H.matmul_quant(q[i:i + 1], s[i:i + 1], wq, ws, out=y[i:i + 1])
        assert H.last_kernel() == "matmul_rows_kernel"

    for i in range(steps):
        step(i)
        torch.cuda.synchronize()
    want = y.clone()
    assert bool(want.abs().amin(1).isfinite().all()) and bool((want.abs().amax(1) > 0).all())

    def chain():
        for i in range(steps):
            step(i)

    graph = torch.cuda.CUDAGraph() if captured else None
    if captured:
        with torch.cuda.graph(graph):
            chain()
    for _ in range(20):
        q.view(torch.uint8).fill_(0x7F)                 # NaN codes and scales: what a step left undone shows
        s.fill_(float("nan"))
        y.zero_()
        torch.cuda.synchronize()
        graph.replay() if captured else chain()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    H.device_status()
