"""The 8-bit operators on a stream that is not the current one: what a call allocates (results, the
gradient's workspace) belongs to the stream that the call runs on, so work that the current stream
still has under way does not write into it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import harp_oracle as O
import workloads as W
import structured_rotations_b200 as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLEEP = 200_000_000   # clocks: about 0.1 s


def _plan(d=512, schedule=(8, 8, 8)):
    theta = W.draw_theta(O.theta_count(schedule), 0.2, 7).astype(np.float32)
    return H.Plan(d, schedule, theta=theta, sign_seed=7).materialize()


def _calls():
    plan = _plan()
    x = torch.randn(2048, 512, device=DEV).bfloat16()
    w = torch.randn(512, 512, device=DEV).bfloat16()
    xq, xs = H.quantize(x)
    wq, ws = H.quantize(w, (128, 128))
    return [
        lambda st: H.quantize(x, stream=st),
        lambda st: (H.dequantize(xq, xs, stream=st),),
        lambda st: H.rms_norm_quant(x, None, x, stream=st),
        lambda st: (H.matmul_quant(xq, xs, wq, ws, dtype=torch.float32, stream=st),),
        lambda st: (H.matmul_quant(xq[:3], xs[:3], wq, ws, stream=st),),
        lambda st: plan.apply_quant(x, code="e4m3", stream=st),
        lambda st: plan.apply_quant(x, code="int8", stream=st),
    ]


@pytest.mark.parametrize("handle", [False, True])
def test_results_belong_to_the_stream_of_the_call(handle):
    side = torch.cuda.Stream()
    for i, call in enumerate(_calls()):
        want = call(None)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        # blocks of the results' sizes, freed while the current stream has yet to fill them
        old = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(SLEEP)
        for t in old:
            t.view(torch.uint8).fill_(0x55)
        del old, t
        got = call(side.cuda_stream if handle else side)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), i


@pytest.mark.parametrize("coded", [False, True])
def test_gradient_workspace_belongs_to_the_stream_of_the_call(monkeypatch, coded):
    plan, side, seen = _plan(), torch.cuda.Stream(), []
    x, g = (torch.randn(300, 512, device=DEV).bfloat16() for _ in range(2))
    q, s = H.quantize(x, (1, 128), "int8")
    call = (lambda st: plan.grad_theta_quant(q, s, g, stream=st)) if coded else (lambda st: plan.grad_theta(x, g, stream=st))
    want = call(None)
    torch.cuda.synchronize()
    make = H.Plan.grad_workspace

    def recorded(self, device=None):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return make(self, device)

    monkeypatch.setattr(H.Plan, "grad_workspace", recorded)
    for st in (side, side.cuda_stream):
        got = call(st)
        torch.cuda.synchronize()
        # the order of the tiles' additions differs from call to call: up to 300 tiles, either sum off by 300 u of
        # its terms' magnitudes (sqrt(300) times the sum itself for random signs), 8 of which make a parameter
        assert (got - want).norm() <= 2 * 300 * 2.0 ** -24 * 300 ** 0.5 * 8 * want.norm()
    assert seen == [side.cuda_stream] * 2


def test_int8_call_refuses_e4m3_codes():
    plan = _plan()
    x = torch.randn(4, 512, device=DEV).bfloat16()
    q = torch.empty(4, 512, dtype=torch.float8_e4m3fn, device=DEV)
    with pytest.raises(TypeError):
        plan.apply_quant(x, q=q)
