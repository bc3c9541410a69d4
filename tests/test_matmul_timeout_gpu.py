"""Waits of the e4m3 product's kernels that run out, on the GPU, without a fault: the test hook
harp_test_inject_wait_timeout makes every load's barrier expect a few bytes more than are copied, and every
wait give up after a few clocks.  Nothing waits for longer than that; the kernels report it through the
device's status word, free their tensor memory and end, and the next products are right (twenty of
them, on every SM: tensor memory that stayed taken would run out)."""
import pytest

torch = pytest.importorskip("torch")

import structured_rotations_b200 as H
from structured_rotations_b200 import harp as HB

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _operands(m, n, k):
    g = torch.Generator(device=DEV).manual_seed(m + n)

    def codes(rows):
        q = torch.zeros(rows, -(-k // 16) * 16, dtype=torch.float8_e4m3fn, device=DEV)[:, :k]
        return q.copy_(torch.randint(-2, 3, (rows, k), generator=g, device=DEV).float())

    xq, wq = codes(m), codes(n)
    return (xq, torch.ones(m, -(-k // 128), device=DEV), wq, torch.ones(-(-n // 128), -(-k // 128), device=DEV)), xq.float() @ wq.float().t()


# every tile of the rows kernel, alone and with k split over a cluster, and both tiles of the other
@pytest.mark.parametrize("m,n,k,kernel", [(5, 300, 130, "rows"), (5, 300, 2100, "rows"), (20, 40000, 300, "rows"), (40, 300, 1000, "rows"),
                                          (64, 20000, 260, "rows"), (100, 260, 900, "rows"), (150, 270, 500, "tiles"),
                                          (2560, 1536, 700, "tiles"), (2560, 1536, 2000, "tiles")])
def test_waits_that_run_out(m, n, k, kernel):
    ops, want = _operands(m, n, k)
    H.device_status()
    for calls in (1, 3):
        H.inject_wait_timeout(1000, 16)
        try:
            for _ in range(calls):
                H.matmul_quant(*ops, dtype=torch.float32)
                assert H.last_kernel() == f"matmul_{kernel}_kernel"
        finally:
            H.inject_wait_timeout(0, 0)
        with pytest.raises(HB.HarpError) as e:
            H.device_status()
        assert e.value.status == HB.HARP_ERR_TIMEOUT
        H.device_status()                                 # cleared by the read
        for _ in range(20):
            got = H.matmul_quant(*ops, dtype=torch.float32)
        H.device_status()
        assert torch.equal(got, want)
