"""Which kernel a product runs on: every kernel gives right results for every size, so only the name of the
kernel shows a call that went to the wrong one.  Aligned operands (as quantize makes them) with up to 64
rows take the rows kernel; up to 128 rows too, while the weight has at most an eighth as many tiles of 128 rows as
there are SMs; more rows the tiles kernel; operands that TMA does not take the CUDA cores."""
import pytest

torch = pytest.importorskip("torch")

import structured_rotations_b200 as H

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _wide():
    """The most columns that keep 65 to 128 rows on the rows kernel."""
    return torch.cuda.get_device_properties(0).multi_processor_count // 8 * 128


def _codes(rows, k, ld=None, offset=0):
    buf = torch.zeros(rows * (ld or -(-k // 16) * 16) + offset + k, dtype=torch.uint8, device=DEV)
    return buf.as_strided((rows, k), (ld or -(-k // 16) * 16, 1), offset).view(torch.float8_e4m3fn).fill_(1.0)


def _kernel(xq, wq, out=torch.float32):
    k = xq.shape[1]
    xs = torch.ones(xq.shape[0], -(-k // 128), device=DEV)
    ws = torch.ones(-(-wq.shape[0] // 128), -(-k // 128), device=DEV)
    y = H.matmul_quant(xq, xs, wq, ws, dtype=out)
    assert torch.all(y.float() == float(k))
    return H.last_kernel()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 16, 129, 256])
@pytest.mark.parametrize("m", [1, 2, 16, 17, 33, 63, 64])
@pytest.mark.parametrize("n", [1, 2, 128, 5000])
def test_up_to_64_rows(m, n, k, out):
    assert _kernel(_codes(m, k), _codes(n, k), out) == "matmul_rows_kernel"


@pytest.mark.parametrize("m", [65, 100, 127, 128])
@pytest.mark.parametrize("k", [130, 256])
def test_up_to_128_rows(m, k):
    for n, kernel in ((1, "rows"), (_wide(), "rows"), (_wide() + 1, "tiles")):
        assert _kernel(_codes(m, k), _codes(n, k)) == f"matmul_{kernel}_kernel"


@pytest.mark.parametrize("m", [129, 256, 257, 1000])
@pytest.mark.parametrize("n", [1, 300, 3001])
def test_many_rows(m, n):
    assert _kernel(_codes(m, 200), _codes(n, 200)) == "matmul_tiles_kernel"


@pytest.mark.parametrize("m", [2, 64, 100, 300])
def test_unaligned_operands(m):
    k, n = 200, 130
    ok = _codes(m, k), _codes(n, k)
    assert _kernel(ok[0], _codes(n, k, offset=1)) == "matmul_simple_kernel"
    assert _kernel(_codes(m, k, offset=8), ok[1]) == "matmul_simple_kernel"
    assert _kernel(_codes(m, k, ld=201), ok[1]) == "matmul_simple_kernel"
    assert _kernel(ok[0], _codes(n, k, ld=232)) == "matmul_simple_kernel"
    assert _kernel(*ok) != "matmul_simple_kernel"
    # a single row's leading dimension plays no part, its address does
    assert _kernel(_codes(1, k, ld=201), ok[1]) == "matmul_rows_kernel"
    assert _kernel(_codes(1, k, offset=1), ok[1]) == "matmul_simple_kernel"
