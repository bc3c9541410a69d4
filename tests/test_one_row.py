"""A matrix of one row is never stepped past, so its leading dimension decides nothing: a decode step takes
the kernels that a batch takes, whatever its width, and torch's view of such a matrix (contiguous with any
stride) does not turn it away.  Values are compared with a batch that holds the same row (bit for bit:
the quantizer's and the norm's codes depend on the row alone), products with exact sums."""
import pytest

torch = pytest.importorskip("torch")

import structured_rotations_b200 as H
from structured_rotations_b200 import harp as HB

DEV = "cuda"


def test_a_single_row_of_any_stride_is_taken():
    """torch calls every view of one row contiguous; its stride may be anything, and the binding's leading
    dimension is at least the width."""
    for v in (torch.empty(1, 176)[:, :162], torch.empty(1, 162), torch.empty(162, 1).t(), torch.empty(400).as_strided((1, 162), (7, 1))):
        assert HB._expect(v, (1, 162), torch.float32, -1, "v")[1] >= 162
    assert HB._expect(torch.empty(2, 176)[:, :162], (2, 162), torch.float32, -1, "v")[1] == 176


def _exact(m, n, k, seed):
    # codes -2 .. 2 and scales 1, 2, 1/2: every partial sum is exact in fp32
    g = torch.Generator(device=DEV).manual_seed(seed)

    def codes(rows):
        q = torch.zeros(rows, -(-k // 16) * 16, dtype=torch.float8_e4m3fn, device=DEV)[:, :k]
        return q.copy_(torch.randint(-2, 3, (rows, k), generator=g, device=DEV).float())

    kb, nb = -(-k // 128), -(-n // 128)
    xs = torch.randint(0, 2, (m, kb), generator=g, device=DEV).float() + 1
    ws = (torch.randint(0, 2, (nb, kb), generator=g, device=DEV).float() + 1) / 2
    return codes(m), xs, codes(n), ws


def _want(xq, xs, wq, ws):
    def full(q, s, rows):
        return q.double() * s.double().repeat_interleave(rows, 0)[: q.shape[0]].repeat_interleave(128, 1)[:, : q.shape[1]]
    return full(xq, xs, 1) @ full(wq, ws, 128).t()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1, 300, 4100), (1, 1, 1), (1, 5, 162), (3, 1, 130), (1, 1, 2049), (200, 1, 300), (1, 4096, 17)])
def test_product_of_one_row_takes_the_tensor_cores(m, n, k):
    xq, xs, wq, ws = _exact(m, n, k, m + n + k)
    want = _want(xq, xs, wq, ws).float()
    # as a padded view, as a row on its own, and with a leading dimension that TMA does not take
    views = [(xq, wq)]
    if m == 1:
        views += [(xq.clone(memory_format=torch.contiguous_format).reshape(1, k), wq),
                  (xq.as_strided((1, k), (k + 3, 1)), wq)]
    if n == 1:
        views += [(xq, wq.as_strided((1, k), (k + 3, 1)))]
    for a, b in views:
        assert torch.equal(H.matmul_quant(a, xs, b, ws, dtype=torch.float32), want)
        assert H.last_kernel() == ("matmul_rows_kernel" if m <= 64 else "matmul_tiles_kernel")
    H.device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("k", [4100, 162, 8200])
def test_decode_step_of_any_width(k):
    """What quantize and rms_norm_quant return for one token goes to the rows kernel."""
    g = torch.Generator(device=DEV).manual_seed(k)
    x = torch.randn(1, k, generator=g, device=DEV).bfloat16()
    w = H.quantize(torch.randn(260, k, generator=g, device=DEV), (128, 128))
    for xq, xs in (H.quantize(x), H.rms_norm_quant(x)[:2]):
        y = H.matmul_quant(xq, xs, *w, dtype=torch.float32)
        assert H.last_kernel() == "matmul_rows_kernel"
        want = _want(xq, xs, *w)
        mag = _want(xq.float().abs(), xs, w[0].float().abs(), w[1])
        # the product's bound: 128 + kb + 4 additions of at most one ulp, half an ulp of the result
        assert torch.all((y.double() - want).abs() <= (133 + xs.shape[1]) * 2.0 ** -23 * mag)
    H.device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [8, 100, 1003, 5120])
def test_codes_of_one_row_equal_those_of_a_batch(d, dtype):
    """With leading dimensions that no vector access divides; nothing is written beside the row."""
    g = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn(3, d, generator=g, device=DEV).to(dtype)
    r = torch.randn(3, d, generator=g, device=DEV).to(dtype)
    for code in ("int8", "e4m3"):
        t = torch.int8 if code == "int8" else torch.float8_e4m3fn
        buf = torch.full((1, d + 5), 3, dtype=torch.uint8, device=DEV)
        q = buf.as_strided((1, d), (d + 5, 1)).view(t)
        want, ws = H.quantize(x, (1, 64), code)
        _, s = H.quantize(x[:1].as_strided((1, d), (d + 3, 1)), (1, 64), code, q=q)
        assert torch.equal(q.view(torch.uint8), want[:1].view(torch.uint8)) and torch.equal(s, ws[:1])
        assert torch.all(buf[:, d:] == 3)
        y = H.dequantize(q, s, (1, 64), dtype=dtype)
        assert torch.equal(y, H.dequantize(want, ws, (1, 64), dtype=dtype)[:1])
        buf.fill_(3)
        wn, wns, wh = H.rms_norm_quant(x, None, r, qblock=64, code=code)
        _, s, h = H.rms_norm_quant(x[:1], None, r[:1], qblock=64, code=code, q=q)
        assert torch.equal(q.view(torch.uint8), wn[:1].view(torch.uint8)) and torch.equal(s, wns[:1]) and torch.equal(h, wh[:1])
        assert torch.all(buf[:, d:] == 3)


@pytest.mark.gpu
def test_in_place_sum_of_one_row_with_another_stride():
    """h may be x itself; of one row the two may be views of different strides."""
    x = torch.randn(1, 256, device=DEV).bfloat16()
    r = torch.randn(1, 256, device=DEV).bfloat16()
    want = H.rms_norm_quant(x, None, r)
    buf = torch.empty(1, 300, dtype=torch.bfloat16, device=DEV)
    buf[:, :256] = x
    got = H.rms_norm_quant(buf[:, :256], None, r, h=buf.as_strided((1, 256), (256, 1)))
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_gradient_of_one_row(code):
    """One row with leading dimensions that no vector access divides, against the same row padded to 16
    bytes: one tile, the same order of every sum."""
    plan = H.Plan(512, (8, 8, 8), sign_seed=3).materialize()
    x, g = torch.randn(1, 512, device=DEV), torch.randn(1, 512, device=DEV)
    q, s = H.quantize(x, (1, 64), code)
    want = plan.grad_theta_quant(q, s, g)
    odd = plan.grad_theta_quant(q.as_strided((1, 512), (515, 1)), s, g.as_strided((1, 512), (513, 1)))
    assert torch.equal(odd, want)
    f = plan.grad_theta(x, g)
    assert torch.equal(plan.grad_theta(x.as_strided((1, 512), (513, 1)), g.as_strided((1, 512), (513, 1))), f)


@pytest.mark.gpu
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("direction", ["forward", "inverse"])
def test_rotation_of_one_row_with_any_stride(code, direction):
    """Codes and bf16 rows whose leading dimensions no vector access divides: the same codes, nothing beside them."""
    plan = H.Plan(1024, (8, 8, 8, 2), sign_seed=3).materialize()
    x = torch.randn(1, 1024, device=DEV).bfloat16()
    want, ws = plan.apply_quant(x, 64, direction, code=code)
    buf = torch.full((1, 1031), 3, dtype=torch.uint8, device=DEV)
    q = buf[:, :1024].view(want.dtype)
    _, s = plan.apply_quant(x.as_strided((1, 1024), (1027, 1)), 64, direction, q=q, code=code)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s, ws)
    assert torch.all(buf[:, 1024:] == 3)
