"""The calibration backward on tiles of many rows and on ragged last tiles, from plain rows and from 8-bit
checkpoints, against the float64 oracle, element by element.

The kernel takes tiles of R rows: as many as shared memory holds (two fp32 rows of round_up(d, 32) floats each
in 227 KiB, at most 16), then as few as keep the number of rounds over the SMs, R = ceil(rows / (rounds SMs)).
`_tiles` repeats that rule, so the batches here are sized to reach the largest R, a smaller one, several
rounds, and a last tile of fewer rows.

Bound: test_grad_gpu's, an entry's terms now being added in R rows of a tile and over the tiles: R + ntiles
additions instead of ntiles."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import harp_oracle as O
import workloads as W
import structured_rotations_b200 as H
from tests import _codes as C
from tests.test_grad_gpu import _check

pytestmark = pytest.mark.gpu
DEV = "cuda"

SCHEDULES = [(8, 8), (8, 8, 8), (8, 8, 8, 8), (8, 8, 8, 5, 2), (8, 8, 8, 8, 2), (5, 2, 8), (7, 8), (3, 4, 2), (6, 6), (5, 7, 3),
             (2, 2, 2, 2, 2), (3,), (8, 7, 6, 5, 4), (4, 3, 5, 7)]


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _most(d):
    return min(16, 227 * 1024 // (8 * ((d + 31) // 32 * 32)))


def _tiles(d, rows):
    """(rows per tile, tiles) of the gradient kernel."""
    rounds = -(-rows // (_most(d) * _sms()))
    r = -(-rows // (rounds * _sms()))
    return r, -(-rows // r)


def _batches(d):
    """Batches whose last tile is ragged: the largest tile in one round, about half of it, and two rounds where the
    rows are short enough for the oracle."""
    most, sms = _most(d), _sms()
    full = most * sms
    half = max(2, (most + 1) // 2) * sms
    out = [full - 1 if most < 4 else full - 3, half - 1]
    if d <= 512:
        out.append(2 * full - 5)
    return out


def _plan(schedule):
    d = int(np.prod(schedule))
    theta = W.draw_theta(O.theta_count(schedule), 0.3, 31)
    gp = H.Plan(d, schedule, theta=theta, sign_seed=12).materialize()
    return d, gp, O.make_plan(d, schedule, theta.astype(np.float32).astype(np.float64), sign_seed=12)


def _decoded(q, s, qblock, code):
    return C.decode(C.to_numpy(q), s.cpu().numpy(), 1, qblock, code).astype(np.float32).astype(np.float64)


def _cases(kinds):
    """Every schedule with every kind (a tuple that ends in the batch's number); two rounds for short rows only."""
    return [(s, *k) for s in SCHEDULES for k in kinds if k[-1] < 2 or np.prod(s) <= 512]


@pytest.mark.parametrize("schedule,which", _cases([(0,), (1,), (2,)]), ids=str)
def test_plain_rows(schedule, which):
    d, gp, op = _plan(schedule)
    rows = _batches(d)[which]
    r, n = _tiles(d, rows)
    assert r > 1 and rows % r, (r, rows)
    gen = torch.Generator(device=DEV).manual_seed(d + which)
    x, g = (torch.randn(rows, d, generator=gen, device=DEV) for _ in range(2))
    if which == 1:
        x, g = x.bfloat16(), g.bfloat16()
    got = gp.grad_theta(x, g)
    _check(got.cpu().numpy(), x.double().cpu().numpy(), g.double().cpu().numpy(), op, f"{schedule} {rows} rows, {r} a tile", r + n)
    # the same rows at odd distances: loads one by one, another walk over the tile
    xo, go = torch.zeros(rows, d + 3, dtype=x.dtype, device=DEV), torch.zeros(rows, d + 1, dtype=x.dtype, device=DEV)
    xo[:, 1:d + 1], go[:, 1:] = x, g
    got = gp.grad_theta(xo[:, 1:d + 1], go[:, 1:])
    _check(got.cpu().numpy(), x.double().cpu().numpy(), g.double().cpu().numpy(), op, f"{schedule} {rows} unaligned rows", r + n)


@pytest.mark.parametrize("schedule,code,qblock,which",
                         _cases([("int8", 64, 0), ("e4m3", 32, 0), ("e4m3", 128, 1), ("int8", 32, 2), ("e4m3", 64, 2)]), ids=str)
def test_rows_as_codes(schedule, code, qblock, which):
    d, gp, op = _plan(schedule)
    rows = _batches(d)[which]
    r, n = _tiles(d, rows)
    assert r > 1 and rows % r, (r, rows)
    gen = torch.Generator(device=DEV).manual_seed(d + 10 * which)
    x, g = (torch.randn(rows, d, generator=gen, device=DEV) for _ in range(2))
    if code == "int8":
        g = g.bfloat16()
    q, s = H.quantize(x, (1, qblock), code)
    xh, g64 = _decoded(q, s, qblock, code), g.double().cpu().numpy()
    got = gp.grad_theta_quant(q, s, g, qblock=qblock)
    _check(got.cpu().numpy(), xh, g64, op, f"{schedule} {code} {rows} rows, {r} a tile", r + n)
    go = torch.zeros(rows, d + 5, dtype=g.dtype, device=DEV)
    go[:, 3:d + 3] = g
    qo = torch.zeros(rows, d + 7, dtype=torch.uint8, device=DEV)
    qo[:, 5:d + 5] = q.view(torch.uint8)
    so = torch.zeros(rows, s.shape[1] + 1, device=DEV)
    so[:, 1:] = s
    got = gp.grad_theta_quant(qo[:, 5:d + 5].view(q.dtype), so[:, 1:], go[:, 3:d + 3], qblock=qblock)
    _check(got.cpu().numpy(), xh, g64, op, f"{schedule} {code} {rows} unaligned rows", r + n)


def test_refusals_one_by_one():
    """Each call of a list is refused by itself: codes whose scales tell no block size."""
    _, gp, _ = _plan((8, 8))
    q = torch.zeros(4, 64, dtype=torch.int8, device=DEV)
    g = torch.zeros(4, 64, device=DEV)
    for nb in (0, 3, 4):
        with pytest.raises(ValueError):
            gp.grad_theta_quant(q, torch.zeros(4, nb, device=DEV), g)
    with pytest.raises(ValueError):
        gp.grad_theta_quant(q, torch.zeros(4, device=DEV), g)
    # one scale for 64 coordinates is a block of 64
    assert torch.count_nonzero(gp.grad_theta_quant(q, torch.zeros(4, 1, device=DEV), g)).item() == 0
