"""The operators of the 8-bit linear layer around the rotation, as measured cases.

Five operators, each with a plain form in elementary torch operations and the library's call:

  norm      residual addition, root-mean-square norm, 8-bit codes with one scale per block
  product   matrix product of e4m3 codes with fp32 scales per 1 x 128 (rows) and 128 x 128 (weight) block
  quantize  8-bit codes of a matrix, per 1 x q block (activation checkpoints, restored again) or
            per 128 x 128 tile (the product's weight operand)
  rotate    the rotation with a fused e4m3 quantizer (the product's row operand)
  gradient  dL/dtheta of the rotation from rows that are kept as 8-bit checkpoints

Codes: a = max |v| over a block, scale = a / Q, code = round(v * (Q / a)) with Q = 127 for int8 and
448 for e4m3, each operation rounded to nearest in fp32; a zero block has scale and codes 0.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TOP = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TYPE = {"bfloat16": torch.bfloat16, "float32": torch.float32}
BYTES = {"bfloat16": 2, "float32": 4}

# Schedules of the rotation: the workloads' own, and shorter ones of the same radices.
SCHEDULES = {
    "8x8": (8, 8), "8x8x4": (8, 8, 4), "8x8x8": (8, 8, 8), "8x8x5x2": (8, 8, 5, 2), "8x8x8x4": (8, 8, 8, 4),
    "8x8x8x8": (8, 8, 8, 8), "8x8x8x5x2": (8, 8, 8, 5, 2), "8x8x8x8x2": (8, 8, 8, 8, 2),
}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one token of a decode step entering a layer of width 8192
        dict(name="norm 1x8192", op="norm", rows=1, d=8192, dtype="bfloat16", residual=True, weight=True, code="e4m3", qblock=128),
        # a ragged prefill batch entering a layer of width 5120, folded weight, codes kept as int8 checkpoints
        dict(name="norm 32767x5120 int8", op="norm", rows=32767, d=5120, dtype="bfloat16", residual=True, weight=False, code="int8", qblock=128),
        # one token through the widest weight of the workloads: the weight's bytes count
        dict(name="product 1x28672x8192", op="product", m=1, n=28672, k=8192, out="bfloat16"),
        # a small decode batch through a square layer
        dict(name="product 24x5120x5120", op="product", m=24, n=5120, k=5120, out="bfloat16"),
        # a ragged chunk of prefill, ragged n and k, fp32 result
        dict(name="product 333x4100x4112 f32", op="product", m=333, n=4100, k=4112, out="float32"),
        # prefill through the widest weight
        dict(name="product 4096x28672x8192", op="product", m=4096, n=28672, k=8192, out="bfloat16"),
        # a calibration batch's rows saved as int8 checkpoints and restored
        dict(name="checkpoint 65536x4096 int8", op="quantize", rows=65536, cols=4096, dtype="bfloat16", brows=1, bcols=128, code="int8", restore=True),
        # the rotated weight's quantization into the product's operand, ragged against its tiles
        dict(name="weight 28600x8200 e4m3", op="quantize", rows=28600, cols=8200, dtype="bfloat16", brows=128, bcols=128, code="e4m3", restore=False),
        # a prefill batch rotated in front of the product (the specialized kernel's shape)
        dict(name="rotate 65536x4096", op="rotate", rows=65536, schedule="8x8x8x8", direction="forward", qblock=128),
        # a decode batch rotated by the inverse (the input side of a two-sided rotated weight)
        dict(name="rotate 16x8192 inverse", op="rotate", rows=16, schedule="8x8x8x8x2", direction="inverse", qblock=128),
        # one calibration step of a layer from its int8 checkpoints
        dict(name="gradient 16384x4096 int8", op="gradient", rows=16384, schedule="8x8x8x8", dtype="bfloat16", code="int8", qblock=128),
        # a short, ragged calibration step, mixed radices, e4m3 checkpoints, fp32 upstream gradients
        dict(name="gradient 1001x5120 e4m3", op="gradient", rows=1001, schedule="8x8x8x5x2", dtype="float32", code="e4m3", qblock=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "product", "product", "quantize", "rotate", "gradient"])
    if op == "norm":
        d = _log(rng, 64, 8192)
        d -= d % 8 if rng.random() < 0.8 else 0      # odd widths among them
        rows = _log(rng, 1, min(65536, 160_000_000 // d))
        return dict(op=op, rows=rows, d=d, dtype=rng.choice(["bfloat16", "bfloat16", "float32"]), residual=rng.random() < 0.7,
                    weight=rng.random() < 0.6, code=rng.choice(["e4m3", "int8"]), qblock=rng.choice([32, 64, 128, 256]))
    if op == "product":
        n, k = _log(rng, 64, 28672), _log(rng, 64, 8192)
        m = _log(rng, 1, 8192)
        while m * n * k > 4096 * 28672 * 8192:
            m = (m + 1) // 2
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(["bfloat16", "float32"]))
    if op == "quantize":
        tile = rng.random() < 0.4
        rows, cols = (_log(rng, 1, 28672), _log(rng, 16, 8192)) if tile else (_log(rng, 1, 65536), _log(rng, 16, 8192))
        while rows * cols > 65536 * 4096:
            rows = (rows + 1) // 2
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bfloat16", "float32"]), brows=128 if tile else 1,
                    bcols=128 if tile else rng.choice([32, 64, 128, 256]), code="e4m3" if tile else rng.choice(["int8", "e4m3"]),
                    restore=rng.random() < 0.5)
    schedule = rng.choice(sorted(SCHEDULES))
    d = math.prod(SCHEDULES[schedule])
    q = rng.choice([q for q in (32, 64, 128, 256) if d % q == 0])
    if op == "rotate":
        return dict(op=op, rows=_log(rng, 1, 65536 * 4096 // max(d, 4096)), schedule=schedule, direction=rng.choice(["forward", "inverse"]), qblock=q)
    return dict(op=op, rows=_log(rng, 1, 16384 * 4096 // max(d, 4096)), schedule=schedule, dtype=rng.choice(["bfloat16", "float32"]),
                code=rng.choice(["int8", "e4m3"]), qblock=q)


def _ceil(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op == "norm":
        n, es = case["rows"] * case["d"], BYTES[case["dtype"]]
        reads = n * es * (2 if case["residual"] else 1) + (case["d"] * es if case["weight"] else 0)
        writes = n * (es if case["residual"] else 0) + n + 4 * case["rows"] * _ceil(case["d"], case["qblock"])
        return {"bytes": reads + writes, "flops": 5 * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        kb = _ceil(k, 128)
        return {"bytes": m * k + n * k + 4 * (m * kb + _ceil(n, 128) * kb) + m * n * BYTES[case["out"]], "flops": 2 * m * n * k}
    if op == "quantize":
        n, es = case["rows"] * case["cols"], BYTES[case["dtype"]]
        scales = 4 * _ceil(case["rows"], case["brows"]) * _ceil(case["cols"], case["bcols"])
        return {"bytes": n * es + n + scales + (n * es if case["restore"] else 0), "flops": 2 * n}
    schedule = SCHEDULES[case["schedule"]]
    d = math.prod(schedule)
    n = case["rows"] * d
    scales = 4 * n // case["qblock"]
    blocks = 4 * d * sum(schedule)
    if op == "rotate":
        return {"bytes": 2 * n + n + scales + blocks, "flops": 2 * n * sum(schedule)}
    # the inputs of every stage (all stages but the last applied), the gradients at every stage (all
    # but the first transposed), and one outer product per stage
    return {"bytes": n + scales + n * BYTES[case["dtype"]] + blocks + 4 * _theta_count(schedule),
            "flops": 2 * n * (3 * sum(schedule) - schedule[0] - schedule[-1])}


# ---------------------------------------------------------------- inputs ---

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _rows(gen, rows, cols, dtype, sigma=1.0):
    """Activations as a layer sees them: normal entries, a few outlier channels, rows of differing size."""
    x = torch.randn(rows, cols, generator=gen, device=DEV, dtype=torch.float32)
    channel = 1 + 20 * (torch.rand(cols, generator=gen, device=DEV) < 0.01).float()
    size = torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device=DEV))
    return (x.mul_(channel * sigma).mul_(size)).to(dtype)


def _padded(shape, dtype, multiple):
    """An empty matrix whose rows are `multiple` elements apart, at least."""
    ld = _ceil(shape[1], multiple) * multiple
    return torch.empty(shape[0], ld, dtype=dtype, device=DEV)[:, : shape[1]]


def _block_max(v, brows, bcols):
    r, c = v.shape
    pr, pc = _ceil(r, brows) * brows, _ceil(c, bcols) * bcols
    if (pr, pc) != (r, c):
        v = torch.nn.functional.pad(v, (0, pc - c, 0, pr - r))
    return v.abs().reshape(pr // brows, brows, pc // bcols, bcols).amax(dim=(1, 3))


def _spread(s, brows, bcols, rows, cols):
    return s.repeat_interleave(brows, 0)[:rows].repeat_interleave(bcols, 1)[:, :cols]


def _quantize(v, brows, bcols, code):
    """Codes and scales of fp32 values, every operation rounded to nearest in fp32."""
    top = torch.full((), TOP[code], device=v.device, dtype=torch.float32)
    a = _block_max(v, brows, bcols)
    scale = a / torch.full_like(a, TOP[code])
    inverse = torch.where(a > 0, top / a, torch.zeros_like(a))
    t = v * _spread(inverse, brows, bcols, *v.shape)
    if code == "int8":
        return torch.round(t).clamp(-127, 127).to(torch.int8), scale
    return t.clamp(-448, 448).to(torch.float8_e4m3fn), scale


def _stored(v, brows, bcols, code):
    """Codes (rows a multiple of 16 bytes apart) and scales that an earlier call left."""
    q, s = _quantize(v.float(), brows, bcols, code)
    out = _padded(q.shape, CODE[code], 16)
    out.copy_(q)
    return out, s


def _params(b):
    return 1 if b == 2 else b * (b - 1) // 2


def _theta_count(schedule):
    d = math.prod(schedule)
    return sum(d // b * _params(b) for b in schedule)


def _splitmix(seed, n):
    with np.errstate(over="ignore"):
        z = np.uint64(seed) + np.arange(1, n + 1, dtype=np.uint64) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))


def _mixer(b):
    """G_b in 64 bits: the normalized Sylvester Hadamard, else the sign-fixed QR of a seeded Gaussian."""
    if b & (b - 1) == 0:
        k = np.arange(b)
        ones = np.array([[bin(i & j).count("1") for j in k] for i in k])
        return (1.0 - 2.0 * (ones % 2)) / math.sqrt(b)
    u = (_splitmix(0x4841525000000000 + b, 2 * b * b) >> np.uint64(11)).astype(np.float64) * 2.0 ** -53
    g = np.sqrt(-2 * np.log(1 - u[0::2])) * np.cos(2 * np.pi * u[1::2])
    q, r = np.linalg.qr(g.reshape(b, b))
    return q * np.where(np.diag(r) < 0, -1.0, 1.0)


def _rotation(gen, seed, schedule):
    """theta (fp32, host) and the +-1 diagonal: what a fit leaves of a layer's rotation."""
    theta = (math.sqrt(0.05) * torch.randn(_theta_count(schedule), generator=gen, device=DEV)).cpu()
    sign_seed = 3000 + int(seed) % 100003
    signs = 1.0 - 2.0 * (_splitmix(sign_seed, math.prod(schedule)) >> np.uint64(63)).astype(np.float64)
    return theta, sign_seed, torch.from_numpy(signs).to(DEV)


def _skew(theta, b):
    """[blocks, b, b] skew matrices of [blocks, p] parameters."""
    i, j = torch.triu_indices(b, b, 1, device=theta.device)
    a = torch.zeros(theta.shape[0], b, b, dtype=theta.dtype, device=theta.device)
    a[:, i, j] = theta
    return a - a.transpose(1, 2)


def _stage_thetas(theta, schedule):
    d = math.prod(schedule)
    return torch.split(theta, [d // b * _params(b) for b in schedule])


def _learned(th, b):
    """Q(theta) of a stage's blocks in 64 bits: Givens rotations for b = 2, else Cayley maps."""
    if b == 2:
        c, s = torch.cos(th), torch.sin(th)
        return torch.stack([torch.stack([c, -s], -1), torch.stack([s, c], -1)], -2)
    a = _skew(th.reshape(-1, _params(b)), b)
    eye = torch.eye(b, dtype=th.dtype, device=th.device)
    return torch.linalg.solve(eye - a, eye + a)


def prepare(case, seed):
    gen = _generator(seed)
    state = dict(case)
    op = case["op"]
    if op == "norm":
        rows, d, dtype = case["rows"], case["d"], TYPE[case["dtype"]]
        state["x"] = _rows(gen, rows, d, dtype)
        state["residual"] = _rows(gen, rows, d, dtype, 2.0) if case["residual"] else None
        state["weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(dtype) if case["weight"] else None
        # buffers of the step
        state["h"] = torch.empty(rows, d, dtype=dtype, device=DEV) if case["residual"] else None
        state["q"] = _padded((rows, d), CODE[case["code"]], 16)
        state["s"] = torch.empty(rows, _ceil(d, case["qblock"]), device=DEV)
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        state["xq"], state["xs"] = _stored(_rows(gen, m, k, torch.bfloat16), 1, 128, "e4m3")
        w = torch.randn(n, k, generator=gen, device=DEV) * 0.02
        state["wq"], state["ws"] = _stored(w, 128, 128, "e4m3")
        state["y"] = torch.empty(m, n, dtype=TYPE[case["out"]], device=DEV)
    elif op == "quantize":
        rows, cols, dtype = case["rows"], case["cols"], TYPE[case["dtype"]]
        state["x"] = _rows(gen, rows, cols, dtype)
        state["q"] = _padded((rows, cols), CODE[case["code"]], 16)
        state["s"] = torch.empty(_ceil(rows, case["brows"]), _ceil(cols, case["bcols"]), device=DEV)
        state["back"] = torch.empty(rows, cols, dtype=dtype, device=DEV) if case["restore"] else None
    else:
        schedule = SCHEDULES[case["schedule"]]
        d, rows = math.prod(schedule), case["rows"]
        theta, sign_seed, signs = _rotation(gen, seed, schedule)
        x = _rows(gen, rows, d, torch.bfloat16)
        if op == "rotate":
            state["x"] = x
            state["q"] = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device=DEV)
            state["s"] = torch.empty(rows, d // case["qblock"], device=DEV)
        else:
            state["q"], state["s"] = _stored(x, 1, case["qblock"], case["code"])
            state["g"] = torch.randn(rows, d, generator=gen, device=DEV).to(TYPE[case["dtype"]])
            state["dtheta"] = torch.empty(_theta_count(schedule), device=DEV)
        if own:
            import structured_rotations_b200 as H
            state["plan"] = H.Plan(d, schedule, theta=theta.numpy(), sign_seed=sign_seed).materialize()
            if op == "gradient":
                state["workspace"] = state["plan"].grad_workspace()
        else:
            th = _stage_thetas(theta.to(DEV).double(), schedule)
            state["Q"] = [_learned(t, b) for t, b in zip(th, schedule)]
            state["thetas"] = th
            state["G"] = [torch.from_numpy(_mixer(b)).to(DEV) for b in schedule]
            state["B"] = [(q @ g).float() for q, g in zip(state["Q"], state["G"])]
            state["signs"] = signs.float()
    return state


# ----------------------------------------------------------- plain forms ---

def _plain_norm(s):
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(h.dtype)
    h32 = h.float()
    mean = h32.double().square().sum(-1, keepdim=True) / s["d"]
    u = h32 * (1 / torch.sqrt(mean + 1e-6)).float()
    if s["weight"] is not None:
        u = u * s["weight"].float()
    q, sc = _quantize(u, 1, s["qblock"], s["code"])
    out = {"codes": q, "scales": sc}
    return out if s["residual"] is None else {**out, "h": h}


def _plain_product(s):
    x = s["xq"].float() * _spread(s["xs"], 1, 128, *s["xq"].shape)
    w = s["wq"].float() * _spread(s["ws"], 128, 128, *s["wq"].shape)
    return (x @ w.t()).to(s["y"].dtype)


def _plain_quantize(s):
    q, sc = _quantize(s["x"].float(), s["brows"], s["bcols"], s["code"])
    out = {"codes": q, "scales": sc}
    if s["restore"]:
        out["values"] = (q.float() * _spread(sc, s["brows"], s["bcols"], *q.shape)).to(s["x"].dtype)
    return out


def _stage(x, blocks, b, stride):
    """Every group of b coordinates `stride` apart times its block."""
    rows, d = x.shape
    hi = d // (b * stride)
    y = torch.einsum("hokl,rhlo->rhko", blocks.reshape(hi, stride, b, b), x.reshape(rows, hi, b, stride))
    return y.reshape(rows, d)


def _strides(schedule):
    return [math.prod(schedule[:t]) for t in range(len(schedule))]


def _plain_rotate(s):
    schedule = SCHEDULES[s["schedule"]]
    stages = list(zip(s["B"], schedule, _strides(schedule)))
    y = s["x"].float()
    if s["direction"] == "forward":
        y = y * s["signs"]
        for blocks, b, stride in stages:
            y = _stage(y, blocks, b, stride)
    else:
        for blocks, b, stride in reversed(stages):
            y = _stage(y, blocks.transpose(1, 2), b, stride)
        y = y * s["signs"]
    q, sc = _quantize(y, 1, s["qblock"], "e4m3")
    return {"codes": q, "scales": sc}


def _plain_gradient(s):
    schedule = SCHEDULES[s["schedule"]]
    strides = _strides(schedule)
    x = s["q"].float() * _spread(s["s"], 1, s["qblock"], *s["q"].shape)
    z = [x * s["signs"]]
    for blocks, b, stride in list(zip(s["B"], schedule, strides))[:-1]:
        z.append(_stage(z[-1], blocks, b, stride))
    h = s["g"].float()
    out = []
    for t in reversed(range(len(schedule))):
        b, stride = schedule[t], strides[t]
        rows, d = h.shape
        hi = d // (b * stride)
        hv, zv = h.reshape(rows, hi, b, stride), z.pop().reshape(rows, hi, b, stride)
        d_block = torch.einsum("rhko,rhlo->hokl", hv, zv).reshape(-1, b, b).double()
        d_q = d_block @ s["G"][t].t()
        if b == 2:
            c, sn = torch.cos(s["thetas"][t]), torch.sin(s["thetas"][t])
            out.append(-d_q[:, 0, 0] * sn - d_q[:, 0, 1] * c + d_q[:, 1, 0] * c - d_q[:, 1, 1] * sn)
        else:
            # Q = (I - A)^-1 (I + A): dL/dA = (I - A)^-T dL/dQ (Q + I)^T
            eye = torch.eye(b, dtype=torch.float64, device=h.device)
            a = _skew(s["thetas"][t].reshape(-1, _params(b)), b)
            e = torch.linalg.solve((eye - a).transpose(1, 2), d_q) @ (s["Q"][t] + eye).transpose(1, 2)
            i, j = torch.triu_indices(b, b, 1, device=h.device)
            out.append((e[:, i, j] - e[:, j, i]).reshape(-1))
        if t:
            h = _stage(h, s["B"][t].transpose(1, 2), b, stride)
    return torch.cat(out[::-1]).float()


# ------------------------------------------------------------------- run ---

def run(state):
    s, op = state, state["op"]
    if not own:
        return {"norm": _plain_norm, "product": _plain_product, "quantize": _plain_quantize, "rotate": _plain_rotate,
                "gradient": _plain_gradient}[op](s)
    import structured_rotations_b200 as H
    if op == "norm":
        H.rms_norm_quant(s["x"], s["weight"], s["residual"], eps=1e-6, qblock=s["qblock"], code=s["code"], h=s["h"], q=s["q"], scales=s["s"])
        out = {"codes": s["q"], "scales": s["s"]}
        return out if s["h"] is None else {**out, "h": s["h"]}
    if op == "product":
        return H.matmul_quant(s["xq"], s["xs"], s["wq"], s["ws"], out=s["y"])
    if op == "quantize":
        block = (s["brows"], s["bcols"])
        H.quantize(s["x"], block=block, code=s["code"], q=s["q"], scales=s["s"])
        out = {"codes": s["q"], "scales": s["s"]}
        if s["restore"]:
            out["values"] = H.dequantize(s["q"], s["s"], block=block, out=s["back"])
        return out
    if op == "rotate":
        s["plan"].apply_quant(s["x"], s["qblock"], s["direction"], q=s["q"], scales=s["s"], code="e4m3")
        return {"codes": s["q"], "scales": s["s"]}
    return s["plan"].grad_theta_quant(s["q"], s["s"], s["g"], dtheta=s["dtheta"], workspace=s["workspace"])


# ----------------------------------------------------------------- exact ---

def _exact_codes(v, brows, bcols, code):
    """Scales, and the values that the codes stand for, by the definition in 64 bits."""
    rows, cols = v.shape
    pad = torch.zeros(_ceil(rows, brows) * brows, _ceil(cols, bcols) * bcols, dtype=torch.float64, device=v.device)
    pad[:rows, :cols] = v
    t = pad.unflatten(0, (-1, brows)).unflatten(2, (-1, bcols))
    scale = t.abs().amax(3).amax(1) / TOP[code]
    unit = torch.where(scale > 0, scale, torch.ones_like(scale))[:, None, :, None]
    t = t / unit
    if code == "int8":
        t = t.round()
    else:  # three bits behind the leading one, the smallest step 2^-9
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
        t = (t / step).round() * step
    return scale, t.flatten(2, 3).flatten(0, 1)[:rows, :cols]


def _exact_blocks(theta, schedule):
    """B_t = Q_t(theta) G in 64 bits, differentiable in theta; the Cayley map as 2 (I - A)^-1 - I."""
    out = []
    for th, b in zip(_stage_thetas(theta, schedule), schedule):
        if b == 2:
            turn = torch.tensor([[0.0, -1.0], [1.0, 0.0]], dtype=torch.float64, device=DEV)
            q = torch.cos(th)[:, None, None] * torch.eye(2, dtype=torch.float64, device=DEV) + torch.sin(th)[:, None, None] * turn
        else:
            eye = torch.eye(b, dtype=torch.float64, device=DEV)
            q = 2 * torch.linalg.inv(eye - _skew(th.reshape(-1, _params(b)), b)) - eye
        out.append(q @ torch.from_numpy(_mixer(b)).to(DEV))
    return out


def _exact_transform(x, blocks, schedule, signs, forward=True):
    """The stages as gathers of each block's coordinates."""
    d = math.prod(schedule)
    if forward:
        x = x * signs
    order = range(len(schedule)) if forward else reversed(range(len(schedule)))
    for t in order:
        b, stride = schedule[t], math.prod(schedule[:t])
        c = torch.arange(d // b, device=x.device)
        at = ((c % stride) + (c // stride) * stride * b)[:, None] + stride * torch.arange(b, device=x.device)
        m = blocks[t] if forward else blocks[t].transpose(1, 2)
        parts = torch.matmul(x[:, at].transpose(0, 1), m.transpose(1, 2))  # [block, row, b]
        back = torch.empty(d, dtype=torch.int64, device=x.device)
        back[at.reshape(-1)] = torch.arange(d, device=x.device)
        x = parts.transpose(0, 1).reshape(x.shape[0], d)[:, back]
    return x if forward else x * signs


def _chunks(rows, d):
    step = max(1, (1 << 26) // d)
    return [(r, min(rows, r + step)) for r in range(0, rows, step)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        u = h * torch.rsqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["d"] + 1e-6)
        if s["weight"] is not None:
            u = u * s["weight"].double()
        scale, codes = _exact_codes(u, 1, case["qblock"], case["code"])
        out = {"codes": codes if case["code"] == "e4m3" else None, "scales": scale}
        return out if s["residual"] is None else {**out, "h": h}
    if op == "product":
        k = case["k"]
        y = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
        row_of = torch.arange(case["n"], device=DEV) // 128
        for kb in range(_ceil(k, 128)):
            part = s["xq"][:, 128 * kb : 128 * kb + 128].double() @ s["wq"][:, 128 * kb : 128 * kb + 128].double().t()
            y += part * s["xs"][:, kb].double()[:, None] * s["ws"][row_of, kb].double()[None, :]
        return y
    if op == "quantize":
        scale, codes = _exact_codes(s["x"].double(), case["brows"], case["bcols"], case["code"])
        out = {"codes": codes if case["code"] == "e4m3" else None, "scales": scale}
        if case["restore"]:
            unit = scale.repeat_interleave(case["brows"], 0)[: case["rows"]].repeat_interleave(case["bcols"], 1)[:, : case["cols"]]
            out["values"] = codes * unit
        return out
    schedule = SCHEDULES[case["schedule"]]
    d, rows = math.prod(schedule), case["rows"]
    gen = _generator(seed)
    theta, _, signs = _rotation(gen, seed, schedule)
    theta = theta.to(DEV).double()
    if op == "rotate":
        blocks = _exact_blocks(theta, schedule)
        got = [_exact_codes(_exact_transform(s["x"][a:b].double(), blocks, schedule, signs, case["direction"] == "forward"), 1,
                            case["qblock"], "e4m3") for a, b in _chunks(rows, d)]
        return {"codes": torch.cat([c for _, c in got]), "scales": torch.cat([c for c, _ in got])}
    theta.requires_grad_(True)
    for a, b in _chunks(rows, d):
        x = (s["q"][a:b].double().unflatten(1, (-1, case["qblock"])) * s["s"][a:b].double()[:, :, None]).flatten(1)
        y = _exact_transform(x, _exact_blocks(theta, schedule), schedule, signs)
        (y * s["g"][a:b].double()).sum().backward()
    return theta.grad
