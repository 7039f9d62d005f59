"""Measured cases of the 8-bit product with a scale for each block of 128, of the quantiser that makes its
operands, of its training form, and of the orthogonalised update of a weight.

``listed()`` gives the cases, ``prepare`` their inputs, ``run`` one pass: in plain torch operations in
32 bits, or, with ``own`` set, through the library's entry points.  ``exact`` gives the same outputs
from the definitions in 64 bits.

  quantize  a block is 128 values of a row ("row") or 128 x 128 values ("tile"), cut at the edges:
            scale = the smallest power of two with max|x| <= 448 scale (1 where all are 0, at least
            2^-126), held as its exponent in 8 bits; values e4m3(x / scale).  Of the matrix, and of its
            transpose with blocks of its own.
  product   y = act(sum over blocks of scale_x scale_w (x weight^T) + bias) + residual, x in row blocks,
            weight in tiles; scales as the quantiser makes them, or any numbers in 32 bits.
  train     the product of bf16 x and weight, quantised on the way, and its gradients through products
            of the same kind: grad_x = g weight with g in row blocks; grad_weight = g^T x with g^T in
            row blocks and x^T in tiles; grad_bias the column sums of g.
  ortho     X = G / (norm of G + eps), then five times X <- a X + (b A + c A A) X with A = X X^T.
"""
import math

import torch

own = False
DEV = "cuda"
BF16, F32, E4M3, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu
TYPES = {"bf16": BF16, "f32": F32}
BLOCK = 128
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS, EPS = 5, 1e-7


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # the operand of sixteen sequences that generate one token each: latency
        dict(name="quantize_step", op="quantize", n=16, K=6656, dtype="bf16", blocks="row", transposed="none"),
        # a training step's upstream gradient, for both of its products
        dict(name="quantize_grad", op="quantize", n=8192, K=6656, dtype="bf16", blocks="row", transposed="row"),
        # 32-bit activations at sizes that are no multiple of anything, kept for the weight's gradient
        dict(name="quantize_odd", op="quantize", n=2051, K=4099, dtype="f32", blocks="row", transposed="tile"),
        # a 32-bit weight, for the forward and for its input's gradient
        dict(name="quantize_weight", op="quantize", n=16384, K=4096, dtype="f32", blocks="tile", transposed="tile"),
        # the head of eight generating sequences: the weight is read once
        dict(name="product_step", op="product", n=8, K=6656, M=202048, scales="f32", act="none", bias=False, residual=False),
        # a block's projection of a prompt, residual added in the epilogue; weights scaled by max / 448
        dict(name="product_prompt", op="product", n=4096, K=8192, M=8192, scales="f32", act="none", bias=True, residual=True),
        # a small batch at an odd vocabulary, the last block of K cut
        dict(name="product_odd", op="product", n=77, K=1008, M=50257, scales="e8m0", act="silu", bias=True, residual=False),
        # a training step of a wide projection with its bias
        dict(name="train_wide", op="train", n=4096, K=4096, M=16384, bias=True),
        # few tokens and sizes that are no multiple of anything
        dict(name="train_odd", op="train", n=517, K=1001, M=2051, bias=True),
        # the update of one small matrix: latency
        dict(name="ortho_small", op="ortho", batch=1, r=256, c=1024, dtype="bf16"),
        # four layers' matrices of one odd shape, taller than wide, 32-bit momentum
        dict(name="ortho_odd", op="ortho", batch=4, r=1003, c=517, dtype="f32"),
        # the update of a wide projection
        dict(name="ortho_wide", op="ortho", batch=1, r=4096, c=16384, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "train", "ortho"])
    if op == "quantize":
        K = _log(rng, 64, 16384)
        n = _log(rng, 1, min(65536, max(1, 16384 * 4096 // K)))
        blocks, transposed = rng.choice([("row", "none"), ("row", "row"), ("row", "tile"), ("tile", "none"), ("tile", "tile")])
        return dict(op=op, n=n, K=K, dtype=rng.choice(["bf16", "bf16", "f32"]), blocks=blocks, transposed=transposed)
    if op == "product":
        while True:
            K = max(16, _log(rng, 256, 8192) // 16 * 16)
            M = _log(rng, 256, 202048)
            n = _log(rng, 1, 4096)
            if n * K * M <= 4096 * 8192 * 8192 and K * M <= 6656 * 202048 // 2:
                break
        return dict(op=op, n=n, K=K, M=M, scales=rng.choice(["e8m0", "f32"]),
                    act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.7, residual=rng.random() < 0.5)
    if op == "train":
        while True:
            n, K, M = _log(rng, 1, 8192), _log(rng, 256, 8192), _log(rng, 256, 32768)
            if n * K * M <= 4096 * 4096 * 16384 and K * M <= 8192 * 16384:
                break
        if rng.random() < 0.6:
            n, K, M = -(-n // 8) * 8, K // 8 * 8, M // 8 * 8
        return dict(op=op, n=n, K=K, M=M, bias=rng.random() < 0.7)
    while True:
        r, c, batch = _log(rng, 32, 8192), _log(rng, 32, 16384), _log(rng, 1, 16)
        if batch * r * c * min(r, c) <= 4096 * 4096 * 16384:
            break
    return dict(op=op, batch=batch, r=r, c=c, dtype=rng.choice(["bf16", "f32"]))


# ---- inputs ----------------------------------------------------------------------------------

def _blocked(x, tile, power=True):
    """(values in e4m3, scales) of x in row blocks or tiles; without ``power``, scales of max|x| / 448."""
    n, K = x.shape
    high = BLOCK if tile else 1
    rows, cols = -(-n // high), -(-K // BLOCK)
    padded = torch.nn.functional.pad(x.float(), (0, cols * BLOCK - K, 0, rows * high - n))
    cut = padded.reshape(rows, high, cols, BLOCK)
    m = cut.abs().amax((1, 3))
    scale = m / 448.0
    if power:
        part, exponent = torch.frexp(m)   # 448 = 0.875 2^9
        scale = torch.ldexp(torch.ones_like(m), torch.where(part > 0.875, exponent - 8, exponent - 9))
    scale = torch.where(m > 0, scale.clamp_min(2.0 ** -126), torch.ones_like(m))
    q = (cut * (1.0 / scale)[:, None, :, None]).reshape(rows * high, cols * BLOCK)[:n, :K]
    return q.to(E4M3).contiguous(), scale.to(E8M0) if power else scale


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=F32):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=F32 if dtype == F32 else BF16) * sigma).to(dtype)

    s = dict(case)
    if case["op"] == "quantize":
        # a few channels are far larger than the others
        x = normal(case["n"], case["K"], dtype=TYPES[case["dtype"]])
        channels = torch.where(torch.rand(case["K"], generator=g, device=DEV) < 0.01, 30.0, 1.0)
        s["x"] = (x * channels).to(x.dtype)
    elif case["op"] == "product":
        n, K, M = case["n"], case["K"], case["M"]
        power = case["scales"] == "e8m0"
        s["x"], s["scale_x"] = _blocked(normal(n, K, dtype=BF16), False, power)
        s["weight"], s["scale_w"] = _blocked(normal(M, K, sigma=1.0 / math.sqrt(K), dtype=BF16), True, power)
        s["bias"] = normal(M, sigma=0.3, dtype=BF16) if case["bias"] else None
        s["residual"] = normal(n, M, dtype=BF16) if case["residual"] else None
    elif case["op"] == "train":
        n, K, M = case["n"], case["K"], case["M"]
        s["x"] = normal(n, K, dtype=BF16).requires_grad_()
        s["weight"] = normal(M, K, sigma=1.0 / math.sqrt(K), dtype=BF16).requires_grad_()
        s["bias"] = normal(M, sigma=0.3, dtype=BF16).requires_grad_() if case["bias"] else None
        s["grad_y"] = normal(n, M, sigma=1e-3, dtype=BF16)
    else:
        # a gradient averaged over steps: a few strong directions over noise
        batch, r, c = case["batch"], case["r"], case["c"]
        rank = max(1, min(r, c) // 16)
        strength = torch.arange(1, rank + 1, device=DEV, dtype=F32).rsqrt()
        signal = torch.matmul(normal(batch, r, rank) * strength, normal(batch, rank, c))
        G = (1e-3 * (signal + 0.3 * normal(batch, r, c))).to(TYPES[case["dtype"]])
        s["G"] = G if batch > 1 else G[0]
    return s


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    with torch.no_grad():
        return {"quantize": _quantize, "product": _product, "train": _train, "ortho": _ortho}[s["op"]](s)


def _own(s):
    import vocabulary_cross_entropy_row_amd as lce
    if s["op"] == "quantize":
        r = lce.lce_quantize_blocks(s["x"], blocks=s["blocks"],
                                    transposed=None if s["transposed"] == "none" else s["transposed"])
        return {"values": r.values, "scale": r.scale, "values_t": r.values_t, "scale_t": r.scale_t}
    if s["op"] == "product":
        return {"y": lce.lce_linear_blocks(s["x"], s["scale_x"], s["weight"], s["scale_w"], bias=s["bias"],
                                           activation=s["act"], residual=s["residual"]).out}
    if s["op"] == "train":
        names = [k for k in ("x", "weight", "bias") if s[k] is not None]
        y = lce.linear_blocks(s["x"], s["weight"], s["bias"])
        grads = torch.autograd.grad(y, [s[k] for k in names], s["grad_y"])
        return {"y": y, **{"grad_" + k: v for k, v in zip(names, grads)}}
    return {"X": lce.lce_orthogonalise(s["G"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)}


def _quantize(s):
    out = dict.fromkeys(("values", "scale", "values_t", "scale_t"))
    out["values"], out["scale"] = _blocked(s["x"], s["blocks"] == "tile")
    if s["transposed"] != "none":
        out["values_t"], out["scale_t"] = _blocked(s["x"].t(), s["transposed"] == "tile")
    return out


def _dense(q, scale):
    """The values that 8-bit values and their scales stand for."""
    n, K = q.shape
    full = scale.float().repeat_interleave(BLOCK, 1)[:, :K]
    if scale.shape[0] != n:
        full = full.repeat_interleave(BLOCK, 0)[:n]
    return q.float() * full


_A, _B = math.sqrt(2.0 / math.pi), 0.044715


def _act(kind, z):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_A * (z + _B * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _product(s):
    z = _dense(s["x"], s["scale_x"]) @ _dense(s["weight"], s["scale_w"]).t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(s["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(BF16)}


def _train(s):
    x, w, g = s["x"], s["weight"], s["grad_y"]
    wq = _dense(*_blocked(w, True))
    y = _dense(*_blocked(x, False)) @ wq.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out = {"y": y.to(BF16)}
    out["grad_x"] = (_dense(*_blocked(g, False)) @ wq).to(x.dtype)
    out["grad_weight"] = (_dense(*_blocked(g.t(), False)) @ _dense(*_blocked(x.t(), True)).t()).to(w.dtype)
    if s["bias"] is not None:
        out["grad_bias"] = g.float().sum(0).to(s["bias"].dtype)
    return out


def _ortho(s):
    G = s["G"].float()
    tall = G.shape[-2] > G.shape[-1]
    X = G.transpose(-2, -1).contiguous() if tall else G
    X = X / (X.double().square().sum((-2, -1), keepdim=True).sqrt().float() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        A = X @ X.transpose(-2, -1)
        X = a * X + (b * A + c * (A @ A)) @ X
    return {"X": (X.transpose(-2, -1) if tall else X).to(BF16).contiguous()}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"quantize": _exact_quantize, "product": _exact_product, "train": _exact_train,
                "ortho": _exact_ortho}[case["op"]](s)


def _exact_scale(x, tile):
    """The scale of every value of x, and of every block: the smallest power of two with m <= 448 scale."""
    x = x.double().abs()
    n, K = x.shape
    per = []
    for k in range(0, K, BLOCK):
        m = x[:, k:k + BLOCK].max(1).values
        if tile:
            m = torch.stack([part.max() for part in m.split(BLOCK)])
        per.append(m)
    m = torch.stack(per, 1)
    scale = torch.exp2(torch.ceil(torch.log2(m / 448.0)).clamp_min(-126.0))
    scale = torch.where(m > 448.0 * scale, 2.0 * scale, torch.where(m <= 224.0 * scale, 0.5 * scale, scale))   # next to a border
    scale = scale.clamp_min(2.0 ** -126)
    scale[m == 0] = 1.0
    row = torch.arange(n, device=x.device) // (BLOCK if tile else 1)
    return scale[row][:, torch.arange(K, device=x.device) // BLOCK], scale


def _exact_held(x, tile):
    """x / scale in e4m3 (a 3-bit fraction, the smallest step 2^-9, halves to even), in 64 bits."""
    each, scale = _exact_scale(x, tile)
    v = x.double() / each
    step = torch.exp2(torch.frexp(v)[1].clamp_min(-5).double() - 4.0)
    return torch.round(v / step) * step, each, scale


def _exact_quantize(s):
    out = dict.fromkeys(("values", "scale", "values_t", "scale_t"))
    out["values"], _, out["scale"] = _exact_held(s["x"], s["blocks"] == "tile")
    if s["transposed"] != "none":
        out["values_t"], _, out["scale_t"] = _exact_held(s["x"].t(), s["transposed"] == "tile")
    return out


def _exact_product(s):
    K, M = s["x"].shape[1], s["weight"].shape[0]
    block = torch.arange(K, device=DEV) // BLOCK
    x = s["x"].double() * s["scale_x"].double()[:, block]
    parts = []
    for i in range(0, M, 32768):   # column blocks: 64 bits of a wide head are large
        w = s["weight"][i:i + 32768].double()
        w *= s["scale_w"].double()[(i + torch.arange(w.shape[0], device=DEV)) // BLOCK][:, block]
        z = torch.mm(x, w.t())
        if s["bias"] is not None:
            z += s["bias"][i:i + 32768].double()
        inner = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z.pow(3))
        parts.append({"none": z, "relu": z.clamp_min(0.0), "gelu": z * 0.5 * torch.erfc(-z / math.sqrt(2.0)),
                      "gelu_tanh": z * torch.sigmoid(2.0 * inner), "silu": z * torch.sigmoid(z)}[s["act"]])
    y = torch.cat(parts, 1)
    return {"y": y if s["residual"] is None else y + s["residual"].double()}


def _exact_train(s):
    def stands(x, tile):
        v, each, _ = _exact_held(x, tile)
        return v * each

    x, w, g = s["x"].detach(), s["weight"].detach(), s["grad_y"]
    wq = stands(w, True)
    y = torch.mm(stands(x, False), wq.t().contiguous())
    out = {"y": y if s["bias"] is None else y + s["bias"].detach().double()}
    out["grad_x"] = torch.mm(stands(g, False), wq)
    out["grad_weight"] = torch.mm(stands(g.t(), False), stands(x.t(), True).t().contiguous())
    if s["bias"] is not None:
        out["grad_bias"] = g.double().sum(0)
    return out


def _exact_ortho(s):
    parts = []
    a, b, c = COEFFICIENTS
    for G in s["G"].double().reshape(-1, *s["G"].shape[-2:]):
        wide = G.shape[1] >= G.shape[0]
        Y = (G.t() if wide else G).contiguous()   # no fewer rows than columns
        Y = Y / (Y.norm() + EPS)
        unit = torch.eye(Y.shape[1], dtype=torch.float64, device=Y.device)
        for _ in range(STEPS):
            S = torch.mm(Y.t().contiguous(), Y)
            Y = torch.mm(Y, a * unit + torch.mm(S, b * unit + c * S))
        parts.append(Y.t() if wide else Y)
    return {"X": torch.stack(parts).reshape(s["G"].shape)}


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "f32": 4}

    def scales(n, K, kind):
        return -(-K // BLOCK) * (n if kind == "row" else -(-n // BLOCK))

    if case["op"] == "quantize":
        n, K = case["n"], case["K"]
        moved = n * K * size[case["dtype"]] + n * K + scales(n, K, case["blocks"])
        if case["transposed"] != "none":
            moved += n * K + scales(K, n, case["transposed"])
        return {"bytes": moved, "flops": (2 if case["transposed"] == "none" else 4) * n * K}
    if case["op"] == "product":
        n, K, M = case["n"], case["K"], case["M"]
        moved = (n + M) * K + (scales(n, K, "row") + scales(M, K, "tile")) * (1 if case["scales"] == "e8m0" else 4)
        moved += 2 * n * M * (1 + int(case["residual"])) + 2 * M * int(case["bias"])
        return {"bytes": moved, "flops": 2 * n * K * M}
    if case["op"] == "train":   # x, weight and grad_y read; y and the gradients written
        n, K, M = case["n"], case["K"], case["M"]
        return {"bytes": 4 * (n * K + M * K + n * M + M * int(case["bias"])), "flops": 6 * n * K * M}
    r, c = sorted((case["r"], case["c"]))   # A and A A are symmetric: half of each
    return {"bytes": case["batch"] * r * c * (size[case["dtype"]] + 2), "flops": case["batch"] * STEPS * (3 * r * r * c + r ** 3)}
