"""Measured cases of the operators around the vocabulary cross-entropy: the final norm, the head's
matrix product and the rules on its logits.

``listed()`` gives the cases, ``prepare`` their inputs, ``run`` one pass: in plain torch operations in
32 bits, or, with ``own`` set, through the library's entry points.  ``exact`` gives the same outputs
from the definitions in 64 bits.

  norm     s = x + residual (rounded to the stream's type, which is what the next layer reads);
           y = s / sqrt(mean(s^2) + eps) * weight.  Forward; forward with backward; forward with y in
           8 bits and one scale per row (scale = max|y| / 448, held values y / scale).
  linear   y = act(x weight^T + bias) + residual, for bf16 operands or 8-bit operands with one scale
           per row of x and of weight.  Forward; forward with backward.
  logits   z = softcap(x); tokens already seen: z / r if z > 0 else z r; minus frequency * count and
           presence for those generated; plus the last bias entry of the token; divided by the
           temperature; disallowed tokens set to the mask's value.
"""
import math

import torch

own = False
DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = {"bf16": BF16, "f32": F32, "e4m3": E4M3}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # the final norm of sixteen sequences that generate one token each: latency
        dict(name="norm_step", op="norm", mode="fwd", n=16, H=6656, dtype="bf16", residual=True),
        # a training step's final norm, 8192 tokens of the 6656-wide model
        dict(name="norm_train", op="norm", mode="train", n=8192, H=6656, dtype="bf16", residual=True),
        # 32-bit training at a width that is no multiple of a vector
        dict(name="norm_train_odd", op="norm", mode="train", n=2051, H=4099, dtype="f32", residual=False),
        # a prompt's norm that feeds an 8-bit product
        dict(name="norm_8bit", op="norm", mode="8bit", n=4096, H=8192, dtype="bf16", residual=True),
        # the head of eight generating sequences: the weight is read once
        dict(name="linear_step", op="linear", mode="fwd", n=8, K=6656, M=202048, dtype="bf16", out="bf16", act="none",
             bias=False, residual=False),
        # logits of a scored prompt chunk of 1024 tokens
        dict(name="linear_prompt", op="linear", mode="fwd", n=1024, K=6656, M=202048, dtype="bf16", out="bf16",
             act="none", bias=True, residual=False),
        # a block's projection in 8 bits, residual added in the epilogue
        dict(name="linear_8bit", op="linear", mode="fwd", n=4096, K=8192, M=8192, dtype="e4m3", out="bf16", act="none",
             bias=True, residual=True),
        # a training step of an activated projection with its bias and residual
        dict(name="linear_train", op="linear", mode="train", n=4096, K=4096, M=16384, dtype="bf16", out="bf16",
             act="gelu", bias=True, residual=True),
        # a small batch at an odd vocabulary, 32-bit logits
        dict(name="linear_odd", op="linear", mode="fwd", n=77, K=1000, M=50257, dtype="bf16", out="f32", act="silu",
             bias=True, residual=False),
        # one sequence's logits with every rule on: latency
        dict(name="logits_step", op="logits", n=1, V=32768, dtype="f32", L=57, B=8, mask=True, softcap=0.0),
        # a serving batch at the 128K vocabulary
        dict(name="logits_batch", op="logits", n=256, V=131072, dtype="bf16", L=2048, B=64, mask=True, softcap=30.0),
        # long generations at an odd vocabulary
        dict(name="logits_long", op="logits", n=33, V=50257, dtype="bf16", L=16384, B=0, mask=False, softcap=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "logits"])
    if op == "norm":
        mode = rng.choice(["fwd", "train", "8bit"])
        H = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            H = max(64, H // 8 * 8)
        n = _log(rng, 1, min(65536, max(1, 8192 * 6656 // H)))
        return dict(op=op, mode=mode, n=n, H=H, dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.6)
    if op == "linear":
        mode = rng.choice(["fwd", "fwd", "train"])
        dtype = "bf16" if mode == "train" else rng.choice(["bf16", "e4m3"])
        unit = 16 if dtype == "e4m3" else 8
        while True:
            K = max(unit, _log(rng, 256, 8192) // unit * unit)
            M = _log(rng, 256, 202048)
            M = max(8, M // 8 * 8) if mode == "train" or rng.random() < 0.6 else M
            n = _log(rng, 1, 4096)
            if n * K * M * (3 if mode == "train" else 1) <= 1024 * 6656 * 202048 and K * M <= 6656 * 202048 // 2:
                break
        return dict(op=op, mode=mode, n=n, K=K, M=M, dtype=dtype,
                    out="bf16" if mode == "train" or dtype == "e4m3" else rng.choice(["bf16", "f32"]),
                    act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.7,
                    residual=rng.random() < 0.5)
    V = _log(rng, 4096, 202048)
    if rng.random() < 0.6:
        V = V // 8 * 8
    n = _log(rng, 1, max(1, min(512, 256 * 131072 // V)))
    return dict(op=op, n=n, V=V, dtype=rng.choice(["bf16", "f32"]), L=_log(rng, 1, 8192), B=rng.choice([0, 5, 64, 300]),
                mask=rng.random() < 0.6, softcap=rng.choice([0.0, 0.0, 30.0]))


# ---- inputs ----------------------------------------------------------------------------------

def _quantised(t):
    """t in 8 bits with one scale per row."""
    scale = t.abs().amax(1).clamp_min(1e-12) / 448.0
    return (t / scale[:, None]).to(E4M3), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=F32):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=F32 if dtype == F32 else BF16) * sigma).to(dtype)

    def integers(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=DEV)

    s = dict(case)
    if case["op"] == "norm":
        dt, n, H = TYPES[case["dtype"]], case["n"], case["H"]
        s["x"] = normal(n, H, sigma=2.0, dtype=dt)
        s["residual"] = normal(n, H, sigma=3.0, dtype=dt) if case["residual"] else None
        s["weight"] = (1.0 + normal(H, sigma=0.2)).to(dt)
        s["eps"] = 1e-6
        if case["mode"] == "train":
            s["grad_y"] = normal(n, H, sigma=0.1, dtype=dt)
            s["grad_sum"] = normal(n, H, sigma=0.1, dtype=dt) if case["residual"] else None
            for k in ("x", "residual", "weight"):
                if s[k] is not None:
                    s[k].requires_grad_()
    elif case["op"] == "linear":
        n, K, M, dt, ot = case["n"], case["K"], case["M"], TYPES[case["dtype"]], TYPES[case["out"]]
        s["scale_x"] = s["scale_w"] = None
        if dt == E4M3:
            s["x"], s["scale_x"] = _quantised(normal(n, K))
            s["weight"], s["scale_w"] = _quantised(normal(M, K, sigma=1.0 / math.sqrt(K)))
        else:
            s["x"] = normal(n, K, dtype=dt)
            s["weight"] = normal(M, K, sigma=1.0 / math.sqrt(K), dtype=dt)
        s["bias"] = normal(M, sigma=0.3, dtype=BF16) if case["bias"] else None
        s["residual"] = normal(n, M, dtype=ot) if case["residual"] else None
        if case["mode"] == "train":
            s["grad_y"] = normal(n, M, sigma=0.1, dtype=ot)
            for k in ("x", "weight", "bias", "residual"):
                if s[k] is not None:
                    s[k].requires_grad_()
    else:
        n, V, L, B = case["n"], case["V"], case["L"], case["B"]
        s["x"] = normal(n, V, sigma=4.0, dtype=TYPES[case["dtype"]])
        # text repeats itself: half of the tokens come from a few hundred
        often = integers(0, V, n, min(V, 200))
        some = torch.gather(often, 1, integers(0, often.shape[1], n, L))
        s["history"] = torch.where(integers(0, 2, n, L) == 0, some, integers(0, V, n, L))
        s["history_lens"] = integers(L // 2, L + 1, n)
        s["prompt_lens"] = (s["history_lens"].double() * 0.6).long()
        s["repetition"] = 1.0 + 0.5 * torch.rand(n, generator=g, device=DEV)
        s["presence"] = 0.5 * torch.rand(n, generator=g, device=DEV)
        s["frequency"] = 0.3 * torch.rand(n, generator=g, device=DEV)
        s["temperature"] = 0.5 + torch.rand(n, generator=g, device=DEV)
        s["bias_ids"] = integers(0, V, n, B) if B else None
        s["bias_values"] = normal(n, B, sigma=3.0) if B else None
        s["allowed"] = s["mask_rows"] = None
        if case["mask"]:   # four states of a grammar; one bit a token, 32 to a word
            words = -(-V // 32)
            s["allowed"] = (integers(0, 1 << 32, 4, words) - (1 << 31)).to(torch.int32)
            s["mask_rows"] = integers(-1, 4, n)   # -1: no rule for this sequence
        s["out"] = torch.empty_like(s["x"])
    return s


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    with torch.no_grad():
        return {"norm": _norm, "linear": _linear, "logits": _logits}[s["op"]](s)


def _own(s):
    import vocabulary_cross_entropy_row_amd as lce
    if s["op"] == "norm":
        if s["mode"] == "train":
            leaves = [s[k] for k in ("x", "residual", "weight") if s[k] is not None]
            if s["residual"] is None:
                y = lce.rms_norm(s["x"], s["weight"], eps=s["eps"])
                grads = torch.autograd.grad(y, leaves, s["grad_y"])
                return {"y": y, "grad_x": grads[0], "grad_weight": grads[1]}
            y, total = lce.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=s["eps"])
            grads = torch.autograd.grad((y, total), leaves, (s["grad_y"], s["grad_sum"]))
            return {"y": y, "sum": total, "grad_x": grads[0], "grad_residual": grads[1], "grad_weight": grads[2]}
        r = lce.lce_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=s["eps"],
                             out_dtype=E4M3 if s["mode"] == "8bit" else None)
        return {"y": r.y, "sum": r.sum, "scale": r.scale}
    if s["op"] == "linear":
        if s["mode"] == "train":
            names = [k for k in ("x", "weight", "bias", "residual") if s[k] is not None]
            y = lce.linear(s["x"], s["weight"], s["bias"], activation=s["act"], residual=s["residual"])
            grads = torch.autograd.grad(y, [s[k] for k in names], s["grad_y"])
            return {"y": y, **{"grad_" + k: v for k, v in zip(names, grads)}}
        r = lce.lce_linear(s["x"], s["weight"], bias=s["bias"], activation=s["act"], residual=s["residual"],
                           scale_x=s["scale_x"], scale_w=s["scale_w"], out_dtype=TYPES[s["out"]])
        return {"y": r.out}
    return {"y": lce.lce_logits_process(
        s["x"], history=s["history"], history_lens=s["history_lens"], prompt_lens=s["prompt_lens"],
        repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"],
        bias_values=s["bias_values"], temperature=s["temperature"], allowed=s["allowed"], mask_rows=s["mask_rows"],
        softcap=s["softcap"], out=s["out"])}


def _norm(s):
    x, w = s["x"], s["weight"]
    total = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    h, wf = total.float(), w.float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"])
    y = h * r * wf
    if s["mode"] == "8bit":
        scale = y.abs().amax(1) / 448.0
        q = (y / scale[:, None]).clamp(-448.0, 448.0).to(E4M3)
        return {"y": q, "sum": None if s["residual"] is None else total, "scale": scale}
    out = {"y": y.to(x.dtype)}
    if s["residual"] is not None:
        out["sum"] = total
    if s["mode"] == "train":
        gy = s["grad_y"].float()
        a = gy * wf
        gx = r * (a - h * (r * r) * (a * h).mean(1, keepdim=True))
        if s["grad_sum"] is not None:
            gx = gx + s["grad_sum"].float()
        gx = gx.to(x.dtype)
        out["grad_x"] = gx
        if s["residual"] is not None:
            out["grad_residual"] = gx
        out["grad_weight"] = (gy * h * r).sum(0).to(w.dtype)
    return out


_A, _B = math.sqrt(2.0 / math.pi), 0.044715


def _act(kind, z):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_A * (z + _B * z * z * z)))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_slope(kind, z):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        t = torch.tanh(_A * (z + _B * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _A * (1.0 + 3.0 * _B * z * z)
    if kind == "silu":
        e = torch.sigmoid(z)
        return e * (1.0 + z * (1.0 - e))
    return torch.ones_like(z)


def _linear(s):
    xf, wf = s["x"].float(), s["weight"].float()
    z = xf @ wf.t()
    if s["scale_x"] is not None:
        z = z * s["scale_x"][:, None] * s["scale_w"]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(s["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(TYPES[s["out"]])}
    if s["mode"] == "train":
        dz = s["grad_y"].float() * _act_slope(s["act"], z)
        out["grad_x"] = (dz @ wf).to(s["x"].dtype)
        out["grad_weight"] = (dz.t() @ xf).to(s["weight"].dtype)
        if s["bias"] is not None:
            out["grad_bias"] = dz.sum(0).to(s["bias"].dtype)
        if s["residual"] is not None:
            out["grad_residual"] = s["grad_y"]
    return out


def _logits(s):
    x = s["x"]
    n, V = x.shape
    z = x.float()
    if s["softcap"] > 0:
        z = s["softcap"] * torch.tanh(z / s["softcap"])
    at = torch.arange(s["history"].shape[1], device=x.device)
    there = at < s["history_lens"][:, None]
    made = there & (at >= s["prompt_lens"][:, None])
    zeros = torch.zeros(n, V, device=x.device)
    seen = zeros.scatter_add(1, s["history"], there.float()) > 0
    count = zeros.scatter_add(1, s["history"], made.float())
    r = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
    z = z - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias_ids"] is not None:   # the last entry of a token counts
        entry = torch.arange(1, s["bias_ids"].shape[1] + 1, device=x.device).expand_as(s["bias_ids"])
        last = torch.zeros(n, V, dtype=torch.int64, device=x.device).scatter_reduce(1, s["bias_ids"], entry, "amax")
        z = z + torch.where(last > 0, torch.gather(s["bias_values"], 1, (last - 1).clamp_min(0)), torch.zeros_like(z))
    z = z / s["temperature"][:, None]
    if s["allowed"] is not None:
        column = torch.arange(V, device=x.device)
        bits = (s["allowed"][:, column // 32] >> (column % 32)) & 1
        free = (s["mask_rows"] < 0)[:, None] | (bits[s["mask_rows"].clamp_min(0)] != 0)
        z = torch.where(free, z, torch.full_like(z, -math.inf))
    return {"y": z.to(x.dtype)}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"norm": _exact_norm, "linear": _exact_linear, "logits": _exact_logits}[case["op"]](s)


def _exact_norm(s):
    h = s["x"].double()
    if s["residual"] is not None:   # the sum is held in the stream's type, and the norm is taken of that
        h = (h + s["residual"].double()).to(s["x"].dtype).double()
    w = s["weight"].double()
    rms = (h.square().sum(1, keepdim=True) / h.shape[1] + s["eps"]).sqrt()
    unit = h / rms
    y = unit * w
    total = None if s["residual"] is None else s["x"].double() + s["residual"].double()
    if s["mode"] == "8bit":
        scale = y.abs().max(1).values / 448.0
        return {"y": y / scale[:, None], "sum": total, "scale": scale}
    out = {"y": y}
    if total is not None:
        out["sum"] = total
    if s["mode"] == "train":
        gy = s["grad_y"].double()
        # d unit / d h is (1 - unit unit^T / H) / rms
        a = gy * w
        gx = (a - unit * ((a * unit).sum(1, keepdim=True) / h.shape[1])) / rms
        if s["grad_sum"] is not None:
            gx = gx + s["grad_sum"].double()
        out["grad_x"] = gx
        if total is not None:
            out["grad_residual"] = gx
        out["grad_weight"] = (gy * unit).sum(0)
    return out


def _exact_linear(s):
    x, w = s["x"].double(), s["weight"].double()
    if s["scale_x"] is not None:
        x, w = x * s["scale_x"].double()[:, None], w * s["scale_w"].double()[:, None]
    b = 0.0 if s["bias"] is None else s["bias"].double()
    c = 0.0 if s["residual"] is None else s["residual"].double()
    train = s["mode"] == "train"
    parts, slopes = [], []
    for i in range(0, w.shape[0], 32768):   # column blocks: 64 bits of a wide head are large
        z = torch.mm(x, w[i:i + 32768].t())
        z += b[i:i + 32768] if s["bias"] is not None else 0.0
        normal = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        k = math.sqrt(2.0 / math.pi)
        inner = k * (z + 0.044715 * z.pow(3))
        gate = 1.0 / (1.0 + torch.exp(-2.0 * inner))   # (1 + tanh) / 2
        sig = 1.0 / (1.0 + torch.exp(-z))
        parts.append({"none": z, "relu": z.clamp_min(0.0), "gelu": z * normal, "gelu_tanh": z * gate,
                      "silu": z * sig}[s["act"]])
        if train:
            slopes.append({"none": torch.ones_like(z), "relu": (z > 0).double(),
                           "gelu": normal + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi),
                           "gelu_tanh": gate + z * 2.0 * gate * (1.0 - gate) * k * (1.0 + 3 * 0.044715 * z * z),
                           "silu": sig + z * sig * (1.0 - sig)}[s["act"]])
    out = {"y": torch.cat(parts, 1) + c}
    if train:
        dz = s["grad_y"].double() * torch.cat(slopes, 1)
        out["grad_x"] = torch.mm(dz, w)
        out["grad_weight"] = torch.mm(dz.t().contiguous(), x)
        if s["bias"] is not None:
            out["grad_bias"] = dz.sum(0)
        if s["residual"] is not None:
            out["grad_residual"] = s["grad_y"].double()
    return out


def _exact_logits(s):
    n, V = s["x"].shape
    L = s["history"].shape[1]
    z = s["x"].double()
    if s["softcap"] > 0:
        u = z / s["softcap"]
        z = s["softcap"] * (1.0 - 2.0 / (1.0 + torch.exp(2.0 * u)))
    row = torch.arange(n, device=z.device)[:, None].expand(n, L)
    at = torch.arange(L, device=z.device)[None].expand(n, L)
    inside, prompt = at < s["history_lens"][:, None], at < s["prompt_lens"][:, None]
    key = row * V + s["history"]
    every = torch.bincount(key[inside], minlength=n * V).reshape(n, V)
    made = torch.bincount(key[inside & ~prompt], minlength=n * V).reshape(n, V).double()
    r = s["repetition"].double()[:, None].expand(n, V)
    factor = torch.where(z > 0, 1.0 / r, r)
    z = torch.where(every > 0, z * factor, z)
    z = z - made * s["frequency"].double()[:, None] - made.clamp_max(1.0) * s["presence"].double()[:, None]
    if s["bias_ids"] is not None:
        ids = s["bias_ids"]
        order = torch.arange(ids.shape[1], device=z.device)
        again = ((ids[:, :, None] == ids[:, None, :]) & (order[None, :] > order[:, None])).any(2)
        rows, cols = torch.nonzero(~again, as_tuple=True)
        z[rows, ids[rows, cols]] += s["bias_values"].double()[rows, cols]
    z = z / s["temperature"].double()[:, None]
    if s["allowed"] is not None:
        words = s["allowed"].long() & 0xFFFFFFFF
        table = torch.stack([(words >> k) & 1 for k in range(32)], 2).reshape(words.shape[0], -1)[:, :V]
        for state in range(words.shape[0]):
            z[(s["mask_rows"] == state)[:, None] & (table[state] == 0)[None]] = -math.inf
    return {"y": z}


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    if case["op"] == "norm":
        n, H, e, r = case["n"], case["H"], size[case["dtype"]], int(case["residual"])
        moved = n * H * e * (1 + 2 * r) + H * e          # x, residual, sum, weight
        if case["mode"] == "8bit":
            return {"bytes": moved + n * H + 4 * n, "flops": 8 * n * H}
        moved += n * H * e
        if case["mode"] == "train":   # grad_y, grad_sum and the stream read, grad_x and grad_weight written
            moved += n * H * e * (3 + r) + 2 * H * e
        return {"bytes": moved, "flops": (18 if case["mode"] == "train" else 5) * n * H}
    if case["op"] == "linear":
        n, K, M, e, o = case["n"], case["K"], case["M"], size[case["dtype"]], size[case["out"]]
        moved = (n * K + M * K) * e + n * M * o * (1 + int(case["residual"])) + 2 * M * int(case["bias"])
        if case["dtype"] == "e4m3":
            moved += 4 * (n + M)
        if case["mode"] == "train":   # grad_y and the operands read, the gradients written
            moved += n * M * o + 2 * (n * K + M * K) * e
            moved += 2 * M * int(case["bias"])
        return {"bytes": moved, "flops": 2 * n * K * M * (3 if case["mode"] == "train" else 1)}
    n, V, e = case["n"], case["V"], size[case["dtype"]]
    moved = 2 * n * V * e + 8 * n * case["L"] + 12 * n * case["B"] + (4 * -(-V // 32) * 4 if case["mask"] else 0)
    return {"bytes": moved, "flops": (12 if case["softcap"] else 4) * n * V}
