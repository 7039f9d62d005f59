"""The operators around the cross-entropy run together, as a program has them: a serving step from the
residual stream to the next token and its log-probability, and a training step from the stream through
the norm and a projection to the fused linear loss."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _rand(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s, t=F32: torch.randn(*s, generator=g, device=DEV).to(t)


@pytest.mark.parametrize("eight_bits", [False, True])
@pytest.mark.parametrize("n,H,V", [(1, 512, 4099), (7, 1024, 50257), (40, 768, 8192)])
def test_serving_step(n, H, V, eight_bits):
    r = _rand(n + H)
    x, res, w = r(n, H, t=BF16), r(n, H, t=BF16), 1 + 0.1 * r(H)
    head = r(V, H) * 4 / math.sqrt(H)
    s64 = (x.float() + res.float()).to(BF16).double()
    y64 = s64 / (s64.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    if eight_bits:
        scale_w = head.abs().amax(1) / 448
        head8 = (head / scale_w[:, None]).to(E4M3)
        a = lce.lce_rms_norm(x, w, residual=res, out_dtype=E4M3)
        logits = lce.lce_linear(a.y, head8, scale_x=a.scale, scale_w=scale_w).out
        z64 = y64 @ (head8.double() * scale_w.double()[:, None]).t()
        step = 2.0 ** -4   # of each e4m3 value of x
    else:
        head = head.to(BF16)
        a = lce.lce_rms_norm(x, w, residual=res)
        logits = lce.lce_linear(a.y, head, out_dtype=F32).out
        z64 = y64 @ head.double().t()
        step = torch.finfo(BF16).eps / 2
    assert torch.equal(a.sum.double(), s64)
    # roundings of the row's values are independent: the logits' error is at most a step of the whole
    assert float((logits.double() - z64).norm() / z64.norm()) <= step
    history = torch.randint(0, V, (n, 33), device=DEV)
    allowed = torch.full((1, (V + 31) // 32), 0x55555555, dtype=torch.int32, device=DEV)
    before = logits.double().clone()
    z = lce.lce_logits_process(logits, history=history, repetition=torch.full((n,), 1.3, device=DEV),
                               allowed=allowed, mask_rows=torch.zeros(n, dtype=torch.int64, device=DEV), mask_value=-1e4)
    for i in range(n):
        h = history[i].unique()
        v = before[i, h]
        before[i, h] = torch.where(v > 0, v / 1.3, v * 1.3)
    before[:, 1::2] = float(torch.tensor(-1e4, dtype=logits.dtype))   # as the logits hold it
    token, _ = lce.lce_ce_argmax(z)
    assert bool((token % 2 == 0).all())
    assert torch.equal(token, z.float().argmax(1))
    if V % 8 == 0:   # the statistics take whole 16 bytes of logits
        rows = lce.lce_ce_combine(lce.lce_ce_stats(z, token), token, V)
        want = torch.log_softmax(z.double(), 1).gather(1, token[:, None])[:, 0]
        assert torch.allclose(rows.logprob.double(), want, atol=1e-4)
    assert float((z.double() - before).abs().max()) <= 1e-2 * float(before[:, ::2].abs().max())


def test_serving_step_captured():
    n, H, V = 5, 512, 4096
    r = _rand(1)
    x, res, w, head = r(n, H, t=BF16), r(n, H, t=BF16), r(H), (r(V, H) / 8).to(BF16)
    bias_ids = torch.randint(0, V, (n, 9), device=DEV)
    bias = torch.randn(n, 9, device=DEV)

    def step():
        a = lce.lce_rms_norm(x, w, residual=res)
        z = lce.lce_linear(a.y, head, out_dtype=F32).out
        lce.lce_logits_process(z, bias_ids=bias_ids, bias_values=bias, softcap=30.0)
        return a.sum, z, lce.lce_ce_argmax(z)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(4):
        x.copy_(torch.randn(n, H, device=DEV))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_training_step():
    """norm -> activated projection with residual -> norm -> fused linear cross-entropy: every gradient
    against the same step in 64 bits.  Four bf16 tensors lie between the loss and the first leaf, each
    rounded by at most 2^-8 of itself, forward and backward: 2-norms within 8 half steps."""
    n, H, V = 96, 256, 1024
    r = _rand(4)
    leaves = dict(x=r(n, H, t=BF16), res=r(n, H, t=BF16), w1=1 + 0.1 * r(H), proj=(r(H, H) / 16).to(BF16), b=0.1 * r(H),
                  w2=(1 + 0.1 * r(H)).to(BF16), head=(r(V, H) / 8).to(BF16))
    for t in leaves.values():
        t.requires_grad_()
    y = torch.randint(0, V, (n,), device=DEV)
    y[::7] = -100
    p = leaves
    a, stream = lce.rms_norm(p["x"], p["w1"], residual=p["res"])
    h = lce.linear(a, p["proj"], p["b"], activation="gelu", residual=stream)
    loss = lce.linear_cross_entropy(lce.rms_norm(h, p["w2"]), p["head"], y)[0]
    got = torch.autograd.grad(loss, list(p.values()))

    d = {k: t.detach().double().requires_grad_() for k, t in leaves.items()}

    def norm(s, w):
        return s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * w

    s = d["x"] + d["res"]
    z = norm(s, d["w1"]) @ d["proj"].t() + d["b"]
    h64 = torch.nn.functional.gelu(z) + s
    loss64 = torch.nn.functional.cross_entropy(norm(h64, d["w2"]) @ d["head"].t(), y)
    want = torch.autograd.grad(loss64, list(d.values()))
    assert abs(float(loss) - float(loss64)) <= 2.0 ** -7 * float(loss64)
    for k, g, e in zip(leaves, got, want):
        assert g.dtype == leaves[k].dtype
        rel = float((g.double() - e).norm() / e.norm())
        assert rel <= 8 * 2.0 ** -8, (k, rel)


def test_training_step_captured():
    """norm -> activated projection with residual and their backward, captured through autograd: every
    replay gives the eager step's bits.  The leaves have no eager graph when the capture is made: the
    warm-up and the comparison take clones."""
    n, H = 130, 264
    r = _rand(9)
    static = [r(n, H, t=BF16), r(n, H, t=BF16), 1 + 0.1 * r(H), (r(H, H) / 16).to(BF16), 0.1 * r(H)]
    g = r(n, H, t=BF16)

    def step(leaves):
        x, res, w1, proj, b = leaves
        a, stream = lce.rms_norm(x, w1, residual=res)
        out = lce.linear(a, proj, b, activation="gelu", residual=stream)
        return [out.detach(), *torch.autograd.grad(out, leaves, g)]

    def eager():
        return step([t.detach().clone().requires_grad_() for t in static])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            eager()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step([t.requires_grad_() for t in static])
    for k in range(4):
        with torch.no_grad():
            static[0].copy_(r(n, H))
            g.copy_(r(n, H) * (k + 1))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager()))
