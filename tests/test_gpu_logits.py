"""The rules on logits on the GPU against a plain loop in 64 bits.

Tolerance: half a step of the logits' type for the one rounding, and fp32 arithmetic before it: at
most 16 operations, each off by 2^-24 of the magnitudes that enter (the hardware exponential and
reciprocal of the softcap by 2^-22 of the cap's slope region, covered by the same 16)."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
INF = math.inf


def _plain(x, r):
    """The rules in 64 bits, row by row: (out, bound on the fp32 arithmetic's error)."""
    n, V = x.shape
    z = x.double().cpu().clone()
    get = lambda k, i, d: d if r.get(k) is None else float(r[k][i])  # noqa: E731
    T = r.get("softcap", 0.0)
    size = z.abs()
    if T > 0:
        z = T * torch.tanh(z / T)
    for i in range(n):
        seen, made = set(), {}
        if r.get("history") is not None:
            h = r["history"][i].tolist()
            m = len(h) if r.get("history_lens") is None else max(0, min(len(h), int(r["history_lens"][i])))
            p = 0 if r.get("prompt_lens") is None else int(r["prompt_lens"][i])
            for k, t in enumerate(h[:m]):
                if 0 <= t < V:
                    seen.add(t)
                    if k >= p:
                        made[t] = made.get(t, 0) + 1
        rep = get("repetition", i, 1.0)
        for t in seen:
            z[i, t] = z[i, t] / rep if z[i, t] > 0 else z[i, t] * rep
            size[i, t] *= max(rep, 1 / rep)
        for t, c in made.items():
            f, q = get("frequency", i, 0.0), get("presence", i, 0.0)
            z[i, t] -= f * c + q
            size[i, t] += abs(f * c) + abs(q)
        if r.get("bias_ids") is not None:
            last = {t: v for t, v in zip(r["bias_ids"][i].tolist(), r["bias_values"][i].tolist()) if 0 <= t < V}
            for t, v in last.items():
                z[i, t] += v
                size[i, t] += abs(v)
        t = get("temperature", i, 0.0)
        if t > 0:
            z[i] /= t
            size[i] /= t
        if r.get("allowed") is not None:
            m = i if r.get("mask_rows") is None else int(r["mask_rows"][i])
            if 0 <= m < r["allowed"].shape[0]:
                words = r["allowed"][m].long().cpu() & 0xFFFFFFFF
                bits = ((words[:, None] >> torch.arange(32)) & 1).reshape(-1)[:V]
                z[i, bits == 0] = r.get("mask_value", -INF)
                size[i, bits == 0] = 0
    return z, size


def _check(got, x, rules):
    want, size = _plain(x, rules)
    got = got.double().cpu()
    dt = x.dtype
    flat = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~flat & ~torch.isnan(want)], want[~flat & ~torch.isnan(want)])
    tol = torch.finfo(dt).eps / 2 * want.abs() + 16 * 2.0 ** -24 * size + torch.finfo(dt).tiny
    off = ((got - want).abs() - tol)[flat]
    assert off.numel() == 0 or float(off.max()) <= 0, f"{int((off > 0).sum())} outside, worst by {float(off.max()):.3g}"


def _rules(n, V, L, B, seed, *, ids=torch.int64, masks=3, softcap=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV)  # noqa: E731
    rf = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    r = dict(softcap=softcap)
    if L:
        hist = ri(-2, V + 2, n, L)                 # ids outside [0, V) are padding
        hist[:, ::3] = hist[:, :1].clone()                 # and some tokens come often
        lens = ri(0, L + 1, n)
        lens[-1], lens[0] = 0, L
        r.update(history=hist.to(ids), history_lens=lens, prompt_lens=ri(0, L + 3, n), repetition=0.5 + rf(n) * 1.5,
                 presence=rf(n) - 0.5, frequency=rf(n) - 0.3)
    if B:
        bids = ri(-1, V + 1, n, B)
        if B > 2:
            bids[:, -1] = bids[:, 0].clone()             # the same token twice: the last entry counts
        r.update(bias_ids=bids.to(ids), bias_values=rf(n, B) * 20 - 10)
    if masks:
        words = (V + 31) // 32
        allowed = (ri(0, 1 << 32, masks, words) - (1 << 31)).to(torch.int32)
        allowed[masks - 1] = 0                     # a mask that allows nothing
        rows = ri(-1, masks + 1, n)                # -1 and `masks`: no mask
        r.update(allowed=allowed, mask_rows=rows)
    t = 0.3 + rf(n)
    t[0] = 0.0                                     # left as it is
    r["temperature"] = t
    return r


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,V,L,B", [(1, 1, 1, 1), (2, 7, 5, 3), (3, 33, 0, 2), (9, 1000, 40, 0), (2, 4096, 300, 9),
                                     (5, 8192, 1, 5), (4, 8193, 700, 64), (11, 50257, 97, 7), (3, 40000, 5000, 300)])
def test_all_rules(n, V, L, B, dtype):
    for k, (ids, softcap, masks) in enumerate([(torch.int64, 0.0, 3), (torch.int32, 20.0, 0), (torch.int64, 5.0, 2)]):
        g = torch.Generator(device=DEV).manual_seed(n * V + k)
        x = (torch.randn(n, V, generator=g, device=DEV) * 6).to(dtype)
        r = _rules(n, V, L, B, n + V + k, ids=ids, masks=masks, softcap=softcap)
        out = torch.empty_like(x)
        before = x.clone()
        assert lce.lce_logits_process(x, out=out, **r) is out
        assert torch.equal(x, before)
        _check(out, x, r)
        assert lce.lce_logits_process(x, **r) is x        # in place: the same bits
        assert torch.equal(x.view(torch.uint8), out.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V,ld,first,out_first", [(100, 131, 1, 1), (100, 131, 3, 0), (8195, 8200, 5, 5),
                                                  (16384, 16384, 0, 0), (4096, 4104, 8, 1)])
def test_strides_and_what_lies_beside(V, ld, first, out_first, dtype):
    n = 3
    x = (torch.randn(n, V, device=DEV) * 4).to(dtype)
    r = _rules(n, V, 50, 4, V, softcap=0.0)

    def wide(t, first):
        b = torch.full((n * ld + 64,), 7.0, dtype=dtype, device=DEV)
        v = b[first:first + n * ld].view(n, ld)[:, :V]
        if t is not None:
            v.copy_(t)
        return b, v

    (_, xv), (ob, ov) = wide(x, first), wide(None, out_first)
    lce.lce_logits_process(xv, out=ov, **r)
    ref = lce.lce_logits_process(x.clone(), **r)
    assert torch.equal(ov.contiguous().view(torch.uint8), ref.view(torch.uint8))
    inside = torch.zeros(ob.numel(), dtype=torch.bool, device=DEV)
    inside[out_first:out_first + n * ld].view(n, ld)[:, :V] = True
    assert bool((ob[~inside] == 7.0).all())


def test_one_list_for_all_rows_and_wider_lists():
    n, V = 6, 500
    x = torch.randn(n, V, device=DEV)
    r = _rules(n, V, 40, 8, 5)
    shared = dict(r, history=r["history"][:1].expand(n, 40), bias_ids=r["bias_ids"][:1].expand(n, 8),
                  bias_values=r["bias_values"][:1].expand(n, 8))
    _check(lce.lce_logits_process(x, out=torch.empty_like(x), **shared), x, shared)
    wide = torch.randint(0, V, (n, 64), device=DEV)
    part = dict(r, history=wide[:, 8:48], history_lens=None, prompt_lens=None)
    _check(lce.lce_logits_process(x, out=torch.empty_like(x), **part), x, part)
    own = dict(r, allowed=(torch.randint(0, 1 << 32, (n, 20), device=DEV) - (1 << 31)).to(torch.int32), mask_rows=None)
    _check(lce.lce_logits_process(x, out=torch.empty_like(x), **own), x, own)   # row i uses mask i


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_infinities_nans_and_masks_that_leave_nothing(dtype):
    n, V = 4, 300
    x = torch.randn(n, V, device=DEV).to(dtype)
    x[0, 3], x[0, 4], x[0, 5], x[0, 6] = INF, -INF, float("nan"), torch.finfo(dtype).min
    x[1] = float("nan")
    x[2] = -INF
    words = (V + 31) // 32
    allowed = torch.zeros(2, words, dtype=torch.int32, device=DEV)
    allowed[1] = -1
    rows = torch.tensor([1, 0, 1, 0], device=DEV)
    for value in (-INF, -1e30):
        out = lce.lce_logits_process(x, allowed=allowed, mask_rows=rows, mask_value=value, out=torch.empty_like(x))
        assert torch.equal(out[0].view(torch.uint8), x[0].view(torch.uint8))      # nothing is hidden from row 0
        want = torch.full((V,), value, dtype=dtype, device=DEV)
        assert torch.equal(out[1], want) and torch.equal(out[3], want)            # rows that allow nothing
        assert bool((out[2] == -INF).all())
    # penalties of infinite logits keep their sign
    r = dict(history=torch.tensor([[3, 4, 6, 6]], device=DEV).expand(n, 4), repetition=torch.full((n,), 2.0, device=DEV),
             presence=torch.ones(n, device=DEV))
    out = lce.lce_logits_process(x, out=torch.empty_like(x), **r)
    assert float(out[0, 3]) == INF and float(out[0, 4]) == -INF and bool(torch.isnan(out[0, 5]))
    # softcap: bounded by the cap, NaN kept
    out = lce.lce_logits_process(x, softcap=30.0, out=torch.empty_like(x))
    assert float(out[0, 3]) == 30 and float(out[0, 4]) == -30 and float(out[0, 6]) == -30
    assert bool(torch.isnan(out[0, 5])) and bool((out[2] == -30).all())


def test_a_vanishing_temperature_keeps_zeros():
    x = torch.tensor([[0.0, 1.0, -1.0, 1e-30]], device=DEV)
    out = lce.lce_logits_process(x, temperature=torch.tensor([1e-39], device=DEV), out=torch.empty_like(x))
    assert float(out[0, 0]) == 0 and float(out[0, 1]) > 1e38 and float(out[0, 2]) < -1e38 and float(out[0, 3]) > 0


def test_no_rule_leaves_the_bits():
    for dtype in (BF16, F32):
        x = torch.randn(3, 999, device=DEV).to(dtype)
        assert torch.equal(lce.lce_logits_process(x, out=torch.empty_like(x)), x)
        none = torch.empty((3, 0), dtype=torch.int64, device=DEV)
        r = dict(history=none, bias_ids=none, bias_values=torch.empty((3, 0), device=DEV))
        assert torch.equal(lce.lce_logits_process(x, out=torch.empty_like(x), **r), x)
    x = torch.empty((0, 64), device=DEV)
    assert lce.lce_logits_process(x).shape == (0, 64)


def test_a_long_history_counts_every_token():
    n, V, L = 2, 20000, 200_001
    x = torch.zeros(n, V, device=DEV)
    h = torch.full((n, L), 12345, dtype=torch.int32, device=DEV)
    h[1, ::2] = 7
    out = lce.lce_logits_process(x, history=h, frequency=torch.ones(n, device=DEV))
    assert float(out[0, 12345]) == -L and float(out[1, 7]) == -((L + 1) // 2) and float(out[1, 12345]) == -(L // 2)
    assert int((out != 0).sum()) == 3


@pytest.mark.parametrize("L,B", [(32767, 65535), (32768, 9), (50, 65536), (0, 70000), (33000, 0)])
def test_long_lists(L, B):
    """Both sides of the sizes at which the counts and entries of a column share a word."""
    n, V = 2, 9000
    x = torch.randn(n, V, device=DEV)
    r = _rules(n, V, L, B, L + B, masks=0)         # most columns are listed: more than a slice's list holds
    if L:
        r["history"][0] = 77                       # one token as often as the list is long
        r["prompt_lens"][0] = 0
    _check(lce.lce_logits_process(x, out=torch.empty_like(x), **r), x, r)


def test_offsets_past_32_bits():
    """A row stride that puts the second row 2^31 elements (4 GiB) away."""
    V, ld = 1000, (1 << 31) + 8
    big = torch.zeros(ld + V, dtype=BF16, device=DEV)
    x = big.as_strided((2, V), (ld, 1))
    x.copy_(torch.randn(2, V, device=DEV))
    r = _rules(2, V, 20, 3, 1)
    want = lce.lce_logits_process(x.contiguous(), **r)
    lce.lce_logits_process(x, **r)
    assert torch.equal(x, want)


def test_captured_and_replayed_on_other_streams():
    n, V = 9, 5001
    x = torch.randn(n, V, device=DEV)
    r = _rules(n, V, 120, 6, 2)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lce.lce_logits_process(x, out=out, stream=side, **r)
    side.synchronize()
    _check(out, x, r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lce.lce_logits_process(x, out=out, **r)
    for k in range(4):
        x.copy_(torch.randn(n, V, device=DEV) * (k + 1))
        r["history"].copy_(torch.randint(0, V, r["history"].shape, device=DEV))
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        _check(got, x, r)


def test_then_argmax_and_log_probability():
    """As a serving step uses them together: rules, then the greedy token and its log-probability."""
    n, V = 8, 32000
    x = (torch.randn(n, V, device=DEV) * 3).to(BF16)
    r = _rules(n, V, 64, 5, 3, masks=2)
    r["mask_rows"].fill_(0)                       # every row keeps something
    hidden = lce.lce_logits_process(x, out=torch.empty_like(x), **r)
    assert bool((hidden == -INF).any())
    z = lce.lce_logits_process(x, mask_value=-1e4, **r)
    token, _ = lce.lce_ce_argmax(z)
    assert torch.equal(token, lce.lce_ce_argmax(hidden)[0])
    rows = lce.lce_ce_combine(lce.lce_ce_stats(z, token), token, V)
    assert torch.equal(token, z.float().argmax(1))
    logp = torch.log_softmax(z.double(), 1)
    assert torch.allclose(rows.logprob.double(), logp.gather(1, token[:, None])[:, 0], atol=1e-4)
    entropy = -(logp.exp() * logp).sum(1)
    assert torch.allclose(rows.entropy.double(), entropy, atol=1e-3) and bool(torch.isfinite(rows.loss_tok).all())
