"""Refusals of the operators around the cross-entropy, on the CPU: the C entry points reject bad
arguments before any HIP call, and the binding refuses host tensors and mismatched operands."""
import pytest

torch = pytest.importorskip("torch")

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

P = 0x10000   # never dereferenced: validation must reject the call first
OK, ARG, UNSUPPORTED = lce.LCE_OK, lce.LCE_ERR_INVALID_ARG, lce.LCE_ERR_UNSUPPORTED


def _call(fn, defaults, over):
    unknown = set(over) - set(defaults)
    assert not unknown
    return getattr(lce.lib(), fn)(*{**defaults, **over}.values()), lce.lce_last_error()


NORM = dict(x=P, ldx=64, dtype=lce.LCE_BF16, residual=None, ldr=0, weight=P, weight_dtype=lce.LCE_BF16, offset=0.0,
            eps=1e-6, n=4, H=64, sum=None, lds=0, y=P, ldy=64, y_dtype=lce.LCE_BF16, scale=None, rstd=None, stream=None)


@pytest.mark.parametrize("over,needle,status", [
    (dict(n=-1), "n must be", ARG), (dict(H=0), "H must be", ARG), (dict(dtype=9), "dtype", ARG),
    (dict(dtype=lce.LCE_E4M3), "dtype", ARG), (dict(weight_dtype=7), "weight dtype", ARG),
    (dict(offset=float("nan")), "weight_offset", ARG), (dict(eps=-1.0), "eps", ARG),
    (dict(eps=float("inf")), "eps", ARG), (dict(eps=float("nan")), "eps", ARG),
    (dict(y_dtype=lce.LCE_F32), "y must have", ARG), (dict(x=None), "x is required", ARG),
    (dict(y=None), "y is required", ARG), (dict(ldx=63), "row stride of x", ARG), (dict(ldy=8), "row stride of y", ARG),
    (dict(residual=P, ldr=63), "row stride of residual", ARG), (dict(sum=P, lds=1), "row stride of sum", ARG),
    (dict(x=P + 1), "aligned", ARG), (dict(weight=P + 1), "aligned", ARG),
    (dict(y_dtype=lce.LCE_E4M3), "scale is required", ARG),
    (dict(H=16385, ldx=16385, ldy=16385), "H must be <=", UNSUPPORTED), (dict(n=2 ** 31), "2^31", UNSUPPORTED),
])
def test_norm_rejects(over, needle, status):
    st, msg = _call("lce_rms_norm", NORM, over)
    assert st == status and needle in msg and msg.startswith("lce_rms_norm: ")


NORM_BWD = dict(grad_y=P, ldg=64, s=P, lds=64, dtype=lce.LCE_F32, weight=P, weight_dtype=lce.LCE_F32, offset=0.0,
                rstd=P, grad_sum=None, ldgs=0, n=4, H=64, grad_x=P, ldgx=64, grad_weight=P,
                grad_weight_dtype=lce.LCE_F32, workspace=P, workspace_bytes=4 * 64 * 4, stream=None)


@pytest.mark.parametrize("over,needle,status", [
    (dict(n=-1), "n must be", ARG), (dict(rstd=None), "rstd", ARG), (dict(s=None), "s is required", ARG),
    (dict(grad_y=None), "grad_y is required", ARG), (dict(grad_x=None), "grad_x is required", ARG),
    (dict(ldgx=3), "row stride of grad_x", ARG), (dict(grad_sum=P, ldgs=3), "row stride of grad_sum", ARG),
    (dict(grad_weight_dtype=lce.LCE_E4M3), "grad_weight dtype", ARG), (dict(workspace=None), "workspace_bytes", ARG),
    (dict(workspace_bytes=4 * 64 * 4 - 1), "workspace_bytes", ARG), (dict(workspace=P + 4), "16-byte aligned", ARG),
    (dict(grad_weight=P + 2), "aligned", ARG), (dict(H=20000, ldg=20000), "H must be <=", UNSUPPORTED),
])
def test_norm_backward_rejects(over, needle, status):
    st, msg = _call("lce_rms_norm_backward", NORM_BWD, over)
    assert st == status and needle in msg


def test_norm_workspace():
    assert lce.lce_rms_norm_workspace_bytes(4, 64) == 4 * 64 * 4
    assert lce.lce_rms_norm_workspace_bytes(10 ** 6, 64) == 1024 * 64 * 4
    assert lce.lce_rms_norm_workspace_bytes(0, 64) == lce.lce_rms_norm_workspace_bytes(5, 0) == 0


RULES = dict(logits=P, ldx=100, dtype=lce.LCE_F32, n=4, V=100, history=None, ldh=0, L=0, history_lens=None,
             prompt_lens=None, bias_ids=None, ldbi=0, bias_values=None, ldbv=0, B=0, wide=1, repetition=None,
             presence=None, frequency=None, temperature=None, allowed=None, ldm=0, masks=0, mask_rows=None,
             mask_value=float("-inf"), softcap=0.0, out=P, ldo=100, stream=None)


@pytest.mark.parametrize("over,needle,status", [
    (dict(n=-1), "n must be", ARG), (dict(V=0), "V must be", ARG), (dict(dtype=lce.LCE_E4M3), "dtype", ARG),
    (dict(ldx=99), "row stride of logits", ARG), (dict(ldo=99), "row stride of out", ARG),
    (dict(out=None), "out is required", ARG), (dict(logits=None), "logits is required", ARG),
    (dict(softcap=-1.0), "softcap", ARG), (dict(softcap=float("inf")), "softcap", ARG),
    (dict(mask_value=float("nan")), "mask_value", ARG), (dict(history=P, L=-1), "L must be", ARG),
    (dict(history=P, L=8, ldh=7), "row stride of history", ARG), (dict(history=P + 4, L=8, ldh=8), "aligned", ARG),
    (dict(bias_ids=P), "go together", ARG), (dict(bias_values=P), "go together", ARG),
    (dict(bias_ids=P, bias_values=P, B=-1), "B must be", ARG),
    (dict(bias_ids=P, bias_values=P, B=4, ldbi=3), "row strides of the biases", ARG),
    (dict(allowed=P, ldm=3, masks=4), "row stride of allowed", ARG), (dict(allowed=P, ldm=4, masks=3), "without mask_rows", ARG),
    (dict(allowed=P, ldm=4, masks=-1), "mask_count", ARG), (dict(allowed=P + 2, ldm=4, masks=4), "aligned", ARG),
    (dict(V=2 ** 31, ldx=2 ** 31, ldo=2 ** 31), "V must be <", UNSUPPORTED), (dict(n=2 ** 31), "2^31", UNSUPPORTED),
    (dict(history=P, L=2 ** 31, ldh=2 ** 31), "L and B", UNSUPPORTED),
])
def test_rules_reject(over, needle, status):
    st, msg = _call("lce_logits_process", RULES, over)
    assert st == status and needle in msg


def test_no_rows_need_no_buffers():
    none = dict(n=0, x=None, y=None)
    assert _call("lce_rms_norm", NORM, none)[0] == OK
    assert _call("lce_logits_process", RULES, dict(n=0, logits=None, out=None))[0] == OK


def test_host_tensors_are_refused():
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    w = torch.zeros(16, dtype=torch.bfloat16)
    for call in (lambda: lce.lce_rms_norm(x, w), lambda: lce.rms_norm(x, w), lambda: lce.rms_norm(x, w, residual=x),
                 lambda: lce.lce_rms_norm_backward(x, x, w, torch.zeros(4)), lambda: lce.lce_logits_process(x)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


def test_operand_checks():
    from vocabulary_cross_entropy_row_amd import head
    t = torch.zeros((4, 8))
    cpu = t.device
    assert head._rows(t, "t", torch.float32, 4, 8, cpu) == 8
    assert head._rows(t[:, :5], "t", torch.float32, 4, 5, cpu) == 8
    assert head._rows(t[:1], "t", torch.float32, 1, 8, cpu) == 8
    for bad, err, needle in ((t.t(), ValueError, r"\[4, 8\]"), (t.double(), TypeError, "float32"),
                             (torch.zeros((8, 4)).t(), ValueError, "unit column stride"), ([1], TypeError, "tensor")):
        with pytest.raises(err, match=needle):
            head._rows(bad, "t", torch.float32, 4, 8, cpu)
    with pytest.raises(ValueError, match="required"):
        head._rows(None, "t", torch.float32, 4, 8, cpu, required=True)
    with pytest.raises(TypeError, match="int32 or int64"):
        head._ids(t, "history", 4, cpu)
    with pytest.raises(ValueError, match="length"):
        head._ids(t.long(), "history", 5, cpu)
    assert head._ids(t.long()[:1].expand(4, 8), "history", 4, cpu) == (0, 8)
    rows = head._rows_of(torch.zeros(2, 3, 8).transpose(0, 1), 8)
    assert rows.shape == (6, 8) and rows.stride() == (8, 1)
    assert head._rows_of(torch.zeros(1, 8).expand(5, 8), 8).stride(0) == 8


LINEAR = dict(x=P, ldx=64, weight=P, ldw=64, in_dtype=lce.LCE_BF16, scale_x=None, scale_w=None, bias=None,
              bias_dtype=lce.LCE_F32, act=0, residual=None, ldr=0, n=4, K=64, M=40, out=P, ldo=40,
              out_dtype=lce.LCE_BF16, preact=None, ldp=0, workspace=None, bytes=0, stream=None)


@pytest.mark.parametrize("over,needle,status", [
    (dict(n=-1), "n must be", ARG), (dict(K=0), "K must be", ARG), (dict(M=0), "M must be", ARG),
    (dict(in_dtype=lce.LCE_F32), "must be bf16 or e4m3", ARG), (dict(act=5), "activation", ARG),
    (dict(act=-1), "activation", ARG), (dict(weight=None), "weight is required", ARG), (dict(x=None), "x is required", ARG),
    (dict(ldx=56), "row strides of x", ARG), (dict(ldw=56), "row strides of x", ARG),
    (dict(scale_x=P), "scales go with e4m3", ARG), (dict(out_dtype=lce.LCE_E4M3), "output dtype", ARG),
    (dict(bias=P, bias_dtype=lce.LCE_E4M3), "bias dtype", ARG), (dict(bias=P + 2), "bias must be", ARG),
    (dict(out=None), "out is required", ARG), (dict(ldo=39), "row stride of out", ARG),
    (dict(residual=P, ldr=39), "row stride of residual", ARG), (dict(preact=P, ldp=39), "row stride of preact", ARG),
    (dict(K=60), "multiples of 8", UNSUPPORTED), (dict(ldx=68), "multiples of 8", UNSUPPORTED),
    (dict(in_dtype=lce.LCE_E4M3, K=56), "multiples of 16", UNSUPPORTED), (dict(x=P + 8), "16-byte aligned", UNSUPPORTED),
    (dict(in_dtype=lce.LCE_E4M3, out_dtype=lce.LCE_F32), "bf16 output", UNSUPPORTED),
    (dict(weight=P + 2), "16-byte aligned", UNSUPPORTED), (dict(ldx=1 << 23), "4 GiB", UNSUPPORTED),
    (dict(n=1 << 23), "2^23", UNSUPPORTED), (dict(M=1 << 23, ldo=1 << 23), "2^23", UNSUPPORTED),
    (dict(n=200, K=4096, ldx=4096, ldw=4096, M=256, ldo=256), "workspace_bytes", ARG),
])
def test_linear_rejects(over, needle, status):
    st, msg = _call("lce_linear", LINEAR, over)
    assert st == status and needle in msg


LINEAR_BWD = dict(grad_out=P, ldg=40, grad_dtype=lce.LCE_BF16, x=P, ldx=64, weight=P, ldw=64, preact=P, ldp=40, act=2,
                  n=4, K=64, M=40, grad_x=P, ldgx=64, grad_weight=P, wdtype=lce.LCE_F32, grad_bias=P,
                  bdtype=lce.LCE_F32, workspace=P, bytes=1 << 20, stream=None)


@pytest.mark.parametrize("over,needle,status", [
    (dict(n=-1), "n must be", ARG), (dict(M=36, ldg=36, ldp=36), "M must be a multiple", UNSUPPORTED),
    (dict(K=60), "multiples of 8", UNSUPPORTED), (dict(grad_dtype=lce.LCE_E4M3), "grad_out dtype", ARG),
    (dict(wdtype=9), "grad_weight dtype", ARG), (dict(bdtype=lce.LCE_E4M3), "grad_bias dtype", ARG),
    (dict(preact=None), "preact is required", ARG), (dict(grad_out=None), "grad_out is required", ARG),
    (dict(ldg=39), "row stride of grad_out", ARG), (dict(ldgx=56), "row stride of grad_x", ARG),
    (dict(grad_x=P + 2), "grad_x must be 16-byte", UNSUPPORTED), (dict(ldgx=68), "whole 16 bytes", UNSUPPORTED),
    (dict(grad_weight=P + 4), "grad_weight must be 16-byte", UNSUPPORTED), (dict(grad_bias=P + 2), "grad_bias", ARG),
    (dict(workspace=None), "workspace_bytes", ARG), (dict(bytes=100), "workspace_bytes", ARG),
    (dict(workspace=P + 16), "256-byte aligned", ARG), (dict(x=None), "x is required", ARG),
])
def test_linear_backward_rejects(over, needle, status):
    st, msg = _call("lce_linear_backward", LINEAR_BWD, over)
    assert st == status and needle in msg


def test_linear_sizes_and_host_tensors():
    assert _call("lce_linear", LINEAR, dict(n=0, x=None, out=None))[0] == OK
    assert lce.lce_linear_workspace_bytes(4096, 4096, 16384) == 0      # enough tiles without splits
    assert lce.lce_linear_workspace_bytes(200, 4096, 256) % (200 * 256 * 4) == 0 < lce.lce_linear_workspace_bytes(200, 4096, 256)
    assert lce.lce_linear_workspace_bytes(4, 0, 8) == lce.lce_linear_backward_workspace_bytes(4, 8, 0) == 0
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((8, 64), dtype=torch.bfloat16)
    for call in (lambda: lce.lce_linear(x, w), lambda: lce.linear(x, w), lambda: lce.lce_linear_backward(x[:, :8], x, w)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


@pytest.mark.parametrize("over,needle", [
    (dict(out=P), "out and preact must not be x or weight"), (dict(weight=2 * P), "out and preact must not be x"),
    (dict(x=2 * P), "out and preact must not be x"), (dict(out=2 * P, preact=P, ldp=40), "must not be x or weight"),
    (dict(out=2 * P, preact=2 * P, ldp=40), "preact must not be residual or out"),
    (dict(out=2 * P, preact=3 * P, ldp=40, residual=3 * P, ldr=40), "preact must not be residual"),
])
def test_linear_rejects_outputs_that_it_still_reads(over, needle):
    st, msg = _call("lce_linear", LINEAR, over)
    assert st == ARG and needle in msg


@pytest.mark.parametrize("over", [dict(n=(1 << 23) - 511), dict(n=(1 << 23) - 1),
                                  dict(M=(1 << 23) - 504, ldg=1 << 23, ldp=1 << 23)])
def test_linear_backward_rejects_rows_past_its_offsets(over):
    """n and M are the row lengths of the transposed operands: 256 such rows stay below 4 GiB."""
    st, msg = _call("lce_linear_backward", LINEAR_BWD, over)
    assert st == UNSUPPORTED and "2^23 - 512" in msg
