"""Refusals of the quantiser into blocks of 128 and of the products that read it: the C entry points
before any HIP call, the binding before any library call."""
import inspect

import pytest

torch = pytest.importorskip("torch")

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

A, B, C, D, E, F, WS = (0x10000 * (i + 1) for i in range(7))   # never dereferenced
INVALID, UNSUPPORTED = lce.LCE_ERR_INVALID_ARG, lce.LCE_ERR_UNSUPPORTED


def quantize(**over):
    a = dict(x=A, ldx=300, dtype=lce.LCE_BF16, n=40, K=300, v=B, ldv=304, kind=0, s=C, s_row=1, s_col=40, vt=D, ldvt=48,
             kind_t=0, st=E, st_row=1, st_col=300, scale=lce.LCE_E8M0)
    a.update(over)
    return lce.lib().lce_quantize_blocks(a["x"], a["ldx"], a["dtype"], a["n"], a["K"], a["v"], a["ldv"], a["kind"], a["s"],
                                         a["s_row"], a["s_col"], a["vt"], a["ldvt"], a["kind_t"], a["st"], a["st_row"],
                                         a["st_col"], a["scale"], None), lce.lce_last_error()


@pytest.mark.parametrize("over,status,needle", [
    (dict(n=-1), INVALID, "n must be"), (dict(K=0), INVALID, "K must be"), (dict(dtype=2), INVALID, "dtype"),
    (dict(kind=2), INVALID, "blocks"), (dict(kind_t=-1), INVALID, "blocks"), (dict(x=None), INVALID, "x is required"),
    (dict(ldx=299), INVALID, "row stride of x"), (dict(ldv=299), INVALID, "row stride of values"),
    (dict(ldvt=39), INVALID, "row stride of values_t"), (dict(v=None, vt=None), INVALID, "values or values_t"),
    (dict(s=None), INVALID, "scale is required"), (dict(st=None), INVALID, "scale_t is required"),
    (dict(scale=1), INVALID, "fp32 or e8m0"), (dict(s_row=1, s_col=39), INVALID, "one place"),
    (dict(s_row=0, s_col=0), INVALID, "one place"), (dict(s_row=-1), INVALID, "strides of scale"),
    (dict(scale=0, s=C + 2), INVALID, "aligned"), (dict(x=A + 1), INVALID, "aligned"),
    (dict(v=A), INVALID, "must not be x"), (dict(vt=B), INVALID, "same buffer"), (dict(st=C), INVALID, "same buffer"),
    (dict(n=1 << 40, K=1 << 40, ldx=1 << 41), UNSUPPORTED, "2^24"), (dict(n=1 << 24, K=1 << 14, ldx=1 << 14), UNSUPPORTED, "2^24"),
])
def test_quantiser_refuses(over, status, needle):
    st, msg = quantize(**over)
    assert st == status and needle in msg, msg


def test_nothing_to_do():
    assert quantize(n=0, x=None, v=None, s=None, vt=None, st=None)[0] == lce.LCE_OK
    assert product(n=0, x=None, sx=None, out=None)[0] == lce.LCE_OK


def product(**over):
    a = dict(x=A, ldx=304, sx=B, sx_row=1, sx_col=40, sx_t=3, w=C, ldw=304, sw=D, sw_row=3, sw_col=1, sw_t=3, bias=None,
             bias_t=0, act=0, res=None, ldr=500, n=40, K=300, M=500, out=E, ldo=500, pre=None, ldp=500, ws=WS, wsb=1 << 30)
    a.update(over)
    return lce.lib().lce_linear_blocks(a["x"], a["ldx"], a["sx"], a["sx_row"], a["sx_col"], a["sx_t"], a["w"], a["ldw"], a["sw"],
                                       a["sw_row"], a["sw_col"], a["sw_t"], a["bias"], a["bias_t"], a["act"], a["res"], a["ldr"],
                                       a["n"], a["K"], a["M"], a["out"], a["ldo"], a["pre"], a["ldp"], a["ws"], a["wsb"],
                                       None), lce.lce_last_error()


@pytest.mark.parametrize("over,status,needle", [
    (dict(n=-1), INVALID, "n must be"), (dict(K=0), INVALID, "K must be"), (dict(M=0), INVALID, "M must be"),
    (dict(n=1 << 23), UNSUPPORTED, "2^23"), (dict(M=1 << 23), UNSUPPORTED, "2^23"), (dict(act=9), INVALID, "activation"),
    (dict(x=None), INVALID, "x is required"), (dict(w=None), INVALID, "weight is required"),
    (dict(ldx=299), INVALID, "row stride of x"), (dict(ldx=301), UNSUPPORTED, "16-byte"), (dict(x=A + 8), UNSUPPORTED, "16-byte"),
    (dict(w=C + 1), UNSUPPORTED, "16-byte"), (dict(ldw=1 << 24), UNSUPPORTED, "4 GiB"), (dict(sx=None), INVALID, "scale_x is required"),
    (dict(sw_t=1), INVALID, "fp32 or e8m0"), (dict(sw_row=-3), INVALID, "strides of scale_w"),
    (dict(sx_t=0, sx=B + 1), INVALID, "aligned"), (dict(bias=F, bias_t=2), INVALID, "bias dtype"), (dict(bias=F + 2), INVALID, "bias must be"),
    (dict(out=None), INVALID, "out is required"), (dict(ldo=499), INVALID, "row stride of out"), (dict(res=F, ldr=1), INVALID, "residual"),
    (dict(out=A), INVALID, "must not be x"), (dict(pre=D), INVALID, "must not be x"), (dict(pre=E), INVALID, "preact"),
    (dict(bias=E), INVALID, "must not be bias"), (dict(n=64, K=8192, ldx=8192, ldw=8192, sx_col=64, sw_row=64, M=256, ws=None), INVALID, "workspace"),
])
def test_product_refuses(over, status, needle):
    st, msg = product(**over)
    assert st == status and needle in msg, msg


def backward(**over):
    a = dict(g=A, ldg=500, g_t=1, xt=B, ldxt=48, sxt=C, sxt_row=1, sxt_col=1, wt=D, ldwt=512, swt=E, swt_row=4, swt_col=1, n=40,
             K=300, M=500, gx=F, ldgx=300, gw=F + 0x1000, gb=F + 0x2000, gb_t=0, ws=WS, wsb=1 << 30)
    a.update(over)
    return lce.lib().lce_linear_blocks_backward(a["g"], a["ldg"], a["g_t"], a["xt"], a["ldxt"], a["sxt"], a["sxt_row"], a["sxt_col"],
                                                a["wt"], a["ldwt"], a["swt"], a["swt_row"], a["swt_col"], a["n"], a["K"], a["M"],
                                                a["gx"], a["ldgx"], a["gw"], a["gb"], a["gb_t"], a["ws"], a["wsb"],
                                                None), lce.lce_last_error()


@pytest.mark.parametrize("over,status,needle", [
    (dict(n=-1), INVALID, "n must be"), (dict(K=1 << 23), UNSUPPORTED, "2^23"), (dict(n=(1 << 23) - 1000), UNSUPPORTED, "2^23 - 1024"),
    (dict(n=1 << 22, M=1 << 22), UNSUPPORTED, "2^24"), (dict(g=None), INVALID, "grad_out is required"), (dict(g_t=2), INVALID, "grad_out dtype"),
    (dict(gb_t=3), INVALID, "grad_bias dtype"), (dict(xt=None), INVALID, "xt is required"), (dict(wt=None), INVALID, "wt is required"),
    (dict(ldxt=47), UNSUPPORTED, "16-byte"), (dict(ldwt=496), INVALID, "row stride of wt"), (dict(sxt=None), INVALID, "scale_xt"),
    (dict(swt=None), INVALID, "scale_wt"), (dict(wsb=100), INVALID, "workspace_bytes"), (dict(ws=WS + 16), INVALID, "256-byte"),
    (dict(gx=A), INVALID, "an operand"), (dict(gw=D), INVALID, "an operand"), (dict(gb=C), INVALID, "an operand"),
    (dict(gw=F + 1), INVALID, "aligned"), (dict(ldgx=299), INVALID, "grad_x"), (dict(gw=F), INVALID, "same buffer"),
])
def test_backward_refuses(over, status, needle):
    st, msg = backward(**over)
    assert st == status and needle in msg, msg


def forward(**over):
    a = dict(x=A, ldx=300, w=B, ldw=300, bias=None, bias_t=0, res=None, ldr=500, n=40, K=300, M=500, out=C, ldo=500, xt=D,
             ldxt=48, sxt=D + 0x8000, wt=E, ldwt=512, swt=E + 0x8000, ws=WS, wsb=1 << 30)
    a.update(over)
    return lce.lib().lce_linear_blocks_forward(a["x"], a["ldx"], a["w"], a["ldw"], a["bias"], a["bias_t"], a["res"], a["ldr"],
                                               a["n"], a["K"], a["M"], a["out"], a["ldo"], a["xt"], a["ldxt"], a["sxt"], a["wt"],
                                               a["ldwt"], a["swt"], a["ws"], a["wsb"], None), lce.lce_last_error()


@pytest.mark.parametrize("over,status,needle", [
    (dict(n=-1), INVALID, "n must be"), (dict(K=0), INVALID, "K must be"), (dict(M=0), INVALID, "M must be"),
    (dict(n=(1 << 23) - 1000), UNSUPPORTED, "2^23 - 1024"), (dict(M=1 << 22, K=1 << 22), UNSUPPORTED, "2^24"),
    (dict(x=None), INVALID, "x is required"), (dict(w=None), INVALID, "weight is required"), (dict(ldx=299), INVALID, "row stride of x"),
    (dict(ldw=299), INVALID, "row stride of weight"), (dict(x=A + 1), INVALID, "aligned"), (dict(out=None), INVALID, "out is required"),
    (dict(ldo=499), INVALID, "row stride of out"), (dict(bias=F, bias_t=2), INVALID, "bias dtype"), (dict(bias=F + 2), INVALID, "bias must be"),
    (dict(res=F, ldr=499), INVALID, "residual"), (dict(ldxt=47), UNSUPPORTED, "16-byte"), (dict(ldwt=496), INVALID, "row stride of wt"),
    (dict(xt=D + 8), UNSUPPORTED, "16-byte"), (dict(sxt=None), INVALID, "scale_xt"), (dict(swt=None), INVALID, "scale_wt"),
    (dict(ws=None), INVALID, "workspace"), (dict(wsb=1000), INVALID, "workspace_bytes"), (dict(ws=WS + 16), INVALID, "256-byte"),
    (dict(out=A), INVALID, "an operand"), (dict(xt=B), INVALID, "an operand"), (dict(wt=D), INVALID, "same buffer"),
    (dict(swt=C), INVALID, "same buffer"), (dict(bias=C), INVALID, "an operand"), (dict(res=D), INVALID, "an operand"),
])
def test_forward_refuses(over, status, needle):
    st, msg = forward(**over)
    assert st == status and needle in msg, msg


X = torch.zeros((4, 16), dtype=torch.bfloat16)
Q, S = torch.zeros((4, 16), dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones((4, 1))


@pytest.mark.parametrize("call", [
    lambda: lce.lce_quantize_blocks(x=X), lambda: lce.lce_quantize_blocks(X),
    lambda: lce.lce_linear_blocks(x=Q, scale_x=S, weight=Q, scale_w=S[:1]),
    lambda: lce.lce_linear_blocks_backward(grad_out=X, xt=Q, scale_xt=S), lambda: lce.linear_blocks(X, X)])
def test_host_tensors(call):
    with pytest.raises(ValueError, match="GPU tensor"):
        call()


def test_workspaces_and_signatures():
    assert lce.lce_linear_blocks_workspace_bytes(4096, 8192, 8192) == 0
    assert lce.lce_linear_blocks_workspace_bytes(-1, 8, 8) == lce.lce_linear_blocks_workspace_bytes(1, 0, 8) == 0
    small, more = (lce.lce_linear_blocks_backward_workspace_bytes(n, 300, 500) for n in (40, 400))
    assert 0 < small < more
    assert list(inspect.signature(lce.lce_linear_blocks).parameters)[:4] == ["x", "scale_x", "weight", "scale_w"]
    assert "lce_quantize_blocks" in dir(lce)
