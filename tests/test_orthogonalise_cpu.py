"""Refusals of the orthogonalised update, before any HIP call."""
import pytest

torch = pytest.importorskip("torch")

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

G, OUT, WS = 0x10000, 0x20000, 0x30000   # never dereferenced
INVALID, UNSUPPORTED = lce.LCE_ERR_INVALID_ARG, lce.LCE_ERR_UNSUPPORTED
INF, NAN = float("inf"), float("nan")


def call(**over):
    a = dict(g=G, ldg=70, gb=7000, dtype=lce.LCE_BF16, batch=3, rows=100, cols=70, steps=5, a=3.4, b=-4.8, c=2.0, eps=1e-7,
             out=OUT, ldo=70, ob=7000, ws=WS, wsb=1 << 30)
    a.update(over)
    return lce.lib().lce_orthogonalise(a["g"], a["ldg"], a["gb"], a["dtype"], a["batch"], a["rows"], a["cols"], a["steps"],
                                       a["a"], a["b"], a["c"], a["eps"], a["out"], a["ldo"], a["ob"], a["ws"], a["wsb"],
                                       None), lce.lce_last_error()


@pytest.mark.parametrize("over,status,needle", [
    (dict(batch=-1), INVALID, "batch must be"), (dict(rows=0), INVALID, "rows and cols"), (dict(cols=0), INVALID, "rows and cols"),
    (dict(cols=(1 << 20) + 1), UNSUPPORTED, "2^20"), (dict(batch=70000), UNSUPPORTED, "65535"),
    (dict(rows=1 << 18, cols=1 << 18, ldg=1 << 18, ldo=1 << 18), UNSUPPORTED, "tiles"),
    (dict(dtype=2), INVALID, "dtype"), (dict(steps=0), INVALID, "steps"), (dict(steps=101), INVALID, "steps"),
    (dict(a=INF), INVALID, "coefficients"), (dict(b=NAN), INVALID, "coefficients"), (dict(eps=-1.0), INVALID, "eps"),
    (dict(eps=NAN), INVALID, "eps"), (dict(g=None), INVALID, "g is required"), (dict(out=None), INVALID, "out is required"),
    (dict(ldg=69), INVALID, "row stride of g"), (dict(ldo=69), INVALID, "row stride of out"), (dict(g=G + 1), INVALID, "aligned"),
    (dict(gb=-1), INVALID, "batch stride of g"), (dict(ob=6999), INVALID, "overlap"), (dict(ob=0), INVALID, "overlap"),
    (dict(out=G), INVALID, "must not be g"), (dict(ws=None), INVALID, "workspace"), (dict(wsb=1000), INVALID, "workspace_bytes"),
    (dict(ws=WS + 16), INVALID, "256-byte"),
])
def test_refuses(over, status, needle):
    st, msg = call(**over)
    assert st == status and needle in msg, msg


def test_nothing_to_do_and_workspace():
    assert call(batch=0, g=None, out=None, ws=None, wsb=0)[0] == lce.LCE_OK
    assert lce.lce_orthogonalise_workspace_bytes(0, 5, 5) == lce.lce_orthogonalise_workspace_bytes(1, 0, 5) == 0
    one, two = (lce.lce_orthogonalise_workspace_bytes(b, 300, 500) for b in (1, 2))
    assert 0 < one < two and lce.lce_orthogonalise_workspace_bytes(1, 500, 300) == one


def test_binding_refuses():
    with pytest.raises(ValueError, match="GPU tensor"):
        lce.lce_orthogonalise(torch.zeros(4, 4))
    with pytest.raises(TypeError, match="torch tensor"):
        lce.lce_orthogonalise(g=None)
