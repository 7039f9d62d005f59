"""What the quantiser allocates beside the outputs that a caller brings."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible to torch", allow_module_level=True)

import vocabulary_cross_entropy_row_amd as lce  # noqa: E402

DEV = torch.device("cuda:0")


def allocated(call):
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    call()
    return torch.cuda.max_memory_allocated() - before


@pytest.mark.parametrize("blocks", ["row", "tile"])
def test_only_what_is_missing_is_allocated(blocks):
    n, K = 1024, 4096
    x = torch.randn(n, K, device=DEV)
    want = lce.lce_quantize_blocks(x, blocks=blocks, transposed=blocks)
    given = dict(values=torch.empty_like(want.values), scale=torch.empty_like(want.scale),
                 values_t=torch.empty_like(want.values_t), scale_t=torch.empty_like(want.scale_t))
    assert allocated(lambda: lce.lce_quantize_blocks(x, blocks=blocks, transposed=blocks, **given)) == 0
    for got, was in ((given["values"], want.values), (given["scale"], want.scale), (given["values_t"], want.values_t),
                     (given["scale_t"], want.scale_t)):
        assert torch.equal(got.view(torch.uint8), was.view(torch.uint8))
    room = allocated(lambda: lce.lce_quantize_blocks(x, blocks=blocks, values=given["values"]))
    assert 0 < room <= 2 * want.scale.numel() + 512
    room = allocated(lambda: lce.lce_quantize_blocks(x, blocks=blocks, scale=given["scale"]))
    assert n * K <= room <= n * K + 2 ** 21


@pytest.mark.parametrize("name", ["values", "scale", "values_t", "scale_t"])
def test_outputs_that_are_no_tensors_are_refused(name):
    with pytest.raises(TypeError, match=f"{name} must be a torch tensor"):
        lce.lce_quantize_blocks(torch.zeros(4, 130, device=DEV), transposed="row", **{name: [1.0]})
