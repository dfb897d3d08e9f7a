"""What the operators of include/lora_base8.h hand back: a Block8 made without its __init__ is one like any other."""
import copy
import dataclasses

import pytest

torch = pytest.importorskip("torch")

from test_gpu_block8 import F32, F8, _built, b8, rnd, same  # noqa: E402,F401
from test_gpu_distill import bwd, fwd, make  # noqa: E402

pytestmark = pytest.mark.gpu


def is_whole(p, rows, cols, tile):
    assert type(p) is b8().Block8 and p.cols == cols and p.tile == tile
    assert p.codes.dtype == F8 and p.codes.shape == (rows, -(-cols // 16) * 16) and p.codes.is_contiguous()
    assert p.scales.dtype == F32 and p.scales.shape == (-(-rows // tile), -(-cols // 128)) and p.scales.is_contiguous()
    assert [f.name for f in dataclasses.fields(p)] == ["codes", "scales", "cols", "tile"]
    for q in (dataclasses.replace(p), copy.copy(p), copy.deepcopy(p)):
        assert same(q.codes, p.codes) and same(q.scales, p.scales) and (q.cols, q.tile) == (p.cols, p.tile)
        assert same(b8().unblock8(q), b8().unblock8(p))


# small ones share an allocation, large ones do not
@pytest.mark.parametrize("rows,cols", [(5, 300), (1, 1), (700, 2001)])
@pytest.mark.parametrize("tile", [1, 128])
def test_a_block8(rows, cols, tile):
    is_whole(b8().block8(rnd(rows, cols), tile=tile), rows, cols, tile)


@pytest.mark.parametrize("m,v", [(7, 130), (600, 4001)])
def test_a_gradient_in_blocks(m, v):
    c = make(m, v, 5)
    _, probs, stats = fwd(c)
    is_whole(bwd(c, torch.ones(m, device="cuda"), probs, stats, block8=True), m, v, 1)
    for t, shape in ((probs, (m, 5)), (stats, (m, 4))):
        assert t.dtype == F32 and t.shape == shape and t.is_contiguous() and t.data_ptr() % 16 == 0
