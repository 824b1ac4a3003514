"""Masks that would leave rows free without a word are refused, by the library and by the binding (CPU)."""
import pytest

import q8_block_quantized_gemv_gb300 as q8
from test_w4_host import ARG, P, SHAPE, choose, lib  # noqa: F401
from test_w4_wide_sizes import Like

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("bad,want", [(dict(mask=P, mask_count=3, mask_pitch=4), SHAPE), (dict(mask=P, mask_count=1, mask_pitch=4), SHAPE),
                                      (dict(mask=P, mask_rows=P + 4096, mask_count=0, mask_pitch=4), SHAPE),
                                      (dict(mask_rows=P), ARG)])
def test_the_library_refuses(lib, bad, want):  # noqa: F811
    assert choose(lib, **bad) == want  # of four rows


def test_the_binding_refuses(lib):  # noqa: F811
    x, rows = Like((4, 100), torch.float32), Like((4,), torch.int32)
    for kw in (dict(mask=Like((1, 4), torch.int32)), dict(mask=Like((3, 4), torch.int32)), dict(mask=Like((0, 4), torch.int32)),
               dict(mask=Like((0, 4), torch.int32), mask_rows=rows), dict(mask_rows=rows)):
        with pytest.raises(ValueError, match="mask"):
            q8.choose(x, **kw)
