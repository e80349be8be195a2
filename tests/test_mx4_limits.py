"""How large the 4-bit calls may be: the bounds that include/fsdp_mx4.h states,
refused with their code before any device work (CPU only)."""

import os
import re

import pytest

from rank_step_amd import binding as B
from tests.test_mx4_host import product, quantize

HEADER = re.sub(r"[\s*]+", " ", open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                                                  "fsdp_mx4.h")).read())
FAR = dict(x=1 << 40, codes=1 << 44, scales=1 << 46, codes_t=1 << 47, scales_t=1 << 49)


@pytest.mark.parametrize("m,n", [(1, 1), (1, 8), (4, 1), (300, 300)])
def test_the_longest_contraction(m, n):
    """Of a single row as well, whose stride says nothing."""
    assert "m and n are at most 2^30, k at most 2^23" in HEADER
    with pytest.raises(B.FsdpError) as e:
        product(m=m, n=n, k=(1 << 23) + 1, a=1 << 40, a_scales=1 << 42, b=1 << 43, b_scales=1 << 45, y=1 << 46)
    assert e.value.name == "FSDP_E_CAPACITY" and "k exceeds 2^23" in str(e.value), str(e.value)


@pytest.mark.parametrize("rows,cols,both", [(1 << 30, 1, True), (1 << 30, 128, False), (1 << 28, 513, True), (1, 1 << 30, True)])
def test_the_most_tiles_of_a_transpose(rows, cols, both):
    """A launch's 2^22 - 1 tiles; the copy along rows has no such bound."""
    assert "2^22 - 1 tiles of 256 x 128" in HEADER
    row_tiles, col_tiles = -(-rows // 512) * 2, -(-cols // 512) * 4 if both else -(-cols // 128)
    assert row_tiles * col_tiles > (1 << 22) - 1
    with pytest.raises(B.FsdpError) as e:
        quantize(rows=rows, cols=cols, **{**FAR, **({} if both else dict(codes=None, scales=None))})
    assert e.value.name == "FSDP_E_CAPACITY", str(e.value)
