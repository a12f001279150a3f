"""What the binding of the rotary operators makes of its arguments; on the CPU."""
import ctypes

import pytest
import torch

from fp8_mla_kv_gb300 import build as B
from fp8_mla_kv_gb300 import mlasparse as M

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.load()


def test_positions_are_passed_with_their_own_stride():
    wide = torch.arange(60, dtype=torch.int32).view(3, 20)
    for n in (1, 2, 20):
        assert M._positions(wide[:, :n], n, 3) == 20
        # one row for all axes: text in a model whose positions have three
        assert M._positions(wide[:1, :n].expand(3, n), n, 3) == 0
        assert M._positions(wide[0, :n].expand(3, n), n, 3) == 0
    assert M._positions(wide[:, :1].t().contiguous().t(), 1, 3) == 1
    for stride in (1, 4, 6):                                # rows that overlap
        with pytest.raises(ValueError):
            M._positions(torch.as_strided(wide, (3, 7), (stride, 1)), 7, 3)
    with pytest.raises(ValueError):
        M._positions(wide[0], 20, 3)
    # one axis: the stride is not used
    M._positions(wide[0], 20, 1)
    M._positions(wide[:1].expand(3, 20), 20, 1)


def test_axes_that_overlap_are_refused_by_the_library(lib):
    s = ctypes.byref(M.rope_spec([1.0] * 32, axis=[i % 3 for i in range(32)]))
    kv = M.KVCache(256, 16, 656)
    for stride in (1, 3):
        assert lib.mla_rope(P(256), 64, 64, P(256), 64, 64, 4, 1, P(256), stride, s, None) == M.MLA_EINVAL
        assert lib.mla_rope_kv_write(kv, P(256), P(256), P(256), 4, 0, P(256), stride, s, None, 0, 0, None, 0, 0, 0,
                                     None) == M.MLA_EINVAL


@pytest.mark.parametrize("row,head,n,heads", [(0, 64, 4, 2), (128, 0, 4, 2), (56, 1024, 4, 2), (1024, 8, 4, 2), (64, 64, 4, 2),
                                              (-64, 64, 4, 2), (128, 64, 4, 3), (192, 128, 4, 4), (320, 192, 9, 9), (0, 0, 2, 1),
                                              (0, 0, 1, 2)])
def test_views_that_overlap_themselves_are_not_written(lib, row, head, n, heads):
    """In place, a broadcast head would be turned once for each of its copies."""
    s = ctypes.byref(M.rope_spec([1.0] * 32))
    kv = M.KVCache(256, 16, 656)
    assert lib.mla_rope(P(256), 1024, 64, P(256), row, head, n, heads, P(256), 0, s, None) == M.MLA_EINVAL
    assert lib.mla_rope_kv_write(kv, P(256), P(256), P(256), n, 0, P(256), 0, s, P(256), 1024, 64, P(256), row, head, heads,
                                 None) == M.MLA_EINVAL
