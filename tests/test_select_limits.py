"""Rows that one launch of a selection does not hold are refused on the host (a launch that fails
leaves its error to whatever launches next in the process)."""
import ctypes

import pytest

from tests.test_quant_cache_refusals import lib, p  # noqa: F401


@pytest.mark.parametrize("rows,P_max,code", [(65536, 1024, -2), (70000, 16, -2), (2 ** 31 - 1, 1024, -2), (65535, 131073, -2),
                                             (7, 262145, -2), (65535, 131072, 0), (7, 262144, 0)])
def test_rows_of_a_selection(lib, p, rows, P_max, code):  # noqa: F811
    size = ctypes.c_size_t(0)
    assert lib.vsd_select_workspace_size(rows, 8, P_max, 64, ctypes.byref(size)) == code
    assert lib.vsd_select_hybrid_workspace_size(rows, P_max, ctypes.byref(size)) == code
    # (what is supported goes on to its pointers: no indices are given)
    rest = -2 if code else -1
    assert lib.vsd_select_topk(rows, 8, p, p, P_max, 64, 4, 16, None, p, None, None, 0, None) == rest
    assert lib.vsd_select_topk_hybrid(rows, 8, p, 8, p, p, P_max, 64, 8, 4, 16, None, p, None, 0, None) == rest
