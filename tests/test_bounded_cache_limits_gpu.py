"""The window, weighing and eviction calls at the ends of what they take."""
import pytest

from gqa_attention_forward_gb300 import binding
from packed_util import offsets
from paged_util import build
from test_tree_gpu import i32, queries, status, trees
from test_window_gpu import check_trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(None, 0), (None, 300), (1, None), (700, None), (None, None)])
def test_windows_of_the_widest_table(window, sinks):
    """None: one less than the table's positions, the largest value that is not the plain call's."""
    page, width = 4096, (2 ** 30 - 1) // 4096
    cache = build([5000, 40], page, 2, 64, "f16", seed=93, width=width)
    most, T = page * width - 1, [9, 1]
    window, sinks = (most if x is None else x for x in (window, sinks))
    par = trees(T, 94)
    q = queries(10, 4, 64, "f16", 95)
    o, lse = binding.attention_tree(q, cache, offsets(T), parents=i32([x for p in par for x in p]), window=window, sinks=sinks)
    assert status() == binding.ATTN_OK
    check_trees(q, cache, o, lse, range(2), par, "f16", 1 / 8, window, sinks)
