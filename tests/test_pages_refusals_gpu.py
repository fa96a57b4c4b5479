"""Wrong lists and wrong tables: the page operators report them and leave the sequence, its pages
and the pools as they were."""
import pytest
import torch

from gqa_attention_forward_gb300 import binding
from paged_util import Model, build

pytestmark = pytest.mark.gpu

LOWEST = -2 ** 31


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    return binding.attn_last_device_error(torch.cuda.current_stream())


@pytest.mark.parametrize("path", [[-1], [-1, 0], [-2, -1], [-5, -3, -1, 0], [LOWEST, -2 * 10 ** 9], [LOWEST, LOWEST + 1, 0, 1],
                                  [0, LOWEST], [-1, -1], [3, -7, -6, 2], [0, 2 ** 31 - 1], [2 ** 31 - 1, LOWEST]])
def test_paths_of_no_tree(path):
    """Paths that ascend, but from before the tree, and others that leave it on either side."""
    c = build([40, 5, 33], 16, 2, 64, "f16", 2, n_rows=6)
    m = Model(c)
    for s in (0, 1, 2):
        binding.kv_accept(c, i32([0, 5]), i32([path]), i32([len(path)]), i32([s]))
        assert status() == binding.ATTN_ERR_SHAPE
        m.same(c)
    # one such sequence does not keep the others from being served
    w = max(3, len(path))
    binding.kv_accept(c, i32([0, 5, 9, 12]), i32([x + [-1] * (w - len(x)) for x in ([1, 4], path, [0, 2])]),
                      i32([2, len(path), 2]), i32([0, 1, 2]))
    assert status() == binding.ATTN_ERR_SHAPE
    m.accept([0, 2], [5, 3], [[1, 4], [0, 2]])
    m.same(c)
