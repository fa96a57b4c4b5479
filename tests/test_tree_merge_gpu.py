"""attn_fwd_tree where a unit is cut into pieces of very different weight."""
import math

import pytest
import torch

from gqa_attention_forward_gb300 import binding
from packed_util import offsets
from paged_util import build
from test_tree_gpu import check, queries, sees, trees

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("Hq,Hkv,T", [(4, 1, 1), (4, 1, 20), (32, 8, 20), (64, 8, 128)])  # the last merges by CTAs
@pytest.mark.parametrize("peak", [5, 39990])
def test_non_finite_values_of_a_piece_without_weight(Hq, Hkv, T, peak):
    """One key outweighs all others by far more than fp32 holds, so that every piece but its own
    has the weight 0: infinities and NaN in the others still reach the rows that see them."""
    base, D, page = 40000, 128, 64
    cache = build([base + T], page, Hkv, D, "bf16", seed=81)
    par = trees([T], 82)[0]

    def at(pos):
        return int(cache.table[0, pos // page]), pos % page

    q = queries(T, Hq, D, "bf16", 83).abs() + 1
    p, r = at(peak)
    cache.k[0, p, :, r] = 60.0  # a score past 60 sqrt(D) = 678, the others' about 10
    # before the tree, far from the peak on either side, and at two tokens of the tree
    node = min(3, T - 1)
    for pos, col, x in ((20000, 3, math.inf), (20000, 7, math.nan), (12345, 9, -math.inf), (base + node, 64, math.inf),
                        (base + T - 1, 100, math.nan)):
        p, r = at(pos)
        cache.v[0, p, :, r, col] = x
    o, lse = binding.attention_tree(q, cache, offsets([T]), parents=i32(par))
    assert binding.attn_last_device_error(torch.cuda.current_stream()) == binding.ATTN_OK
    see = sees(par, base + T)[:, base:].cuda()
    for col in (3, 7, 9):
        assert not bool(torch.isfinite(o[:, :, col]).any())
    for col, t in ((64, node), (100, T - 1)):
        for h in range(Hq):
            assert torch.equal(torch.isfinite(o[:, h, col]), ~see[:, t])
    # the other columns are as without them
    cols = [3, 7, 9, 64, 100]
    cache.v[..., cols] = 0
    o[..., cols] = 0
    check(q, cache, o, lse, [0], [par], "bf16", 1 / math.sqrt(D), heads=[0, Hq - 1])
