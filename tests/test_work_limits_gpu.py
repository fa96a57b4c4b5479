"""Offsets that ask for more work than ascending ones can: what lies behind the limit is not done,
seen by the rows that stay as they were."""
import pytest
import torch

from gqa_attention_forward_gb300 import binding
from handover_model import blocks_in_order
from packed_util import offsets
from paged_util import build

pytestmark = pytest.mark.gpu


def status():
    return binding.attn_last_device_error(torch.cuda.current_stream())


@pytest.mark.parametrize("Hq,Hkv,block", [(4, 2, 128), (3, 1, 256)])
def test_packed_blocks_end_at_what_ascending_offsets_can_have(Hq, Hkv, block):
    """40 sequences over the same 600 rows and one of one row: the rows of the order's first
    total_q / block + n_seqs blocks are written and no others, that one row not among them."""
    cu = [0, 600] * 40 + [601]
    n = len(cu) - 1
    lens = [max(0, b - a) for a, b in zip(cu, cu[1:])]
    order = blocks_in_order(lens, lens, block, True)
    limit = 601 // block + n
    assert order[-1] == (n - 1, 0) and len(order) > limit
    torch.manual_seed(95)
    q = torch.randn(601, Hq, 64, device="cuda").half()
    k = torch.randn(601, Hkv, 64, device="cuda").half()
    for given in (cu, [0, 600, 601]):  # and ascending ones, with which all rows are written
        o, lse = torch.full_like(q, 7.0), torch.full((Hq, 601), 7.0, device="cuda")
        binding.attention_varlen(q, k, k, torch.tensor(given, dtype=torch.int32, device="cuda"), out=o, lse_out=lse)
        written = torch.zeros(601, dtype=torch.bool, device="cuda")
        if given is cu:
            assert status() == binding.ATTN_ERR_SHAPE
            for s, b in order[:limit]:
                written[cu[s] + b * block:min(cu[s] + (b + 1) * block, cu[s] + lens[s])] = True
            assert not bool(written[600])
        else:
            assert status() == binding.ATTN_OK
            written[:] = True
        assert torch.equal(~(o == 7).all(2), written[:, None].expand(601, Hq))
        assert torch.equal(lse != 7, written.expand(Hq, 601))


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (128, 2)])
def test_trees_end_at_128_tokens(Hq, Hkv):
    """A tree of 300 tokens is cut: the queries behind its first 128 are not computed."""
    cache = build([1000, 500], 32, Hkv, 64, "f16", seed=91)
    torch.manual_seed(96)
    q = torch.randn(305, Hq, 64, device="cuda").half()
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, 305), 7.0, device="cuda")
    binding.attention_tree(q, cache, offsets([300, 5]), out=o, lse_out=lse)
    assert status() == binding.ATTN_ERR_SHAPE
    assert bool((o[128:300] == 7).all()) and bool((lse[:, 128:300] == 7).all())
    assert not bool((o[:128] == 7).all(2).any()) and not bool((o[300:] == 7).all(2).any())
