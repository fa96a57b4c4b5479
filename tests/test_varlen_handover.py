"""The hand-over of units in attn_fwd_varlen_kernel, on a model of its barriers: every role comes
to its end whatever mix of units with and without keys a CTA gets, as it does not where units
without keys are handed out like the others."""
import itertools
import os
import random
import re

import pytest

import handover_model
from gqa_attention_forward_gb300 import build
from handover_model import Cta, blocks_in_order, units_of_ctas

KINDS = [(0, 0, 0), (1, 1, 0), (2, 2, 1), (0, 1, 0), (1, 0, 0), (2, 3, 1), (3, 3, 3)]


def finishes(units, hand_out_all=False):
    c = Cta(units, hand_out_all)
    done = c.run()
    if done:  # every unit stored once by either tile, in the order of the list, or by the scheduler
        assert len(c.units) + len(c.blind) == len(units)
        for i in range(2):
            assert [t for x, t in c.stored if x == i] == list(range(len(c.units)))
            assert c.scores[i] == [(t, j) for t, u in enumerate(c.units) for j in range(u[i])]
    return done


def test_the_model_has_the_kernels_numbers():
    with open(os.path.join(build.CSRC, "attn_fwd_varlen.cuh")) as f:
        text = f.read()
    with open(os.path.join(build.CSRC, "attn_fwd_ws.cuh")) as f:
        text += f.read()
    for name, value in (("kVlSlots", handover_model.SLOTS), ("kStagesWs", handover_model.STAGES)):
        assert int(re.search(rf"constexpr int {name} = (\d+);", text).group(1)) == value


@pytest.mark.parametrize("count", range(6))
def test_every_mix_finishes(count):
    for mix in itertools.product(KINDS, repeat=count):
        assert finishes(mix), mix


def test_long_lists_finish():
    rng = random.Random(1)
    for _ in range(300):
        kinds = rng.sample(KINDS, rng.randint(1, len(KINDS)))
        mix = rng.choices(kinds, k=rng.randint(6, 60))
        assert finishes(mix), mix


@pytest.mark.parametrize("tiles,ends", [([3, 0, 0], True), ([3, 0, 0, 0], False), ([3, 2, 1, 0, 0, 0, 0], False),
                                        ([0, 0, 0, 0, 0, 0], True), ([1, 0, 0, 0, 1], False)])
def test_a_look_past_units_without_keys_does_not_end(tiles, ends):
    """Handed out like the others, three of them behind a unit with keys make it wait for its own slot."""
    units = [(n, n, max(0, n - 1)) for n in tiles]
    assert finishes(units, hand_out_all=True) == ends
    assert finishes(units)


@pytest.mark.parametrize("lens_q,lens_k,causal", [
    ([8192], [512], True),                              # many queries, few keys
    ([6144], [1024], True),
    ([100] * 41, [300] + [0] * 40, False),              # one sequence with keys among many without
    ([1] * 64, [0] * 40 + [700] * 8 + [0] * 16, True),  # decoding rows, most without keys
    ([700, 260, 5, 130] * 20, [1, 300, 0, 131] * 20, True),
])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (6, 2)])
def test_calls_with_units_without_keys_finish(lens_q, lens_k, causal, Hq, Hkv):
    lists = units_of_ctas(lens_q, lens_k, Hq, Hkv, causal, 152)
    assert any(max(u[:2]) == 0 for x in lists for u in x)
    assert all(finishes(x) for x in lists)


def test_handing_out_all_units_would_not_finish_them():
    lists = units_of_ctas([8192], [512], 32, 8, True, 152)
    assert sum(not finishes(x, hand_out_all=True) for x in lists) == 64


@pytest.mark.parametrize("causal", [True, False])
def test_levels_hold_every_block_once(causal):
    rng = random.Random(2)
    for _ in range(50):
        n = rng.randint(1, 20)
        lens_q, lens_k = ([rng.choice([0, 1, 127, 128, 129, 300, 1000]) for _ in range(n)] for _ in range(2))
        order = blocks_in_order(lens_q, lens_k, 128, causal)
        assert sorted(order) == [(s, b) for s, x in enumerate(lens_q) for b in range(-(-x // 128))]
