"""Sizes that the weighing and the eviction do not number in 32 bits are refused before a device is touched."""
import pytest

from gqa_attention_forward_gb300 import binding, build
from test_bounded_cache_host import evict, weigh
from test_packed_paged_host import NODEVICE, SHAPE, cache, no_gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


# rows, entries, layers, heads: their product is the number of evictions of one head; 2^28 of them are too many
MANY = dict(n_layers=1 << 10, Hkv=1 << 9, page=16, D=64, n_rows=1 << 10, table_width=4)


def test_evictions_are_numbered_in_32_bits():
    assert evict(cache(**MANY), n=1 << 9) == SHAPE
    assert evict(cache(**MANY), n=1 << 10, heavy=0, weights=None) == SHAPE
    assert evict(cache(n_layers=1, n_pages=1 << 20, Hkv=1, page=4096, D=64), n=1) == SHAPE  # 2^32 rows in a layer


def test_units_of_a_weighing_are_numbered_in_32_bits():
    c = dict(n_layers=1, Hkv=1 << 9, page=4096, D=64, n_rows=1 << 12, table_width=1 << 8)
    assert weigh(cache(**c), n=1 << 9, Hq=1 << 9) == SHAPE


def test_the_largest_reach_the_device_check():
    no_gpu()
    assert evict(cache(**MANY), n=(1 << 9) - 1) == NODEVICE
    assert evict(cache(n_layers=1, n_pages=(1 << 20) - 1, Hkv=1, page=4096, D=64), n=1) == NODEVICE
    c = dict(n_layers=1, Hkv=1 << 9, page=4096, D=64, n_rows=1 << 12, table_width=1 << 8)
    assert weigh(cache(**c), n=(1 << 9) - 1, Hq=1 << 9) == NODEVICE
