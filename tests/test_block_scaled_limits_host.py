"""Sizes at which the block-scaled calls' index arithmetic ends, refused on the host
(nothing is dereferenced or launched)."""

import pytest

from test_block_scaled_host import EUNSUPPORTED, P, at, pk  # noqa: F401


@pytest.mark.parametrize("hkv", [2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1])
def test_copy_of_scales_of_more_heads_than_a_cache_has(pk, hkv):  # noqa: F811
    """Twice the heads, a pair's elements, is a 32-bit number."""
    c = pk.CacheDesc(1, 16, hkv, 64)
    assert pk.lib.pkv_copy_block_scales(at(1), at(2), c, at(3), 1, P(0)) == EUNSUPPORTED
