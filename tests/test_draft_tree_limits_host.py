"""Refusals of the speculative step's calls that need no GPU: sizes whose index
arithmetic would leave 32 bits, and arguments that lie over one another."""

import ctypes

import pytest

NULL, DUMMY = ctypes.c_void_p(0), ctypes.c_void_p(1 << 20)  # DUMMY is never dereferenced


@pytest.fixture(scope="module")
def pk():
    import os
    from paged_kv_cache_52_gb300 import build as b
    if not os.path.exists(b.LIB_PATH):
        b.build()
    from paged_kv_cache_52_gb300 import pagedkv
    return pagedkv


@pytest.mark.parametrize("seqs,blocks,heads,nodes,status", [
    # the workspace is too small throughout: -4 where the sizes are taken
    (1 << 28, 1, 2, 8, -4),             # 2^29 items of one tile: 3 places each
    ((1 << 28) + (1 << 27), 1, 2, 8, -2),
    (1 << 29, 7, 2, 8, -2),
    (1 << 20, 8, 2, 64, -4),            # one row group a tree
    (1 << 20, 16000, 2, 8, -2),
    (2, 112_000_000, 2, 8, -4),         # positions up to 1.8e9
    (2, (1 << 27) - 1, 2, 8, -2),       # their last tile's number times that of SMs
    (1, (1 << 31) - 1, 1, 1, -2),
])
def test_tree_attention_refuses_sizes_beyond_32_bits(pk, seqs, blocks, heads, nodes, status):
    desc = pk.CacheDesc(64, 16, heads, 64)
    for fn in (pk.lib.pkv_paged_tree_attention, pk.lib.pkv_paged_tree_attention_bf16out):
        assert fn(DUMMY, DUMMY, seqs, 9, nodes, 2 * heads, DUMMY, DUMMY, DUMMY, desc, DUMMY, blocks,
                  DUMMY, 0.1, DUMMY, DUMMY, 1000, NULL) == status


LAYER = 64 * 16 * 128 * 2  # bytes of a pool of the descriptor below


def _accept(pk, layers, k, kstep, v, vstep, new=1 << 24, tables=1 << 26):
    return pk.lib.pkv_kv_accept_rows(
        ctypes.c_void_p((1 << 30) + k), kstep // 2, ctypes.c_void_p((1 << 30) + v), vstep // 2,
        layers, pk.CacheDesc(64, 16, 2, 64), 2, ctypes.c_void_p(tables), 8, DUMMY, DUMMY, 2, DUMMY,
        4, DUMMY, ctypes.c_void_p(new), NULL)


# only layouts that are refused: the others would be launched
@pytest.mark.parametrize("layers,k,kstep,v,vstep", [
    (1, 0, 0, 0, 0),                              # one pool as both
    (1, 0, 0, LAYER - 16, 0),
    (1, LAYER - 16, 0, 0, 0),
    (5, 0, 2 * LAYER, LAYER + 16, 2 * LAYER),     # K and V of a layer side by side, but
    (5, 0, 2 * LAYER, LAYER - 16, 2 * LAYER),
    (5, 0, LAYER, 4 * LAYER, LAYER),              # all K, then all V, but
    (5, 8 * LAYER, LAYER, 0, 2 * LAYER),
    (3, 0, 4 * LAYER, LAYER, 3 * LAYER),          # K at 0 4 8, V at 1 4 7
])
def test_accept_rows_refuses_pools_that_lie_over_one_another(pk, layers, k, kstep, v, vstep):
    assert _accept(pk, layers, k, kstep, v, vstep) == -1


def test_accept_rows_refuses_lengths_that_lie_over_the_block_table(pk):
    for new in (1 << 24, (1 << 24) + 60):
        assert _accept(pk, 1, 0, 0, LAYER, 0, new=new, tables=1 << 24) == -1


@pytest.mark.parametrize("kstep,vstep", [(1 << 60, 2 * LAYER), (2 * LAYER, 1 << 60)])
def test_accept_rows_refuses_layers_that_no_address_reaches(pk, kstep, vstep):
    # the last of 64 layers would lie 2^66 bytes on
    assert _accept(pk, 64, 0, kstep, LAYER, vstep) == -1
