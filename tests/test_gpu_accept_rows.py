"""The accepted path's rows moved in place, bit for bit against the oracle."""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_52_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"
BS = 16


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_52_gb300 import pagedkv
    pagedkv.get_device_error(clear=True)
    return pagedkv


def _case(layers, hkv, d, dtype, nodes, lens, counts, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    need = sum(-(-x // BS) for x in lens) + 3
    tables, _ = wl.build_block_tables(lens, torch.randperm(need, generator=g))
    pools = [torch.randint(0, 255, (layers, need, BS, hkv, d), generator=g, dtype=torch.uint8)
             for _ in range(2)]
    if dtype == torch.bfloat16:
        pools = [torch.randn(layers, need, BS, hkv, d, generator=g).bfloat16() for _ in range(2)]
    width = max(counts + [1])
    accepted = np.full((len(nodes), width), 99, dtype=np.int32)  # past the count: not read
    for s, (n, c) in enumerate(zip(nodes, counts)):
        accepted[s, :c] = np.sort(rng.choice(n, size=c, replace=False))
    q_start = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    return pools, tables, np.array(lens, dtype=np.int32), q_start, accepted, np.array(counts, dtype=np.int32)


def _dev(*xs):
    return [(torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(DEV) for x in xs]


def _np(t):
    t = t.cpu()
    return t.view(torch.int16).numpy() if t.dtype == torch.bfloat16 else t.numpy()


@pytest.mark.parametrize("layers,hkv,d", [(1, 8, 128), (3, 2, 64), (2, 32, 128), (1, 1, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8])
def test_rows_move_in_place(pk, layers, hkv, d, dtype):
    nodes = [64, 64, 10, 1, 1, 0, 33, 20]
    counts = [64, 13, 10, 0, 1, 0, 17, 9]      # whole trees, none, and paths that overlap themselves
    lens = [64, 100, 40, 17, 1, 5, 161, 300]
    pools, tables, lens, q_start, accepted, counts = _case(layers, hkv, d, dtype, nodes, lens,
                                                           counts, layers + hkv)
    (k, v) = pools
    k_ref, new = oracle.accept_rows(_np(k), tables.numpy(), lens, q_start, accepted, counts)
    v_ref, _ = oracle.accept_rows(_np(v), tables.numpy(), lens, q_start, accepted, counts)
    kd, vd = k.to(DEV), v.to(DEV)
    if layers == 1:
        kd, vd = kd[0], vd[0]
    got = pk.kv_accept_rows(kd, vd, *_dev(tables, lens, q_start, accepted, counts))
    torch.cuda.synchronize()
    assert pk.get_device_error(clear=True) == 0
    assert np.array_equal(_np(kd).reshape(k_ref.shape), k_ref)
    assert np.array_equal(_np(vd).reshape(v_ref.shape), v_ref)
    assert got.cpu().tolist() == new.tolist()


def test_layers_interleaved_in_one_tensor(pk):
    # one tensor [layers, 2, ...]: K and V of a layer side by side
    pools, tables, lens, q_start, accepted, counts = _case(4, 2, 64, torch.bfloat16, [9, 30],
                                                           [50, 90], [4, 8], 5)
    kv = torch.stack(pools, 1).to(DEV)
    refs = [oracle.accept_rows(_np(p), tables.numpy(), lens, q_start, accepted, counts)[0]
            for p in pools]
    pk.kv_accept_rows(kv[:, 0], kv[:, 1], *_dev(tables, lens, q_start, accepted, counts))
    for i in range(2):
        assert np.array_equal(_np(kv[:, i].contiguous()), refs[i])


def test_bad_paths_change_nothing_and_are_flagged(pk):
    nodes, lens = [6] * 7, [40] * 7
    pools, tables, lens, q_start, accepted, counts = _case(1, 2, 64, torch.bfloat16, nodes, lens,
                                                           [3] * 7, 6)
    accepted[:] = [0, 2, 5]
    accepted[1] = [2, 2, 5]     # the same node twice
    accepted[2] = [3, 2, 5]     # not increasing
    accepted[3] = [0, 2, 6]     # beyond the tree
    accepted[4] = [-1, 2, 5]
    counts[5] = 4               # more than accepted holds
    counts[6] = -1
    k, v = (p[0].to(DEV) for p in pools)
    new = pk.kv_accept_rows(k, v, *_dev(tables, lens, q_start, accepted, counts))
    torch.cuda.synchronize()
    assert pk.get_device_error(clear=True) == 0x400
    assert new.tolist() == [37] + [40] * 6
    good = counts.copy()
    good[1:] = 0
    ref, _ = oracle.accept_rows(_np(pools[0]), tables.numpy(), lens, q_start, accepted, good)
    assert np.array_equal(_np(k), ref[0])


def test_bad_block_ids_are_skipped_and_flagged(pk):
    pools, tables, lens, q_start, accepted, counts = _case(1, 2, 64, torch.bfloat16, [20], [40],
                                                           [2], 7)
    accepted[0] = [5, 15]       # positions 25 -> 20 and 35 -> 21
    tables[0, 2] = 10 ** 6      # positions 32 .. 47
    k, v = (p[0].to(DEV) for p in pools)
    new = pk.kv_accept_rows(k, v, *_dev(tables, lens, q_start, accepted, counts))
    torch.cuda.synchronize()
    assert pk.get_device_error(clear=True) == 0x2 and new.tolist() == [22]
    ref = _np(pools[0][0]).copy()
    ref[tables[0, 1], 4] = ref[tables[0, 1], 9]
    assert np.array_equal(_np(k), ref)


def test_refusals_and_empty_calls(pk):
    pools, tables, lens, q_start, accepted, counts = _case(2, 2, 64, torch.bfloat16, [5, 5],
                                                           [20, 20], [2, 2], 8)
    k, v = (p.to(DEV) for p in pools)
    args = _dev(tables, lens, q_start, accepted, counts)
    with pytest.raises(pk.PagedKVError):            # the lengths in place
        pk.kv_accept_rows(k, v, *args, new_context_lens=args[1])
    for bad in ((k, v.to(torch.uint8)), (k.float(), v.float()), (k[:, :, ::2], v[:, :, ::2]),
                (k[0], v)):
        with pytest.raises(ValueError):
            pk.kv_accept_rows(*bad, *args)
    with pytest.raises(ValueError):
        pk.kv_accept_rows(k, v, args[0], args[1].long(), *args[2:])
    none = pk.kv_accept_rows(k, v, args[0][:0], args[1][:0], args[2][:1], args[3][:0], args[4][:0])
    assert none.numel() == 0
    no_path = pk.kv_accept_rows(k, v, *args[:3], args[3][:, :0].contiguous(), args[4] * 0)
    assert no_path.tolist() == [15, 15] and torch.equal(k.cpu(), pools[0])
