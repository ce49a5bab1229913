"""Accepted rows where the layers' K and V pools lie in one buffer in different
orders: every order in which no pool lies over another is taken."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda"
BS = 16


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_52_gb300 import pagedkv
    pagedkv.get_device_error(clear=True)
    return pagedkv


def _bits(t):
    return t.contiguous().cpu().view(torch.int16).numpy()


@pytest.mark.parametrize("layers,k,kstep,v,vstep", [
    (4, 0, 2, 1, 2), (4, 1, 2, 0, 2), (4, 0, 1, 4, 1), (4, 4, 1, 0, 1), (4, 7, 1, 0, 2),
    (3, 0, 4, 1, 2), (3, 1, 2, 0, 4), (1, 0, 1, 1, 1), (1, 1, 1, 0, 1)])
def test_pools_in_one_buffer(pk, layers, k, kstep, v, vstep):
    # starts and steps in pools
    shape = (9, BS, 2, 64)
    pool = int(np.prod(shape))
    g = torch.Generator().manual_seed(layers + k)
    count = 1 + max(k + (layers - 1) * kstep, v + (layers - 1) * vstep)
    flat = torch.randn(count * pool, generator=g).bfloat16().to(DEV)
    stride = (BS * 128, 128, 64, 1)
    kc, vc = (flat.as_strided((layers, *shape), (step * pool, *stride), at * pool)
              for at, step in ((k, kstep), (v, vstep)))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    tables, lens, start = i32([[2, 7, 1], [3, 0, 8]]), i32([40, 33]), i32([0, 20, 30])
    path, n = i32([[1, 3, 4, 9, 19], [0, 5, 6, 0, 0]]), i32([5, 3])
    host = [x.cpu().numpy() for x in (tables, lens, start, path, n)]
    want_k, want = oracle.accept_rows(_bits(kc), *host)
    want_v, _ = oracle.accept_rows(_bits(vc), *host)
    before = flat.clone()
    if layers == 1:
        kc, vc = kc[0], vc[0]
    new = pk.kv_accept_rows(kc, vc, tables, lens, start, path, n)
    assert new.tolist() == want.tolist()
    assert np.array_equal(_bits(kc).reshape(want_k.shape), want_k)
    assert np.array_equal(_bits(vc).reshape(want_v.shape), want_v)
    used = {k + i * kstep for i in range(layers)} | {v + i * vstep for i in range(layers)}
    for i in set(range(count)) - used:  # pools between them that are not the call's
        assert torch.equal(flat[i * pool:(i + 1) * pool], before[i * pool:(i + 1) * pool])
    assert pk.get_device_error(clear=True) == 0
