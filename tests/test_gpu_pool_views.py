"""The speculative step's calls take every view of a pool that is contiguous, and
refuse pools without layers."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_52_gb300 import pagedkv
    pagedkv.get_device_error(clear=True)
    return pagedkv


def _views(pool):
    """``pool [NB, 16, 1, d]`` and views of it with other strides in dimensions of one
    element: heads before tokens, and a part of more heads."""
    nb, bs, _, d = pool.shape
    heads_first = pool.view(nb, 1, bs, d).transpose(1, 2)
    unsqueezed = pool.view(nb, bs, d).as_strided((nb, bs, 1, d), (bs * d, d, 7, 1))
    for x in (heads_first, unsqueezed):
        assert x.is_contiguous() and x.stride() != pool.stride()
    return [pool, heads_first, unsqueezed]


def test_one_kv_head_in_any_contiguous_view(pk):
    d, n = 64, 5
    g = torch.Generator().manual_seed(0)
    k0, v0 = (torch.randn(6, 16, 1, d, generator=g).bfloat16().to(DEV) for _ in range(2))
    q = torch.randn(n, 4, d, generator=g).bfloat16().to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    start, lens, tables = i32([0, n]), i32([40]), i32([[4, 0, 2]])
    mask = torch.tensor([1, 3, 5, 9, 17], device=DEV)
    table = torch.randn(64, d, generator=g).to(DEV)
    slots = torch.tensor([3, 17, 40, -1, 95], device=DEV)
    got = []
    for i in range(3):
        kc, vc = k0.clone(), v0.clone()
        kv, vv = _views(kc)[i], _views(vc)[i]
        x = pk.qk_norm_rope_append(q, q[:, :1], q[:, 1:2], slots * 0 + 9, table, slots, kv, vv)
        out = pk.paged_tree_attention(x, start, mask, kv, vv, tables, lens, 0.1, max_q_len=n)
        new = pk.kv_accept_rows(kv, vv, tables, lens, start, i32([[0, 2, 4]]), i32([3]))
        layer = pk.kv_accept_rows(kv[None], vv[None], tables, lens, start, i32([[1, 2, 3]]), i32([2]))
        got.append([x, out, new, layer, kc, vc])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(other, got[0]))
    assert not torch.equal(got[0][4], k0)
    assert pk.get_device_error(clear=True) == 0


def test_pools_without_layers_and_strided_ones_are_refused(pk):
    k = torch.zeros(2, 6, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    args = (i32([[0]]), i32([4]), i32([0, 2]), i32([[1]]), i32([1]))
    for bad in (k[:0], k[:, ::2], k[:, :, :, :1], k[..., :32]):
        with pytest.raises(ValueError):
            pk.kv_accept_rows(bad, bad.clone() if bad.is_contiguous() else bad, *args)


@pytest.mark.parametrize("T", [3, 700])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_norm_for_queries_or_keys_alone(pk, T, fp8):
    # the side with a weight is as with both, the side without as with none
    g = torch.Generator().manual_seed(T)
    hq, hkv, d = 8, 4, 128
    qkv = torch.randn(T, hq + 2 * hkv, d, generator=g).bfloat16().to(DEV)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    table = torch.randn(64, d, generator=g).to(DEV)
    pos = torch.randint(0, 64, (T,), generator=g).to(DEV)
    slots = torch.randperm(T, generator=g).to(DEV)
    w = (torch.rand(d, generator=g) + 0.5).bfloat16().to(DEV)
    blocks = -(-T // 16)

    def run(qw, kw):
        kc, vc = (torch.zeros(blocks, 16, hkv, d, device=DEV,
                              dtype=torch.uint8 if fp8 else torch.bfloat16) for _ in range(2))
        call = pk.qk_norm_rope_append_fp8 if fp8 else pk.qk_norm_rope_append
        scales = (0.02, 0.03) if fp8 else ()
        return call(q, k, v, pos, table, slots, kc, vc, *scales, q_weight=qw, k_weight=kw), kc, vc

    both, none, q_only, k_only = run(w, w), run(None, None), run(w, None), run(None, w)
    assert not torch.equal(both[0], none[0]) and not torch.equal(both[1], none[1])
    for got, want_q, want_k in ((q_only, both, none), (k_only, none, both)):
        assert torch.equal(got[0], want_q[0]) and torch.equal(got[1], want_k[1])
        assert torch.equal(got[2], both[2])
    assert pk.get_device_error(clear=True) == 0
