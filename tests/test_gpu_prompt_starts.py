"""Packed rows whose starts are out of order, sequences with nothing new, and a scale of
0, in prompt attention, the block-scaled prefill and append.  Where starts fall, the
sequence that ends before it begins and all behind it are left out, so that no two
write one row (and the CTAs that share an item have one item each).  Tolerances:
test_gpu_prompt.py."""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_52_gb300 import workloads as wl
from test_gpu_prompt import BS, DEV, _cached, _check, _inputs, _prefill, _run, _start

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_52_gb300 import pagedkv
    pagedkv.get_device_error(clear=True)
    return pagedkv


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _check_taken(out, x, start, taken, hq, hkv, scale, step):
    """Sequences `taken` against float64 at every `step`-th row and the last; rows of
    no such sequence still 3."""
    free = np.ones(out.shape[0], bool)
    got = out.double().cpu().numpy()
    for s in taken:
        a, b = start[s], start[s + 1]
        free[a:b] = False
        k, v = x[a:b, hq:hq + hkv], x[a:b, hq + hkv:]
        for i in sorted(set(range(0, b - a, step)) | {b - a - 1}):
            _check(got[a + i:a + i + 1], x[a + i:a + i + 1, :hq], k, v, scale, i)
    assert (got[free] == 3.0).all()


@pytest.mark.parametrize("start,taken", [
    ([0, 2000, 100, 2100], [0]),              # the third begins inside the first
    ([0, 10000, 0, 10000], [0]),              # more items than the starts in order could have
    ([0, 300, 1200, 1100, 1900, 1950], [0, 1]),
    ([500, 400, 900, 800, 1000, 2000], []),
    ([0, 900, 5000, 1, 700, 2000], [0]),      # one beyond the rows before the fall
])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts_that_begin_inside_another(pk, start, taken, d):
    T = 10000 if max(start) == 10000 else 2100
    qkv = _inputs([T], 1, 1, d, seed=len(start))
    q, k, v = qkv.to(DEV).split(1, 1)
    out = torch.full((T, 1, d), 3.0, dtype=torch.bfloat16, device=DEV)
    pk.prompt_attention(q, _i32(start), k, v, True, 0.1, out=out)
    assert pk.get_device_error(clear=True) == 0x10
    _check_taken(out, qkv.double().numpy(), start, taken, 1, 1, 0.1, 331)


@pytest.mark.parametrize("count,at", [(40, 7), (40, 33), (700, 3), (700, 511), (700, 600)])
def test_many_prompts_with_one_start_out_of_order(pk, count, at):
    """Sequence `at` begins where it should, but the start after it is put back by 30
    rows: it and all behind it are left out, the others are there."""
    start = [10 * i for i in range(count + 1)]
    start[at + 1] -= 30
    qkv = _inputs([10 * count], 2, 1, 64, seed=at)
    q, k, v = qkv.to(DEV).split([2, 1, 1], 1)
    out = torch.full((10 * count, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    pk.prompt_attention(q, _i32(start), k, v, True, 0.1, out=out)
    assert pk.get_device_error(clear=True) == 0x10
    _check_taken(out, qkv.double().numpy(), start, range(at), 2, 1, 0.1, 9)


@pytest.mark.parametrize("hkv,d", [(1, 128), (2, 64)])
def test_prefill_of_chunks_that_begin_inside_another(pk, hkv, d):
    g = torch.Generator().manual_seed(d)
    lens, start = [2000, 40, 2050], [0, 2000, 100, 2100]
    cache = _cached(lens, hkv, d, g)
    q = torch.randn(2100, hkv, d, generator=g).bfloat16()
    tables, codes, scales = cache
    out = torch.full((2100, hkv, d), 3.0, dtype=torch.bfloat16, device=DEV)
    pk.paged_prefill_attention_fp8_block_scaled(
        q.to(DEV), _i32(start), *(x.to(DEV) for x in codes + scales), tables.to(DEV), _i32(lens),
        True, 0.02, out=out)
    assert pk.get_device_error(clear=True) == 0x10
    k, v = (oracle.dequantize_blocks(a.numpy(), b.numpy())[tables[0, :125].tolist()]
            .reshape(-1, hkv, d) for a, b in zip(codes, scales))
    got, x = out.double().cpu().numpy(), q.double().numpy()
    for i in list(range(0, 2000, 173)) + [1999]:
        _check(got[i:i + 1], x[i:i + 1], k, v, 0.02, i)
    assert (got[2000:] == 3.0).all()


@pytest.mark.parametrize("start,taken", [
    ([0, 20] * 20, [0]),
    ([0, 40, 30, 35, 41, 45, 60], [0]),
    ([5, 5, 2, 9, 8, 9, 30], []),
    ([10 * i if i != 301 else 2980 for i in range(700)], list(range(300))),
])
def test_append_of_sequences_that_begin_inside_another(pk, start, taken):
    hkv, d, S = 2, 64, len(start) - 1
    T = max(start) + 3
    lens = [max(0, b - a) + (7 * s) % 40 for s, (a, b) in enumerate(zip(start, start[1:]))]
    g = torch.Generator().manual_seed(S)
    tables, codes, scales = _cached(lens, hkv, d, g)
    k = torch.randn(T, hkv, d, generator=g).bfloat16()
    host = [codes[0].numpy(), codes[1].numpy(), scales[0].numpy(), scales[1].numpy()]
    bits = wl.bf16_bits(k)
    for s in taken:
        a, b = start[s], start[s + 1]
        host = oracle.append_block_scaled(bits[a:b], bits[a:b], [0, b - a], tables[s:s + 1].tolist(),
                                          lens[s:s + 1], *host)
    got = [x.to(DEV) for x in codes + scales]
    pk.kv_append_fp8_block_scaled(k.to(DEV), k.to(DEV), _i32(start), tables.to(DEV), _i32(lens), *got)
    assert pk.get_device_error(clear=True) == 0x10
    for a, b in zip(got, host):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_does_not_look_at_pages_of_sequences_without_rows(pk, d):
    """Their block tables may name anything, and their part of the workspace stays."""
    g = torch.Generator().manual_seed(d)
    counts, lens = [5, 0, 9, 0], [60, 100, 33, 500]
    c = dict(cache=_cached(lens, 2, d, g, width=32), counts=counts, lens=lens, scale=0.02,
             q=torch.randn(14, 4, d, generator=g).bfloat16())
    want = _prefill(pk, c)
    assert pk.get_device_error(clear=True) == 0
    c["cache"][0][1, :] = 10 ** 6
    c["cache"][0][3, :] = -7
    ws = pk.prefill_fp8_block_scaled_workspace(4, 32, 2, d, DEV)
    ws.fill_(0xa5)
    got = _prefill(pk, c, workspace=ws)
    assert pk.get_device_error(clear=True) == 0
    assert torch.equal(got, want)
    rows = ws.view(2, 4, -1)
    assert (rows[:, 1] == 0xa5).all() and (rows[:, 3] == 0xa5).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_scale_of_0_weighs_all_alike_whatever_the_scores(pk, d):
    lens = [200, 1, 700]
    qkv = _inputs(lens, 2, 1, d)
    qkv[:, :3] *= 2.0 ** 55                     # q k up to 2^120
    got = _run(pk, qkv, lens, 2, 1, scale=0.0).double().cpu().numpy()
    x = qkv.double().numpy()
    start = _start(lens).tolist()
    for s, n in enumerate(lens):
        for i in sorted({0, n // 3, n - 1}):
            a = start[s]
            _check(got[a + i:a + i + 1], x[a + i:a + i + 1, :2], x[a:a + n, 2:3], x[a:a + n, 3:],
                   0.0, i)
    assert pk.get_device_error(clear=True) == 0


def test_a_call_again_gives_the_same_bits(pk):
    for lens, hq, hkv, d in (([700, 3, 129], 8, 2, 128), ([4000], 2, 1, 128), ([90] * 60, 4, 4, 64)):
        qkv = _inputs(lens, hq, hkv, d)
        first = _run(pk, qkv, lens, hq, hkv)
        for _ in range(5):
            assert torch.equal(_run(pk, qkv, lens, hq, hkv), first)
