"""Prompt attention and the block-scaled prefill where scores are large.

Scores are float32.  Where those of a row are equal its weights are equal whatever
their size, so it is the mean of what it sees: weights of one value, which bf16 may
round by 2^-8 (and all alike), float32 sums of n additions, and an output rounded to
bf16, 2^-8 of itself."""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_prompt import DEV, _cached, _inputs, _prefill, _run, _start

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_52_gb300 import pagedkv
    pagedkv.get_device_error(clear=True)
    return pagedkv


# eight bits, all of bf16's, which no power of two's product has: scores times a scale
# are rounded
ODD = 149 / 128


def _is_mean(got, v, n):
    tol = (2.0 ** -8 + n * 2.0 ** -23 + 2.0 ** -18) * np.abs(v).mean(0)
    tol = (tol + 2.0 ** -8 * np.abs(v.mean(0))) * (1 + 2.0 ** -6)
    assert (np.abs(got - v.mean(0)) <= tol).all(), (got, v.mean(0))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [20, 26, 31, 45, 60])
@pytest.mark.parametrize("lens", [[200, 1, 37], [2100], [300] * 40])
def test_equal_scores_of_any_size_give_the_mean(pk, d, size, lens):
    """Scores of -2^size and 2^size, about, in log2 units, by the head."""
    qkv = _inputs(lens, 2, 1, d, seed=size)
    qkv[:, 0], qkv[:, 1] = ODD * 2.0 ** (size - 20), -ODD * 2.0 ** (size - 20)
    qkv[:, 2] = 1
    scale = 1.2345 * 2.0 ** 20 / d
    got = _run(pk, qkv, lens, 2, 1, scale=scale).double().cpu().numpy()
    v = qkv[:, 3].double().numpy()
    start = _start(lens).tolist()
    for s in range(0, len(lens), 7):
        for i in sorted({0, lens[s] // 2, lens[s] - 1}):
            for h in range(2):
                _is_mean(got[start[s] + i, h], v[start[s]:start[s] + i + 1], i + 1)
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_become_large_late(pk, d):
    """Keys of ordinary scores, then one in each of several tiles that outweighs all
    before it: from it on rows are its value, until the next."""
    n = 900
    qkv = _inputs([n], 1, 1, d)
    qkv[:, 0], qkv[:, 1] = 1, 2.0 ** -10
    peaks = {150: 2.0 ** 5, 300: 2.0 ** 15, 500: 2.0 ** 30, 511: 2.0 ** 31, 700: 2.0 ** 40}
    for i, size in peaks.items():
        qkv[i, 1] = ODD * size
    got = _run(pk, qkv, [n], 1, 1, scale=1.2345).double().cpu().numpy()
    v = qkv[:, 2].double().numpy()
    for i in list(range(0, 150, 13)):
        _is_mean(got[i, 0], v[:i + 1], i + 1)
    for i in list(range(150, n, 11)) + [299, 300, 499, 500, 511, 699, 700, n - 1]:
        last = max(x for x in peaks if x <= i)
        _is_mean(got[i, 0], v[last:last + 1], 1)
    # rows beside them in a tile are what they are without them
    calm = qkv.clone()
    for i in peaks:
        calm[i, 1] = 2.0 ** -10
    assert torch.equal(_run(pk, calm, [n], 1, 1, scale=1.2345)[:150].double().cpu(),
                       torch.from_numpy(got[:150]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("counts,lens", [([8], [5000]), ([20, 1], [700, 3])])
def test_prefill_of_large_equal_scores(pk, d, counts, lens):
    g = torch.Generator().manual_seed(d)
    tables, (kc, vc), (ks, vs) = _cached(lens, 1, d, g)
    kc, ks = torch.full_like(kc, 0x38), torch.ones_like(ks)
    q = torch.full((sum(counts), 2, d), ODD * 2.0 ** 12).bfloat16()
    q[:, 1] *= -1
    c = dict(cache=(tables, (kc, vc), (ks, vs)), counts=counts, lens=lens, q=q,
             scale=1.2345 * 2.0 ** 20 / d)
    got = _prefill(pk, c).double().cpu().numpy()
    vd = oracle.dequantize_blocks(vc.numpy(), vs.numpy())
    start = _start(counts).tolist()
    for s, (n, L) in enumerate(zip(counts, lens)):
        v = vd[tables[s, :-(-L // 16)].tolist()].reshape(-1, d)[:L]
        for i in range(n):
            for h in range(2):
                _is_mean(got[start[s] + i, h], v[:L - n + i + 1], L - n + i + 1)
    assert pk.get_device_error(clear=True) == 0
