"""The block-scaled decode where scores are large, keys are many and scales lie far
apart, through all three of its splits.

Splits: a table of up to 32 pages and few pairs give a cluster a pair; many pairs a
warp each; a table of more than 32 pages with many pairs (or a long one) the
flat split.  ``WAYS`` reaches each.

Scores are float32.  Where the scores of a row are equal their weights are
equal whatever their size, so such a row is the mean of its values: the weights,
1 times a power of two, enter P V as they are, and what is left is the float32 sums
(n additions of 2^-23 each at most), and the factors and divisions of the joins
(2^-19).
"""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_block_scaled import BS, DEV, _check_rows, _decode, _decode_case, _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_52_gb300 import pagedkv
    pagedkv.get_device_error(clear=True)
    return pagedkv


MANY = [(29 * i) % 200 for i in range(260)]
WAYS = {"cluster": ([300, 90, 1, 17], None), "pairs": (MANY, None), "flat": (MANY, 40)}


def _bounded(pk, c, **more):
    return _decode(pk, c, max_context_len=BS * c["tables"].shape[1], **more)


def _values(c, s, x="v"):
    n = c["lens"][s]
    pages = c["tables"][s, :-(-n // BS)].long()
    v = oracle.dequantize_blocks(c[x + "c"][pages].numpy(), c[x + "s"][pages].numpy())
    return v.reshape(-1, *v.shape[2:])[:n]


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [20, 31, 60])
@pytest.mark.parametrize("power", [-100, -30, 20, 100])
def test_equal_scores_of_any_size_give_the_mean(pk, way, d, size, power):
    """Every key's score is -2^size or 2^size in log2 units, V's scales about 2^power."""
    lens, width = WAYS[way]
    c = _decode_case(lens, 8, 2, d, seed=d, width=width)
    c["kc"] = torch.full_like(c["kc"], 0x38)                    # 1.0
    c["ks"] = torch.ones_like(c["ks"])
    c["vs"] = torch.exp2((torch.arange(c["vs"].shape[0]) % 5 + power).float())[:, None].repeat(1, 2)
    c["q"] = torch.full_like(c["q"], 2.0 ** (size - 20))
    c["q"][:, ::2] *= -1
    c["scale"] = 2.0 ** 20 / d / np.log2(np.e)
    got = _bounded(pk, c).double().cpu().numpy()
    assert pk.get_device_error(clear=True) == 0
    for s in range(0, len(lens), 5 if len(lens) > 9 else 1):
        n = lens[s]
        if n == 0:
            assert not got[s].any()
            continue
        v = _values(c, s)
        want = np.repeat(v.mean(0), 4, axis=0)
        tol = np.repeat(np.abs(v).mean(0), 4, axis=0) * (n * 2.0 ** -23 + 2.0 ** -19)
        assert (np.abs(got[s] - want) <= tol).all(), (s, n, got[s, :, 0], want[:, 0])
