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


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("power", [-126, -130, -140])
def test_v_scales_down_to_subnormal_numbers(pk, way, power):
    """Equal weights, V's scales of 2^power: the mean, in float32's steps of 2^-149 and
    twice that for a piece's rounding before it is joined."""
    lens, width = WAYS[way]
    c = _decode_case(lens, 8, 2, 64, width=width)
    c["kc"] = torch.zeros_like(c["kc"])
    c["vs"] = torch.full_like(c["vs"], 2.0 ** power)
    assert (c["vs"] > 0).all()
    got = _bounded(pk, c).double().cpu().numpy()
    assert pk.get_device_error(clear=True) == 0
    for s in range(0, len(lens), 5 if len(lens) > 9 else 1):
        n = lens[s]
        if n:
            v = _values(c, s)
            want = np.repeat(v.mean(0), 4, axis=0)
            tol = np.repeat(np.abs(v).mean(0), 4, axis=0) * (n * 2.0 ** -23 + 2.0 ** -19)
            assert (np.abs(got[s] - want) <= tol + 3 * 2.0 ** -149).all(), (s, n)
            assert np.abs(got[s]).max() > 0


@pytest.mark.parametrize("S,n,width", [(1, 3000, None), (2, 60000, None), (300, 600, 40),
                                       (300, 500, 32)])
def test_many_small_weights_beside_a_large_one(pk, S, n, width):
    """One key of weight 1 and value 0, and n - 1 of weight 2^-26 and value 1.  A weight
    times its V scale is off by half a step of f16, 2^-11 of itself, or by 2^-39 of the
    row's largest such product; the score -26 and its exponential by 2^-17, a piece's
sum of 512 keys or fewer by 2^-14."""
    hkv, d = 2, 64
    lens = [n] * S
    g = torch.Generator().manual_seed(n)
    tables, blocks = _tables(lens, g, width)
    kc = torch.zeros(blocks, BS, hkv, d, dtype=torch.uint8)
    kc[..., 0] = 0xdd                                           # -26
    vc = torch.full_like(kc, 0x38)                              # 1
    first = tables[:, 0].long()
    kc[first, 3] = 0
    vc[first, 3] = 0
    one = torch.ones(blocks, hkv)
    q = torch.zeros(S, 4, d, dtype=torch.bfloat16)
    q[..., 0] = 1
    c = dict(q=q, kc=kc, vc=vc, ks=one, vs=one, tables=tables, lens=lens, scale=float(np.log(2.0)))
    got = _bounded(pk, c).double().cpu().numpy()
    assert oracle.dequantize_blocks(kc[:1].numpy(), one[:1].numpy()).min() == -26
    part = (n - 1) * 2.0 ** -26
    want = part / (1 + part)
    tol = want * (2.0 ** -11 + 2.0 ** -14 + 2.0 ** -17) + n * 2.0 ** -39
    assert np.abs(got - want).max() <= tol, (got.min(), got.max(), want)


# ------------------------------------------------- the flat split's own paths
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (8, 4, 128)])
def test_flat_decode_of_more_sequences_than_one_launch_holds(pk, hq, hkv, d):
    """Three launches of up to 1024 sequences, each joining its own pieces over the
    workspace of the one before."""
    lens = [(13 * i) % 50 for i in range(2100)]
    for s in (5, 1022, 1023, 1024, 1500, 2047, 2048, 2099):
        lens[s] = 500 + s % 37
    c = _decode_case(lens, hq, hkv, d, width=33)
    got = _bounded(pk, c)
    _check_rows(got.cpu().numpy(), c, list(range(0, 2100, 97)) +
                [5, 1022, 1023, 1024, 1025, 1500, 2047, 2048, 2049, 2098, 2099])
    assert torch.equal(_bounded(pk, c, out_dtype=torch.bfloat16), got.bfloat16())
    assert not got[torch.tensor(lens) == 0].any()
    assert pk.get_device_error(clear=True) == 0


def test_flat_decode_of_tables_whose_pages_pass_32_bits(pk):
    """17 sequences that might be of 2^27 - 1 pages each, 2^31 together and more: 16 to a
    launch, for the page counts' sums are 32-bit numbers."""
    lens = [300, 1, 0, 16, 17, 90] * 3
    lens = lens[:17]
    c = _decode_case(lens, 4, 2, 64)
    want = _decode(pk, c, max_context_len=300)
    wide = torch.empty(17, 2 ** 27 - 1, dtype=torch.int32, device=DEV)
    wide[:, :c["tables"].shape[1]] = c["tables"].to(DEV)
    got = pk.paged_decode_attention_fp8_block_scaled(
        *(c[x].to(DEV) for x in ("q", "kc", "vc", "ks", "vs")), wide,
        torch.tensor(lens, dtype=torch.int32, device=DEV), c["scale"],
        max_context_len=2 ** 31 - 1)
    _check_rows(got.cpu().numpy(), c, range(17))
    _check_rows(want.cpu().numpy(), c, range(17))
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("q_size", [1e-12, 2e-3, 3e4, 1e30])
def test_flat_decode_of_queries_outside_the_range_of_f16(pk, q_size):
    c = _decode_case(MANY, 8, 2, 128, q_size=q_size, width=40)
    _check_rows(_bounded(pk, c).cpu().numpy(), c, range(0, len(MANY), 9))
    assert pk.get_device_error(clear=True) == 0


def test_flat_decode_of_scales_far_apart(pk):
    c = _decode_case(MANY, 8, 2, 128, width=40)
    order = torch.arange(c["vs"].shape[0]) % 61
    c["vs"] = torch.exp2((order - 70).float())[:, None].expand(-1, 2).contiguous()
    _check_rows(_bounded(pk, c).cpu().numpy(), c, range(0, len(MANY), 9))
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_flat_decode_of_large_values_that_weigh_nothing(pk, d):
    """Every other block's values are 2^40 times the others' and its weights below
    2^-1000: the others' values come out."""
    c = _decode_case(MANY, 8, 2, d, spread=0.5, width=40)
    c["q"] = c["q"].abs() + 0.5
    low = torch.arange(c["kc"].shape[0]) % 2 == 0
    low[c["tables"][:, 0].clamp(min=0).long()] = False
    c["kc"] = torch.where(low[:, None, None, None], 0xf8, 0x38).to(torch.uint8).expand_as(
        c["kc"]).contiguous()                                   # -256 or 1
    c["ks"] = torch.where(low, 4.0, 2.0 ** -9)[:, None].repeat(1, 2)
    c["vs"] = torch.where(low, 2.0 ** 30, 2.0 ** -10)[:, None].repeat(1, 2)
    c["scale"] = 1.0                                            # scores of -d 1024 / 2 ln2 or less
    got = _bounded(pk, c).double().cpu().numpy()
    assert pk.get_device_error(clear=True) == 0
    for s in range(0, len(MANY), 9):
        if MANY[s]:
            c1 = dict(c, vc=torch.where(low[:, None, None, None], 0, c["vc"]).to(torch.uint8))
            k, v, kept = _values(c, s, "k"), _values(c1, s), _values(c, s, "k")[:, 0, 0] > 0
            want = np.repeat(v[kept].mean(0), 4, axis=0)        # their scores are equal
            tol = np.repeat(np.abs(v[kept]).mean(0), 4, axis=0) * (MANY[s] * 2.0 ** -23 + 2.0 ** -19)
            assert k[~kept].max(initial=-1024) == -1024
            assert (np.abs(got[s] - want) <= tol).all(), s


def test_a_call_again_gives_the_same_bits(pk):
    for lens, width in WAYS.values():
        c = _decode_case(lens, 8, 2, 128, width=width)
        first = _bounded(pk, c)
        for _ in range(5):
            assert torch.equal(_bounded(pk, c), first)
