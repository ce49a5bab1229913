"""Prompt attention and the block-scaled prefill, against float64.

Tolerance: weights enter P V as bf16, off by 2^-8 of themselves (half a step of its 8 bits); scores are
float32 sums of exact products, d additions off by d 2^-24 sum |q k|, which
moves a weight (and their sum) by that times the scale; the exponential, the
sums and the division are within 2^-18; the output is rounded to bf16, 2^-8 of
itself.  |error| <= sum w |V| (2^-8 + 2 d 2^-24 max_j sum |q k_j| scale + 2^-18)
+ 2^-8 |out|, times 1 + 2^-6 for the products of these.
"""

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


def _start(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def _inputs(lens, hq, hkv, d, seed=0, extra=0):
    g = torch.Generator().manual_seed(seed)
    rows = int(sum(lens)) + extra
    qkv = torch.randn(rows, hq + 2 * hkv, d, generator=g)
    qkv[:, hq:] *= torch.exp2(0.7 * torch.randn(1, 2 * hkv, 1, generator=g))
    return qkv.bfloat16()


def _run(pk, qkv, lens, hq, hkv, causal=True, scale=None, **more):
    d = qkv.shape[-1]
    dev = qkv.to(DEV)
    q, k, v = dev.split([hq, hkv, hkv], 1)
    return pk.prompt_attention(q, _start(lens).to(DEV), k, v, causal,
                               d ** -0.5 if scale is None else scale, **more)


def _check(got, q, k, v, scale, first):
    """got, q [n, Hq, d] over k, v [L, Hkv, d], all float64 numpy."""
    d = q.shape[-1]
    want, size = oracle.attend(q, k, v, scale, first)
    g = q.shape[1] // k.shape[1]
    dots = np.stack([(np.abs(q[:, h]) @ np.abs(k[:, h // g]).T).max(1)
                     for h in range(q.shape[1])], 1)
    rel = 2.0 ** -8 + 2 * d * 2.0 ** -24 * dots * abs(scale) + 2.0 ** -18
    tol = (size * rel[..., None] + 2.0 ** -8 * np.abs(want)) * (1 + 2.0 ** -6) + 1e-38
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), float((err / tol).max())


def _check_prompts(got, qkv, lens, hq, hkv, causal=True, scale=None, rows=None):
    x = qkv.double().numpy()
    got = got.double().cpu().numpy()
    d = x.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    start = _start(lens).tolist()
    for s, n in enumerate(lens):
        a = start[s]
        k, v = x[a:a + n, hq:hq + hkv], x[a:a + n, hq + hkv:]
        for i in (range(0, n, 64) if rows is None else [r for r in rows if r < n]):
            b = min(n, i + (64 if rows is None else 1))
            _check(got[a + i:a + b], x[a + i:a + b, :hq], k, v, scale, i if causal else None)


SHAPES = [(1, 1, 128), (4, 4, 64), (8, 4, 128), (8, 2, 64), (16, 4, 128), (8, 1, 128), (16, 2, 64),
          (16, 1, 128), (16, 1, 64)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[1], [0, 37, 1, 0], [127, 128, 129]])
def test_short_prompts(pk, hq, hkv, d, causal, lens):
    qkv = _inputs(lens, hq, hkv, d, seed=hq + d)
    _check_prompts(_run(pk, qkv, lens, hq, hkv, causal), qkv, lens, hq, hkv, causal)
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (4, 1, 128), (8, 1, 64), (2, 2, 64)])
def test_prompts_of_many_tiles(pk, hq, hkv, d):
    lens = [1500, 3, 700, 256, 1025]
    qkv = _inputs(lens, hq, hkv, d, seed=1)
    rows = [0, 1, 31, 63, 64, 127, 128, 255, 256, 511, 512, 640, 699, 1024, 1279, 1499]
    _check_prompts(_run(pk, qkv, lens, hq, hkv), qkv, lens, hq, hkv, rows=rows)
    _check_prompts(_run(pk, qkv, lens, hq, hkv, False), qkv, lens, hq, hkv, False, rows=rows)
    assert pk.get_device_error(clear=True) == 0


def test_many_prompts(pk):
    lens = [(i * i * 7) % 150 for i in range(400)]
    qkv = _inputs(lens, 4, 2, 64)
    got = _run(pk, qkv, lens, 4, 2)
    start = _start(lens).tolist()
    x = qkv.double().numpy()
    out = got.double().cpu().numpy()
    for s in range(0, 400, 23):
        a, n = start[s], lens[s]
        if n:
            _check(out[a:a + n], x[a:a + n, :4], x[a:a + n, 4:6], x[a:a + n, 6:], 0.125, 0)
    # each prompt's rows do not depend on its neighbours
    s = 201
    alone = _run(pk, qkv[start[s]:start[s + 1]], [lens[s]], 4, 2)
    assert torch.equal(alone, got[start[s]:start[s + 1]])
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("causal", [True, False])
def test_more_prompts_than_one_warp_holds(pk, causal):
    """The items of the first 512 sequences are held, the others' found again."""
    lens = [(i * i * 11) % 70 for i in range(1100)]
    lens[700] = 400
    qkv = _inputs(lens, 4, 2, 64)
    got = _run(pk, qkv, lens, 4, 2, causal)
    start = _start(lens).tolist()
    for s in [0, 1, 31, 32, 33, 511, 512, 513, 700, 701, 1023, 1024, 1099]:
        alone = _run(pk, qkv[start[s]:start[s + 1]], [lens[s]], 4, 2, causal)
        assert torch.equal(alone, got[start[s]:start[s + 1]])
    rows = list(range(0, sum(lens), 501))
    _check_prompts(got, qkv, lens, 4, 2, causal, rows=rows)
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_maxima_that_rise_late(pk, d):
    """Scores far above the first keys' in every tile: the running maximum moves
    in the first and the second half of tiles, by more than the weights' range."""
    lens = [900]
    qkv = _inputs(lens, 2, 1, d, seed=4)
    for i, key in enumerate([40, 70, 127, 128, 200, 320, 500, 511, 650, 899]):
        qkv[key, 2] = qkv[key, 2] * (4 + 3 * i)
    _check_prompts(_run(pk, qkv, lens, 2, 1, scale=1.0), qkv, lens, 2, 1, scale=1.0)
    _check_prompts(_run(pk, qkv, lens, 2, 1, False, scale=-0.7), qkv, lens, 2, 1, False, scale=-0.7)
    _check_prompts(_run(pk, qkv, lens, 2, 1, scale=0.0), qkv, lens, 2, 1, scale=0.0)
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (2, 2, 64), (16, 1, 128)])
def test_what_a_row_does_not_see_never_reaches_it(pk, hq, hkv, d):
    """NaN and infinities in other prompts, behind the last one, and in V of later
    tokens; rows of no prompt keep what they held."""
    lens = [130, 200, 61]
    extra = 150
    qkv = _inputs(lens, hq, hkv, d, seed=2, extra=extra)
    want = _run(pk, qkv, lens, hq, hkv)
    bad = qkv.clone()
    bad[130:330] = float("nan")          # the whole second prompt
    bad[391:] = float("inf")             # nobody's rows
    bad[100, hq + hkv:] = float("nan")   # V of token 100 of the first
    bad[350, hq + hkv:, 5] = float("-inf")   # an element of V of token 20 of the third
    out = torch.full((391 + extra, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    got = _run(pk, bad, lens, hq, hkv, out=out)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(got[:100], want[:100])
    assert torch.isnan(got[100:130]).all()
    assert torch.isnan(got[130:330]).all()
    assert torch.equal(got[330:350], want[330:350])
    seen, ref = got[350:391], want[350:391]
    assert (seen[..., 5] == float("-inf")).all()
    assert torch.equal(seen[..., :5], ref[..., :5]) and torch.equal(seen[..., 6:], ref[..., 6:])
    assert (got[391:] == 7.0).all()
    assert pk.get_device_error(clear=True) == 0


def test_nan_in_a_visible_key_or_query(pk):
    lens = [300]
    qkv = _inputs(lens, 2, 1, 128)
    want = _run(pk, qkv, lens, 2, 1)
    bad = qkv.clone()
    bad[150, 2] = float("nan")      # K of token 150
    got = _run(pk, bad, lens, 2, 1)
    assert torch.equal(got[:150], want[:150]) and torch.isnan(got[150:]).all()
    bad = qkv.clone()
    bad[70, 1, 3] = float("nan")    # an element of a query
    got = _run(pk, bad, lens, 2, 1)
    assert torch.isnan(got[70, 1]).all()
    got[70, 1] = want[70, 1]
    assert torch.equal(got, want)


def test_contiguous_inputs_equal_views(pk):
    lens = [77, 130]
    qkv = _inputs(lens, 8, 2, 128)
    want = _run(pk, qkv, lens, 8, 2)
    q, k, v = (x.contiguous() for x in qkv.to(DEV).split([8, 2, 2], 1))
    assert torch.equal(pk.prompt_attention(q, _start(lens).to(DEV), k, v, True, 128 ** -0.5), want)


def test_starts_out_of_order_leave_their_sequences_out(pk):
    qkv = _inputs([100], 4, 2, 64).to(DEV)
    q, k, v = qkv.split([4, 2, 2], 1)
    out = torch.full((100, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    start = torch.tensor([0, 20, 10, 40, 101], dtype=torch.int32, device=DEV)
    pk.prompt_attention(q, start, k, v, True, 0.1, out=out)
    assert pk.get_device_error(clear=True) == 0x10
    want = pk.prompt_attention(q[:20], start[:2], k[:20], v[:20], True, 0.1)
    assert torch.equal(out[:10], want[:10])
    assert torch.isfinite(out).all() and (out[40:] == 3.0).all()


# ------------------------------------------------ over a block-scaled cache
def _cached(lens, hkv, d, g, width=None):
    need = [-(-int(x) // BS) for x in lens]
    blocks = sum(need) + 3
    perm = (torch.randperm(blocks - 1, generator=g) + 1).to(torch.int32)
    tables = torch.full((len(lens), width or max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = perm[at:at + n]
        at += n
    codes = [torch.randint(0, 256, (blocks, BS, hkv, d), generator=g, dtype=torch.int32)
             .to(torch.uint8) for _ in range(2)]
    codes = [torch.where((c & 0x7f) == 0x7f, c - 1, c) for c in codes]
    scales = [torch.exp2(torch.randint(-9, -4, (blocks, hkv), generator=g).float())
              for _ in range(2)]
    for s, n in enumerate(lens):  # behind the end: NaN
        if n % BS:
            for c in codes:
                c[int(tables[s, n // BS]), n % BS:] = 0x7f
    return tables, codes, scales


def _prefill(pk, c, causal=True, **more):
    tables, (kc, vc), (ks, vs) = c["cache"]
    dev = lambda x: x.to(DEV)
    return pk.paged_prefill_attention_fp8_block_scaled(
        dev(c["q"]), dev(_start(c["counts"])), dev(kc), dev(vc), dev(ks), dev(vs), dev(tables),
        torch.tensor(c["lens"], dtype=torch.int32, device=DEV), causal, c["scale"], **more)


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (4, 1, 64), (16, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("counts,lens", [([1], [1]), ([5, 0, 1, 130], [21, 40, 16, 500]),
                                         ([64, 129, 3], [64, 300, 1030])])
def test_prefill_over_a_block_scaled_cache(pk, hq, hkv, d, causal, counts, lens):
    g = torch.Generator().manual_seed(hq + len(lens))
    c = dict(cache=_cached(lens, hkv, d, g, width=70), counts=counts, lens=lens, scale=0.02,
             q=torch.randn(sum(counts), hq, d, generator=g).bfloat16())
    ws = pk.prefill_fp8_block_scaled_workspace(len(lens), 70, hkv, d, DEV)
    ws.fill_(0xff)  # NaN wherever the pages are not widened
    got = _prefill(pk, c, causal, workspace=ws).double().cpu().numpy()
    tables, (kc, vc), (ks, vs) = c["cache"]
    kd, vd = (oracle.dequantize_blocks(a.numpy(), b.numpy()) for a, b in ((kc, ks), (vc, vs)))
    start = _start(counts).tolist()
    for s, (n, L) in enumerate(zip(counts, lens)):
        pages = tables[s, :-(-L // BS)].tolist()
        k, v = (x[pages].reshape(-1, hkv, d)[:L] for x in (kd, vd))
        q = c["q"][start[s]:start[s + 1]].double().numpy()
        if n:
            _check(got[start[s]:start[s + 1]], q, k, v, 0.02, L - n if causal else None)
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (2, 2, 64), (16, 1, 64)])
@pytest.mark.parametrize("counts,lens", [([8], [5000]), ([1], [1025]), ([300], [2000]),
                                         ([20, 1], [700, 3])])
def test_items_shared_by_several_ctas(pk, hq, hkv, d, counts, lens):
    """Few rows against many keys, so that CTAs share an item: some of them without a
    key that a row sees, or without a tile of the second half of the rows."""
    g = torch.Generator().manual_seed(hq)
    c = dict(cache=_cached(lens, hkv, d, g), counts=counts, lens=lens, scale=0.03,
             q=torch.randn(sum(counts), hq, d, generator=g).bfloat16())
    got = _prefill(pk, c).double().cpu().numpy()
    tables, (kc, vc), (ks, vs) = c["cache"]
    kd, vd = (oracle.dequantize_blocks(a.numpy(), b.numpy()) for a, b in ((kc, ks), (vc, vs)))
    start = _start(counts).tolist()
    for s, (n, L) in enumerate(zip(counts, lens)):
        pages = tables[s, :-(-L // BS)].tolist()
        k, v = (x[pages].reshape(-1, hkv, d)[:L] for x in (kd, vd))
        q = c["q"][start[s]:start[s + 1]].double().numpy()
        for i in range(0, n, 37):
            _check(got[start[s] + i:start[s] + i + 1], q[i:i + 1], k, v, 0.03, L - n + i)
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_nonfinite_values_in_shared_items(pk, d):
    lens = [1900]
    qkv = _inputs(lens, 2, 1, d)
    want = _run(pk, qkv, lens, 2, 1)
    bad = qkv.clone()
    bad[1850, 3, 7] = float("inf")
    got = _run(pk, bad, lens, 2, 1)
    assert torch.equal(got[:1850], want[:1850])
    assert (got[1850:, :, 7] == float("inf")).all()
    assert torch.equal(got[1850:, :, :7], want[1850:, :, :7])


def test_prefill_rejects_bad_sequences(pk):
    g = torch.Generator().manual_seed(0)
    lens = [40, 100, 64, 32]
    cache = _cached(lens, 2, 64, g, width=7)
    counts = [8, 8, 8, 8]
    q = torch.randn(32, 4, 64, generator=g).bfloat16()
    c = dict(cache=cache, counts=counts, lens=lens, scale=0.02, q=q)
    want = _prefill(pk, c)
    assert pk.get_device_error(clear=True) == 0
    c["lens"] = [7, 113, 64, 0]      # shorter than the chunk, beyond the table, -, none
    out = torch.full((32, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    _prefill(pk, c, out=out)
    assert pk.get_device_error(clear=True) & 0x10
    assert torch.equal(out[16:24], want[16:24])
    assert (out[:16] == 5.0).all() and (out[24:] == 5.0).all()
    c["lens"] = lens
    cache[0][2, 1] = 10 ** 6
    got = _prefill(pk, c)
    assert pk.get_device_error(clear=True) == 0x2
    assert torch.equal(got[:16], want[:16]) and torch.isfinite(got).all()
