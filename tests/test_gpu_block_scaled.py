"""The block-scaled FP8 cache on the GPU: the append bit for bit, the decode
against float64.

Tolerance of the decode: the weights (at most 1 before they are divided by
their sum, which is at least 1) enter the second product as f16, off by 2^-11
of themselves, and by 2^-25 of the largest V scale times 448 where they are
subnormal, at most 2 max|V| for each of the n keys.  Scores are float32 sums
of exact products: d additions are off by d 2^-24 of sum |q k|, which moves a
weight by that times the scale.  The exponential and the final division are
within 2^-20.  So |error| <= sum w |V| (2^-11 + 2 d 2^-24 max_j sum |q k_j|
scale + 2^-18) + n 2^-24 max |V|; a bf16 output is that float32 rounded.
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


def _tables(lens, g, width=None, spare=3):
    need = [-(-int(x) // BS) for x in lens]
    blocks = sum(need) + spare
    perm = (torch.randperm(blocks - 1, generator=g) + 1).to(torch.int32)
    tables = torch.full((len(lens), width or max(1, max(need, default=1))), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = perm[at:at + n]
        at += n
    return tables, blocks


def _cache(blocks, hkv, d, g, spread=3.0):
    """Random codes (NaN among them where no test looks) and power-of-two scales."""
    codes = [torch.randint(0, 256, (blocks, BS, hkv, d), generator=g, dtype=torch.int32)
             .to(torch.uint8) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-9, -9 + int(2 * spread), (blocks, hkv), generator=g)
                         .float()) for _ in range(2)]
    return codes, scales


def _no_nan(codes):
    return torch.where((codes & 0x7f) == 0x7f, codes - 1, codes)


def _start(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


def _append(pk, counts, lens, hkv, d, seed=0, spread=6, extra_rows=0, edit=None):
    """One call against the oracle, every byte of pools and scales compared."""
    g = torch.Generator().manual_seed(seed)
    tables, blocks = _tables(lens, g)
    (kc, vc), (ks, vs) = _cache(blocks, hkv, d, g)
    kc, vc = _no_nan(kc), _no_nan(vc)
    rows = int(sum(counts)) + extra_rows
    kv = torch.randn(rows, 2 * hkv + 1, d, generator=g)  # a fused projection's rows
    kv = (kv * torch.exp2(spread * torch.randn(rows, 2 * hkv + 1, 1, generator=g))).bfloat16()
    if edit is not None:
        edit(kv)
    q_start = _start(counts)
    k, v = kv[:, :hkv], kv[:, hkv:2 * hkv]
    want = oracle.append_block_scaled(
        wl.bf16_bits(k.contiguous()), wl.bf16_bits(v.contiguous()), q_start.tolist(),
        tables.tolist(), lens, kc.numpy(), vc.numpy(), ks.numpy(), vs.numpy())
    dev = kv.to(DEV)
    got = [x.to(DEV) for x in (kc, vc, ks, vs)]
    pk.kv_append_fp8_block_scaled(dev[:, :hkv], dev[:, hkv:2 * hkv], q_start.to(DEV),
                                  tables.to(DEV), torch.tensor(lens, dtype=torch.int32).to(DEV),
                                  *got)
    torch.cuda.synchronize()
    for name, a, b in zip(("k", "v", "k_scales", "v_scales"), got, want):
        assert np.array_equal(a.cpu().numpy(), b), name
    return got


@pytest.mark.parametrize("hkv,d", [(1, 64), (2, 128), (8, 128), (5, 64), (32, 128)])
@pytest.mark.parametrize("counts,lens", [
    ([1], [1]),                                   # the first token of a first block
    ([1, 1, 1, 1], [16, 17, 500, 32]),            # decodes: last of a block, first, inside
    ([0, 1, 0, 7, 0], [5, 9, 0, 7, 33]),          # sequences with nothing new
    ([16, 32, 15, 17], [16, 32, 15, 17]),         # whole prompts
    ([40, 3, 100], [53, 34, 109]),                # chunks that start and end inside blocks
])
def test_append_is_the_oracles_bit_for_bit(pk, hkv, d, counts, lens):
    _append(pk, counts, lens, hkv, d, seed=hkv + len(counts))
    assert pk.get_device_error(clear=True) == 0


def test_append_of_many_single_tokens_and_of_long_prompts(pk):
    _append(pk, [1] * 700, [1 + (7 * i) % 40 for i in range(700)], 2, 64)
    _append(pk, [1000, 1, 333], [1000, 77, 350], 4, 128)
    assert pk.get_device_error(clear=True) == 0


def test_append_of_rows_without_a_sequence(pk):
    """Padding behind the last sequence is read by nobody."""
    _append(pk, [3, 5], [20, 5], 2, 128, extra_rows=40)
    assert pk.get_device_error(clear=True) == 0


def test_append_of_extreme_values(pk):
    def edit(kv):
        kv[0] = 0                                     # nothing but zeros in a fresh block
        kv[1, :, 0] = float("inf")                    # left out of the maximum, saturated
        kv[1, :, 1] = float("-inf")
        kv[2, :, 3] = float("nan")
        kv[3] = torch.finfo(torch.bfloat16).max
        kv[4] = 1e-40                                 # subnormal: the least scale
        kv[5] = 0
        kv[5, :, 7] = 448.0                           # exactly the largest code
        kv[6] = 0
        kv[6, :, 7] = 450.0                           # the next bf16: the next scale
        kv[7] = float("inf")                          # no finite element at all
    got = _append(pk, [1] * 8, [1, 5, 6, 16, 1, 1, 1, 17], 2, 64, spread=0, edit=edit)
    assert pk.get_device_error(clear=True) == 0
    assert torch.isfinite(got[2]).all()


def test_append_twice_gives_the_same_cache(pk):
    g = torch.Generator().manual_seed(5)
    lens, counts = [37, 70], [10, 33]
    tables, blocks = _tables(lens, g)
    (kc, vc), (ks, vs) = _cache(blocks, 2, 128, g)
    pools = [x.to(DEV) for x in (_no_nan(kc), _no_nan(vc), ks, vs)]
    k = torch.randn(43, 2, 128, generator=g).bfloat16().to(DEV)
    args = (k, k, _start(counts).to(DEV), tables.to(DEV), torch.tensor(lens).int().to(DEV))
    pk.kv_append_fp8_block_scaled(*args, *pools)
    once = [x.clone() for x in pools]
    pk.kv_append_fp8_block_scaled(*args, *pools)
    assert all(torch.equal(a, b) for a, b in zip(once, pools))


def test_append_leaves_bad_sequences_out(pk):
    """A context shorter than the rows, one beyond the table, a bad block id:
    those sequences' rows go nowhere, the others' arrive."""
    g = torch.Generator().manual_seed(9)
    lens = [20, 20, 20, 20]
    tables, blocks = _tables(lens, g)
    (kc, vc), (ks, vs) = _cache(blocks, 2, 64, g)
    k = torch.randn(12, 2, 64, generator=g).bfloat16()
    want = oracle.append_block_scaled(
        wl.bf16_bits(k[9:]), wl.bf16_bits(k[9:]), [0, 0, 0, 0, 3], tables.tolist(), lens,
        kc.numpy(), vc.numpy(), ks.numpy(), vs.numpy())
    broken = tables.clone()
    broken[2, 1] = blocks
    got = [x.to(DEV) for x in (kc, vc, ks, vs)]
    pk.kv_append_fp8_block_scaled(
        k.to(DEV), k.to(DEV), torch.tensor([0, 3, 6, 9, 12]).int().to(DEV), broken.to(DEV),
        torch.tensor([2, 33, 20, 20]).int().to(DEV), *got)
    word = pk.get_device_error(clear=True)
    assert word == 0x10 | 0x2
    for a, b in zip(got, want):
        assert np.array_equal(a.cpu().numpy(), b)


# ------------------------------------------------------------------- decode
def _decode_case(lens, hq, hkv, d, seed=0, width=None, q_size=1.0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    tables, blocks = _tables(lens, g, width)
    (kc, vc), (ks, vs) = _cache(blocks, hkv, d, g, spread)
    kc, vc = _no_nan(kc), _no_nan(vc)
    for s, n in enumerate(lens):  # what lies behind a sequence's end is nobody's: NaN
        if n % BS:
            b = int(tables[s, n // BS])
            kc[b, n % BS:] = 0x7f
            vc[b, n % BS:] = 0x7f
    q = (torch.randn(len(lens), hq, d, generator=g) * q_size).bfloat16()
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, tables=tables, lens=lens, scale=0.02 / q_size)


def _decode(pk, c, **more):
    return pk.paged_decode_attention_fp8_block_scaled(
        *(c[x].to(DEV) for x in ("q", "kc", "vc", "ks", "vs", "tables")),
        torch.tensor(c["lens"], dtype=torch.int32, device=DEV), c["scale"], **more)


def _check_rows(got, c, seqs):
    """Rows of `seqs` within the tolerance above."""
    kd, vd = (oracle.dequantize_blocks(c[x].numpy(), c[y].numpy())
              for x, y in (("kc", "ks"), ("vc", "vs")))
    q = c["q"].double().numpy()
    d = q.shape[-1]
    for s in seqs:
        n = c["lens"][s]
        if n == 0:
            assert not got[s].any()
            continue
        pages = c["tables"][s, :-(-n // BS)].tolist()
        k = kd[pages].reshape(-1, *kd.shape[2:])[:n]
        v = vd[pages].reshape(-1, *vd.shape[2:])[:n]
        want, size = oracle.attend(q[s:s + 1], k, v, c["scale"], None)
        g = q.shape[1] // k.shape[1]
        dots = np.stack([np.abs(k[:, h // g]) @ np.abs(q[s, h]) for h in range(q.shape[1])])
        rel = 2.0 ** -11 + 2 * d * 2.0 ** -24 * dots.max(1) * abs(c["scale"]) + 2.0 ** -18
        tol = size[0] * rel[:, None] + n * 2.0 ** -24 * np.abs(v).max()
        err = np.abs(got[s] - want[0])
        assert (err <= tol).all(), (s, n, float((err / tol).max()))


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (8, 2, 128), (16, 8, 64), (32, 2, 128),
                                      (64, 8, 128), (16, 1, 64), (5, 5, 128)])
@pytest.mark.parametrize("lens", [[1], [0, 16, 17, 0, 31], [500], [1030, 3, 260]])
def test_decode_of_small_batches(pk, hq, hkv, d, lens):
    c = _decode_case(lens, hq, hkv, d, seed=hq + len(lens))
    got = _decode(pk, c)
    _check_rows(got.cpu().numpy(), c, range(len(lens)))
    assert torch.equal(_decode(pk, c, out_dtype=torch.bfloat16), got.bfloat16())
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (16, 4, 128), (16, 16, 128), (128, 8, 128),
                                      (4, 2, 64)])
def test_decode_of_batches_over_one_wave(pk, hq, hkv, d):
    """Enough pairs for the flat split, some sequences empty."""
    lens = [(37 * i * i) % 300 for i in range(300)]
    c = _decode_case(lens, hq, hkv, d, seed=hq)
    got = _decode(pk, c)
    _check_rows(got.cpu().numpy(), c, range(0, 300, 7))
    assert torch.equal(_decode(pk, c, out_dtype=torch.bfloat16), got.bfloat16())
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d", [(32, 32, 128), (128, 8, 64)])
@pytest.mark.parametrize("lens", [[1] * 227, [(5 * i) % 34 for i in range(254)]])
@pytest.mark.parametrize("width", [None, 40])
def test_decode_of_many_short_contexts(pk, hq, hkv, d, lens, width):
    """A warp each; or, where contexts might be of 40 pages, fewer pages than warps:
    ranges of two pages, over several sequences and within one."""
    c = _decode_case(lens, hq, hkv, d, seed=hq, width=width)
    bound = BS * c["tables"].shape[1]
    got = _decode(pk, c, max_context_len=bound)
    _check_rows(got.cpu().numpy(), c, range(0, len(lens), 11))
    assert torch.equal(_decode(pk, c, max_context_len=bound, out_dtype=torch.bfloat16),
                       got.bfloat16())
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (16, 4, 128), (16, 16, 128), (128, 8, 128),
                                      (4, 2, 64), (4, 2, 128), (16, 1, 64), (32, 4, 64)])
@pytest.mark.parametrize("width", [32, 33])
def test_decode_of_ranges_and_of_whole_pairs(pk, hq, hkv, d, width):
    """Tables of up to 32 pages give a warp a whole pair, wider ones a range of pages;
    one sequence fills its table, another's length is below 0."""
    lens = [(41 * i * i) % 330 for i in range(460)]
    lens[7] = BS * width
    c = _decode_case(lens, hq, hkv, d, seed=hq, width=width)
    got = _decode(pk, c, max_context_len=BS * width)
    _check_rows(got.cpu().numpy(), c, list(range(0, 460, 23)) + [7])
    assert torch.equal(_decode(pk, c, max_context_len=BS * width, out_dtype=torch.bfloat16),
                       got.bfloat16())
    assert pk.get_device_error(clear=True) == 0
    bad = dict(c, lens=lens[:9] + [-1] + lens[10:])
    bad["tables"] = c["tables"].clone()
    bad["tables"][11, 0] = -5
    lens_11 = lens[11]
    other = _decode(pk, bad, max_context_len=BS * width)
    assert pk.get_device_error(clear=True) == 0x4 | (0x2 if lens_11 else 0)
    assert not other[9].any() and torch.isfinite(other).all()
    rest = [s for s in range(460) if s not in (9, 11)]
    if width == 32:  # (ranges move with the lengths before them)
        assert torch.equal(other[rest], got[rest])


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (2, 2, 64)])
def test_decode_of_long_contexts(pk, hq, hkv, d):
    lens = [20000, 16, 17001]
    c = _decode_case(lens, hq, hkv, d)
    _check_rows(_decode(pk, c).cpu().numpy(), c, range(3))
    assert pk.get_device_error(clear=True) == 0


def test_decode_of_more_sequences_than_one_launch_holds(pk):
    lens = [(13 * i) % 50 for i in range(2100)]
    c = _decode_case(lens, 4, 1, 64)
    _check_rows(_decode(pk, c).cpu().numpy(), c, [0, 1, 1023, 1024, 1025, 2047, 2048, 2099])
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("lens", [[300, 90], [(29 * i) % 200 for i in range(260)]])
@pytest.mark.parametrize("q_size", [1e-12, 2e-3, 3e4, 1e30])
def test_decode_of_queries_outside_the_range_of_f16(pk, lens, q_size):
    c = _decode_case(lens, 8, 2, 128, q_size=q_size)
    _check_rows(_decode(pk, c).cpu().numpy(), c, range(0, len(lens), 9))
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("lens", [[300, 90], [(29 * i) % 200 for i in range(260)]])
def test_decode_of_queries_at_the_end_of_bf16(pk, lens):
    """Rows whose largest element is 2^127 or more, against keys of small scales."""
    c = _decode_case(lens, 8, 2, 128)
    q = (c["q"].double() * 8e37).clamp(-3.3e38, 3.3e38)
    q[..., 0] = 2.0 ** 127
    c["q"] = q.bfloat16()
    c["ks"] = c["ks"] * 2.0 ** -60
    c["scale"] = 0.02 / 8e37 * 2.0 ** 60
    _check_rows(_decode(pk, c).cpu().numpy(), c, range(0, len(lens), 9))
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("lens", [[300, 90], [(29 * i) % 200 for i in range(260)]])
def test_decode_of_scales_far_apart(pk, lens):
    """V scales over 60 powers of two, in rising and falling order, all small in
    another sequence."""
    c = _decode_case(lens, 8, 2, 128)
    order = torch.arange(c["vs"].shape[0]) % 61
    c["vs"] = torch.exp2((order - 70).float())[:, None].expand(-1, 2).contiguous()
    pages = c["tables"][1][c["tables"][1] >= 0].long()
    c["vs"][pages] = 2.0 ** -100
    _check_rows(_decode(pk, c).cpu().numpy(), c, range(0, len(lens), 9))
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[300, 90], [(29 * i) % 200 for i in range(260)]])
def test_decode_of_large_values_that_weigh_nothing(pk, lens, d):
    """Every other block has V scales 2^40 times the others' and scores so low that
    it gives the rows next to nothing: the others' values come out.  A weight times
    its block's scale is off by half a step of f16 (2^-11), or 2^-25 of the row's
    largest such product where that is more."""
    c = _decode_case(lens, 8, 2, d, spread=0.5)
    c["q"] = c["q"].abs() + 0.5
    low = torch.arange(c["kc"].shape[0]) % 2 == 0
    low[c["tables"][:, 0].long()] = False       # the first block of each is one of the others
    sign = torch.where(low, 0x80, 0).to(torch.uint8)[:, None, None, None]
    nan = (c["kc"] & 0x7f) == 0x7f
    c["kc"] = torch.where(nan, c["kc"], (c["kc"] & 0x7f) | sign)
    c["ks"] = torch.where(low, 2.0, 2.0 ** -9)[:, None].expand(-1, 2).contiguous()
    c["vs"] = torch.where(low, 2.0 ** 30, 2.0 ** -10)[:, None].expand(-1, 2).contiguous()
    got = _decode(pk, c).cpu().numpy()
    assert pk.get_device_error(clear=True) == 0
    kd, vd = (oracle.dequantize_blocks(c[x].numpy(), c[y].numpy())
              for x, y in (("kc", "ks"), ("vc", "vs")))
    q = c["q"].double().numpy()
    for s in range(0, len(lens), 9):
        n = lens[s]
        if n == 0:
            continue
        pages = c["tables"][s, :-(-n // BS)].tolist()
        k = kd[pages].reshape(-1, *kd.shape[2:])[:n]
        v = vd[pages].reshape(-1, *vd.shape[2:])[:n]
        vscale = np.repeat(c["vs"][pages].double().numpy(), BS, axis=0)[:n]
        for h in range(8):
            x = (k[:, h // 4] @ q[s, h]) * c["scale"]
            w = np.exp(x - x.max())
            l = w.sum()
            want = w @ v[:, h // 4] / l
            dots = (np.abs(k[:, h // 4]) @ np.abs(q[s, h]))
            own = w > 1e-30
            rel = 2.0 ** -11 + 2 * d * 2.0 ** -24 * dots[own].max() * c["scale"] + 2.0 ** -18
            tol = rel * (w @ np.abs(v[:, h // 4]) / l)
            tol = tol + n * 2.0 ** -25 * 448 * (w * vscale[:, h // 4]).max() / l
            part = w * vscale[:, h // 4]
            assert part[vscale[:, h // 4] > 1].max(initial=0) < 2.0 ** -10  # the others' largest
            assert (np.abs(got[s, h] - want) <= tol).all(), (s, h, n)


def test_decode_of_context_bounds_and_block_ids(pk):
    c = _decode_case([40, 100, 30], 8, 2, 64, width=7)
    want = _decode(pk, c)
    assert pk.get_device_error(clear=True) == 0
    got = _decode(pk, c, max_context_len=64)       # the second is cut at 64
    assert pk.get_device_error(clear=True) == 0x4
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    cut = dict(c, lens=[40, 64, 30])
    assert torch.equal(_decode(pk, cut, max_context_len=64)[1], got[1])
    c["tables"][0, 1] = 10 ** 6
    got = _decode(pk, c)
    assert pk.get_device_error(clear=True) == 0x2
    assert torch.equal(got[1:], want[1:]) and torch.isfinite(got).all()


def test_decode_of_nan_in_view_gives_nan(pk):
    c = _decode_case([40, 100], 8, 2, 64)
    c["kc"][int(c["tables"][0, 1]), 2] = 0x7f
    got = _decode(pk, c)
    assert torch.isnan(got[0]).all() and torch.isfinite(got[1]).all()


def test_copied_blocks_take_their_scales_along(pk):
    g = torch.Generator().manual_seed(3)
    for hkv, d in ((1, 64), (3, 128)):
        (kc, vc), (ks, vs) = _cache(9, hkv, d, g)
        t = [x.to(DEV) for x in (kc, vc, ks, vs)]
        pairs = torch.tensor([[1, 5], [2, 8]], dtype=torch.int32, device=DEV)
        pk.copy_blocks(t[0], t[1], pairs, k_scales=t[2], v_scales=t[3])
        for new, old in zip(t, (kc, vc, ks, vs)):
            old = old.clone()
            old[5], old[8] = old[1], old[2]
            assert torch.equal(new.cpu(), old)
    pairs = torch.tensor([[1, 9]], dtype=torch.int32, device=DEV)
    pk.copy_blocks(t[0], t[1], pairs, k_scales=t[2], v_scales=t[3])
    assert pk.get_device_error(clear=True) == 0x2
