"""Attention of drafted trees over the paged cache on the GPU against the
float64 oracle, and the layout kernel that makes its masks.

Tolerance of a float32 output element, from the arithmetic alone: a score is
off by at most e = (d + 4) 2^-23 |scale| |q| |k| (float32 accumulation of d
products, by Cauchy-Schwarz on the magnitudes), so a weight by a factor
exp(2 e) at most (numerator and sum); P as bf16 hi + lo adds 2^-16, the base-2
exponential 2^-21, and the float32 accumulation of L / 16 + 8 partial products
and the pieces' join (L / 16 + 40) 2^-23.  Each acts on a convex combination of V
rows, so the output is off by at most their sum times max|V|.  A bf16 output
adds half a step, 2^-8 of its value.
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


class Batch:
    """Ragged trees over a shuffled pool, on the host, and their oracle."""

    def __init__(self, hq, hkv, d, nodes, lens, seed=0, masks="tree", k_scale=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.n, self.lens = np.array(nodes), np.array(lens)
        self.q_start = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        total = int(self.q_start[-1])
        blocks = [-(-x // BS) for x in lens]
        perm = torch.randperm(sum(blocks) + 5, generator=g)
        self.tables, _ = wl.build_block_tables(lens, perm)
        shape = (sum(blocks) + 5, BS, hkv, d)
        self.k = (torch.randn(shape, generator=g) * k_scale).bfloat16()
        self.v = torch.randn(shape, generator=g).bfloat16()
        self.q = torch.randn((total, hq, d), generator=g).bfloat16()
        self.scale = d ** -0.5
        self.parents = np.full(total, -1, dtype=np.int32)
        for s in range(len(nodes)):
            for t in range(nodes[s]):
                self.parents[self.q_start[s] + t] = rng.integers(-1, t)
        if masks == "tree":
            self.mask, self.positions = oracle.tree_layout(self.parents, self.q_start, self.lens)
        else:  # any bits, those of other sequences' nodes and empty words among them
            self.mask = rng.integers(0, 2 ** 64, total, dtype=np.uint64)
            self.mask[rng.random(total) < 0.3] = 0

    def slot(self, s, pos):
        return int(self.tables[s, pos // BS]), pos % BS

    def ref(self):
        return oracle.tree_attention(wl.bf16_bits(self.q), self.q_start, self.mask,
                                     wl.bf16_bits(self.k), wl.bf16_bits(self.v),
                                     self.tables.numpy(), self.lens, self.scale)

    def tolerance(self):
        d = self.q.shape[2]
        q = float(self.q.float().norm(dim=-1).max()) if self.q.numel() else 0.0
        k = float(self.k.float().nan_to_num(0, 0, 0).norm(dim=-1).max())
        v = float(self.v.float().nan_to_num(0, 0, 0).abs().max())
        e = (d + 4) * 2.0 ** -23 * abs(self.scale) * q * k
        L = int(self.lens.max())
        return v * (np.expm1(2 * e) + 2.0 ** -16 + 2.0 ** -21 + (L / 16 + 40) * 2.0 ** -23)

    def dev(self):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        return dict(q=self.q.to(DEV), q_start=t(self.q_start), tree_mask=t(self.mask.view(np.int64)),
                    k_cache=self.k.to(DEV), v_cache=self.v.to(DEV), block_tables=self.tables.to(DEV),
                    context_lens=t(self.lens.astype(np.int32)), scale=self.scale)

    def run(self, pk, **kw):
        out = pk.paged_tree_attention(**self.dev(), max_q_len=int(self.n.max()), **kw)
        torch.cuda.synchronize()
        return out


def check(b, out, what):
    ref, got = b.ref(), out.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    tol = b.tolerance()
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    diff = np.abs(got - ref)
    assert (diff <= tol).all(), f"{what}: max {diff.max():.3e}, tolerance {np.max(tol):.3e}"


NODES = [1, 7, 64, 16, 33, 2, 0, 17]
LENS = [1, 300, 64, 16, 1000, 130, 40, 273]


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (4, 2, 128), (8, 2, 64), (16, 2, 128),
                                      (16, 1, 64), (3, 3, 64), (64, 8, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tree_ragged_batch(pk, hq, hkv, d, dtype):
    b = Batch(hq, hkv, d, NODES, LENS, seed=hq + d)
    check(b, b.run(pk, out_dtype=dtype), f"{hq}/{hkv} d{d} {dtype}")
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,n", [(8, 1, 16), (8, 1, 17), (16, 1, 8), (16, 1, 64), (1, 1, 64)])
@pytest.mark.parametrize("L", [64, 127, 128, 129, 191, 192, 193, 256, 2049])
def test_tree_across_tile_borders(pk, hq, hkv, n, L):
    # one sequence: the tree inside a key tile, across two, and at its end
    b = Batch(hq, hkv, 128, [n], [L], seed=L + n)
    check(b, b.run(pk), f"n {n} L {L}")
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("nodes,lens", [([5], [40000]), ([64, 3], [9000, 20011]),
                                        ([4] * 400, [20 + i % 90 for i in range(400)]),
                                        ([1] * 700, [1 + i % 40 for i in range(700)])])
def test_tree_long_contexts_and_many_sequences(pk, nodes, lens):
    # items cut over many SMs, and many items on each
    b = Batch(8, 2, 64, nodes, lens, seed=3)
    check(b, b.run(pk), f"{len(nodes)} sequences")
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq", [2, 16])
def test_arbitrary_masks_and_rows_that_see_nothing(pk, hq):
    # contexts that are all tree: a row with an empty word sees no key
    b = Batch(hq, 1, 128, [64, 9, 30, 1], [64, 9, 200, 1], seed=5, masks="any")
    out = b.run(pk)
    check(b, out, f"hq {hq}")
    word = b.mask.copy()
    for s in range(4):
        lo, hi, n = b.q_start[s], b.q_start[s + 1], int(b.n[s])
        if n < 64:
            word[lo:hi] &= np.uint64((1 << n) - 1)
    empty = [r for s in (0, 1, 3) for r in range(b.q_start[s], b.q_start[s + 1]) if word[r] == 0]
    assert empty and (out[torch.tensor(empty, device=DEV)] == 0).all()


def test_large_scores_move_the_running_maximum(pk):
    b = Batch(8, 1, 128, [16, 16], [700, 1400], seed=6, k_scale=20.0)
    for key, f in ((300, 10), (690, 30)):
        blk, off = b.slot(0, key)
        b.k[blk, off] *= f
    check(b, b.run(pk), "large scores")
    b.scale = -b.scale
    check(b, b.run(pk), "negative scale")
    b.scale = 0.0
    check(b, b.run(pk), "scale 0: the mean of the visible rows")


@pytest.mark.parametrize("hq", [2, 16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_masked_rows_may_hold_anything(pk, hq, value):
    # stale rows behind the context, and the K and V rows of two drafted nodes,
    # hold NaN or an infinity: rows that do not see those nodes do not change
    b = Batch(hq, 1, 128, [40, 5], [333, 37], seed=7)
    clean = b.run(pk)
    assert (b.lens % BS != 0).all()
    for s in range(2):
        blk, off = b.slot(s, int(b.lens[s]) - 1)
        b.k[blk, off + 1:] = value
        b.v[blk, off + 1:] = value
    assert torch.equal(b.run(pk), clean)
    bad = [3, 17]
    for t in bad:
        blk, off = b.slot(0, int(b.lens[0]) - 40 + t)
        b.k[blk, off] = value
        b.v[blk, off, :, 5] = value
    out = b.run(pk)
    sees = np.array([int(b.mask[r]) >> t & 1 for r in range(45) for t in bad]).reshape(45, 2)
    sees[40:] = 0
    hidden = torch.from_numpy(sees.sum(1) == 0).to(DEV)
    assert 10 < int(hidden.sum()) < 43
    assert torch.equal(out[hidden], clean[hidden])
    assert pk.get_device_error(clear=True) == 0


def test_visible_infinity_of_v_reaches_its_rows(pk):
    b = Batch(2, 1, 128, [20], [150], seed=8)
    clean = b.run(pk)
    blk, off = b.slot(0, 130 + 2)
    b.v[blk, off, 0, 77] = float("inf")
    b.v[blk, off, 0, 12] = float("nan")
    out = b.run(pk)
    for r in range(20):
        if int(b.mask[r]) >> 2 & 1:
            assert (out[r, :, 77] == float("inf")).all() and out[r, :, 12].isnan().all()
            keep = [c for c in range(128) if c not in (12, 77)]
            assert torch.isfinite(out[r][:, keep]).all()
        else:
            assert torch.equal(out[r], clean[r])


def test_single_nodes_match_the_decode(pk):
    # a tree of one node is a decode step
    lens = [900, 33, 1, 2500, 128]
    b = Batch(64, 8, 128, [1] * 5, lens, seed=9)
    got = b.run(pk)
    a = b.dev()
    ref = pk.paged_decode_attention(a["q"], a["k_cache"], a["v_cache"], a["block_tables"],
                                    a["context_lens"], b.scale, max_context_len=2500)
    assert float((got - ref).abs().max()) <= 2 * b.tolerance()


def test_chains_match_the_linear_verification(pk):
    lens, n = [300, 64, 1000], 4
    b = Batch(64, 8, 128, [n] * 3, lens, seed=10)
    b.mask = np.array([(1 << (t + 1)) - 1 for _ in lens for t in range(n)], dtype=np.uint64)
    got = b.run(pk)
    a = b.dev()
    ref = pk.paged_verify_attention(a["q"].view(3, n, 64, 128), a["k_cache"], a["v_cache"],
                                    a["block_tables"], a["context_lens"], b.scale,
                                    max_context_len=1000)
    assert float((got - ref.view_as(got)).abs().max()) <= 2 * b.tolerance()


def test_rounded_output_is_the_float32_one_and_repeats_bitwise(pk):
    b = Batch(16, 2, 128, [30, 64, 5], [700, 3000, 90], seed=11)
    ws = pk.tree_attention_workspace(3, 64, 16, 2, 128, DEV)
    ws.fill_(0xFF)  # NaN everywhere: its contents do not matter
    a = b.run(pk, workspace=ws)
    assert torch.equal(a, b.run(pk, workspace=ws))
    assert torch.equal(b.run(pk, out_dtype=torch.bfloat16), a.bfloat16())


def test_rejected_sequences_and_rows_behind_the_last_keep_their_contents(pk):
    b = Batch(4, 2, 64, [5, 6, 7, 3], [100, 40, 50, 33], seed=12)
    ref = b.ref()
    a = b.dev()
    a["context_lens"][1] = 4                      # fewer positions than nodes
    a["context_lens"][2] = 16 * b.tables.shape[1] + 1  # beyond the block table
    a["q"] = torch.cat([a["q"], a["q"][:4]])      # rows of no sequence
    a["tree_mask"] = torch.cat([a["tree_mask"], a["tree_mask"][:4]])
    out = torch.full((25, 4, 64), 7.0, device=DEV)
    pk.get_device_error(clear=True)
    pk.paged_tree_attention(**a, max_q_len=7, out=out)
    torch.cuda.synchronize()
    assert pk.get_device_error(clear=True) == 0x10
    assert (out[5:18] == 7).all() and (out[21:] == 7).all()
    got = out.double().cpu().numpy()
    for rows in (slice(0, 5), slice(18, 21)):
        assert np.abs(got[rows] - ref[rows]).max() <= b.tolerance()
    # a tree larger than the bound, and a q_start that runs backwards
    a = b.dev()
    a["q_start"] = torch.tensor([0, 5, 3, 18, 21], dtype=torch.int32, device=DEV)
    out.fill_(7.0)
    pk.paged_tree_attention(**a, max_q_len=7, out=out[:21])
    torch.cuda.synchronize()
    assert pk.get_device_error(clear=True) == 0x10
    assert (out[5:18] == 7).all() and not (out[18:21] == 7).any()


def test_block_ids_outside_the_pool_read_as_zeros(pk):
    b = Batch(4, 2, 64, [5], [100], seed=13)
    a = b.dev()
    a["block_tables"][0, 1] = b.k.shape[0] + 3
    out = pk.paged_tree_attention(**a, max_q_len=5)
    torch.cuda.synchronize()
    assert pk.get_device_error(clear=True) == 0x2
    blk = int(b.tables[0, 1])
    b.k[blk], b.v[blk] = 0, 0
    check(b, out, "zeros")


def test_graph_replay_with_other_lengths_and_two_streams(pk):
    one = Batch(16, 2, 128, [20, 1, 64], [500, 900, 70], seed=14)
    two = Batch(16, 2, 128, [64, 20, 1], [70, 31, 1000], seed=15)
    blocks = max(one.k.shape[0], two.k.shape[0])
    width = max(one.tables.shape[1], two.tables.shape[1])

    def padded(b):
        a = b.dev()
        for n in ("k_cache", "v_cache"):
            x = a[n]
            a[n] = torch.cat([x, x.new_zeros(blocks - x.shape[0], *x.shape[1:])])
        t = a["block_tables"]
        a["block_tables"] = torch.cat([t, t.new_full((3, width - t.shape[1]), -1)], 1).contiguous()
        return a

    st, other = padded(one), padded(two)
    ws = pk.tree_attention_workspace(3, 64, 16, 2, 128, DEV)
    out = torch.empty(85, 16, 128, device=DEV)
    pk.paged_tree_attention(**st, max_q_len=64, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.paged_tree_attention(**st, max_q_len=64, out=out, workspace=ws)
    for b, a in ((one, padded(one)), (two, other), (one, padded(one))):
        for n, x in a.items():
            if torch.is_tensor(x):
                st[n].copy_(x)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check(b, out, "replay")
    # two calls at once, each with its workspace
    side = [torch.cuda.Stream() for _ in range(2)]
    args = [padded(one), padded(two)]
    wss = [torch.empty_like(ws) for _ in range(2)]
    outs = [torch.empty_like(out) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                pk.paged_tree_attention(**args[i], max_q_len=64, out=outs[i], workspace=wss[i])
    torch.cuda.synchronize()
    check(one, outs[0], "stream 0")
    check(two, outs[1], "stream 1")
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("nodes", [[1], [64], [63, 0, 1, 30, 64], [5] * 300])
def test_layout(pk, nodes):
    b = Batch(1, 1, 64, nodes, [n + 10 * i % 100 + 1 for i, n in enumerate(nodes)], seed=16)
    if nodes[0] == 64:
        b.parents = np.arange(-1, 63, dtype=np.int32)  # a chain: the deepest tree
    masks, positions = oracle.tree_layout(b.parents, b.q_start, b.lens)
    a = b.dev()
    got, pos = pk.draft_tree_layout(torch.from_numpy(b.parents).to(DEV), a["q_start"],
                                    a["context_lens"])
    assert np.array_equal(got.cpu().numpy().view(np.uint64), masks)
    assert np.array_equal(pos.cpu().numpy(), positions)
    assert pk.get_device_error(clear=True) == 0


def test_layout_flags_bad_parents_and_ranges(pk):
    parents = torch.tensor([-1, 1, 0, -2, 0, -1], dtype=torch.int32, device=DEV)
    q_start = torch.tensor([0, 4, 6], dtype=torch.int32, device=DEV)
    lens = torch.tensor([9, 1], dtype=torch.int32, device=DEV)  # the second: 2 nodes, 1 position
    masks = torch.full((6,), 55, dtype=torch.int64, device=DEV)
    pos = torch.full((6,), 55, dtype=torch.int64, device=DEV)
    pk.draft_tree_layout(parents, q_start, lens, max_q_len=4, tree_mask=masks, positions=pos)
    torch.cuda.synchronize()
    assert pk.get_device_error(clear=True) == 0x410
    assert masks.tolist() == [1, 2, 5, 8, 55, 55] and pos.tolist() == [5, 5, 6, 5, 55, 55]


@pytest.mark.parametrize("hq,hkv,d", [(6, 3, 64), (5, 5, 128), (12, 6, 128), (28, 7, 64),
                                      (32, 32, 128), (48, 3, 64)])
def test_head_counts_that_share_the_grid_unevenly(pk, hq, hkv, d):
    b = Batch(hq, hkv, d, [33, 1, 64], [2100, 5000, 700], seed=hkv)
    check(b, b.run(pk), f"{hq}/{hkv}")
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 128), (8, 1, 64), (4, 4, 128)])
def test_many_sequences_with_little_and_with_uneven_work(pk, hq, hkv, d):
    # more sequences than the short split takes: empty ones, single tiles, and
    # two long ones between them that are cut over many SMs
    n = [i % 3 for i in range(45)]
    lens = [max(m, (i * 37) % 100) for i, m in enumerate(n)]
    few = Batch(hq, hkv, d, n, lens, seed=hq)
    check(few, few.run(pk), "little")
    n[20], lens[20], n[31], lens[31] = 64, 9000, 17, 4001
    uneven = Batch(hq, hkv, d, n, lens, seed=hq)
    check(uneven, uneven.run(pk), "uneven")
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,nodes,lens", [(8, [9, 3], [100, 60]), (32, [64, 20], [300, 5000])])
def test_output_that_starts_between_32_byte_borders(pk, dtype, hq, nodes, lens):
    b = Batch(hq, 2, 128, nodes, lens, seed=20)
    want = b.run(pk, out_dtype=dtype)
    shift = 16 // want.element_size()
    flat = torch.full((want.numel() + 2 * shift,), 7.0, dtype=dtype, device=DEV)
    out = flat[shift:-shift].view(want.shape)
    assert out.data_ptr() % 32 == 16
    pk.paged_tree_attention(**b.dev(), max_q_len=max(nodes), out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert (flat[:shift] == 7).all() and (flat[-shift:] == 7).all()


@pytest.mark.parametrize("lens", [[300, 40], [9000, 5000]])
def test_rounded_output_with_visible_infinities_and_nan(pk, lens):
    # whole and cut items: what a non-finite V element makes of a row rounds to itself
    b = Batch(16, 2, 128, [40, 20], lens, seed=21)
    for s, node, col, value in [(0, 0, 3, np.inf), (0, 7, 3, -np.inf), (0, 7, 90, -np.inf),
                                (0, 30, 127, np.nan), (1, 0, 64, np.inf)]:
        blk, row = b.slot(s, b.lens[s] - b.n[s] + node)
        b.v[blk, row, 1, col] = value
    full, rounded = b.run(pk), b.run(pk, out_dtype=torch.bfloat16)
    assert not full.isfinite().all()
    assert torch.equal(full.bfloat16().nan_to_num(3e38), rounded.nan_to_num(3e38))
    assert torch.equal(full.isnan(), rounded.isnan())
