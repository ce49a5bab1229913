"""Attention of drafted trees over many items of several key tiles each, so that
the rings of tiles run on across the items of a CTA: rows that nobody sees may
hold anything wherever in the stream their tile comes.

The reference is the definition in float64 on the GPU.  Tolerance of a float32
output element, from the arithmetic alone: a score is off by at most
e = (d + 4) 2^-24 * 2 |scale| |q| |k| (float32 accumulation of d products,
Cauchy-Schwarz on the magnitudes), a weight and the sum so by a factor
exp(2 e); P as bf16 hi + lo adds 2^-16, the base-2 exponential 2^-21, the
accumulation of L / 16 + 8 partial products and the join (L / 16 + 40) 2^-23;
all of it times max|V|.
"""

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BS = 16


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_52_gb300 import pagedkv
    pagedkv.get_device_error(clear=True)
    return pagedkv


class Batch:
    """Trees of any mask over a shuffled pool on the GPU."""

    def __init__(self, hq, hkv, d, nodes, lens, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.n, self.lens = np.array(nodes), np.array(lens)
        self.start = np.concatenate([[0], np.cumsum(self.n)])
        total = int(self.start[-1])
        need = -(-self.lens // BS)
        blocks = int(need.sum()) + 3
        perm = rng.permutation(blocks)
        tables = np.full((len(nodes), int(need.max())), -1, dtype=np.int32)
        at = 0
        for s, b in enumerate(need):
            tables[s, :b] = perm[at:at + b]
            at += b
        self.tables = torch.from_numpy(tables).to(DEV)
        self.k = torch.randn(blocks, BS, hkv, d, device=DEV, generator=g).bfloat16()
        self.v = torch.randn(blocks, BS, hkv, d, device=DEV, generator=g).bfloat16()
        self.q = torch.randn(total, hq, d, device=DEV, generator=g).bfloat16()
        self.mask = rng.integers(0, 2 ** 64, total, dtype=np.uint64)
        self.scale = d ** -0.5

    def row(self, s, pos):
        return int(self.tables[s, pos // BS]), pos % BS

    def run(self, pk, **kw):
        i32 = lambda x: torch.from_numpy(x.astype(np.int32)).to(DEV)  # noqa: E731
        kw = dict(max_q_len=int(self.n.max())) | kw
        return pk.paged_tree_attention(
            self.q, i32(self.start), torch.from_numpy(self.mask.view(np.int64)).to(DEV), self.k,
            self.v, self.tables, i32(self.lens), self.scale, **kw)

    def ref(self, s):
        """Sequence s's rows in float64, from its visible keys."""
        n, L = int(self.n[s]), int(self.lens[s])
        pages = self.tables[s, :-(-L // BS)].long()
        k, v = (x[pages].flatten(0, 1)[:L].double() for x in (self.k, self.v))
        q = self.q[self.start[s]:self.start[s + 1]].double()
        q = q.view(n, k.shape[1], -1, q.shape[2])
        word = torch.from_numpy(self.mask[self.start[s]:self.start[s + 1]].view(np.int64)).to(DEV)
        seen = torch.ones(n, L, dtype=torch.bool, device=DEV)
        seen[:, L - n:] = (word[:, None] >> torch.arange(n, device=DEV)) & 1 == 1
        x = torch.einsum("thgd,lhd->thgl", q, k) * float(np.float32(self.scale))
        p = x.masked_fill(~seen[:, None, None, :], -math.inf).softmax(-1).nan_to_num(0.0)
        return torch.einsum("thgl,lhd->thgd", p, v).flatten(1, 2)

    def tolerance(self):
        d, L = self.q.shape[2], int(self.lens.max())
        q, k = (float(x.float().norm(dim=-1).max()) for x in (self.q, self.k))
        e = (d + 4) * 2.0 ** -23 * abs(self.scale) * q * k
        return float(self.v.float().abs().max()) * (
            math.expm1(2 * e) + 2.0 ** -16 + 2.0 ** -21 + (L / 16 + 40) * 2.0 ** -23)

    def check(self, out, what=""):
        tol = self.tolerance()
        for s in np.flatnonzero(self.n):
            diff = (out[self.start[s]:self.start[s + 1]].double() - self.ref(s)).abs()
            assert bool((diff <= tol).all()), (what, s, float(diff.max()), tol)


# (query heads, KV heads, d, nodes): one row tile, and two
SHAPES = [(8, 4, 128, 8), (8, 4, 64, 8), (4, 4, 64, 33), (32, 4, 128, 16), (32, 4, 128, 40),
          (16, 4, 64, 64)]


@pytest.mark.parametrize("hq,hkv,d,n", SHAPES)
@pytest.mark.parametrize("seqs", [31, 40])
def test_unseen_rows_may_hold_anything_wherever_in_the_stream(pk, hq, hkv, d, n, seqs):
    # contexts of 9 to 17 key tiles whose last page is never full, items enough
    # for every SM to take several pieces in turn
    rng = np.random.default_rng(seqs + d + n)
    lens = [int(x) * BS + 5 for x in rng.integers(70, 132, seqs)]
    b = Batch(hq, hkv, d, [n] * seqs, lens, seed=n)
    hidden = np.array([rng.integers(0, n) for _ in range(seqs)])
    for s in range(seqs):  # one node of each tree that no row sees, itself included
        b.mask[b.start[s]:b.start[s + 1]] &= ~np.uint64(1 << int(hidden[s]))
    clean = b.run(pk)
    b.check(clean)
    for value in (float("nan"), float("inf"), -float("inf")):
        for s in range(seqs):
            blk, off = b.row(s, lens[s] - 1)
            b.k[blk, off + 1:] = value
            b.v[blk, off + 1:] = value
            blk, off = b.row(s, lens[s] - n + int(hidden[s]))
            b.k[blk, off] = value
            b.v[blk, off] = value
        for _ in range(4):
            out = b.run(pk)
            assert torch.equal(out, clean), value
    assert pk.get_device_error(clear=True) == 0


# Where a sequence's scores climb, (key, height): within the first tile, in each
# half of a later one, several times, and in the tree.
CLIMBS = [[(70, 30.0)], [(200, 15.0)], [(330, 20.0)], [(130, 14.0), (700, 50.0)],
          [(64, 45.0), (128, 90.0)], [(400, 12.0), (460, 24.0), (900, 37.0), (970, 60.0)],
          [(5, 60.0), (640, 70.0)], [(1297, 25.0)], [(1291, 100.0)], []]


@pytest.mark.parametrize("hq,hkv,d,n", SHAPES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("big", [1.0, 2.0 ** 96])
def test_climbing_scores(pk, hq, hkv, d, n, sign, big):
    """Scores that are exact, a_row s_key: with q = a u, k = s u, u of d signs and
    the scale 1 / d.  What is left of a score's error, in units of X, the largest
    score times log2 e: the scale's product and constant, the multiply-add and up
    to 12 differences of references and log-sum-exps, 2^-24 X each.  A weight is so
    off by a factor E = exp(2 * 16 * 2^-24 X), by two roundings to hi + lo (2^-16
    each) and up to eight exponentials of references (2^-21 each).  Every error
    is relative to a key's weight or, from accumulating, to the sum of |p v|, so
    an element is off by at most twice that part of sum p |v|; weights beyond
    2^-126 of the largest are lost.  V up to 2^96 times 6.2: below 2^110 / (L + 64)."""
    seqs, L = 40, 1301
    b = Batch(hq, hkv, d, [n] * seqs, [L] * seqs, seed=d + n)
    g = torch.Generator().manual_seed(3)
    u = (torch.randint(0, 2, (d,), generator=g) * 2 - 1).float()
    a = 2.0 ** -torch.randint(0, 3, b.q.shape[:2], generator=g).float()
    b.q = (a[..., None] * u).bfloat16().to(DEV)
    for s in range(seqs):
        height = torch.randint(-2, 3, (L,), generator=g) / 2
        for key, h in CLIMBS[s % len(CLIMBS)]:
            height[key] += h
        pages = b.tables[s].long()
        rows = torch.zeros(len(pages) * BS, d)
        rows[:L] = sign * height[:, None] * u
        b.k[pages] = rows.bfloat16().to(DEV).view(-1, BS, 1, d).expand(-1, -1, hkv, -1)
    b.v = (b.v.float() * big).bfloat16()
    assert float(b.v.float().abs().max()) * (L + 64) < 2.0 ** 110
    b.scale = sign / d
    out = b.run(pk)
    assert bool(out.isfinite().all())
    X = 103 * 1.4427
    part = (math.expm1(2 * 16 * 2.0 ** -24 * X) + 2 * 2.0 ** -16 + 8 * 2.0 ** -21
            + (L / 16 + 40) * 2.0 ** -23)
    values = b.v
    for s in range(seqs):
        got = out[b.start[s]:b.start[s + 1]].double()
        want = b.ref(s)
        b.v = values.abs()
        tol = 2 * part * b.ref(s) + 2.0 ** -100 * big
        b.v = values
        bad = (got - want).abs() > tol
        assert not bool(bad.any()), (s, CLIMBS[s % len(CLIMBS)], int(bad.sum()),
                                     float(((got - want).abs() / tol).max()))
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d,n", SHAPES)
def test_non_finite_values_of_committed_keys_stay_in_their_element(pk, hq, hkv, d, n):
    lens = [700 + 31 * s for s in range(40)]
    b = Batch(hq, hkv, d, [n] * 40, lens, seed=n + 1)
    clean = b.run(pk)
    want = clean.isfinite()
    assert bool(want.all())
    group = hq // hkv
    for s, (pos, head, col, value) in {0: (0, 0, 5, math.inf), 7: (300, 1, d - 1, -math.inf),
                                       21: (lens[21] - n - 1, hkv - 1, 32, math.nan)}.items():
        blk, off = b.row(s, pos)
        b.v[blk, off, head, col] = value
        want[b.start[s]:b.start[s + 1], head * group:(head + 1) * group, col] = False
    out = b.run(pk)
    assert torch.equal(out.isfinite(), want)
    assert torch.equal(out[want], clean[want])
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d", [(64, 8, 128), (32, 8, 64), (4, 4, 128), (16, 1, 64)])
@pytest.mark.parametrize("seqs", [12, 40])
def test_bound_above_the_trees(pk, hq, hkv, d, seqs):
    # a bucket's bound instead of the largest tree's nodes: the second row tile has
    # rows for some of the trees, for a part of its rows, or for none
    for small in (True, False):
        nodes = [1 + (5 * s) % 16 if small else (0, 1, 15, 17, 33, 40, 48, 64)[s % 8]
                 for s in range(seqs)]
        lens = [n + (97 * s) % 1500 for s, n in enumerate(nodes)]
        b = Batch(hq, hkv, d, nodes, lens, seed=seqs + small)
        out = torch.full((int(b.start[-1]), hq, d), float("nan"), device=DEV)
        ws = pk.tree_attention_workspace(seqs, 64, hq, hkv, d, DEV)
        b.run(pk, max_q_len=64, out=out, workspace=ws)
        b.check(out, f"bound 64, small trees {small}")
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 128), (8, 8, 128), (64, 4, 64), (3, 3, 64)])
@pytest.mark.parametrize("seqs", [385, 900])
def test_more_sequences_than_threads(pk, hq, hkv, d, seqs):
    nodes = [(7 * s) % 12 for s in range(seqs)]
    lens = [n + (53 * s) % 200 for s, n in enumerate(nodes)]
    nodes[seqs // 2], lens[seqs // 2] = 64, 5000   # one of them long
    b = Batch(hq, hkv, d, nodes, lens, seed=seqs)
    b.check(b.run(pk))
    assert pk.get_device_error(clear=True) == 0


def test_pools_of_more_than_2_31_elements(pk):
    # the step's calls on the last blocks of pools of 2.6e9 elements, against the same
    # blocks in small pools
    hq, hkv, d, n, L = 16, 8, 128, 20, 150
    far, need = 160_000, -(-L // BS)
    g = torch.Generator(device=DEV).manual_seed(1)
    qkv = torch.randn(n, hq + 2 * hkv, d, device=DEV, generator=g).bfloat16()
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    small = [torch.randn(need, BS, hkv, d, device=DEV, generator=g).bfloat16() for _ in range(2)]
    large = [torch.empty(far, BS, hkv, d, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    assert large[0].numel() > 2 ** 31
    for a, b in zip(large, small):
        a[far - need:] = b
    angles = torch.rand(L, d // 2, device=DEV, generator=g)
    table = torch.cat([angles.cos(), angles.sin()], 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    start, lens = i32([0, n]), i32([L])
    parents = i32([-1] + [t // 2 for t in range(n - 1)])
    mask, pos = pk.draft_tree_layout(parents, start, lens, max_q_len=n)
    path, count = i32([[0, 2, 5, 12]]), i32([4])
    got = []
    for pools, first in ((small, 0), (large, far - need)):
        slots = first * BS + torch.arange(L - n, L, device=DEV)
        tables = torch.arange(first, first + need, device=DEV, dtype=torch.int32)[None].contiguous()
        x = pk.qk_norm_rope_append(q, k, v, pos, table, slots, *pools)
        out = pk.paged_tree_attention(x, start, mask, *pools, tables, lens, 0.09, max_q_len=n)
        pools[1].view(-1, hkv, d)[slots[3], 2, 7] = float("inf")  # a visible node's V
        inf = pk.paged_tree_attention(x, start, mask, *pools, tables, lens, 0.09, max_q_len=n)
        new = pk.kv_accept_rows(*pools, tables, lens, start, path, count)
        got.append([x, out, inf, new] + [p[first:first + need].clone() for p in pools])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert not torch.equal(got[0][1], got[0][2])
    assert pk.get_device_error(clear=True) == 0
