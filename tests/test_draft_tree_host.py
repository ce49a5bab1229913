"""The speculative step without a GPU: drafts in the block manager against the
oracle model, argument checks at the C entries, and the oracle against plain
identities."""

import ctypes
import random

import numpy as np
import pytest

import oracle
from oracle.block_manager import BlockManager as OracleBM, NoFreeBlocks as OracleNoFree

BS = 16


@pytest.fixture(scope="module")
def pk():
    import os
    from paged_kv_cache_52_gb300 import build as b
    if not os.path.exists(b.LIB_PATH):
        b.build()
    from paged_kv_cache_52_gb300 import pagedkv
    return pagedkv


def _state(bm, ids, num_blocks, native):
    return ({s: bm.block_table(s) for s in ids}, {s: bm.seq_len(s) for s in ids},
            [bm.refcount(b) for b in range(num_blocks)],
            bm.free_list() if native else list(bm.free))


@pytest.mark.parametrize("seed,num_blocks", [(0, 30), (1, 60), (2, 18)])
def test_drafts_match_the_oracle_operation_by_operation(pk, seed, num_blocks):
    rng = random.Random(seed)
    nat, ref = pk.BlockManager(num_blocks, BS), OracleBM(num_blocks, BS)
    live, drafts, next_id, seen = [], {}, 0, dict(full=0, cow=0, freed=0, hit=0)
    base = [rng.randrange(30) for _ in range(60)]
    for _ in range(500):
        op = rng.random()
        idle = [s for s in live if s not in drafts]
        if op < 0.2 or not live:
            call, sid = ("add_sequence", next_id, base[:rng.randrange(60)] +
                         [rng.randrange(30) for _ in range(rng.randrange(6))]), next_id
            next_id += 1
        elif op < 0.3 and idle:
            call, sid = ("fork", rng.choice(idle), next_id), next_id
            next_id += 1
        elif op < 0.45 and idle:
            sid = rng.choice(idle)
            call = ("append_tokens", sid, [rng.randrange(30) for _ in range(rng.randrange(1, 9))])
        elif op < 0.7 and idle:
            sid = rng.choice(idle)
            call = ("reserve_draft", sid, rng.randrange(1, 65))
        elif op < 0.9 and drafts:
            sid = rng.choice(sorted(drafts))
            call = ("commit_draft", sid, [rng.randrange(30) for _ in
                                          range(rng.randrange(0, drafts[sid] + 1))])
        else:
            sid = rng.choice(live)
            call = ("free_sequence", sid)
        name, *args = call
        free = nat.num_free_blocks()
        try:
            want, err = getattr(ref, name)(*args), None
        except OracleNoFree:
            want, err = None, "full"
        try:
            got, got_err = getattr(nat, name)(*args), None
        except pk.NoFreeBlocks:
            got, got_err = None, "full"
        assert (got, got_err) == (want, err), call
        if err:
            seen["full"] += 1
        elif name in ("add_sequence", "fork"):
            live.append(sid)
            seen["hit"] += name == "add_sequence" and want > 0
        elif name == "free_sequence":
            live.remove(sid)
            drafts.pop(sid, None)
        elif name == "reserve_draft":
            drafts[sid] = args[1]
            seen["cow"] += bool(want[1])
        elif name == "commit_draft":
            del drafts[sid]
            seen["freed"] += nat.num_free_blocks() > free
        assert _state(nat, live, num_blocks, True) == _state(ref, live, num_blocks, False), call
    assert all(seen.values()), seen
    if live:
        tables, lens = nat.block_tables(live, num_blocks)
        assert lens.tolist() == [ref.seq_len(s) + drafts.get(s, 0) for s in live]
    nat.close()


def test_draft_refusals_change_nothing(pk):
    bm = pk.BlockManager(6, BS)
    bm.add_sequence(1, range(20))
    bm.fork(1, 2)

    def state():
        return bm.free_list(), bm.block_table(2), bm.seq_len(2), [bm.refcount(b) for b in range(6)]

    before = state()
    for bad in (lambda: bm.reserve_draft(9, 4), lambda: bm.reserve_draft(2, 0),
                lambda: bm.commit_draft(2, []), lambda: bm.commit_draft(9, [])):
        with pytest.raises(pk.PagedKVError) as e:
            bad()
        assert e.value.status == -1
    with pytest.raises(pk.NoFreeBlocks):
        bm.reserve_draft(2, 61)             # a copy and four blocks more: 5 of 4
    slots, n = (ctypes.c_int64 * 4)(), ctypes.c_int32()
    assert pk.lib.pkv_bm_reserve_draft(bm._h, 2, 4, slots, None, 0, ctypes.byref(n)) == -1
    assert pk.lib.pkv_bm_reserve_draft(bm._h, 2, 4, None, None, 0, ctypes.byref(n)) == -1
    assert state() == before
    slots, copies = bm.reserve_draft(2, 30)
    assert copies == [(1, 2)] and slots[0] == 2 * BS + 4 and len(slots) == 30
    during = state()
    for bad in (lambda: bm.reserve_draft(2, 1), lambda: bm.append_tokens(2, [5]),
                lambda: bm.fork(2, 3), lambda: bm.commit_draft(2, range(31))):
        with pytest.raises(pk.PagedKVError):
            bad()
    assert state() == during
    bm.commit_draft(2, [])                  # nothing accepted: the copied block stays
    assert bm.block_table(2) == [0, 2] and bm.seq_len(2) == 20 and bm.num_free_blocks() == 3
    bm.reserve_draft(2, 30)
    bm.free_sequence(2)                     # a draft goes with its sequence
    assert bm.num_free_blocks() == 4
    bm.close()


def test_rejected_nodes_are_never_shared(pk):
    # a draft fills a block, a few of its nodes are accepted: only blocks of
    # committed tokens can be hit by another prompt
    bm = pk.BlockManager(20, BS)
    bm.add_sequence(1, range(10))
    bm.reserve_draft(1, 40)
    assert bm.add_sequence(2, list(range(10)) + [7] * 40) == 0
    bm.commit_draft(1, [100, 101, 102, 103, 104, 105, 106])
    assert bm.seq_len(1) == 17
    assert bm.add_sequence(3, list(range(10)) + [100, 101, 102, 103, 104, 105, 106, 9]) == BS
    bm.close()


def _desc(pk, nb=64, bs=16, hkv=2, d=64):
    return pk.CacheDesc(nb, bs, hkv, d)


NULL, DUMMY = ctypes.c_void_p(0), ctypes.c_void_p(1 << 20)  # DUMMY is never dereferenced


def test_rope_append_host_validation(pk):
    def call(T=4, hq=4, q=DUMMY, qs=256, kst=128, pos=DUMMY, table=DUMMY, rows=100, rot=64,
             eps=1e-6, out=ctypes.c_void_p(1 << 30), kc=DUMMY, qw=NULL, desc=None):
        return pk.lib.pkv_qk_norm_rope_append(q, qs, DUMMY, kst, DUMMY, kst, T, hq, pos, table,
                                              rows, rot, 0, qw, NULL, eps, DUMMY, out, kc, DUMMY,
                                              desc or _desc(pk), NULL)
    assert call(T=0) == 0
    odd = ctypes.c_void_p((1 << 20) + 4)
    for kw in (dict(T=-1), dict(hq=0), dict(q=NULL), dict(pos=NULL), dict(table=NULL),
               dict(out=NULL), dict(kc=NULL), dict(qs=248), dict(qs=257), dict(kst=120),
               dict(rows=0), dict(eps=float("inf")), dict(q=odd), dict(table=odd), dict(qw=odd),
               dict(out=ctypes.c_void_p((1 << 20) + 512)), dict(desc=_desc(pk, nb=0))):
        assert call(**kw) == -1, kw
    for kw in (dict(rot=0), dict(rot=24), dict(rot=80), dict(desc=_desc(pk, d=96)),
               dict(desc=_desc(pk, bs=32))):
        assert call(**kw) == -2, kw
    for ks, vs in ((0.0, 1.0), (1.0, -1.0), (float("nan"), 1.0), (1.0, float("inf"))):
        assert pk.lib.pkv_qk_norm_rope_append_fp8(
            DUMMY, 256, DUMMY, 128, DUMMY, 128, 4, 4, DUMMY, DUMMY, 100, 64, 0, NULL, NULL, 1e-6,
            DUMMY, ctypes.c_void_p(1 << 30), DUMMY, DUMMY, _desc(pk), ks, vs, NULL) == -1


def test_layout_host_validation(pk):
    def call(parents=DUMMY, S=2, total=9, most=8, out=DUMMY):
        return pk.lib.pkv_draft_tree_layout(parents, DUMMY, S, total, most, DUMMY, out, DUMMY, NULL)
    assert call(S=0) == call(total=0) == call(most=0) == 0
    assert call(parents=NULL) == call(S=-1) == call(out=ctypes.c_void_p((1 << 20) + 4)) == -1
    assert call(most=65) == -2


def test_tree_attention_host_validation(pk):
    def call(S=2, total=9, most=8, hq=4, mask=DUMMY, mb=16, scale=0.1, ws=DUMMY, nws=1 << 40,
             desc=None, out=DUMMY, fn=pk.lib.pkv_paged_tree_attention):
        return fn(DUMMY, DUMMY, S, total, most, hq, mask, DUMMY, DUMMY, desc or _desc(pk), DUMMY,
                  mb, DUMMY, scale, out, ws, nws, NULL)
    for fn in (pk.lib.pkv_paged_tree_attention, pk.lib.pkv_paged_tree_attention_bf16out):
        assert call(S=0, fn=fn) == call(total=0, fn=fn) == 0
        for kw in (dict(S=-1), dict(mask=NULL), dict(out=NULL), dict(mb=0),
                   dict(scale=float("nan")), dict(out=ctypes.c_void_p((1 << 20) + 8)),
                   dict(ws=ctypes.c_void_p((1 << 20) + 16))):
            assert call(fn=fn, **kw) == -1, kw
        for kw in (dict(most=65), dict(hq=6), dict(desc=_desc(pk, d=96)),
                   dict(desc=_desc(pk, bs=8)), dict(mb=1 << 28)):
            assert call(fn=fn, **kw) == -2, kw
        assert call(ws=NULL, fn=fn) == call(nws=1000, fn=fn) == -4
    assert pk.lib.pkv_tree_attention_workspace_bytes(2, 65, 8, 2, 64) == 0
    small = pk.lib.pkv_tree_attention_workspace_bytes(2, 16, 8, 1, 64)   # 128 rows a pair
    large = pk.lib.pkv_tree_attention_workspace_bytes(900, 17, 8, 1, 64)
    assert 0 < small < large < 2 * small + 1024


def test_accept_rows_host_validation(pk):
    out = ctypes.c_void_p(1 << 24)

    def call(layers=1, stride=64 * 16 * 128, eb=2, S=2, A=4, mb=16, new=out, desc=None, acc=DUMMY):
        return pk.lib.pkv_kv_accept_rows(DUMMY, stride, DUMMY, stride, layers, desc or _desc(pk),
                                         eb, DUMMY, mb, DUMMY, DUMMY, S, acc, A, DUMMY, new, NULL)
    assert call(layers=0) == call(S=0) == 0
    for kw in (dict(layers=-1), dict(S=-1), dict(A=-1), dict(eb=4), dict(mb=0), dict(new=NULL),
               dict(new=DUMMY), dict(acc=NULL), dict(layers=2, stride=64 * 16 * 128 - 8),
               dict(layers=2, stride=64 * 16 * 128 + 4), dict(desc=_desc(pk, nb=-1))):
        assert call(**kw) == -1, kw
    assert call(desc=_desc(pk, bs=32)) == -2
    assert call(desc=_desc(pk, hkv=1, d=3)) == -2
    assert call(layers=1 << 20, stride=64 * 16 * 128, S=1 << 12) == -2


def test_oracle_tree_of_a_chain_is_the_causal_prefill():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 9, BS, 2, 8))
    tables, lens, n = np.array([[3, 1, 4, 0], [5, 8, 2, 6]]), [50, 37], [5, 3]
    q_start = np.array([0, 5, 8])
    q = rng.standard_normal((8, 4, 8))
    parents = np.concatenate([np.arange(-1, 4), np.arange(-1, 2)])
    masks, positions = oracle.tree_layout(parents, q_start, lens)
    assert positions.tolist() == [45, 46, 47, 48, 49, 34, 35, 36]
    got = oracle.tree_attention(q, q_start, masks, k, v, tables, lens, 0.25)
    want = oracle.paged_prefill_attention(q, q_start, k, v, tables, lens, True, 0.25)
    assert np.allclose(got, want, atol=1e-12)


def test_oracle_rotation_keeps_products_of_equal_distance():
    # the point of the rotation: q . k depends on the distance of the positions
    rng = np.random.default_rng(1)
    table = oracle.rope_table(400, 16)
    q, k = rng.standard_normal((2, 1, 1, 24))
    for inter in (False, True):
        dots = []
        for p in (10, 300):
            a = oracle.norm_rope(q, None, np.array([p + 7]), table, 0.0, inter)
            b = oracle.norm_rope(k, None, np.array([p]), table, 0.0, inter)
            dots.append(float((a * b).sum()))
        assert abs(dots[0] - dots[1]) < 1e-5        # the table is float32
        assert np.array_equal(oracle.norm_rope(q, None, np.array([5]), table, 0.0, inter)[..., 16:],
                              q[..., 16:])
