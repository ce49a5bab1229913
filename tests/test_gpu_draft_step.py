"""Whole speculative steps: pages reserved for a tree, its layout, the rotated
append and the tree attention of two layers, the accepted path moved up and
committed -- over several steps, with forks that share pages, rejections of
everything, and sequences that leave.  After every step each sequence's cache
must hold exactly the rows of its committed tokens, in order."""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_52_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"
BS = 16
LAYERS = 2


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_52_gb300 import pagedkv
    pagedkv.get_device_error(clear=True)
    return pagedkv


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (16, 2, 128)])
def test_speculative_steps_end_to_end(pk, hq, hkv, d):
    rng = np.random.default_rng(d)
    g = torch.Generator(device=DEV).manual_seed(d)
    blocks, width = 120, 20
    bm = pk.BlockManager(blocks, BS)
    shape = (LAYERS, blocks, BS, hkv, d)
    kc = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)  # unused rows hold NaN
    vc = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.from_numpy(oracle.rope_table(400, d)).to(DEV)
    weights = [(torch.rand(d, device=DEV) + 0.5).bfloat16() for _ in range(2)]
    ws = pk.tree_attention_workspace(8, 64, hq, hkv, d, DEV)
    truth = {}   # sequence -> [(K rows, V rows) of all layers] of its committed tokens

    def append(positions, slots, layer):
        """A layer's rotated append of random projections; returns its queries."""
        qkv = torch.randn(len(slots), hq + 2 * hkv, d, device=DEV, generator=g).bfloat16()
        q, k, v = qkv.split([hq, hkv, hkv], 1)
        return pk.qk_norm_rope_append(q, k, v, positions, table, slots, kc[layer], vc[layer],
                                      *weights)

    def rows_at(slots):
        at = torch.tensor(slots, device=DEV)
        return [(kc.view(LAYERS, -1, hkv, d)[:, s].clone(), vc.view(LAYERS, -1, hkv, d)[:, s].clone())
                for s in at]

    def check_cache(live):
        for s in live:
            slots = bm.slots(s, 0, bm.seq_len(s))
            assert len(truth[s]) == len(slots)
            for have, want in zip(rows_at(slots), truth[s]):
                assert torch.equal(have[0], want[0]) and torch.equal(have[1], want[1]), s

    for s, n in enumerate([1, 37, 16, 90]):   # prompts
        bm.add_sequence(s, rng.integers(0, 50, n).tolist())
        slots = bm.slots(s, 0, n)
        for layer in range(LAYERS):
            append(torch.arange(n, device=DEV), torch.tensor(slots, device=DEV), layer)
        truth[s] = rows_at(slots)
    bm.fork(1, 4)                             # shares a partly filled page
    truth[4] = list(truth[1])
    live = [0, 1, 2, 3, 4]

    for step in range(5):
        nodes = [int(n) for n in rng.integers(1, 33, len(live))]
        if step == 1:
            nodes[2] = 64
        slots = []
        for s, n in zip(live, nodes):
            got, copies = bm.reserve_draft(s, n)
            if copies:
                for layer in range(LAYERS):
                    pk.copy_blocks(kc[layer], vc[layer], _i32(copies))
            slots += got
        parents = np.concatenate([[rng.integers(-1, t) for t in range(n)] for n in nodes])
        q_start = np.concatenate([[0], np.cumsum(nodes)])
        tables, lens = bm.block_tables(live, width)
        assert lens.tolist() == [bm.seq_len(s) + n for s, n in zip(live, nodes)]
        dev = dict(tables=tables.to(DEV), lens=lens.to(DEV), q_start=_i32(q_start))
        mask, positions = pk.draft_tree_layout(_i32(parents), dev["q_start"], dev["lens"],
                                               max_q_len=64)
        want_mask, want_pos = oracle.tree_layout(parents, q_start, lens.numpy())
        assert np.array_equal(mask.cpu().numpy().view(np.uint64), want_mask)
        assert np.array_equal(positions.cpu().numpy(), want_pos)
        slot_t = torch.tensor(slots, device=DEV)
        for layer in range(LAYERS):
            q = append(positions, slot_t, layer)
            out = pk.paged_tree_attention(q, dev["q_start"], mask, kc[layer], vc[layer],
                                          dev["tables"], dev["lens"], d ** -0.5, max_q_len=64,
                                          workspace=ws)
            ref = oracle.tree_attention(wl.bf16_bits(q), q_start, want_mask,
                                        wl.bf16_bits(kc[layer]), wl.bf16_bits(vc[layer]),
                                        tables.numpy(), lens.numpy(), d ** -0.5)
            diff = np.abs(out.double().cpu().numpy() - ref).max()
            # as the decode's and verification's outputs: 2e-3 absolute
            assert diff <= 2e-3, (step, layer, diff)
        drafted = rows_at(slots)

        # a random root-to-node path of each tree is accepted, sometimes none
        paths = []
        for i, n in enumerate(nodes):
            t, path = int(rng.integers(0, n)), []
            while t >= 0:
                path.insert(0, t)
                t = int(parents[q_start[i] + t])
            paths.append([] if rng.random() < 0.2 else path)
        most = max(1, max(map(len, paths)))
        accepted = [p + [0] * (most - len(p)) for p in paths]
        new = pk.kv_accept_rows(kc, vc, dev["tables"], dev["lens"], dev["q_start"],
                                _i32(accepted), _i32([len(p) for p in paths]))
        for i, (s, path) in enumerate(zip(live, paths)):
            truth[s] = truth[s] + [drafted[q_start[i] + t] for t in path]
            bm.commit_draft(s, rng.integers(0, 50, len(path)).tolist())
            assert bm.seq_len(s) == int(new[i])
        check_cache(live)
        if step == 2:
            bm.fork(2, 5)
            truth[5] = list(truth[2])
            live.append(5)
        if step == 3:
            bm.free_sequence(3)
            live.remove(3)
    assert pk.get_device_error(clear=True) == 0
    # what remains decodes as any other cache
    slots = [bm.append_tokens(s, [1]) for s in live]
    for _, copies in slots:
        if copies:
            pk.copy_blocks(kc[0], vc[0], _i32(copies))
    tables, lens = bm.block_tables(live, width)
    pos = torch.tensor([n - 1 for n in lens.tolist()], device=DEV)
    q = append(pos, torch.tensor([x[0] for x, _ in slots], device=DEV), 0)
    out = pk.paged_decode_attention(q, kc[0], vc[0], tables.to(DEV), lens.to(DEV), d ** -0.5)
    ref = oracle.paged_decode_attention(wl.bf16_bits(q), wl.bf16_bits(kc[0]), wl.bf16_bits(vc[0]),
                                        tables.numpy(), lens.numpy(), d ** -0.5)
    assert np.abs(out.double().cpu().numpy() - ref).max() <= 2e-3
    for s in live:
        bm.free_sequence(s)
    assert bm.num_free_blocks() == blocks
    bm.close()


def test_captured_step_replays_with_other_trees(pk):
    # layout, append, attention and acceptance of one step in one graph: replayed
    # with other trees, positions and paths it gives what the calls give eagerly
    S, n, hq, hkv, d = 3, 12, 8, 2, 128
    rng = np.random.default_rng(3)
    lens0 = [40, 130, 12]
    tables, used = wl.build_block_tables([x + 20 for x in lens0], torch.randperm(40))
    table = torch.from_numpy(oracle.rope_table(300, d)).to(DEV)
    base_k = torch.randn(40, BS, hkv, d, device=DEV).bfloat16()
    base_v = torch.randn(40, BS, hkv, d, device=DEV).bfloat16()
    q_start = _i32(np.arange(S + 1) * n)
    ws = pk.tree_attention_workspace(S, n, hq, hkv, d, DEV)
    st = dict(parents=_i32(np.full(S * n, -1)), lens=_i32(lens0), tables=tables.to(DEV),
              slots=torch.full((S * n,), -1, device=DEV), k=base_k.clone(), v=base_v.clone(),
              qkv=torch.zeros(S * n, hq + 2 * hkv, d, dtype=torch.bfloat16, device=DEV),
              path=_i32(np.tile(np.arange(4), (S, 1))), count=_i32([1] * S))

    def step():
        mask, pos = pk.draft_tree_layout(st["parents"], q_start, st["lens"], max_q_len=n)
        q, k, v = st["qkv"].split([hq, hkv, hkv], 1)
        q = pk.qk_norm_rope_append(q, k, v, pos, table, st["slots"], st["k"], st["v"])
        out = pk.paged_tree_attention(q, q_start, mask, st["k"], st["v"], st["tables"], st["lens"],
                                      0.1, max_q_len=n, workspace=ws)
        new = pk.kv_accept_rows(st["k"], st["v"], st["tables"], st["lens"], q_start, st["path"],
                                st["count"])
        return mask, pos, q, out, new

    def fill(seed):
        r = np.random.default_rng(seed)
        lens = [int(x + r.integers(0, 8)) for x in lens0]
        parents = np.concatenate([[r.integers(-1, t) for t in range(n)] for _ in range(S)])
        slots = [int(tables[s, p // BS]) * BS + p % BS for s in range(S)
                 for p in range(lens[s] - n, lens[s])]
        st["parents"].copy_(_i32(parents))
        st["lens"].copy_(_i32(lens))
        st["slots"].copy_(torch.tensor(slots, device=DEV))
        st["qkv"].copy_(torch.randn(st["qkv"].shape, generator=torch.Generator().manual_seed(seed)))
        st["path"].copy_(_i32([np.sort(r.choice(n, 4, replace=False)) for _ in range(S)]))
        st["count"].copy_(_i32(r.integers(0, 5, S)))
        st["k"].copy_(base_k)
        st["v"].copy_(base_v)

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (1, 2, 1):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured] + [st["k"].clone(), st["v"].clone()]
        fill(seed)
        want = list(step()) + [st["k"], st["v"]]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert pk.get_device_error(clear=True) == 0
