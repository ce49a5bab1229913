"""The operators of a speculative serving step over the paged KV cache, as they are timed and compared.

One step, in the order a user's program runs it: the shape of each sequence's
tree of drafted tokens becomes ancestor masks and positions (``layout``); every
layer normalises and rotates the new queries and keys and writes keys and
values into the pages (``append``), then attends each drafted token over its
sequence's cache and its own ancestors (``tree``); after sampling, the rows of
the accepted path move up behind the committed ones (``accept``).

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end), or, where ``own`` is true, through this
package's call.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 16


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of a 7B-MHA model (32 heads of 128): the smallest decode step
        dict(name="append one token", op="append", tokens=1, hq=32, hkv=32, d=128, rot=128,
             interleaved=False, pool="bf16", norm=True),
        # a decode step of the 70B-GQA shape, 256 sequences, some of them padding of a graph bucket
        dict(name="append 256 tokens", op="append", tokens=256, hq=64, hkv=8, d=128, rot=128,
             interleaved=False, pool="bf16", norm=True),
        # drafted tokens of a small-head model, interleaved pairs over half of the head
        dict(name="append 1801 tokens d64", op="append", tokens=1801, hq=16, hkv=4, d=64, rot=32,
             interleaved=True, pool="bf16", norm=False),
        # a prefill step's worth of prompt chunks into an FP8 cache
        dict(name="append 16384 tokens fp8", op="append", tokens=16384, hq=64, hkv=8, d=128,
             rot=128, interleaved=False, pool="fp8", norm=True),
        # one user's tree of 63 nodes, and a batch with trees of other sizes
        dict(name="layout one tree", op="layout", seqs=1, nodes=63, ragged=False),
        dict(name="layout 256 trees", op="layout", seqs=256, nodes=64, ragged=True),
        # one user, a short context, a small tree, no shared KV heads
        dict(name="tree 1 x 500, 8 nodes", op="tree", seqs=1, nodes=8, ctx=500, hq=32, hkv=32,
             d=128, ragged=False),
        # an ordinary batch of the 70B-GQA shape: 16 nodes a sequence
        dict(name="tree 16 x 4096, 16 nodes", op="tree", seqs=16, nodes=16, ctx=4096, hq=64,
             hkv=8, d=128, ragged=True),
        # wide trees on a full batch: the most arithmetic for each byte of cache
        dict(name="tree 64 x 8192, 64 nodes", op="tree", seqs=64, nodes=64, ctx=8192, hq=64,
             hkv=8, d=128, ragged=True),
        # two long documents, heads of 64
        dict(name="tree 2 x 131072, 27 nodes", op="tree", seqs=2, nodes=27, ctx=131072, hq=32,
             hkv=8, d=64, ragged=False),
        # one layer's rows of a few sequences
        dict(name="accept 8 sequences", op="accept", layers=1, seqs=8, nodes=16, ctx=300, hkv=8,
             d=128, pool="bf16"),
        # every layer's rows of a full batch at once, in an FP8 cache
        dict(name="accept 64 x 32 layers fp8", op="accept", layers=32, seqs=64, nodes=64, ctx=200,
             hkv=8, d=128, pool="fp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "layout", "tree", "tree", "accept"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 32])
    group = rng.choice([1, 2, 4, 8, 16]) if hkv <= 8 else 1
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 8000), hq=hkv * group, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.4,
                    pool=rng.choice(["bf16", "bf16", "fp8"]), norm=rng.random() < 0.7)
    if op == "layout":
        return dict(op=op, seqs=_log(rng, 1, 400), nodes=rng.randint(1, 64),
                    ragged=rng.random() < 0.5)
    if op == "accept":
        return dict(op=op, layers=_log(rng, 1, 24), seqs=_log(rng, 1, 64), nodes=rng.randint(4, 64),
                    ctx=_log(rng, 70, 400), hkv=min(hkv, 8), d=d,
                    pool=rng.choice(["bf16", "fp8"]))
    nodes = rng.randint(1, 64)
    ctx = _log(rng, nodes + 1, 60000)
    most = (1 << 19) // (ctx * max(1, hkv // 8))  # the largest listed case's cache
    most = min(48, most, int(1.4e9 // (ctx * nodes * hkv * group * (d // 64))))  # and its products
    most = max(1, most)
    return dict(op=op, seqs=_log(rng, 1, most), nodes=nodes, ctx=ctx, hq=hkv * group, hkv=hkv, d=d,
                ragged=rng.random() < 0.6)


# ---------------------------------------------------------------- sizes that a case fixes
def _sizes(case):
    """Nodes and context length (tree included) of each sequence."""
    s = np.arange(case["seqs"], dtype=np.int64)
    nodes, ctx = case["nodes"], case.get("ctx", 1000)
    n = np.full_like(s, nodes)
    lens = np.full_like(s, ctx)
    if case.get("ragged"):  # every eighth tree smaller, down to one node; contexts down to a half
        n = np.where(s % 8 == 7, 1 + (s * 13) % nodes, n)
        lens = np.maximum(ctx - (s * 7919) % (ctx // 2 + 1), n)
    if case["op"] == "accept":
        lens = np.maximum(ctx - (s * 37) % (ctx // 2 + 1), n)
    return n, lens


def _accepted(case):
    """How many nodes of each sequence are accepted, at most half of its tree."""
    s = np.arange(case["seqs"], dtype=np.int64)
    return (s * 5 + 3) % (min(8, case["nodes"] // 2) + 1)


def _keeps_root(case):
    return np.arange(case["seqs"]) % 2 == 0  # the first accepted node is node 0: nothing to move


# ---------------------------------------------------------------- inputs
def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(int(seed))


def _randn(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pool(shape, g, kind):
    """A pool in use: every row holds something."""
    if kind == "bf16":
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return (x * 20).to(torch.float8_e4m3fn).view(torch.uint8)


def _tables(lens, g):
    """Block tables over a shuffled pool; block 0 belongs to nobody."""
    need = -(-lens // BLOCK)
    total = int(need.sum())
    blocks = total + total // 4 + 2
    perm = torch.randperm(blocks - 1, generator=g)[:total] + 1
    tables = torch.full((len(lens), int(need.max())), -1, dtype=torch.int32)
    at = torch.arange(tables.shape[1])[None, :] < torch.from_numpy(need)[:, None]
    tables[at] = perm.to(torch.int32)
    return tables, blocks


def _trees(n, rng):
    """Parents of random trees in the order they were drafted: -1 or an earlier node."""
    parents = np.full(int(n.sum()), -1, dtype=np.int32)
    start = np.concatenate([[0], np.cumsum(n)])
    for s in range(len(n)):
        t = np.arange(n[s])
        back = rng.integers(1, 1 + np.minimum(np.maximum(t, 1), 6))
        parents[start[s]:start[s + 1]] = np.where(t < 3, -1, t - back)
    return parents


def _masks(n, parents):
    start = np.concatenate([[0], np.cumsum(n)])
    words = np.zeros(int(n.sum()), dtype=np.uint64)
    for s in range(len(n)):
        for t in range(int(n[s])):
            p = parents[start[s] + t]
            up = words[start[s] + p] if p >= 0 else np.uint64(0)
            words[start[s] + t] = up | (np.uint64(1) << np.uint64(t))
    return words.view(np.int64)


def prepare(case, seed):
    g, cpu, rng = _gen(seed), _gen(seed, "cpu"), np.random.default_rng(seed)
    st = dict(case=case)
    if case["op"] == "append":
        T, hq, hkv, d, rot = (case[k] for k in ("tokens", "hq", "hkv", "d", "rot"))
        qkv = _randn((T, hq + 2 * hkv, d), g)  # the rows of a fused projection
        qkv[:, :hq + hkv] *= 3
        st["q"], st["k"], st["v"] = qkv.split([hq, hkv, hkv], dim=1)
        far = 32768
        inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        angle = torch.arange(far, dtype=torch.float64)[:, None] * inv
        st["table"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        st["positions"] = torch.randint(0, far, (T,), generator=cpu).cuda()
        blocks = -(-T // BLOCK) + -(-T // (4 * BLOCK)) + 1
        slots = torch.randperm((blocks - 1) * BLOCK, generator=cpu)[:T] + BLOCK
        if T >= 256:
            slots[torch.randperm(T, generator=cpu)[:T // 64]] = -1  # padding of a graph bucket
        st["slots"] = slots.cuda()
        st["kc"] = _pool((blocks, BLOCK, hkv, d), g, case["pool"])
        st["vc"] = _pool((blocks, BLOCK, hkv, d), g, case["pool"])
        st["qw"] = (1 + 0.2 * _randn((d,), g, torch.float32)).bfloat16() if case["norm"] else None
        st["kw"] = (1 + 0.2 * _randn((d,), g, torch.float32)).bfloat16() if case["norm"] else None
        st["scales"] = (0.03125, 0.0234375)
        return st

    n, lens = _sizes(case)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    st["q_start"] = torch.from_numpy(start).cuda()
    st["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    st["nodes"] = int(n.max())
    if case["op"] == "layout":
        st["parents"] = torch.from_numpy(_trees(n, rng)).cuda()
        return st
    tables, blocks = _tables(lens, cpu)
    st["tables"] = tables.cuda()
    if case["op"] == "tree":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        st["kc"] = _pool((blocks, BLOCK, hkv, d), g, "bf16")
        st["vc"] = _pool((blocks, BLOCK, hkv, d), g, "bf16")
        hot = torch.randint(0, blocks * BLOCK, (max(1, blocks // 8),), generator=cpu).cuda()
        st["kc"].view(-1, hkv * d)[hot] *= 4  # keys that draw a lot of attention
        st["q"] = _randn((int(start[-1]), hq, d), g)
        st["mask"] = torch.from_numpy(_masks(n, _trees(n, rng))).cuda()
        st["scale"] = d ** -0.5
        return st
    shape = (case["layers"], blocks, BLOCK, case["hkv"], case["d"])
    st["kc"], st["vc"] = _pool(shape, g, case["pool"]), _pool(shape, g, case["pool"])
    count = np.minimum(_accepted(case), n // 2)
    keep = np.zeros((case["seqs"], max(1, int(count.max()))), dtype=np.int32)
    root = _keeps_root(case)
    for s in range(case["seqs"]):  # the path's nodes come behind the rows they move to
        path = np.sort(rng.choice(np.arange(count[s], n[s]), size=count[s], replace=False))
        keep[s, :count[s]] = path
        if root[s] and count[s]:
            keep[s, 0] = 0
    st["accepted"] = torch.from_numpy(keep).cuda()
    st["count"] = torch.from_numpy(count.astype(np.int32)).cuda()
    return st


# ---------------------------------------------------------------- the framework's calls
def _call(st):
    from paged_kv_cache_52_gb300 import pagedkv

    case = st["case"]
    if case["op"] == "append":
        args = (st["q"], st["k"], st["v"], st["positions"], st["table"], st["slots"], st["kc"],
                st["vc"])
        more = dict(q_weight=st["qw"], k_weight=st["kw"], eps=1e-6,
                    interleaved=case["interleaved"])
        if case["pool"] == "fp8":
            q = pagedkv.qk_norm_rope_append_fp8(*args, *st["scales"], **more)
        else:
            q = pagedkv.qk_norm_rope_append(*args, **more)
        return _appended(st, q)
    if case["op"] == "layout":
        mask, positions = pagedkv.draft_tree_layout(st["parents"], st["q_start"], st["lens"],
                                                    max_q_len=st["nodes"])
        return dict(mask=mask, positions=positions)
    if case["op"] == "tree":
        if "workspace" not in st:  # kept by the program from step to step
            st["workspace"] = pagedkv.tree_attention_workspace(
                case["seqs"], st["nodes"], case["hq"], case["hkv"], case["d"], st["q"].device)
        return pagedkv.paged_tree_attention(
            st["q"], st["q_start"], st["mask"], st["kc"], st["vc"], st["tables"], st["lens"],
            st["scale"], max_q_len=st["nodes"], workspace=st["workspace"],
            out_dtype=torch.bfloat16)
    lens = pagedkv.kv_accept_rows(st["kc"], st["vc"], st["tables"], st["lens"], st["q_start"],
                                  st["accepted"], st["count"])
    return _moved(st, lens)


def _values(pool):
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def _appended(st, q):
    return dict(q=q, k=_values(st["kc"]), v=_values(st["vc"]))


def _moved(st, lens):
    return dict(k=_values(st["kc"]), v=_values(st["vc"]), lens=lens)


# ---------------------------------------------------------------- the plain forms
def _normed(x, w):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.to(x.dtype)


def _rotated(x, cos, sin, interleaved):
    half = cos.shape[-1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _write_rows(pool, slots, rows, scale):
    flat = _values(pool).view(-1, *pool.shape[2:])
    if pool.dtype == torch.uint8:
        rows = (rows * (1.0 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        rows = rows.to(torch.bfloat16)
    at = slots.clamp(min=0)
    bits = torch.uint8 if pool.dtype == torch.uint8 else torch.int16
    flat, rows = flat.view(bits), rows.view(bits)
    flat[at] = torch.where((slots >= 0)[:, None, None], rows, flat[at])


def _append_plain(st):
    case = st["case"]
    half = case["rot"] // 2
    row = st["table"][st["positions"]]
    cos, sin = row[:, :half], row[:, half:]
    q = _rotated(_normed(st["q"].float(), st["qw"]), cos, sin, case["interleaved"])
    k = _rotated(_normed(st["k"].float(), st["kw"]), cos, sin, case["interleaved"])
    _write_rows(st["kc"], st["slots"], k, st["scales"][0])
    _write_rows(st["vc"], st["slots"], st["v"].float(), st["scales"][1])
    return _appended(st, q.to(torch.bfloat16))


def _padded(st):
    """Row numbers [sequences, nodes] of each sequence's tree, and which of them exist."""
    start = st["q_start"].long()
    t = torch.arange(st["nodes"], device=start.device)
    n = start[1:] - start[:-1]
    there = t[None, :] < n[:, None]
    return torch.where(there, start[:-1, None] + t, 0), there, n


def _twice(m):
    return (m @ m).clamp(max=1)


def _layout_plain(st):
    rows, there, n = _padded(st)
    parent = torch.where(there, st["parents"].long()[rows], -1)
    t = torch.arange(st["nodes"], device=parent.device)
    up = (parent[:, :, None] == t).float() + torch.eye(st["nodes"], device=parent.device)
    up = _twice(_twice(_twice(_twice(_twice(_twice(up))))))  # ancestors up to 64 steps away
    seen = up > 0
    word = (seen.long() << t).sum(-1)
    depth = seen.sum(-1) - 1
    base = st["lens"].long() - n
    return dict(mask=word[there], positions=(base[:, None] + depth)[there])


def _tree_plain(st, dtype=torch.float32):
    case = st["case"]
    hkv, d = case["hkv"], case["d"]
    group = case["hq"] // hkv
    rows, there, n = _padded(st)
    S, N = rows.shape
    tables = st["tables"].clamp(min=0).long()
    k = st["kc"][tables].view(S, -1, hkv, d).permute(0, 2, 1, 3).to(dtype)
    v = st["vc"][tables].view(S, -1, hkv, d).permute(0, 2, 1, 3).to(dtype)
    q = st["q"][rows].view(S, N, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(S, hkv, -1, d)
    x = (q.to(dtype) @ k.transpose(-1, -2)) * st["scale"]  # [S, hkv, N * group, keys]
    key = torch.arange(k.shape[2], device=q.device)
    base = (st["lens"].long() - n)[:, None, None]
    node = key - base
    word = st["mask"][rows][:, :, None]
    sees = (node < 0) | ((node < n[:, None, None]) & ((word >> node.clamp(0, 63)) & 1).bool())
    x = x.view(S, hkv, N, group, -1)
    x = x.masked_fill(~sees[:, None, :, None, :], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = (x - top.masked_fill(top == float("-inf"), 0)).exp()
    total = p.sum(-1, keepdim=True)
    p = p / total.masked_fill(total == 0, 1)
    out = (p.view(S, hkv, N * group, -1) @ v).view(S, hkv, N, group, d)
    out = out.permute(0, 2, 1, 3, 4).reshape(S, N, hkv * group, d)[there]
    return out.to(torch.bfloat16) if dtype == torch.float32 else out


def _accept_plain(st):
    tables, n = st["tables"].long(), (st["q_start"][1:] - st["q_start"][:-1]).long()
    lens, count, keep = st["lens"].long(), st["count"].long(), st["accepted"].long()
    i = torch.arange(keep.shape[1], device=keep.device)[None, :]
    base = (lens - n)[:, None]
    moved = i < count[:, None]
    last = (lens - 1)[:, None]  # beyond the path: the last row onto itself

    def slot(pos):
        return torch.gather(tables, 1, pos // BLOCK) * BLOCK + pos % BLOCK

    src = slot(torch.where(moved, base + keep, last)).view(-1)
    dst = slot(torch.where(moved, base + i, last)).view(-1)
    k, v = (st[x].view(st[x].shape[0], -1, *st[x].shape[3:]) for x in ("kc", "vc"))
    k[:, dst] = k[:, src]
    v[:, dst] = v[:, src]
    return _moved(st, (lens - n + count).int())


PLAIN = dict(append=_append_plain, layout=_layout_plain, tree=_tree_plain, accept=_accept_plain)


def run(state):
    if own:
        return _call(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "append":
        T, hq, hkv, d, rot = (case[k] for k in ("tokens", "hq", "hkv", "d", "rot"))
        elem = 1 if case["pool"] == "fp8" else 2
        rows = T * (hq + 2 * hkv) * d * 2 + T * hq * d * 2 + 2 * T * hkv * d * elem
        return dict(bytes=rows + T * (16 + 4 * rot), flops=8 * T * (hq + hkv) * d)
    n, lens = _sizes(case)
    if case["op"] == "layout":
        return dict(bytes=int(n.sum()) * 20 + 8 * len(n), flops=int(n.sum()))
    if case["op"] == "tree":
        cache = int(lens.sum()) * case["hkv"] * case["d"] * 4
        rows = int(n.sum()) * case["hq"] * case["d"] * 4
        pairs = int((n * (lens - n + 1)).sum())  # a node sees the committed keys and itself at least
        return dict(bytes=cache + rows, flops=4 * pairs * case["hq"] * case["d"])
    count = np.minimum(_accepted(case), n // 2)
    moved = int((count - (_keeps_root(case) & (count > 0))).sum())
    elem = 1 if case["pool"] == "fp8" else 2
    return dict(bytes=4 * case["layers"] * moved * case["hkv"] * case["d"] * elem
                + 16 * case["seqs"], flops=0)


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _append_exact(st)
    if case["op"] == "layout":
        return None  # whole numbers: equal or wrong
    if case["op"] == "accept":
        return _accept_exact(st)
    return _tree_exact(st)


def _append_exact(st):
    case = st["case"]
    rot, inter = case["rot"], case["interleaved"]
    # each element's partner, its sign, and the angle's column, element by element
    e = torch.arange(rot)
    if inter:
        partner, sign, col = e ^ 1, torch.where(e % 2 == 0, -1.0, 1.0), e // 2
    else:
        partner = (e + rot // 2) % rot
        sign, col = torch.where(e < rot // 2, -1.0, 1.0), e % (rot // 2)
    partner, sign, col = partner.cuda(), sign.double().cuda(), col.cuda()
    row = st["table"].double()[st["positions"]]
    cos, sin = row[:, None, col], row[:, None, rot // 2 + col]

    def turn(x, w):
        x = x.double()
        if w is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
        y = x.clone()
        y[..., :rot] = x[..., :rot] * cos + sign * x[..., partner] * sin
        return y

    def put(pool, rows, scale):
        out = _values(pool).double().view(-1, *pool.shape[2:])
        if pool.dtype == torch.uint8:
            rows = (rows / scale).clamp(-448, 448)
        keep = st["slots"] >= 0
        out[st["slots"][keep]] = rows[keep]
        return out.view(pool.shape)

    return dict(q=turn(st["q"], st["qw"]), k=put(st["kc"], turn(st["k"], st["kw"]), st["scales"][0]),
                v=put(st["vc"], st["v"].double(), st["scales"][1]))


def _accept_exact(st):
    k, v = (_values(st[x]).double() for x in ("kc", "vc"))
    tables, lens, start, keep, count = (st[x].cpu().tolist() for x in
                                        ("tables", "lens", "q_start", "accepted", "count"))
    before = k.clone(), v.clone()
    for s in range(len(lens)):
        base = lens[s] - (start[s + 1] - start[s])
        for i in range(count[s]):
            a, b = base + i, base + keep[s][i]
            for new, old in zip((k, v), before):
                new[:, tables[s][a // BLOCK], a % BLOCK] = old[:, tables[s][b // BLOCK], b % BLOCK]
    return dict(k=k, v=v, lens=None)


def _tree_exact(st):
    case = st["case"]
    group, scale = case["hq"] // case["hkv"], st["scale"]
    start, lens, tables = (st[x].cpu().tolist() for x in ("q_start", "lens", "tables"))
    mask = st["mask"].cpu().tolist()
    out = []
    for s in range(len(lens)):
        n, L = start[s + 1] - start[s], lens[s]
        pages = torch.tensor(tables[s][:-(-L // BLOCK)], device="cuda")
        k = st["kc"][pages].flatten(0, 1)[:L].double()
        v = st["vc"][pages].flatten(0, 1)[:L].double()
        q = st["q"][start[s]:start[s + 1]].double()
        hidden = torch.zeros(n, L, dtype=torch.bool)
        for t in range(n):
            for j in range(n):
                hidden[t, L - n + j] = not (mask[start[s] + t] >> j) & 1
        hidden = hidden.cuda()
        heads = []
        for h in range(case["hkv"]):
            x = torch.einsum("tgd,ld->tgl", q[:, h * group:(h + 1) * group], k[:, h]) * scale
            x = x.masked_fill(hidden[:, None, :], -math.inf)
            heads.append(torch.einsum("tgl,ld->tgd", torch.softmax(x, -1), v[:, h]))
        out.append(torch.cat(heads, 1))
    return torch.cat(out)
