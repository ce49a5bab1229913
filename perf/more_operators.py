"""The operators of serving over a paged KV cache of 8-bit codes with a scale for each block of tokens and
head, as they are timed and compared.

A prompt's life, in the order a user's program runs it: its tokens attend to one another over the keys and
values that have just been computed, many prompts packed behind one another (``prompt``); the rows are then
quantised into the pages, every page of a head getting the power of two that its largest value needs
(``append``); each later step appends one token per sequence and attends it over the pages (``decode``); a
chunk of tokens that continues a cached prefix attends over the pages too (``prefill``).

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once at the
end), or, where ``own`` is true, through this package's call.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 16
TOP = 448.0  # the largest e4m3 value


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of a 7B-MHA model (32 heads of 128) into a page in use: the smallest append
        dict(name="append one token", op="append", seqs=1, new=1, prior=499, hkv=32, d=128, ragged=False),
        # a decode step's tokens of a full batch of the 70B-GQA shape, each into a page of its own
        dict(name="append 256 tokens", op="append", seqs=256, new=1, prior=200, hkv=8, d=128, ragged=True),
        # a prefill step's prompt chunks, some of them starting inside a page
        dict(name="append 8 x 2048 tokens", op="append", seqs=8, new=2048, prior=100, hkv=8, d=128, ragged=True),
        # one short question to a 7B-MHA model
        dict(name="prompt 1 x 37", op="prompt", seqs=1, new=37, hq=32, hkv=32, d=128, ragged=False),
        # a batch of ordinary prompts of a small model, packed, heads of 64
        dict(name="prompt 24 x 700 d64", op="prompt", seqs=24, new=700, hq=16, hkv=4, d=64, ragged=True),
        # one long document
        dict(name="prompt 1 x 16384", op="prompt", seqs=1, new=16384, hq=32, hkv=8, d=128, ragged=False),
        # one user, a short context, no shared KV heads
        dict(name="decode 1 x 500", op="decode", seqs=1, ctx=500, hq=32, hkv=32, d=128, ragged=False),
        # an ordinary batch of a small model, heads of 64
        dict(name="decode 24 x 2500 d64", op="decode", seqs=24, ctx=2500, hq=16, hkv=4, d=64, ragged=True),
        # a full batch of the 70B-GQA shape
        dict(name="decode 256 x 6000", op="decode", seqs=256, ctx=6000, hq=64, hkv=8, d=128, ragged=True),
        # two long documents
        dict(name="decode 2 x 131072", op="decode", seqs=2, ctx=131072, hq=32, hkv=8, d=128, ragged=False),
        # short turns that continue cached conversations, heads of 64
        dict(name="prefill 6 x 90 after 1000 d64", op="prefill", seqs=6, new=90, prior=1000, hq=16, hkv=4, d=64,
             ragged=True),
        # a step of prompt chunks of the 70B-GQA shape
        dict(name="prefill 8 x 512 after 4096", op="prefill", seqs=8, new=512, prior=4096, hq=64, hkv=8, d=128,
             ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "prompt", "decode", "decode", "prefill"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 32])
    hq = hkv * (rng.choice([1, 2, 4, 8, 16]) if hkv <= 8 else 1)
    ragged = rng.random() < 0.7
    if op == "append":
        new = _log(rng, 1, 4000)
        seqs = _log(rng, 1, max(1, min(300, (1 << 14) * 8 // (new * hkv))))
        return dict(op=op, seqs=seqs, new=new, prior=rng.choice([0, rng.randint(1, 400)]), hkv=hkv, d=d, ragged=ragged)
    if op == "prompt":
        new = _log(rng, 1, 12000)
        most = max(1, min(64, int(8.0e9 // (hq * new * new))))
        return dict(op=op, seqs=_log(rng, 1, most), new=new, hq=hq, hkv=hkv, d=d, ragged=ragged)
    if op == "decode":
        ctx = _log(rng, 1, 100000)
        most = max(1, min(300, (1 << 20) * 8 // (ctx * hkv)))
        return dict(op=op, seqs=_log(rng, 1, most), ctx=ctx, hq=hq, hkv=hkv, d=d, ragged=ragged)
    new, prior = _log(rng, 1, 1500), _log(rng, 16, 20000)
    most = max(1, min(32, int(1.0e9 // (new * hq * (prior + new))), (1 << 19) // (prior * max(1, hkv // 8))))
    return dict(op=op, seqs=_log(rng, 1, most), new=new, prior=prior, hq=hq, hkv=hkv, d=d, ragged=ragged)


# ---------------------------------------------------------------- sizes that a case fixes
def _sizes(case):
    """New tokens of each sequence, and its context length with them."""
    s = np.arange(case["seqs"], dtype=np.int64)
    new, prior = case.get("new", 1), case.get("prior", 0)
    if case["op"] == "decode":
        prior = case["ctx"] - 1
    n, before = np.full_like(s, new), np.full_like(s, prior)
    if case["ragged"]:  # lengths down to a half, every eighth shorter still
        n = np.where(s % 8 == 7, 1 + (s * 13) % new, new - (s * 7919) % (new // 2 + 1))
        before = prior - (s * 6151) % (prior // 2 + 1)
    return n, before + n


# ---------------------------------------------------------------- inputs
def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(int(seed))


def _randn(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _need(amax):
    """The smallest power of two (from 2^-126 on) that takes amax to 448 or less."""
    part, power = torch.frexp(amax)  # amax = part * 2^power, part in [0.5, 1)
    power = power - 9 + (part > TOP / 512).int()
    power = torch.where(amax > 0, power, -126).clamp(min=-126)
    return torch.ldexp(torch.ones_like(amax), power)


def _codes(x):
    """32-bit values within 448 -> e4m3 codes (nearest, ties to even)."""
    return x.clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)


def _pool(blocks, hkv, d, g, outliers):
    """A pool in use: codes and scales of rows whose size differs from page to page and head to head."""
    size = torch.exp2(0.7 * _randn((blocks, 1, hkv, 1), g, torch.float32)).bfloat16()
    x = _randn((blocks, BLOCK, hkv, d), g) * size
    if outliers:  # a few tokens' keys draw a lot of attention
        hot = torch.randint(0, blocks * BLOCK, (max(1, blocks // 8),), generator=g, device="cuda")
        x.view(-1, hkv * d)[hot] *= 3
    scales = _need(x.abs().amax((1, 3)).float())
    codes = _codes(x / scales.bfloat16()[:, None, :, None])
    return codes, scales


def _tables(lens, g):
    """Block tables over a shuffled pool; block 0 belongs to nobody."""
    need = -(-lens // BLOCK)
    total = int(need.sum())
    blocks = total + total // 8 + 2
    perm = torch.randperm(blocks - 1, generator=g)[:total] + 1
    tables = torch.full((len(lens), max(1, int(need.max()))), -1, dtype=torch.int32)
    tables[torch.arange(tables.shape[1])[None, :] < torch.from_numpy(need)[:, None]] = perm.to(torch.int32)
    return tables, blocks


def prepare(case, seed):
    g, cpu = _gen(seed), _gen(seed, "cpu")
    op, hkv, d = case["op"], case["hkv"], case["d"]
    n, lens = _sizes(case)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    st = dict(case=case, q_start=torch.from_numpy(start).cuda(), new=int(n.max()), scale=d ** -0.5)
    rows = int(start[-1])
    if op in ("prompt", "append"):  # the rows of a fused projection
        hq = case.get("hq", hkv)
        qkv = _randn((rows, hq + 2 * hkv, d), g)
        qkv[:, hq:] *= torch.exp2(0.7 * _randn((1, 2 * hkv, 1), g))
        st["q"], st["k"], st["v"] = qkv.split([hq, hkv, hkv], dim=1)
    else:
        st["q"] = _randn((rows, case["hq"], d), g)
    if op != "prompt":
        tables, blocks = _tables(lens, cpu)
        st["tables"], st["lens"] = tables.cuda(), torch.from_numpy(lens.astype(np.int32)).cuda()
        st["longest"] = int(lens.max())
        st["kc"], st["ks"] = _pool(blocks, hkv, d, g, True)
        st["vc"], st["vs"] = _pool(blocks, hkv, d, g, False)
    return st


# ---------------------------------------------------------------- the framework's calls
def _call(st):
    from paged_kv_cache_52_gb300 import pagedkv

    case = st["case"]
    if case["op"] == "append":
        pagedkv.kv_append_fp8_block_scaled(st["k"], st["v"], st["q_start"], st["tables"], st["lens"], st["kc"],
                                           st["vc"], st["ks"], st["vs"])
        return _appended(st)
    if case["op"] == "prompt":
        return pagedkv.prompt_attention(st["q"], st["q_start"], st["k"], st["v"], True, st["scale"])
    S, hq, hkv, d = case["seqs"], case["hq"], case["hkv"], case["d"]
    if case["op"] == "decode":
        if "workspace" not in st:  # kept by the program from step to step
            st["workspace"] = pagedkv.decode_fp8_block_scaled_workspace(S, hq, hkv, d, st["q"].device)
        return pagedkv.paged_decode_attention_fp8_block_scaled(
            st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["tables"], st["lens"], st["scale"],
            max_context_len=st["longest"], workspace=st["workspace"], out_dtype=torch.bfloat16)
    if "workspace" not in st:
        st["workspace"] = pagedkv.prefill_fp8_block_scaled_workspace(S, st["tables"].shape[1], hkv, d, st["q"].device)
    return pagedkv.paged_prefill_attention_fp8_block_scaled(
        st["q"], st["q_start"], st["kc"], st["vc"], st["ks"], st["vs"], st["tables"], st["lens"], True, st["scale"],
        workspace=st["workspace"])


def _appended(st):
    kind = torch.float8_e4m3fn
    return dict(k=st["kc"].view(kind), v=st["vc"].view(kind), k_scales=st["ks"], v_scales=st["vs"])


# ---------------------------------------------------------------- the plain forms
def _append_plain(st):
    start, lens, tables = st["q_start"].long(), st["lens"].long(), st["tables"].clamp(min=0).long()
    n = start[1:] - start[:-1]
    base = lens - n
    row = torch.arange(st["k"].shape[0], device=start.device)
    seq = torch.searchsorted(start[1:].contiguous(), row, right=True)
    pos = base[seq] + row - start[seq]
    page = tables[seq, pos // BLOCK]
    # the page that each sequence's first new token lies in, where older rows of its own are before it
    held = (n > 0) & (base % BLOCK > 0)
    first = torch.where(held, torch.gather(tables, 1, (base // BLOCK)[:, None]).squeeze(1), 0)
    for rows, codes, scales in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
        rows = rows.float()
        amax = torch.zeros_like(scales).index_reduce_(0, page, rows.abs().amax(-1), "amax")
        old = torch.zeros_like(scales)
        old[first] = scales[first]  # block 0 is nobody's
        scale = torch.maximum(old, _need(amax))
        ratio = (old / scale)[first]
        older = codes[first]
        kept = (older.view(torch.float8_e4m3fn).float() * ratio[:, None, :, None])
        mine = (torch.arange(BLOCK, device=start.device) < (base % BLOCK)[:, None]) & held[:, None]
        codes[first] = torch.where(mine[:, :, None, None], _codes(kept), older)
        codes.view(-1, *codes.shape[2:])[page * BLOCK + pos % BLOCK] = _codes(rows / scale[page][:, :, None])
        touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=start.device)
        touched[page] = True
        scales.copy_(torch.where(touched[:, None], scale, scales))
    return _appended(st)


def _padded(st):
    """Row numbers [sequences, longest] of each sequence's new tokens, and which of them exist."""
    start = st["q_start"].long()
    t = torch.arange(st["new"], device=start.device)
    n = start[1:] - start[:-1]
    there = t[None, :] < n[:, None]
    return torch.where(there, start[:-1, None] + t, 0), there, n


def _attend(q, k, v, sees, scale):
    """q [S, N, Hq, d] over k, v [S, L, Hkv, d]; sees [S, N, L]."""
    S, N, hq, d = q.shape
    hkv = k.shape[2]
    q = q.float().view(S, N, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(S, hkv, -1, d)
    k, v = k.permute(0, 2, 3, 1), v.permute(0, 2, 1, 3)
    x = (q @ k).view(S, hkv, hq // hkv, N, -1).mul_(scale)
    x.masked_fill_(~sees[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x.sub_(top.masked_fill(top == float("-inf"), 0)).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x.view(S, hkv, -1, x.shape[-1]) @ v).view(S, hkv, hq // hkv, N, d)
    out = out / total.masked_fill(total == 0, 1)
    return out.permute(0, 3, 1, 2, 4).reshape(S, N, hq, d).bfloat16()


def _prompt_plain(st):
    rows, there, _ = _padded(st)
    t = torch.arange(st["new"], device=rows.device)
    sees = (t[None, :, None] >= t[None, None, :]) & there[:, None, :]
    return _attend(st["q"][rows], st["k"][rows].float(), st["v"][rows].float(), sees, st["scale"])[there]


def _cached(st):
    """Keys and values of every sequence from its pages, [S, positions, Hkv, d]."""
    tables = st["tables"].clamp(min=0).long()
    return [(c[tables].view(torch.float8_e4m3fn).float() * s[tables][:, :, None, :, None]).flatten(1, 2)
            for c, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"]))]


def _cached_plain(st):
    rows, there, n = _padded(st)
    k, v = _cached(st)
    t = torch.arange(st["new"], device=rows.device)
    last = (st["lens"].long() - n)[:, None] + t  # the last position each new token sees
    sees = torch.arange(k.shape[1], device=rows.device) <= torch.where(there, last, 0)[:, :, None]
    return _attend(st["q"][rows], k, v, sees, st["scale"])[there]


PLAIN = dict(append=_append_plain, prompt=_prompt_plain, decode=_cached_plain, prefill=_cached_plain)


def run(state):
    if own:
        return _call(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    n, lens = _sizes(case)
    rows, hkv, d = int(n.sum()), case["hkv"], case["d"]
    pages = -(-lens // BLOCK)
    if case["op"] == "append":
        touched = int((pages - (lens - n) // BLOCK).sum())
        return dict(bytes=rows * hkv * d * 6 + touched * hkv * 16, flops=4 * rows * hkv * d)
    pairs = int((n * (lens - n) + n * (n + 1) // 2).sum())  # (query, visible key)
    rows_bytes = rows * case["hq"] * d * 4
    if case["op"] == "prompt":
        return dict(bytes=rows_bytes + rows * hkv * d * 4, flops=4 * pairs * case["hq"] * d)
    cache = int(lens.sum()) * hkv * d * 2 + int(pages.sum()) * (hkv * 8 + 4)
    return dict(bytes=cache + rows_bytes, flops=4 * pairs * case["hq"] * d)


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _append_exact(st)
    start = st["q_start"].tolist()
    out = []
    for s in range(case["seqs"]):
        q = st["q"][start[s]:start[s + 1]].double()
        if case["op"] == "prompt":
            k, v = (st[x][start[s]:start[s + 1]].double() for x in "kv")
        else:
            L = int(st["lens"][s])
            pages = st["tables"][s, :-(-L // BLOCK)].long()
            k, v = ((st[c][pages].view(torch.float8_e4m3fn).double() * st[f][pages].double()[:, None, :, None])
                    .flatten(0, 1)[:L] for c, f in (("kc", "ks"), ("vc", "vs")))
        out.append(_rows_exact(q, k, v, st["scale"]))
    return torch.cat(out)


def _rows_exact(q, k, v, scale):
    """The last rows of a sequence, [n, Hq, d], over all of it, some rows and one KV head at a time."""
    n, hq, d = q.shape
    L, hkv = k.shape[:2]
    group = hq // hkv
    out = torch.empty_like(q)
    for a in range(0, n, 1024):
        b = min(n, a + 1024)
        seen = L - n + b  # no row of these sees further
        hidden = torch.arange(seen, device=q.device) > torch.arange(L - n + a, L - n + b, device=q.device)[:, None]
        for h in range(hkv):
            x = torch.einsum("tgd,ld->tgl", q[a:b, h * group:(h + 1) * group], k[:seen, h]) * scale
            x = x.masked_fill(hidden[:, None, :], -math.inf)
            out[a:b, h * group:(h + 1) * group] = torch.einsum("tgl,ld->tgd", torch.softmax(x, -1), v[:seen, h])
    return out


def _nearest(x):
    """The e4m3 value nearest to x (64 bits), ties to the even code."""
    _, power = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (power - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def _append_exact(st):
    start, lens, tables = (st[x].tolist() for x in ("q_start", "lens", "tables"))
    out = {}
    for name, rows, codes, scales in (("k", st["k"], st["kc"], st["ks"]), ("v", st["v"], st["vc"], st["vs"])):
        value, factor = codes.view(torch.float8_e4m3fn).double(), scales.double()
        for s, length in enumerate(lens):
            pos = length - (start[s + 1] - start[s])
            row = start[s]
            while pos < length:  # page by page
                page, a = tables[s][pos // BLOCK], pos % BLOCK
                b = min(BLOCK, a + length - pos)
                x = rows[row:row + b - a].double()
                # the least p from -126 on with 448 2^p at least the largest value: near its logarithm
                top = x.abs().amax((0, 2))
                p = torch.round(torch.log2(top / TOP).clamp(min=-126)) - 1
                p = (p + (TOP * torch.exp2(p) < top).double()).clamp(min=-126)
                p = p + (TOP * torch.exp2(p) < top).double()
                f = torch.maximum(torch.exp2(p), factor[page]) if a else torch.exp2(p)
                value[page, :a] = _nearest(value[page, :a] * (factor[page] / f)[:, None])
                value[page, a:b] = _nearest(x / f[:, None])
                factor[page] = f
                pos, row = pos + b - a, row + b - a
        out[name], out[name + "_scales"] = value, factor
    return dict(k=out["k"], v=out["v"], k_scales=out["k_scales"], v_scales=out["v_scales"])
