"""Prompts and steps over a block-scaled FP8 cache as a whole: norm + rotation into a
staging pool, prompt attention, quantizing append, decode steps, forks with
copied blocks and a chunk that continues a cached prefix, with the block manager's
tables; the same captured into graphs and replayed, and on two streams.
Tolerances are those of the single operators' tests."""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_52_gb300 import workloads as wl
from test_gpu_block_scaled import _check_rows
from test_gpu_prompt import _check

pytestmark = pytest.mark.gpu

DEV = "cuda"
BS = 16


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_52_gb300 import pagedkv
    pagedkv.get_device_error(clear=True)
    return pagedkv


def _start(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Cache:
    """One layer's block-scaled pools, and what they hold by the oracle's append."""

    def __init__(self, blocks, hkv, d):
        self.t = [torch.zeros(blocks, BS, hkv, d, dtype=torch.uint8, device=DEV) for _ in range(2)]
        self.t += [torch.zeros(blocks, hkv, device=DEV) for _ in range(2)]
        self.host = [x.cpu().numpy() for x in self.t]

    def append(self, pk, k, v, counts, tables, lens):
        pk.kv_append_fp8_block_scaled(k, v, _start(counts), tables.to(DEV), _i32(lens), *self.t)
        bits = [wl.bf16_bits(x.contiguous()) for x in (k, v)]
        self.host = list(oracle.append_block_scaled(*bits, _start(counts).tolist(),
                                                    tables.tolist(), lens, *self.host))
        for a, b in zip(self.t, self.host):
            assert np.array_equal(a.cpu().numpy(), b)

    def copy(self, pk, pairs):
        if pairs:
            pk.copy_blocks(self.t[0], self.t[1], _i32(pairs), k_scales=self.t[2],
                           v_scales=self.t[3])
            for x in self.host:
                for a, b in pairs:
                    x[b] = x[a]

    def case(self, q, tables, lens, scale):
        kc, vc, ks, vs = (torch.from_numpy(np.array(x)) for x in self.host)
        return dict(q=q.cpu(), kc=kc, vc=vc, ks=ks, vs=vs, tables=tables, lens=lens, scale=scale)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64)])
def test_a_prompts_life(pk, hq, hkv, d):
    g = torch.Generator().manual_seed(hq)
    rnd = lambda *shape: torch.randn(*shape, generator=g).bfloat16().to(DEV)
    scale = d ** -0.5
    bm = pk.BlockManager(80, BS)
    cache = Cache(80, hkv, d)
    width = 12
    prompts = [37, 100, 16, 5]
    ids = list(range(4))
    for s, n in zip(ids, prompts):
        bm.add_sequence(s, [1000 * s + i for i in range(n)])

    # the prompts: projections normed and rotated into a staging pool slot by slot
    T = sum(prompts)
    rows = -(-T // BS) * BS
    qkv = rnd(T, hq + 2 * hkv, d)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    stage = [torch.zeros(rows // BS, BS, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    table = torch.from_numpy(oracle.rope_table(200, d)).to(DEV)
    pos = torch.cat([torch.arange(n) for n in prompts]).to(DEV)
    qr = pk.qk_norm_rope_append(q, k, v, pos, table, torch.arange(T, device=DEV), *stage)
    kr, vr = (x.view(rows, hkv, d)[:T] for x in stage)
    out = pk.prompt_attention(qr, _start(prompts), kr, vr, True, scale).double().cpu().numpy()
    start = _start(prompts).tolist()
    f64 = [x.double().cpu().numpy() for x in (qr, kr, vr)]
    for s, n in enumerate(prompts):
        a, b = start[s], start[s + 1]
        _check(out[a:b], f64[0][a:b], f64[1][a:b], f64[2][a:b], scale, 0)
    tables, lens = bm.block_tables(ids, width)
    cache.append(pk, kr, vr, prompts, tables, lens.tolist())

    # a fork that shares its last block until one of the two writes into it
    bm.fork(1, 4)
    ids.append(4)
    for step in range(20):
        pairs = []
        for s in ids:
            pairs += bm.append_tokens(s, [7 * step + s])[1]
        cache.copy(pk, pairs)
        tables, lens = bm.block_tables(ids, width)
        lens = lens.tolist()
        kv = rnd(len(ids), 2 * hkv, d) * 2.0 ** (step % 5 - 2)   # scales that grow
        cache.append(pk, kv[:, :hkv], kv[:, hkv:], [1] * len(ids), tables, lens)
        q1 = rnd(len(ids), hq, d)
        got = pk.paged_decode_attention_fp8_block_scaled(q1, *cache.t, tables.to(DEV), _i32(lens),
                                                         scale)
        _check_rows(got.cpu().numpy(), cache.case(q1, tables, lens, scale), range(len(ids)))

    # a chunk on top of each sequence; one sequence has nothing new
    counts = [30, 0, 1, 17, 8]
    for s, n in zip(ids, counts):
        if n:
            cache.copy(pk, bm.append_tokens(s, [9000 + i for i in range(n)])[1])
    tables, lens = bm.block_tables(ids, width)
    lens = lens.tolist()
    kv, q2 = rnd(sum(counts), 2 * hkv, d), rnd(sum(counts), hq, d)
    cache.append(pk, kv[:, :hkv], kv[:, hkv:], counts, tables, lens)
    got = pk.paged_prefill_attention_fp8_block_scaled(
        q2, _start(counts), *cache.t, tables.to(DEV), _i32(lens), True, scale)
    kd, vd = (oracle.dequantize_blocks(cache.host[i], cache.host[i + 2]) for i in (0, 1))
    start = _start(counts).tolist()
    for s, (n, L) in enumerate(zip(counts, lens)):
        if n:
            kk, vv = (x[tables[s, :-(-L // BS)].tolist()].reshape(-1, hkv, d)[:L] for x in (kd, vd))
            a, b = start[s], start[s + 1]
            _check(got[a:b].double().cpu().numpy(), q2[a:b].double().cpu().numpy(), kk, vv, scale,
                   L - n)
    assert pk.get_device_error(clear=True) == 0
    bm.close()


def _step_state(pk, lens, hq, hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    S = len(lens)
    width = 40
    tables = (torch.randperm(S * width, generator=g) + 1).int().view(S, width)
    cache = Cache(S * width + 1, hkv, d)
    for x, y in zip(cache.t[:2], cache.t[2:]):
        x.copy_((torch.randint(0, 127, x.shape, generator=g)).to(torch.uint8))
        y.copy_(torch.exp2(torch.randint(-9, -6, y.shape, generator=g).float()))
    cache.host = [x.cpu().numpy() for x in cache.t]
    return dict(cache=cache, tables=tables, lens=_i32(lens), S=S,
                kv=torch.randn(S, 2 * hkv, d, generator=g).bfloat16().to(DEV),
                q=torch.randn(S, hq, d, generator=g).bfloat16().to(DEV), hkv=hkv, d=d,
                dev_tables=tables.to(DEV), start=_start([1] * S),
                ws=pk.decode_fp8_block_scaled_workspace(S, hq, hkv, d, DEV),
                out=torch.zeros(S, hq, d, device=DEV))


def _step(pk, st):
    k, v = st["kv"].split([st["hkv"]] * 2, 1)
    pk.kv_append_fp8_block_scaled(k, v, st["start"], st["dev_tables"], st["lens"], *st["cache"].t)
    pk.paged_decode_attention_fp8_block_scaled(
        st["q"], *st["cache"].t, st["dev_tables"], st["lens"], st["d"] ** -0.5, out=st["out"],
        max_context_len=640, workspace=st["ws"])


def _check_step(st, lens):
    c = st["cache"]
    k, v = (wl.bf16_bits(x.contiguous()) for x in st["kv"].split([st["hkv"]] * 2, 1))
    c.host = list(oracle.append_block_scaled(k, v, st["start"].tolist(), st["tables"].tolist(),
                                             lens, *c.host))
    for a, b in zip(c.t, c.host):
        assert np.array_equal(a.cpu().numpy(), b)
    _check_rows(st["out"].cpu().numpy(), c.case(st["q"], st["tables"], lens, st["d"] ** -0.5),
                range(0, st["S"], max(1, st["S"] // 8)))


@pytest.mark.parametrize("S,hkv,d", [(3, 2, 128), (300, 2, 64)])
def test_a_captured_step_replays_with_other_lengths(pk, S, hkv, d):
    """The cluster split and the flat one; every replay sees what the step before wrote."""
    lens = [1 + (37 * i) % 600 for i in range(S)]
    st = _step_state(pk, lens, 4 * hkv, hkv, d, S)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        warm = _step_state(pk, lens, 4 * hkv, hkv, d, S + 1)
        _step(pk, warm)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            _step(pk, st)
    for step in range(3):
        now = [n + step for n in lens]
        st["lens"].copy_(_i32(now))
        st["kv"].mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        _check_step(st, now)
    assert pk.get_device_error(clear=True) == 0


def test_steps_on_two_streams(pk):
    """Two batches at once, each with a workspace of its own."""
    a = _step_state(pk, [(11 * i) % 500 + 1 for i in range(200)], 8, 4, 128, 1)
    b = _step_state(pk, [(17 * i) % 600 + 1 for i in range(30)], 16, 2, 64, 2)
    first = [x["lens"].tolist() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):  # the same step again: the same cache
        for st, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                _step(pk, st)
    torch.cuda.synchronize()
    for st, lens in zip((a, b), first):
        _check_step(st, lens)
    assert pk.get_device_error(clear=True) == 0


def test_prompts_captured_beside_other_work(pk):
    """Prompt attention in a graph, replayed with other starts, beside a decode stream."""
    g = torch.Generator().manual_seed(8)
    hq, hkv, d = 4, 2, 128
    qkv = torch.randn(400, hq + 2 * hkv, d, generator=g).bfloat16().to(DEV)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    start = _start([100, 200, 50])
    out = torch.zeros(400, hq, d, dtype=torch.bfloat16, device=DEV)
    other = _step_state(pk, [(17 * i) % 600 + 1 for i in range(30)], 16, 2, 64, 2)
    stream, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        pk.prompt_attention(q, start, k, v, True, 0.1, out=out)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            pk.prompt_attention(q, start, k, v, True, 0.1, out=out)
    for counts in ([100, 200, 50], [1, 0, 399], [130, 130, 130]):
        start.copy_(_start(counts))
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            _step(pk, other)
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        x = [t.double().cpu().numpy() for t in (q, k, v)]
        s = _start(counts).tolist()
        for i in range(3):
            a, b = s[i], s[i + 1]
            if b > a:
                _check(out[a:b].double().cpu().numpy(), x[0][a:b], x[1][a:b], x[2][a:b], 0.1, 0)
        assert not out[s[3]:].any()
    assert pk.get_device_error(clear=True) == 0


@pytest.mark.parametrize("lens", [[40, 1, 333], [17] * 300])
def test_pools_past_32_bits(pk, lens):
    """Blocks at the far end of pools of 4.3 GB: as in small ones, bit for bit."""
    hq, hkv, d = 16, 8, 128
    g = torch.Generator().manual_seed(5)
    need = [-(-n // BS) for n in lens]
    near = torch.arange(sum(need) + 1, dtype=torch.int32)
    tables = torch.zeros(len(lens), max(need), dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = near[at:at + n]
        at += n
    blocks = (1 << 32) // (BS * hkv * d) + 512
    kv = torch.randn(sum(lens), 2 * hkv, d, generator=g).bfloat16().to(DEV)
    q = torch.randn(len(lens), hq, d, generator=g).bfloat16().to(DEV)
    rows = torch.randn(sum(lens), hq, d, generator=g).bfloat16().to(DEV)
    results = []
    for count, shift in ((at + 1, 0), (blocks, blocks - at - 1)):
        pools = [torch.empty(count, BS, hkv, d, dtype=torch.uint8, device=DEV) for _ in "kv"]
        scales = [torch.empty(count, hkv, device=DEV) for _ in "kv"]
        t = (tables + shift).to(DEV)
        for x in pools:
            x[shift:].zero_()
        pk.kv_append_fp8_block_scaled(*kv.split([hkv] * 2, 1), _start(lens).to(DEV), t,
                                      _i32(lens), *pools, *scales)
        pairs = torch.tensor([[shift, shift + at]], dtype=torch.int32, device=DEV)
        pk.copy_blocks(*pools, pairs, *scales)
        results.append([x[shift:].clone() for x in pools + scales] + [
            pk.paged_decode_attention_fp8_block_scaled(q, *pools, *scales, t, _i32(lens), 0.1),
            pk.paged_prefill_attention_fp8_block_scaled(rows, _start(lens).to(DEV), *pools, *scales,
                                                        t, _i32(lens), True, 0.1)])
        assert pk.get_device_error(clear=True) == 0
    for a, b in zip(*results):
        assert torch.equal(a, b)
    for x in results[1][:4]:
        assert torch.equal(x[at], x[0])
