"""Norm + rotation + append in one pass, against the float64 oracle.

Tolerance: with y the exact value and m the largest |x inv w| of its pair,
float32 rounding leaves at most 8 half-steps of 2^-24 on each of the two
products and the sum over d squares adds (d / 2 + 4) 2^-24 to the norm's factor: the
float32 value is off by (d / 2 + 24) 2^-24 * 2 m; the stored bf16 by half a
step more, 2^-8 |y| (plus 2^-134, half the smallest subnormal).
"""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_52_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_52_gb300 import pagedkv
    pagedkv.get_device_error(clear=True)
    return pagedkv


def _inputs(T, hq, hkv, d, rot, norm=True, seed=0, table_rows=5000, fused=True):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, hq + 2 * hkv, d, generator=g) * 2).bfloat16()
    if not fused:
        q, k, v = (x.contiguous() for x in qkv.split([hq, hkv, hkv], 1))
    else:
        q, k, v = qkv.to(DEV).split([hq, hkv, hkv], 1)
    blocks = -(-T // 16) + 3
    slots = torch.randperm(blocks * 16, generator=g)[:T]
    if T > 4:
        slots[::5] = -1
    w = [(1 + 0.3 * torch.randn(d, generator=g)).bfloat16() if norm else None for _ in range(2)]
    return dict(q=q.to(DEV), k=k.to(DEV), v=v.to(DEV),
                positions=torch.randint(0, table_rows, (T,), generator=g).to(DEV),
                table=torch.from_numpy(oracle.rope_table(table_rows, rot)).to(DEV),
                slots=slots.to(DEV), blocks=blocks, g=g,
                qw=w[0].to(DEV) if norm else None, kw=w[1].to(DEV) if norm else None)


def _bits(t):
    return wl.bf16_bits(t.contiguous())


def _want(x, w, a, eps, inter):
    pos, table = a["positions"].cpu().numpy(), a["table"].cpu().numpy()
    return oracle.norm_rope(_bits(x), None if w is None else _bits(w), pos, table, eps, inter)


def _slack(x, w, eps):
    y = oracle.bf16_bits_to_f64(_bits(x))
    d = y.shape[-1]
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * oracle.bf16_bits_to_f64(_bits(w))
    return (d / 2 + 24) * 2.0 ** -24 * 2 * np.abs(y).max(-1, keepdims=True)


def _close(got, want, slack):
    diff = np.abs(oracle.bf16_bits_to_f64(_bits(got)) - want)
    tol = slack + 2.0 ** -8 * (np.abs(want) + slack) + 2.0 ** -134
    assert (diff <= tol).all(), float((diff - tol).max())


CASES = [(1, 32, 32, 128, 128, False), (1, 1, 1, 64, 16, True), (37, 8, 2, 64, 32, False),
         (37, 8, 2, 64, 64, True), (200, 64, 8, 128, 128, False), (33, 5, 3, 128, 48, False),
         (33, 5, 3, 128, 48, True), (700, 16, 1, 128, 64, True), (2049, 12, 4, 64, 64, False)]


@pytest.mark.parametrize("T,hq,hkv,d,rot,inter", CASES)
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope_append(pk, T, hq, hkv, d, rot, inter, norm):
    a = _inputs(T, hq, hkv, d, rot, norm, seed=T + d, fused=T % 2 == 1)
    kc = torch.randn(a["blocks"], 16, hkv, d, generator=a["g"]).bfloat16().to(DEV)
    vc = torch.randn(a["blocks"], 16, hkv, d, generator=a["g"]).bfloat16().to(DEV)
    k0, v0 = kc.clone(), vc.clone()
    eps = 1e-5
    out = pk.qk_norm_rope_append(a["q"], a["k"], a["v"], a["positions"], a["table"], a["slots"],
                                 kc, vc, a["qw"], a["kw"], eps, inter)
    torch.cuda.synchronize()
    assert pk.get_device_error(clear=True) == 0
    _close(out, _want(a["q"], a["qw"], a, eps, inter), _slack(a["q"], a["qw"], eps))
    keep = a["slots"] >= 0
    at = a["slots"][keep]
    want = _want(a["k"], a["kw"], a, eps, inter)[keep.cpu().numpy()]
    _close(kc.view(-1, hkv, d)[at], want, _slack(a["k"][keep], a["kw"], eps))
    assert torch.equal(vc.view(-1, hkv, d)[at], a["v"][keep])
    k0.view(-1, hkv, d)[at] = kc.view(-1, hkv, d)[at]
    v0.view(-1, hkv, d)[at] = a["v"][keep]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)  # nothing else changed


@pytest.mark.parametrize("T,hq,hkv,d,rot,inter", [CASES[0], CASES[2], CASES[4], CASES[7]])
def test_fp8_pools_hold_the_nearest_codes(pk, T, hq, hkv, d, rot, inter):
    # V's codes are the plain append's, bit for bit; K's are the nearest to
    # the exact value, or the neighbour where that lies within the float32
    # slack of the border between two codes
    a = _inputs(T, hq, hkv, d, rot, True, seed=T)
    kc = torch.zeros(a["blocks"], 16, hkv, d, dtype=torch.uint8, device=DEV)
    vc, k8, v8 = (torch.zeros_like(kc) for _ in range(3))
    ks, vs = 0.037, 0.05
    out = pk.qk_norm_rope_append_fp8(a["q"], a["k"], a["v"], a["positions"], a["table"],
                                     a["slots"], kc, vc, ks, vs, a["qw"], a["kw"], 1e-6, inter)
    pk.kv_append_fp8(a["k"], a["v"], a["slots"], k8, v8, ks, vs)
    torch.cuda.synchronize()
    assert pk.get_device_error(clear=True) == 0
    _close(out, _want(a["q"], a["qw"], a, 1e-6, inter), _slack(a["q"], a["qw"], 1e-6))
    assert torch.equal(vc, v8)
    keep = (a["slots"] >= 0).cpu().numpy()
    want = _want(a["k"], a["kw"], a, 1e-6, inter)[keep] * (1 / np.float32(ks)).astype(np.float64)
    want = np.clip(want, -448, 448)
    slack = _slack(a["k"], a["kw"], 1e-6)[keep] / ks + np.abs(want) * 2.0 ** -23
    got = oracle.e4m3_bits_to_f64(kc.view(-1, hkv, d)[a["slots"][a["slots"] >= 0]].cpu().numpy())
    # half a step: 2^-4 of the value, 2^-10 among the subnormals
    assert (np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + slack).all()


def test_far_positions_and_zero_rows(pk):
    a = _inputs(64, 4, 2, 128, 128, True, seed=4, table_rows=200000)
    a["positions"][:3] = torch.tensor([199999, 0, 131072])
    a["q"][1] = 0
    a["k"][2] = 0
    kc = torch.zeros(a["blocks"], 16, 2, 128, dtype=torch.bfloat16, device=DEV)
    out = pk.qk_norm_rope_append(a["q"], a["k"], a["v"], a["positions"], a["table"], a["slots"],
                                 kc, torch.zeros_like(kc), a["qw"], a["kw"])
    _close(out, _want(a["q"], a["qw"], a, 1e-6, False), _slack(a["q"], a["qw"], 1e-6))
    assert (out[1] == 0).all()


def test_infinities_stay_in_their_head(pk):
    # elements beyond the rotated ones pass through, an infinity does not
    # touch the other heads or tokens
    a = _inputs(9, 4, 2, 64, 32, False, seed=5)
    kc = torch.zeros(a["blocks"], 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    clean = pk.qk_norm_rope_append(a["q"], a["k"], a["v"], a["positions"], a["table"],
                                   a["slots"], kc, torch.zeros_like(kc))
    a["q"][3, 1, 40] = float("inf")
    for inter in (False, True):
        out = pk.qk_norm_rope_append(a["q"], a["k"], a["v"], a["positions"], a["table"],
                                     a["slots"], kc, torch.zeros_like(kc), interleaved=inter)
        assert out[3, 1, 40] == float("inf")
        assert torch.equal(out[3, 1, 32:40], a["q"][3, 1, 32:40])
        assert torch.isfinite(out[:, [0, 2, 3]]).all() and int((~torch.isfinite(out)).sum()) == 1
    del clean


def test_bad_positions_and_slots_are_skipped_and_flagged(pk):
    a = _inputs(6, 4, 2, 64, 64, True, seed=6, table_rows=100)
    a["slots"] = torch.tensor([0, 1, 2, 3, 16 * a["blocks"], -2], device=DEV)
    a["positions"][1], a["positions"][2] = -1, 100
    kc = torch.zeros(a["blocks"], 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    out = torch.full((6, 4, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    pk.qk_norm_rope_append(a["q"], a["k"], a["v"], a["positions"], a["table"], a["slots"], kc, vc,
                           a["qw"], a["kw"], out=out)
    torch.cuda.synchronize()
    assert pk.get_device_error(clear=True) == 0x201
    assert (out[1:3] == 9).all() and not (out[[0, 3, 4, 5]] == 9).any()
    written = (vc.view(-1, 128) != 0).any(1).nonzero().flatten().tolist()
    assert written == [0, 3] and torch.equal(kc.view(-1, 128)[1:3], torch.zeros_like(kc.view(-1, 128)[1:3]))


def test_refusals(pk):
    a = _inputs(4, 4, 2, 64, 64, True, seed=7)
    kc = torch.zeros(a["blocks"], 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)

    def call(**kw):
        x = dict(q=a["q"], k=a["k"], v=a["v"], positions=a["positions"], rope_table=a["table"],
                 slot_mapping=a["slots"], k_cache=kc, v_cache=vc, q_weight=a["qw"],
                 k_weight=a["kw"])
        x.update(kw)
        return pk.qk_norm_rope_append(**x)

    for bad in (dict(q=a["q"].float()), dict(k=a["k"][:3]), dict(positions=a["positions"].int()),
                dict(rope_table=a["table"].double()), dict(q_weight=a["qw"].float()),
                dict(slot_mapping=a["slots"].cpu()), dict(v=a["v"].transpose(1, 2)),
                dict(rope_table=a["table"].cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad, status in ((dict(rope_table=a["table"][:, :24].contiguous()), -2),
                        (dict(eps=float("nan")), -1), (dict(eps=-1.0), -1)):
        with pytest.raises(pk.PagedKVError) as e:
            call(**bad)
        assert e.value.status == status
    q = a["q"].contiguous()
    with pytest.raises(pk.PagedKVError) as e:      # in place: another warp's input
        call(q=q, out=q)
    assert e.value.status == -1
    empty = call(q=a["q"][:0], k=a["k"][:0], v=a["v"][:0], positions=a["positions"][:0],
                 slot_mapping=a["slots"][:0])
    assert empty.shape == (0, 4, 64)


def test_replay_side_stream_and_two_calls_at_once(pk):
    # two appends on two streams into their own pools, and one captured and
    # replayed with other tokens, give what plain calls give
    calls = []
    for seed in (1, 2):
        a = _inputs(150, 8, 2, 128, 64, seed=seed)
        pools = [torch.zeros(a["blocks"], 16, 2, 128, dtype=torch.bfloat16, device=DEV)
                 for _ in range(2)]
        calls.append((a, pools))

    def run(a, pools):
        return pk.qk_norm_rope_append(a["q"], a["k"], a["v"], a["positions"], a["table"],
                                      a["slots"], *pools, a["qw"], a["kw"], 1e-6)

    want = []
    for a, pools in calls:
        out = run(a, pools)
        torch.cuda.synchronize()
        want.append([out.clone()] + [p.clone() for p in pools])
        for p in pools:
            p.zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = []
    for (a, pools), s in zip(calls, streams):
        with torch.cuda.stream(s):
            got.append([run(a, pools)] + pools)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))
    # captured with the first call's tensors, replayed with the second's contents
    a, pools = calls[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(a, pools)
    b = calls[1][0]
    for name in ("q", "k", "v", "positions", "table", "slots", "qw", "kw"):
        a[name].copy_(b[name])
    for p in pools:
        p.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip([out] + pools, want[1]))
    assert pk.get_device_error(clear=True) == 0
