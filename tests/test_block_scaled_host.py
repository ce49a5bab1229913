"""The block-scaled cache and prompt attention without a GPU: refusals at the C
entries (nothing is dereferenced or launched), workspace sizes, and the oracle
against plain identities."""

import ctypes

import numpy as np
import pytest

import oracle


@pytest.fixture(scope="module")
def pk():
    import os
    from paged_kv_cache_52_gb300 import build as b
    if not os.path.exists(b.LIB_PATH):
        b.build()
    from paged_kv_cache_52_gb300 import pagedkv
    return pagedkv


OK, EINVAL, EUNSUPPORTED, ENOMEM = 0, -1, -2, -4
P = ctypes.c_void_p


def at(mb, off=0):
    return P((mb << 24) + off)


def desc(pk, nb=64, bs=16, hkv=2, d=64):
    return pk.CacheDesc(nb, bs, hkv, d)


def append(pk, **a):
    c = a.get("cache", desc(pk))
    row = 128
    return pk.lib.pkv_kv_append_fp8_block_scaled(
        a.get("k", at(1)), a.get("ks", row), a.get("v", at(2)), a.get("vs", row), a.get("T", 4),
        a.get("start", at(3)), a.get("S", 2), a.get("tables", at(4)), a.get("width", 8),
        a.get("lens", at(5)), a.get("kc", at(6)), a.get("vc", at(7)), a.get("kscale", at(8)),
        a.get("vscale", at(9)), c, P(0))


def test_append_refusals(pk):
    assert append(pk, T=0, k=P(0)) == OK and append(pk, S=0, start=P(0)) == OK
    assert append(pk, T=-1) == EINVAL and append(pk, S=-1) == EINVAL
    for name in ("k", "v", "start", "tables", "lens", "kc", "vc", "kscale", "vscale"):
        assert append(pk, **{name: P(0)}) == EINVAL, name
    for name, off in (("k", 8), ("v", 2), ("kc", 8), ("vc", 4), ("kscale", 2), ("vscale", 1),
                      ("start", 2), ("tables", 1), ("lens", 2)):
        assert append(pk, **{name: at(30, off)}) == EINVAL, name
    assert append(pk, ks=120) == EINVAL and append(pk, vs=132) == EINVAL
    assert append(pk, width=0) == EINVAL and append(pk, width=2 ** 28) == EUNSUPPORTED
    assert append(pk, cache=desc(pk, bs=8)) == EUNSUPPORTED
    assert append(pk, cache=desc(pk, d=96)) == EUNSUPPORTED
    assert append(pk, cache=desc(pk, hkv=0)) == EINVAL
    assert append(pk, T=2 ** 31) == EUNSUPPORTED
    # pools, or scales, over one another (a pool is 64 x 16 x 128 bytes)
    assert append(pk, vc=at(6, 64 * 16 * 128 - 16)) == EINVAL
    assert append(pk, vscale=at(8, 64 * 2 * 4 - 4)) == EINVAL


def decode(pk, **a):
    fn = (pk.lib.pkv_paged_decode_attention_fp8_block_scaled_bf16out if a.get("bf16")
          else pk.lib.pkv_paged_decode_attention_fp8_block_scaled)
    return fn(a.get("q", at(1)), a.get("S", 2), a.get("hq", 4), a.get("kc", at(2)),
              a.get("vc", at(3)), a.get("kscale", at(4)), a.get("vscale", at(5)),
              a.get("cache", desc(pk)), a.get("tables", at(6)), a.get("width", 8),
              a.get("lens", at(7)), a.get("longest", 100), a.get("scale", 1.0),
              a.get("out", at(8)), a.get("ws", at(9)), a.get("bytes", 1 << 40), P(0))


@pytest.mark.parametrize("bf16", [False, True])
def test_decode_refusals(pk, bf16):
    assert decode(pk, bf16=bf16, S=0, q=P(0)) == OK
    for name in ("q", "kc", "vc", "kscale", "vscale", "tables", "lens", "out"):
        assert decode(pk, bf16=bf16, **{name: P(0)}) == EINVAL, name
    for name, off in (("q", 8), ("kc", 8), ("vc", 1), ("kscale", 2), ("vscale", 2), ("tables", 2),
                      ("lens", 1), ("out", 1)):
        assert decode(pk, bf16=bf16, **{name: at(30, off)}) == EINVAL, name
    assert decode(pk, bf16=bf16, hq=3) == EUNSUPPORTED       # not a multiple
    assert decode(pk, bf16=bf16, hq=6) == EUNSUPPORTED       # a group of 3
    assert decode(pk, bf16=bf16, hq=0) == EINVAL and decode(pk, bf16=bf16, S=-1) == EINVAL
    assert decode(pk, bf16=bf16, longest=-1) == EINVAL
    assert decode(pk, bf16=bf16, scale=float("nan")) == EINVAL
    assert decode(pk, bf16=bf16, width=0) == EINVAL
    assert decode(pk, bf16=bf16, cache=desc(pk, d=32)) == EUNSUPPORTED
    need = pk.lib.pkv_decode_fp8_block_scaled_workspace_bytes(2, 4, 2, 64)
    assert need > 0 and decode(pk, bf16=bf16, bytes=need - 1) == ENOMEM
    assert decode(pk, bf16=bf16, ws=P(0)) == ENOMEM
    assert decode(pk, bf16=bf16, ws=at(9, 128)) == EINVAL


def prompt(pk, **a):
    return pk.lib.pkv_prompt_attention(
        a.get("q", at(1)), a.get("qs", 256), a.get("start", at(2)), a.get("S", 2), a.get("T", 10),
        a.get("hq", 4), a.get("k", at(3)), a.get("ks", 128), a.get("v", at(4)), a.get("vs", 128),
        a.get("hkv", 2), a.get("d", 64), 1, a.get("scale", 1.0), a.get("out", at(5)), P(0))


def test_prompt_refusals(pk):
    assert prompt(pk, T=0, q=P(0)) == OK and prompt(pk, S=0, q=P(0)) == OK
    for name in ("q", "start", "k", "v", "out"):
        assert prompt(pk, **{name: P(0)}) == EINVAL, name
    for name, off in (("q", 8), ("k", 8), ("v", 2), ("out", 16), ("start", 2)):
        assert prompt(pk, **{name: at(30, off)}) == EINVAL, name
    assert prompt(pk, qs=248) == EINVAL and prompt(pk, ks=120) == EINVAL and prompt(pk, vs=132) == EINVAL
    assert prompt(pk, qs=1 << 39) == EUNSUPPORTED
    assert prompt(pk, d=80) == EUNSUPPORTED and prompt(pk, hq=3) == EUNSUPPORTED
    assert prompt(pk, hkv=0) == EINVAL and prompt(pk, T=-1) == EINVAL and prompt(pk, S=-1) == EINVAL
    assert prompt(pk, T=2 ** 31 - 1) == EUNSUPPORTED
    assert prompt(pk, scale=float("inf")) == EINVAL
    for name in ("q", "k", "v"):   # the output over an input
        assert prompt(pk, **{name: at(5, 1024)}) == EINVAL, name


def prefill(pk, **a):
    return pk.lib.pkv_paged_prefill_attention_fp8_block_scaled(
        a.get("q", at(1)), a.get("start", at(2)), a.get("S", 2), a.get("T", 10), a.get("hq", 4),
        a.get("kc", at(3)), a.get("vc", at(4)), a.get("kscale", at(5)), a.get("vscale", at(6)),
        a.get("cache", desc(pk)), a.get("tables", at(7)), a.get("width", 8), a.get("lens", at(8)),
        1, a.get("scale", 1.0), a.get("out", at(9)), a.get("ws", at(10)), a.get("bytes", 1 << 40),
        P(0))


def test_prefill_refusals(pk):
    assert prefill(pk, T=0, q=P(0)) == OK and prefill(pk, S=0, q=P(0)) == OK
    for name in ("q", "start", "kc", "vc", "kscale", "vscale", "tables", "lens", "out"):
        assert prefill(pk, **{name: P(0)}) == EINVAL, name
    for name, off in (("q", 8), ("out", 16), ("kscale", 2), ("vscale", 2), ("kc", 8), ("vc", 8),
                      ("start", 2), ("tables", 2), ("lens", 2)):
        assert prefill(pk, **{name: at(30, off)}) == EINVAL, name
    assert prefill(pk, hq=6) == EUNSUPPORTED and prefill(pk, scale=float("nan")) == EINVAL
    assert prefill(pk, width=2 ** 26) == EUNSUPPORTED and prefill(pk, width=0) == EINVAL
    need = pk.lib.pkv_prefill_fp8_block_scaled_workspace_bytes(2, 8, 2, 64)
    assert need == 2 * 2 * 8 * 16 * 2 * 64 * 2
    assert prefill(pk, bytes=need - 1) == ENOMEM and prefill(pk, ws=P(0)) == ENOMEM
    assert prefill(pk, ws=at(10, 16)) == EINVAL and prefill(pk, out=at(1, 64)) == EINVAL
    assert pk.lib.pkv_prefill_fp8_block_scaled_workspace_bytes(0, 8, 2, 64) == 0
    assert pk.lib.pkv_prefill_fp8_block_scaled_workspace_bytes(2 ** 20, 2 ** 10, 2, 64) == 0


def test_copy_of_scales_refusals(pk):
    fn, c = pk.lib.pkv_copy_block_scales, desc(pk)
    assert fn(P(0), P(0), c, P(0), 0, P(0)) == OK
    assert fn(P(0), at(1), c, at(2), 1, P(0)) == EINVAL
    assert fn(at(1), at(2), c, P(0), 1, P(0)) == EINVAL
    assert fn(at(1, 2), at(2), c, at(3), 1, P(0)) == EINVAL
    assert fn(at(1), at(2), c, at(3), -1, P(0)) == EINVAL


def test_decode_workspace_covers_pairs_and_warps(pk):
    ws = pk.lib.pkv_decode_fp8_block_scaled_workspace_bytes
    assert ws(0, 4, 2, 64) > 0 and ws(5, 4, 2, 64) >= (5 * 2 + 12) * 2 * (64 + 1) * 4
    assert ws(5000, 4, 2, 64) == ws(1024, 4, 2, 64)     # a launch takes 1024 at most
    assert ws(5, 6, 2, 64) == 0 and ws(5, 4, 2, 80) == 0 and ws(-1, 4, 2, 64) == 0
    assert ws(1, 2 ** 20, 2 ** 20, 64) == 0             # more KV heads than warps


# ------------------------------------------------------------------- oracle
def test_the_scale_is_the_least_power_of_two_that_holds_the_block():
    rng = np.random.default_rng(0)
    for x in np.concatenate([rng.standard_normal(50) * 10.0 ** rng.integers(-30, 30, 50),
                             [448.0, 448.0001, 896.0, 2.0 ** -117, 1e-45]]):
        s = oracle.block_scale([x, 0.0])
        assert s == 2.0 ** round(np.log2(s)) and abs(x) <= 448 * s
        assert s == 2.0 ** -126 or abs(x) > 448 * s / 2
    assert oracle.block_scale([0.0]) == oracle.block_scale([np.nan, np.inf]) == 2.0 ** -126


def test_appending_row_by_row_ends_where_appending_at_once_does():
    """Scales only grow, and a power of two moves a code exactly unless it becomes
    subnormal: with values within 2^5 of one another both ways give the same cache."""
    rng = np.random.default_rng(1)
    n, hkv, d = 16, 2, 8
    x = ((1 + rng.integers(0, 8, (n, hkv, d)) / 8) * 2.0 ** rng.integers(0, 5, (n, hkv, d)))
    bits = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    empty = [np.zeros((2, 16, hkv, d), np.uint8)] * 2 + [np.zeros((2, hkv), np.float32)] * 2
    once = oracle.append_block_scaled(bits, bits, [0, n], [[1]], [n], *empty)
    step = empty
    for i in range(n):
        step = oracle.append_block_scaled(bits[i:i + 1], bits[i:i + 1], [0, 1], [[1]], [i + 1],
                                          *step)
    for a, b in zip(once, step):
        assert np.array_equal(a, b)
    assert np.array_equal(oracle.dequantize_blocks(once[0], once[2])[1], x)


def test_attend_is_a_softmax_over_what_a_row_sees():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal(s) for s in ((3, 4, 8), (10, 2, 8), (10, 2, 8)))
    out, size = oracle.attend(q, k, v, 0.5, 7)
    for i in range(3):
        for h in range(4):
            w = np.exp(k[:8 + i, h // 2] @ q[i, h] * 0.5)
            assert np.allclose(out[i, h], w @ v[:8 + i, h // 2] / w.sum())
    assert (size >= np.abs(out) - 1e-12).all()
