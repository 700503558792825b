"""The 8-bit cache on the host: the oracle's pins and every call's refusals.  No call here reaches a CUDA API."""
import numpy as np
import pytest
import torch

import oracle

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from linear_hybrid_attention_b200 import build, _lib
    build.build()
    return _lib.load()


# ------------------------------------------------------------ oracle's pins ----
def test_e4m3_values_are_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oracle.E4M3_VALUES, codes)
    assert oracle.E4M3_VALUES[-1] == 448.0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_oracle_quantiser(fmt):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 64)) * np.exp(rng.standard_normal(64))
    c, s = oracle.quantise_block(x, fmt)
    top = 127.0 if fmt == "int8" else 448.0
    assert np.abs(c).max() == top and s == np.float32(np.abs(x).max() / top)
    if fmt == "int8":
        np.testing.assert_array_equal(c, np.rint(x / s))
    else:  # torch rounds fp64 to e4m3 through fp32: off the ties the nearest is the nearest
        np.testing.assert_array_equal(c, torch.from_numpy(x / s).to(torch.float8_e4m3fn).double().numpy())
    # scale 1: every value of the format stands for itself, ties go to the even code
    top_row = np.zeros((1, 64)); top_row[0, 0] = top
    ties = {"int8": ([0.5, 1.5, 2.5, -3.5], [0, 2, 2, -4]),
            "e4m3": ([17.0, 19.0, 1.0625, 2.0 ** -10, 3 * 2.0 ** -10], [16, 20, 1.0, 0, 2.0 ** -8])}[fmt]
    top_row[0, 1:1 + len(ties[0])] = ties[0]
    c, s = oracle.quantise_block(top_row, fmt)
    assert s == 1.0
    np.testing.assert_array_equal(c[0, 1:1 + len(ties[0])], ties[1])
    c, s = oracle.quantise_block(np.zeros((2, 64)), fmt)
    assert s == 0.0 and not c.any()
    assert np.isnan(oracle.quantise_block(np.full((2, 64), np.inf), fmt)[1])


def test_oracle_attention():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((2, 3, 64)), rng.standard_normal((40, 64)), rng.standard_normal((40, 64))
    O, lse, mass = oracle.cache_attention(q, k, v, 0.125, False, 16)
    want = torch.nn.functional.scaled_dot_product_attention(*(torch.from_numpy(x)[None] for x in
                                                              (q.reshape(1, 6, 64), k[None], v[None])))[0, 0]
    np.testing.assert_allclose(O.reshape(6, 64), want.numpy(), atol=1e-12)
    assert mass.shape == (3,) and mass.sum() == pytest.approx(6)
    # causal: the last query sees everything, each earlier one a key less; alone, it equals a shorter cache
    Oc, lc, mc = oracle.cache_attention(q, k, v, 0.125, True, 16)
    np.testing.assert_allclose(Oc[:, 2], O[:, 2], atol=1e-13)
    np.testing.assert_allclose(Oc[:, 0], oracle.cache_attention(q[:, :1], k[:38], v[:38], 0.125, False, 16)[0][:, 0],
                               atol=1e-13)
    # rows that see nothing
    O, lse, mass = oracle.cache_attention(q, k[:2], v[:2], 0.125, True, 16)
    assert not O[:, 0].any() and np.isneginf(lse[:, 0]).all() and np.isfinite(lse[:, 1:]).all()


def test_oracle_eviction():
    table, mass = [3, 0, 4, 1, 2, 5], [5.0, 1.0, 9.0, 2.0, 2.0, 0.0]   # mass by slot
    # five blocks of 16, the last partial: logical weights 2, 5, 2, 1, 9
    t, n, kept = oracle.evict_blocks(table, mass, 70, 16, 3, 0, 1)
    assert kept == [0, 1, 4] and t == [3, 0, 2, 4, 1, 5] and n == 70 - 32   # block 0 before its equal 2
    t, n, kept = oracle.evict_blocks(table, mass, 70, 16, 3, 1, 2)
    assert kept == [0, 3, 4] and t == [3, 1, 2, 0, 4, 5]
    t, n, kept = oracle.evict_blocks(table, mass, 48, 16, 3, 0, 1)
    assert t == table and n == 48 and kept == [0, 1, 2]


# ---------------------------------------------------------------- refusals ----
def _cache(**over):
    from linear_hybrid_attention_b200._lib import ZbKv8
    d = dict(heads=2, slots=5, head_dim=64, block=64, format=0, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE,
             k_tail=FAKE, v_tail=FAKE, table=FAKE, mass=FAKE)
    d.update(over)
    return ZbKv8(*d.values())


BAD_CACHES = [(dict(heads=0), 2), (dict(slots=0), 2), (dict(head_dim=128), 4), (dict(block=48), 4), (dict(block=8), 4),
              (dict(block=256), 4), (dict(format=2), 4), (dict(heads=65536), 4), (dict(slots=2 ** 25), 4),
              (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
              (dict(table=None), 1), (dict(k=FAKE + 8), 3), (dict(table=FAKE + 4), 3), (dict(mass=FAKE + 4), 3)]


@pytest.mark.parametrize("over,want", BAD_CACHES)
def test_bad_caches(lib, over, want):
    c = _cache(**over)
    assert lib.zb_kv8_append(c, FAKE, FAKE, 1, FAKE, FAKE, None) == want
    assert lib.zb_kv8_read(c, FAKE, 1, FAKE, FAKE, None) == want
    assert lib.zb_kv8_attn(FAKE, 4 if c.heads == 2 else c.heads, 1, c, FAKE, 0, 0.125, FAKE, None, 0, FAKE, 1 << 40,
                           None) == want
    if want in (2, 4):
        assert lib.zb_kv8_attn_workspace_bytes(c, 4, 1, 0) == 0


def test_append_and_read_refusals(lib):
    ap = lambda K=FAKE, V=FAKE, n=3, lens=FAKE, out=FAKE, **o: lib.zb_kv8_append(_cache(**o), K, V, n, lens, out, None)
    assert ap(n=0) == 2 and ap(n=5 * 64 + 1) == 2
    assert ap(K=None) == 1 and ap(V=None) == 1 and ap(lens=None) == 1 and ap(out=None) == 1
    assert ap(k_tail=None) == 1 and ap(v_tail=None) == 1
    assert ap(K=FAKE + 8) == 3 and ap(lens=FAKE + 2) == 3 and ap(out=FAKE + 1) == 3 and ap(v_tail=FAKE + 4) == 3
    rd = lambda n=3, K=FAKE, V=FAKE, lens=FAKE: lib.zb_kv8_read(_cache(), lens, n, K, V, None)
    assert rd(n=0) == 2 and rd(K=None) == 1 and rd(V=FAKE + 8) == 3 and rd(lens=None) == 1 and rd(lens=FAKE + 2) == 3


def test_attn_refusals(lib):
    need = lib.zb_kv8_attn_workspace_bytes(_cache(), 4, 3, 1)
    assert need > lib.zb_kv8_attn_workspace_bytes(_cache(), 4, 3, 0) > 0
    assert lib.zb_kv8_attn_workspace_bytes(_cache(), 5, 3, 1) == 0     # not a multiple of the cache's heads
    assert lib.zb_kv8_attn_workspace_bytes(_cache(), 4, 0, 1) == 0
    at = lambda Q=FAKE, hq=4, n=3, lens=FAKE, scale=0.125, O=FAKE, lse=None, add=1, ws=FAKE, wsb=need, **o: \
        lib.zb_kv8_attn(Q, hq, n, _cache(**o), lens, 0, scale, O, lse, add, ws, wsb, None)
    assert at(hq=5) == 2 and at(hq=0) == 2 and at(n=0) == 2
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert at(scale=s) == 2
    assert at(n=2 ** 31) == 4
    assert at(Q=None) == 1 and at(lens=None) == 1 and at(O=None) == 1 and at(mass=None) == 1
    assert at(Q=FAKE + 2) == 3 and at(O=FAKE + 8) == 3 and at(lse=FAKE + 2) == 3 and at(ws=FAKE + 4) == 3
    assert at(ws=None) == 5 and at(wsb=need - 1) == 5


def test_attn_refuses_its_queries_as_output(lib):
    at = lambda n: lib.zb_kv8_attn(FAKE, 4, n, _cache(), FAKE, 0, 0.125, FAKE, None, 0, FAKE, 1 << 40, None)
    assert at(1) == 2 and at(300) == 2


def test_evict_refusals(lib):
    ev = lambda table=FAKE, mass=FAKE, lens=FAKE, H=2, S=9, B=64, budget=4, sinks=1, recent=2, out=FAKE + 64, lo=FAKE, \
        kept=None: lib.zb_kv8_evict(table, mass, lens, H, S, B, budget, sinks, recent, out, lo, kept, None)
    assert ev(H=0) == 2 and ev(S=0) == 2 and ev(budget=0) == 2 and ev(budget=10) == 2
    assert ev(sinks=-1) == 2 and ev(recent=0) == 2 and ev(sinks=3) == 2 and ev(sinks=2 ** 31 - 1, recent=1) == 2
    assert ev(B=100) == 4 and ev(H=70000) == 4 and ev(S=2 ** 26) == 4
    assert ev(table=None) == 1 and ev(mass=None) == 1 and ev(lens=None) == 1 and ev(out=None) == 1 and ev(lo=None) == 1
    assert ev(out=FAKE) == 2                                            # in place
    assert ev(table=FAKE + 2) == 3 and ev(kept=FAKE + 1) == 3 and ev(lo=FAKE + 3) == 3


def test_bindings_refuse_cpu_tensors():
    import linear_hybrid_attention_b200 as zb
    with pytest.raises(ValueError, match="CUDA"):
        zb.KV8Cache.empty(2, 100, device="cpu")
    x = torch.zeros(2, 10, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        zb.zb_kv8_evict(x, x.float(), x[:, 0], 64, 4)
    with pytest.raises(ValueError, match="heads"):
        zb.CachedAttention(1, 5, 2, 100, device="cpu")
    with pytest.raises(ValueError, match="format"):
        zb.KV8Cache.empty(2, 100, format="int4", device="cpu")


def test_empty_cache_refuses_blocks():
    import linear_hybrid_attention_b200 as zb
    for block in (0, -16, 48):
        with pytest.raises(ValueError, match="block"):
            zb.KV8Cache.empty(2, 100, block, device="cpu")
