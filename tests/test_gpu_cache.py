"""The 8-bit key/value cache on the GPU against the fp64 oracle: append and read exactly, attention and block
weights within derived bounds, eviction exactly, and a run of all of them as a layer in service makes it.

Tolerances of the attention (q and the cached values are the oracle's own inputs, exact).  A logit is a sum of
64 products in fp32: its error is at most d = 64 * 2^-23 * scale * sum |q k|, the largest over the row's keys (the
tensor core may truncate: a whole step, 2^-23, per addition).  A weight p then is off by d plus some ten roundings
of the exponential, the running maxima and the joins (2^-19 in all), and enters the product as fp16: 2^-11.
   |O - ref|    <= 2^-8 |ref| + (2 d + 2^-11 + 2^-18) sum p |v|      (O in bf16; 2 d: numerator and sum)
   |lse - ref|  <= d + 2^-19 + 2^-22 |ref|
   |mass - ref| <= (2 d + 2^-18) mass
"""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import bf16_round_f64, host, sync_ok

pytestmark = pytest.mark.gpu
FMT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def _rand(shape, seed, spread=0.7):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[-1], generator=g))
    return x.bfloat16().cuda()


def _shuffled(cache, seed):
    """The slots of every head in another order."""
    g = torch.Generator().manual_seed(seed)
    cache.table.copy_(torch.stack([torch.randperm(cache.slots, generator=g) for _ in range(cache.heads)]).int())
    return cache


def _ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def _filled(zb, lens, cap, block, fmt, seed, dirty=True):
    """A cache whose head h holds lens[h] tokens, appended one head at a time, and the oracle's caches."""
    H = len(lens)
    c = _shuffled(zb.KV8Cache.empty(H, cap, block, fmt), seed)
    if dirty:  # what lies in unused slots and behind the last token is never looked at
        c.k.view(torch.uint8).fill_(0x7F)
        c.v.view(torch.uint8).fill_(0x7F)
        c.k_scale.fill_(float("nan"))
        c.v_scale.fill_(float("nan"))
    n = max(max(lens), 1)
    K, V = _rand((H, n, 64), seed + 1), _rand((H, n, 64), seed + 2)
    ora = [oracle.Cache8(block, fmt) for _ in range(H)]
    for h, L in enumerate(lens):
        ora[h].append(host(K[h, :L]), host(V[h, :L]))
    # heads of one length at a time: others are past their room and stay (their status is cleared below)
    got = torch.zeros(H, dtype=torch.int32, device="cuda")
    for L in sorted(set(lens) - {0}):
        one = torch.where(_ints(lens) == L, 0, c.capacity + 1).int()
        out = zb.zb_kv8_append(c, K[:, :L].contiguous(), V[:, :L].contiguous(), one)
        got = torch.where(_ints(lens) == L, out, got)
    torch.cuda.synchronize()
    try:
        zb.zb_last_device_status()
    except zb.ZbError as e:
        assert e.status == 9
    assert got.tolist() == list(lens)
    return c, ora


# ------------------------------------------------------------ append, read ----
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_append_and_read_are_exact(fmt, block):
    import linear_hybrid_attention_b200 as zb
    H, N = 3, 517
    K, V = _rand((H, N, 64), 5, 1.5), _rand((H, N, 64), 6, 1.5)
    K[1, 40:60] = 0                                     # rows of zeros, and whole blocks of them
    V[1, 128:256] = 0
    K[2, 3] *= 1e-30                                    # far below their block's scale
    V[2, 300:] *= 2.0 ** -100
    ora = [oracle.Cache8(block, fmt) for _ in range(H)]
    for h in range(H):
        ora[h].append(host(K[h]), host(V[h]))
    ref = [o.values() for o in ora]
    caches = []
    for parts in ([N], [1] * 5 + [130, 127, 1, 254], [block - 1, 1, block, 2 * block + 1, N - 4 * block - 1]):
        c = _shuffled(zb.KV8Cache.empty(H, N + 40, block, fmt), 7)
        c.mass.fill_(3.0)
        lens, at = _ints([0] * H), 0
        for i, n in enumerate(parts):
            k, v = K[:, at:at + n].contiguous(), V[:, at:at + n].contiguous()
            if i % 2:
                zb.zb_kv8_append(c, k, v, lens, lens_out=lens)          # advances in place
            else:
                new = zb.zb_kv8_append(c, k, v, lens)
                assert torch.equal(new, lens + n)
                lens = new
            at += n
        assert at == N and lens.tolist() == [N] * H
        sync_ok()
        Ko, Vo = zb.zb_kv8_read(c, lens, N)
        for h in range(H):
            np.testing.assert_array_equal(host(Ko[h]), bf16_round_f64(ref[h][0]))
            np.testing.assert_array_equal(host(Vo[h]), bf16_round_f64(ref[h][1]))
            live = c.table[h, :-(-N // block)].long()
            np.testing.assert_array_equal(c.k_scale[h, live].double().cpu().numpy(), ref[h][2])
            np.testing.assert_array_equal(c.v_scale[h, live].double().cpu().numpy(), ref[h][3])
            # opened blocks lost their old weight, the others kept theirs
            assert (c.mass[h, live] == 0).all() and (c.mass[h, c.table[h, -(-N // block):].long()] == 3).all()
            tail = c.k[h, live[-1]].view(torch.uint8)[N % block:]
            assert N % block == 0 or not tail.any()      # codes behind the last token
        caches.append(c)
    for c in caches[1:]:                                 # however the tokens were split
        assert torch.equal(c.k.view(torch.uint8), caches[0].k.view(torch.uint8))
        assert torch.equal(c.v.view(torch.uint8), caches[0].v.view(torch.uint8))
    # the newest few; more than there are: zeros before the first token
    k5, _ = zb.zb_kv8_read(c, lens, 5)
    assert torch.equal(k5, Ko[:, -5:])
    kx, vx = zb.zb_kv8_read(c, lens, N + 9)
    assert not kx[:, :9].any() and torch.equal(kx[:, 9:], Ko) and torch.equal(vx[:, 9:], Vo)


def test_values_on_every_tie():
    # every tie between two codes at scale 1, both signs: the even code
    import linear_hybrid_attention_b200 as zb
    grids = {"int8": np.arange(128.0), "e4m3": oracle.E4M3_VALUES}
    for fmt, grid in grids.items():
        ties = (grid[1:] + grid[:-1]) / 2
        x = np.zeros((2, 64, 64))
        flat = x.reshape(2, -1)
        flat[:, 0] = grid[-1]
        flat[0, 1:1 + len(ties)], flat[1, 1:1 + len(ties)] = ties, -ties
        flat[0, 1000:1000 + len(grid)], flat[1, 1000:1000 + len(grid)] = grid, -grid
        X = torch.from_numpy(x).bfloat16().cuda()
        assert np.array_equal(host(X), x)                # bf16 holds them all
        c = zb.KV8Cache.empty(2, 64, 64, fmt)
        lens = zb.zb_kv8_append(c, X, X, _ints([0, 0]))
        K, V = zb.zb_kv8_read(c, lens, 64)
        for h in range(2):
            np.testing.assert_array_equal(host(K[h]), oracle.quantise_block(x[h], fmt)[0])
        assert torch.equal(K, V)
    sync_ok()


def test_scales_that_make_ties_hard():
    # quotients a fraction of a fp32 step off a tie: x = (k + 1/2) s rounded to bf16 for scales s with few bits
    import linear_hybrid_attention_b200 as zb
    rng = np.random.default_rng(11)
    x = np.zeros((64, 64, 64))
    for h in range(64):
        top = float(torch.tensor(rng.uniform(1, 2)).bfloat16())
        s = np.float32(top / 127.0)
        k = rng.integers(0, 126, (64, 64))
        x[h] = np.where(rng.random((64, 64)) < 0.5, 1, -1) * (k + 0.5) * float(s)
        x[h, 0, 0] = top
    X = torch.from_numpy(x).bfloat16().cuda()
    for fmt in FMT:
        c = zb.KV8Cache.empty(64, 64, 64, fmt)
        lens = zb.zb_kv8_append(c, X, X, _ints([0] * 64))
        K, _ = zb.zb_kv8_read(c, lens, 64)
        for h in range(64):
            q, s = oracle.quantise_block(host(X[h]), fmt)
            np.testing.assert_array_equal(host(K[h]), bf16_round_f64(np.asarray(q * s, np.float32)))


def test_not_finite_blocks_and_full_heads():
    import linear_hybrid_attention_b200 as zb
    c = zb.KV8Cache.empty(3, 64, 16, "int8")
    X = _rand((3, 40, 64), 3)
    X[0, 20, 7] = float("inf")
    X[1, 3, 1] = float("nan")
    lens = zb.zb_kv8_append(c, X, X, _ints([0, 0, 0]))
    K, _ = zb.zb_kv8_read(c, lens, 40)
    assert torch.isnan(K[0, 16:32]).all() and torch.isfinite(K[0, :16]).all() and torch.isfinite(K[0, 32:]).all()
    assert torch.isnan(K[1, :16]).all() and torch.isfinite(K[1, 16:]).all() and torch.isfinite(K[2]).all()
    sync_ok()
    # a head without room stays as it was, the others take the rows
    full = _ints([40, 24, 25])
    before = (c.k.clone(), c.k_tail.clone())
    out = zb.zb_kv8_append(c, X, X, full)
    with pytest.raises(zb.ZbError, match="INDEX"):
        sync_ok()
    assert out.tolist() == [40, 64, 25]
    for h in (0, 2):
        assert torch.equal(c.k[h], before[0][h]) and torch.equal(c.k_tail[h], before[1][h])
    # in place over several units of rows, negative lengths
    big = zb.KV8Cache.empty(2, 512, 16, "e4m3")
    Y = _rand((2, 300, 64), 4)
    n = _ints([212, 213])
    zb.zb_kv8_append(big, Y, Y, n, lens_out=n)
    with pytest.raises(zb.ZbError, match="INDEX"):
        sync_ok()
    assert n.tolist() == [512, 213]
    n = _ints([-1, 0])
    zb.zb_kv8_append(big, Y, Y, n, lens_out=n)
    with pytest.raises(zb.ZbError, match="INDEX"):
        sync_ok()
    assert n.tolist() == [-1, 300]


# --------------------------------------------------------------- attention ----
def _check_attention(zb, c, ora, lens, G, n_q, causal, seed, scale=0.125, add_mass=True, big_q=1.5):
    H, block = c.heads, c.block
    Q = _rand((H * G, n_q, 64), seed, 0.3) * big_q
    prior = torch.rand((H, c.slots), generator=torch.Generator().manual_seed(seed)).cuda()
    if add_mass:
        c.mass.copy_(prior)
    got = zb.zb_kv8_attn(Q, c, _ints(lens), causal=causal, scale=scale, want_lse=True, add_mass=add_mass)
    sync_ok()
    O, lse = host(got[0]).reshape(H, G, n_q, 64), got[1].double().cpu().numpy().reshape(H, G, n_q)
    q64 = host(Q).reshape(H, G, n_q, 64)
    for h, L in enumerate(lens):
        K, V = ora[h].values()[:2]
        refO, refl, refm = oracle.cache_attention(q64[h], K[:L], V[:L], scale, causal, block)
        none = np.isneginf(refl)
        assert np.array_equal(none, np.isneginf(lse[h])) and not O[h][none].any()
        if L == 0:
            assert none.all()
            continue
        d = 64 * 2.0 ** -23 * scale * np.max(np.abs(q64[h]) @ np.abs(K[:L]).T, -1)
        absO = oracle.cache_attention(q64[h], K[:L], np.abs(V[:L]), scale, causal, block)[0]
        bound = 2.0 ** -8 * np.abs(refO) + (2 * d[..., None] + 2.0 ** -11 + 2.0 ** -18) * absO + 1e-30
        assert np.all(np.abs(O[h] - refO) <= bound), (h, L, float(np.max(np.abs(O[h] - refO) / bound)))
        ok = ~none
        assert np.all(np.abs(lse[h][ok] - refl[ok]) <= d[ok] + 2.0 ** -19 + 2.0 ** -22 * np.abs(refl[ok])), (h, L)
        if add_mass:
            live = c.table[h, :len(refm)].long()
            add = (c.mass[h, live].double() - prior[h, live].double()).cpu().numpy()
            # the sum with what was there is rounded once more, to half a step of 2^-23 of it
            tol = (2 * d.max() + 2.0 ** -18) * refm + 2.0 ** -23 * (prior[h, live].double().cpu().numpy() + refm)
            assert np.all(np.abs(add - refm) <= tol), (h, L, float(np.max(np.abs(add - refm) / tol)))
            rest = c.table[h, len(refm):].long()
            assert torch.equal(c.mass[h, rest], prior[h, rest])
    return Q, got


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("G,n_q,causal", [(1, 1, False), (8, 1, True), (4, 3, True), (1, 16, False), (2, 16, True),
                                          (31, 1, False), (1, 33, True), (3, 90, False)])
def test_attention_short_lengths(fmt, block, G, n_q, causal):
    import linear_hybrid_attention_b200 as zb
    c, ora = _filled(zb, LENS, 256, block, fmt, 100 + block)
    _check_attention(zb, c, ora, LENS, G, n_q, causal, 7)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("block", [16, 64, 128])
@pytest.mark.parametrize("lens,G,n_q,causal", [([5000, 3, 2049], 4, 1, False), ([9999], 1, 2, True),
                                               ([1, 0, 0, 12000, 700], 5, 4, True), ([2100, 300], 2, 150, True), ([700, 129, 0, 2], 1, 300, True),
                                               ([1030, 40], 3, 130, False), ([3000], 4, 32, True)])
def test_attention_long_lengths(fmt, block, lens, G, n_q, causal):
    import linear_hybrid_attention_b200 as zb
    c, ora = _filled(zb, lens, max(lens) + 300, block, fmt, 200 + block)
    _check_attention(zb, c, ora, lens, G, n_q, causal, 8)


def test_attention_of_many_heads():
    import linear_hybrid_attention_b200 as zb
    lens = [(37 * h) % 150 for h in range(700)]         # more heads than CTAs or threads of one
    c, ora = _filled(zb, lens, 150, 32, "int8", 300)
    _check_attention(zb, c, ora, lens, 2, 1, False, 9)


def test_attention_extreme_logits():
    # one key takes everything; then keys of hardly any weight whose sum counts: 20,000 of 2^-16 each
    import linear_hybrid_attention_b200 as zb
    c, ora = _filled(zb, [3000, 300], 3008, 64, "int8", 400)
    _check_attention(zb, c, ora, [3000, 300], 2, 1, False, 10, scale=4.0)
    n = 20000
    K, V = torch.zeros((1, n, 64)), torch.ones((1, n, 64))
    K[0, 7, 0] = 127.0                                   # scale 1 in its block: code 127
    V[0, 7] = -1.0
    K, V = K.bfloat16().cuda(), V.bfloat16().cuda()
    c = zb.KV8Cache.empty(1, n, 64, "int8")
    lens = zb.zb_kv8_append(c, K, V, _ints([0]))
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 0.125                                    # logits scale * 0.125 * 127 and 0
    scale = 16 * np.log(2.0) / (0.125 * 127)
    O, lse = zb.zb_kv8_attn(q, c, lens, scale=scale, want_lse=True)
    w = (n - 1) * 2.0 ** -16
    sync_ok()
    # all values are +-1 and stand for themselves: the sum is off by fp32 alone (d = 64 * 2^-23 * 11.1)
    assert abs(float(O[0, 0, 0]) - (w - 1) / (w + 1)) <= 2.0 ** -8 * abs((w - 1) / (w + 1)) + 2 * 64 * 2.0 ** -23 * 11.1 + 2.0 ** -17
    assert float(lse[0, 0]) == pytest.approx(16 * np.log(2.0) + np.log1p(w), abs=64 * 2.0 ** -23 * 11.1 + 2.0 ** -18)


def test_attention_query_sizes():
    # queries far outside fp16's range, tiny ones, zeros
    import linear_hybrid_attention_b200 as zb
    c, ora = _filled(zb, [300], 512, 64, "e4m3", 500)
    _check_attention(zb, c, ora, [300], 4, 1, False, 11, big_q=2.0 ** 40, scale=2.0 ** -43)
    _check_attention(zb, c, ora, [300], 4, 1, False, 11, big_q=2.0 ** -60, scale=2.0 ** 57)
    Q = torch.zeros((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    O, lse = zb.zb_kv8_attn(Q, c, _ints([300]), want_lse=True)
    V = ora[0].values()[1]
    assert np.all(np.abs(host(O)[:, 0] - V.mean(0)) <= 2.0 ** -8 * np.abs(V.mean(0)) + (2.0 ** -11 + 2.0 ** -18) * np.abs(V).mean(0))
    np.testing.assert_allclose(lse.cpu().numpy(), np.log(300.0), atol=2.0 ** -18)


def test_not_finite_values_stay_where_they_are_seen():
    import linear_hybrid_attention_b200 as zb
    c, ora = _filled(zb, [100, 100], 128, 16, "int8", 600)
    Q = _rand((2, 8, 64), 12)
    want = zb.zb_kv8_attn(Q, c, _ints([100, 100]), causal=True)
    X = _rand((2, 1, 64), 13)
    X[0, 0, 0] = float("nan")                           # token 100 of head 0: block 6 (96..111) reads as NaN
    lens = zb.zb_kv8_append(c, X, X, _ints([100, 100]))
    O, lse = zb.zb_kv8_attn(Q, c, lens, causal=True, want_lse=True)
    # of 101 tokens, query i sees the first 94 + i: queries 0..2 end before block 6
    assert torch.isfinite(O[0, :3]).all() and torch.isnan(O[0, 3:]).all() and torch.isnan(lse[0, 3:]).all()
    assert torch.isfinite(O[1]).all() and torch.isfinite(lse[0, :3]).all()
    assert torch.equal(O[0, 0], zb.zb_kv8_attn(Q, c, _ints([94 + 7, 101]), causal=True)[0, 0])
    # a query that is not finite spoils its own row alone
    R = Q.clone()
    R[1, 4, 9] = float("inf")
    O2 = zb.zb_kv8_attn(R, c, _ints([100, 100]), causal=True)
    assert torch.isnan(O2[1, 4]).all()
    keep = torch.ones(8, dtype=torch.bool); keep[4] = False
    assert torch.isfinite(O2[1][keep.cuda()]).all() and want.shape == O2.shape
    sync_ok()


def test_attention_is_repeatable_and_bad_tables_are_reported():
    import linear_hybrid_attention_b200 as zb
    lens = [4000, 77, 2500, 1]
    c, ora = _filled(zb, lens, 4096, 64, "int8", 700)
    Q = _rand((16, 1, 64), 14)
    a = zb.zb_kv8_attn(Q, c, _ints(lens), want_lse=True)
    b = zb.zb_kv8_attn(Q, c, _ints(lens), want_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # lengths out of range are cut to what the cache holds
    cut = zb.zb_kv8_attn(Q, c, _ints([2 ** 31 - 1, -5, 2500, 1]))
    assert torch.equal(cut[8:], a[0][8:]) and not cut[4:8].any()
    sync_ok()
    c.table[2, 3] = c.slots
    c.table[0, 1] = -1
    zb.zb_kv8_attn(Q, c, _ints(lens))
    with pytest.raises(zb.ZbError, match="INDEX"):
        sync_ok()


def test_many_rows_are_repeatable_in_graphs_and_streams():
    import linear_hybrid_attention_b200 as zb
    lens = [3000, 70, 900]
    c, ora = _filled(zb, lens, 3008, 64, "int8", 710)
    n = _ints(lens)
    Q = [_rand((6, 150, 64), 15 + i) for i in range(2)]
    want = [zb.zb_kv8_attn(q, c, n, causal=True, want_lse=True) for q in Q]
    streams = [torch.cuda.Stream() for _ in Q]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(zb.zb_kv8_attn(Q[i], c, n, causal=True, want_lse=True))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) for o, l in got[i])
    # a captured call with weights follows the lengths
    c.mass.zero_()
    with torch.cuda.stream(streams[0]):
        zb.zb_kv8_attn(Q[0], c, n, add_mass=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        out = zb.zb_kv8_attn(Q[0], c, n, add_mass=True)
    for now in (lens, [1, 0, 900], [2999, 64, 129]):
        n.copy_(_ints(now))
        c.mass.zero_()
        graph.replay()
        torch.cuda.synchronize()
        mass = c.mass.clone()
        c.mass.zero_()
        assert torch.equal(out, zb.zb_kv8_attn(Q[0], c, n, add_mass=True)) and torch.equal(mass, c.mass)
    sync_ok()


@pytest.mark.parametrize("n_q", [1, 40])
def test_offsets_past_32_bits(n_q):
    # heads of 2^31 bytes of codes and more, their tokens in the last slots
    import linear_hybrid_attention_b200 as zb
    block, fmt, H, N = 128, "int8", 2, 700
    slots = 2 ** 31 // (block * 64) + 40
    c = zb.KV8Cache.empty(H, slots * block, block, fmt)
    assert c.slots == slots
    c.table.copy_(c.table.flip(1))
    K, V = _rand((H, N, 64), 720), _rand((H, N, 64), 721)
    lens = zb.zb_kv8_append(c, K, V, _ints([0] * H))
    ora = [oracle.Cache8(block, fmt) for _ in range(H)]
    for h in range(H):
        ora[h].append(host(K[h]), host(V[h]))
    Ko, Vo = zb.zb_kv8_read(c, lens, N)
    for h in range(H):
        np.testing.assert_array_equal(host(Ko[h]), bf16_round_f64(ora[h].values()[0]))
        np.testing.assert_array_equal(host(Vo[h]), bf16_round_f64(ora[h].values()[1]))
    _check_attention(zb, c, ora, [N] * H, 1, n_q, True, 16)
    table, lens, kept = zb.zb_kv8_evict(c.table, c.mass, lens, block, 3, 1, 1)
    sync_ok()
    for h in range(H):
        assert int(lens[h]) == N - 3 * block and kept[h, 0] == 0 and kept[h, 2] == 5
        assert torch.equal(table[h, 6:], c.table[h, 6:])


# ---------------------------------------------------------------- eviction ----
@pytest.mark.parametrize("slots,block,budget,sinks,recent", [(1, 16, 1, 0, 1), (9, 16, 4, 1, 2), (9, 64, 3, 1, 2),
                                                             (300, 64, 100, 4, 12), (1500, 16, 1499, 0, 1),
                                                             (5000, 128, 660, 0, 1), (50000, 16, 7000, 3, 5)])
@pytest.mark.parametrize("weights", ["spread", "ties", "equal", "odd"])
def test_evict(slots, block, budget, sinks, recent, weights):
    import linear_hybrid_attention_b200 as zb
    H = 5
    rng = np.random.default_rng(slots + budget)
    table = np.stack([rng.permutation(slots) for _ in range(H)]).astype(np.int32)
    mass = np.exp(3 * rng.standard_normal((H, slots))).astype(np.float32)
    if weights == "ties":
        mass = np.floor(mass).astype(np.float32)
    elif weights == "equal":
        mass[:] = 2.5
    elif weights == "odd":                               # zeros of both signs, subnormals, infinities, negatives
        odd = np.array([0.0, -0.0, 1e-42, np.inf, -1.0, 3.4e38, 1e-30], np.float32)
        mass = odd[rng.integers(0, len(odd), mass.shape)]
    lens = np.array([slots * block, max(1, slots * block - 1), min(budget * block + 1, slots * block), budget * block,
                     0], np.int32)
    new, length, kept = zb.zb_kv8_evict(torch.from_numpy(table).cuda(), torch.from_numpy(mass).cuda(), _ints(lens.tolist()),
                                        block, budget, sinks=sinks, recent=recent)
    sync_ok()
    for h in range(H):
        t, n, k = oracle.evict_blocks(table[h].tolist(), mass[h].tolist(), int(lens[h]), block, budget, sinks, recent)
        assert length[h] == n and kept[h].tolist() == k + [-1] * (budget - len(k)) and new[h].tolist() == t


def test_evict_nan_weights_and_bad_tables():
    import linear_hybrid_attention_b200 as zb
    mass = torch.tensor([[1.0, float("nan"), 5.0, -float("nan"), 2.0, 0.0]], device="cuda")
    bits = mass.view(torch.int32)
    bits[0, 1], bits[0, 3] = 0x7FC00000, -0x400000       # a NaN of each sign
    table = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    _, _, kept = zb.zb_kv8_evict(table, mass, _ints([96]), 16, 4)
    assert kept.tolist() == [[1, 2, 4, 5]]               # clear sign: largest; block 5 is the recent one
    _, _, kept = zb.zb_kv8_evict(table, mass, _ints([96]), 16, 5)
    assert kept.tolist() == [[0, 1, 2, 4, 5]]            # set sign: smallest
    sync_ok()
    table[0, 2] = 6
    zb.zb_kv8_evict(table, mass, _ints([96]), 16, 4)
    with pytest.raises(zb.ZbError, match="INDEX"):
        sync_ok()
    # the lengths may be advanced in place
    table[0, 2] = 2
    lens = _ints([95])
    zb.zb_kv8_evict(table, mass, lens, 16, 4, lens_out=lens)
    assert lens.tolist() == [95 - 32]


# ------------------------------------------------------------ all together ----
@pytest.mark.parametrize("fmt,block", [("int8", 16), ("e4m3", 32)])
def test_layer_in_service(fmt, block):
    """Norm, rotation, append, attention and eviction over many steps, against the oracle holding the same."""
    import linear_hybrid_attention_b200 as zb
    B, H, G, budget, sinks, recent = 2, 4, 2, 6, 1, 2
    fr = zb.zb_rope_frequencies(32, scaling="ntk", factor=4.0)
    wq, wk = (1 + 0.1 * torch.randn(64, generator=torch.Generator().manual_seed(i)) for i in (1, 2))
    layer = zb.CachedAttention(B, H, G, 12 * block, block, fmt, freqs=fr, norm="rms", wq=wq.cuda(), wk=wk.cuda(),
                               budget=budget, sinks=sinks, recent=recent)
    blocks = [[oracle.Cache8(block, fmt)] for _ in range(B * G)]     # rows in logical order, one cache a head
    lens, past = [0] * (B * G), 0
    how = dict(layout="half")
    for step, n in enumerate([3 * block + 5, 1, 1, block, 1, 2 * block - 3, 1, 7]):
        X = _rand((B, n, H + 2 * G, 64), 50 + step, 0.4).transpose(1, 2)   # one projection's output
        Q, K, V = X[:, :H], X[:, H:H + G], X[:, H + G:]
        pos = (past + torch.arange(n, dtype=torch.int32))[None, None].contiguous()
        O = layer.step(Q, K, V, pos.cuda())
        sync_ok()
        # the cache takes what the GPU's norm and rotation gave (checked by themselves elsewhere)
        Qo, Ko = zb.zb_qk_norm_rope(Q, K, pos.cuda(), layer.turns, norm="rms", wq=wq.cuda(), wk=wk.cuda())
        near = oracle.qk_norm_rope(host(K), wk.double().numpy(), None, "rms", 1e-6, pos.numpy(), fr.radians.numpy(), **how)
        assert np.max(np.abs(host(Ko) - near)) <= 2.0 ** -8 * np.abs(near).max() + 2.0 ** -18 * np.abs(near).max()
        for b in range(B):
            for g in range(G):
                c = blocks[b * G + g][0]
                c.append(host(Ko[b, g]), host(V[b, g]))
                k, v = c.values()[:2]
                hq = slice(g * (H // G), (g + 1) * (H // G))
                ref, _, mass = oracle.cache_attention(host(Qo[b, hq]), k, v, 0.125, True, block)
                d = 64 * 2.0 ** -23 * 0.125 * np.max(np.abs(host(Qo[b, hq])) @ np.abs(k).T)
                absO = oracle.cache_attention(host(Qo[b, hq]), k, np.abs(v), 0.125, True, block)[0]
                bound = 2.0 ** -8 * np.abs(ref) + (2 * d + 2.0 ** -11 + 2.0 ** -18) * absO
                assert np.all(np.abs(host(O[b, hq]) - ref) <= bound)
                lens[b * G + g] += n
        past += n
        assert layer.lens.tolist() == lens
        if step % 2:
            table, mass = layer.cache.table.tolist(), layer.cache.mass.tolist()
            kept = layer.evict()
            sync_ok()
            for h in range(B * G):
                t, L, k = oracle.evict_blocks(table[h], mass[h], lens[h], block, budget, sinks, recent)
                assert layer.cache.table[h].tolist() == t and kept[h].tolist() == k + [-1] * (budget - len(k))
                c = blocks[h][0]
                rows = np.concatenate([np.arange(i * block, min((i + 1) * block, lens[h])) for i in k])
                c.k, c.v, lens[h] = c.k[rows], c.v[rows], L
            assert layer.lens.tolist() == lens


def test_graph_replay_follows_the_lengths():
    import linear_hybrid_attention_b200 as zb
    make = lambda: zb.CachedAttention(2, 4, 2, 512, 32, "int8", norm="rms", budget=8)
    a, b = make(), make()
    X = [_rand((2, 8, 1, 64), 70 + i, 0.4) for i in range(40)]
    split = lambda x: (x[:, :4], x[:, 4:6], x[:, 6:])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                        # warm up on the capture's stream, then forget it
        a.step(*split(X[0]))
        a.evict()
    torch.cuda.synchronize()
    a.lens.zero_()
    a.cache.mass.zero_()
    a.cache.table.copy_(b.cache.table)
    hold = X[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = a.step(*split(hold))
        a.evict()
    for x in X:
        hold.copy_(x)
        graph.replay()
        want = b.step(*split(x))
        b.evict()
        assert torch.equal(out, want)
    sync_ok()
    assert a.lens.tolist() == b.lens.tolist() == [40] * 4 and torch.equal(a.cache.mass, b.cache.mass)


def test_two_streams_with_workspaces_of_their_own():
    import linear_hybrid_attention_b200 as zb
    lens = [3000, 1700]
    c, _ = _filled(zb, lens, 3008, 64, "int8", 800)
    Q = [_rand((8, 1, 64), 90 + i) for i in range(2)]
    n = _ints(lens)
    want = [zb.zb_kv8_attn(q, c, n) for q in Q]
    streams = [torch.cuda.Stream() for _ in Q]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(zb.zb_kv8_attn(Q[i], c, n))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_binding_refusals():
    import linear_hybrid_attention_b200 as zb
    c = zb.KV8Cache.empty(2, 128, 64, "int8", mass=False)
    X, n = _rand((2, 3, 64), 1), _ints([0, 0])
    for f, err in ((lambda: zb.zb_kv8_append(c, X, X[:, :2], n), ValueError),
                   (lambda: zb.zb_kv8_append(c, X.float(), X, n), TypeError),
                   (lambda: zb.zb_kv8_append(c, X, X, n.long()), ValueError),
                   (lambda: zb.zb_kv8_append(c, X, X, n.cpu()), ValueError),
                   (lambda: zb.zb_kv8_append(c, X[:1], X[:1], n), ValueError),
                   (lambda: zb.zb_kv8_append(c, _rand((2, 129, 64), 1), _rand((2, 129, 64), 1), n), zb.ZbError),
                   (lambda: zb.zb_kv8_attn(X, c, n, add_mass=True), ValueError),
                   (lambda: zb.zb_kv8_attn(X[:, :, :32], c, n), ValueError),
                   (lambda: zb.zb_kv8_attn(_rand((3, 1, 64), 1), c, n), zb.ZbError),
                   (lambda: zb.zb_kv8_attn(X, c, n, scale=0.0), zb.ZbError),
                   (lambda: zb.zb_kv8_attn(X, c, n, out=X[:1]), ValueError),
                   (lambda: zb.zb_kv8_read(c, n, 0), ValueError),
                   (lambda: zb.zb_kv8_evict(c.table, c.k_scale, n, 64, 3), zb.ZbError),
                   (lambda: zb.zb_kv8_evict(c.table, c.k_scale, n, 64, 2, table_out=c.table), zb.ZbError),
                   (lambda: zb.zb_kv8_evict(c.table, c.k_scale[:1], n, 64, 2), ValueError),
                   (lambda: zb.KV8Cache(c.k, c.v, c.k_scale, c.v_scale, c.k_tail, c.v_tail, c.table[:1]), ValueError),
                   (lambda: zb.KV8Cache(c.k, c.v.view(torch.uint8), c.k_scale, c.v_scale, c.k_tail, c.v_tail, c.table), TypeError),
                   (lambda: zb.KV8Cache.empty(2, 100, 48), ValueError),
                   (lambda: zb.CachedAttention(1, 2, 2, 128).evict(), ValueError),
                   (lambda: zb.CachedAttention(1, 2, 2, 128, budget=9), ValueError),
                   (lambda: zb.CachedAttention(1, 2, 2, 128).step(X, X, X), ValueError)):
        with pytest.raises(err):
            f()
