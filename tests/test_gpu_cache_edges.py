"""The 8-bit cache's attention where values, logits and scales are uneven, for every kernel that serves it: few query
rows of a cache head (up to 32) and many (items of 128 rows, and of 256); exact rounding of every scale; calls that
write where they read.

Tolerances.  Logits, sums, log-sum-exp and weights as in test_gpu_cache.py, whose d, 2^-11 and 2^-18 these are.  A
softmax weight enters the product as fp16.  Its largest of a row is there at 2^6 at least, so what is below fp16's
normal numbers is off by half of its smallest step, 2^-25, over 2^6: 2^-31 of the row's largest weight, p_max.
   |O - ref|    <= 2^-8 |ref| + (2 d + 2^-11 + 2^-18) sum p |v| + 2^-31 p_max sum |v|
   |lse - ref|  <= d + 2^-19 + 2^-22 |ref|
   |mass - ref| <= (2 d + 2^-18) mass, and 2^-23 of the sum with what was there
"""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import host, sync_ok
from tests.test_gpu_cache import _ints, _rand, _shuffled

pytestmark = pytest.mark.gpu

ROWS = [(1, 8, True), (2, 16, False), (1, 33, True), (3, 50, False), (2, 150, True), (1, 300, True)]  # G, n_q, causal
MANY = [r for r in ROWS if r[0] * r[1] > 32]


def _made(zb, K, V, block, fmt, seed):
    """A cache that holds K, V [H, n, 64] and the oracle's; unused slots and tokens hold anything."""
    K, V = K.bfloat16().cuda(), V.bfloat16().cuda()
    H, n = K.shape[:2]
    c = _shuffled(zb.KV8Cache.empty(H, n + 2 * block, block, fmt), seed)
    c.k.view(torch.uint8).fill_(0x7F)
    c.v.view(torch.uint8).fill_(0x7F)
    c.k_scale.fill_(float("nan"))
    c.v_scale.fill_(float("nan"))
    lens = zb.zb_kv8_append(c, K, V, _ints([0] * H))
    ora = [oracle.Cache8(block, fmt) for _ in range(H)]
    for h in range(H):
        ora[h].append(host(K[h]), host(V[h]))
    return c, ora, lens


def _check(zb, c, ora, lens, Q, G, causal, scale, rows=None, rel_v=0.0):
    """Attention of Q [H G, n_q, 64] within the bounds above.  rows: the query rows that are looked at (bool, [G, n_q]);
    rel_v: what a value may be off by, relative to the largest value of its feature's head."""
    H, block, n_q = c.heads, c.block, Q.shape[1]
    prior = torch.rand((H, c.slots), generator=torch.Generator().manual_seed(5)).cuda() * 1e-3
    c.mass.copy_(prior)
    O, lse = zb.zb_kv8_attn(Q, c, lens, causal=causal, scale=scale, want_lse=True, add_mass=True)
    sync_ok()
    O, lse = host(O).reshape(H, G, n_q, 64), lse.double().cpu().numpy().reshape(H, G, n_q)
    q64 = host(Q).reshape(H, G, n_q, 64)
    rows = np.ones((G, n_q), bool) if rows is None else rows
    for h in range(H):
        K, V = ora[h].values()[:2]
        L = len(K)
        refO, refl, refm = oracle.cache_attention(q64[h], K, V, scale, causal, block)
        d = 64 * 2.0 ** -23 * scale * np.max(np.abs(q64[h]) @ np.abs(K).T, -1)
        absO = oracle.cache_attention(q64[h], K, np.abs(V), scale, causal, block)[0]
        x = scale * q64[h] @ K.T
        if causal:
            x = np.where(np.arange(L) <= L - n_q + np.arange(n_q)[:, None], x, -np.inf)
        top = np.exp(x.max(-1) - refl)
        bound = 2.0 ** -8 * np.abs(refO) + (2 * d[..., None] + 2.0 ** -11 + 2.0 ** -18) * absO + \
            2.0 ** -31 * top[..., None] * np.abs(V).sum(0) + rel_v * np.abs(V).max() + 1e-38
        err = np.abs(O[h] - refO) / bound
        assert np.all(err[rows] <= 1), (h, float(err[rows].max()))
        el = np.abs(lse[h] - refl) / (d + 2.0 ** -19 + 2.0 ** -22 * np.abs(refl))
        assert np.all(el[rows] <= 1), (h, float(el[rows].max()))
        if rows.all():
            live = c.table[h, :len(refm)].long()
            was = prior[h, live].double().cpu().numpy()
            add = c.mass[h, live].double().cpu().numpy() - was
            tol = (2 * d.max() + 2.0 ** -18) * refm + 2.0 ** -23 * (was + refm)
            assert np.all(np.abs(add - refm) <= tol), (h, float(np.max(np.abs(add - refm) / tol)))
    return O, lse


def _loaded(H, n, logit, seed, at=3, q=4.0, scale=0.125):
    """K and Q rows of which key `at` has `logit` more than the others, and the rest a spread of about 1."""
    K = _rand((H, n, 64), seed, 0.3).float().cpu()
    K[..., 0] = 0.0
    K[:, at, 0] = logit / (q * scale)

    def queries(G, n_q):
        Q = _rand((H * G, n_q, 64), seed + 1, 0.3)
        Q[..., 0] = q
        return Q
    return K, queries


# ---------------------------------------------------------- scales of values ----
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("block", [16, 64, 128])
@pytest.mark.parametrize("G,n_q,causal", ROWS)
def test_blocks_of_zero_values(fmt, block, G, n_q, causal):
    # the first block's values are zeros and one of its keys takes most of the weight: what counts is small
    import linear_hybrid_attention_b200 as zb
    n = 3000
    for size, logit in ((0.01, 14.0), (0.001, 12.0), (0.05, 16.0)):
        K, queries = _loaded(2, n, logit, 21)
        V = _rand((2, n, 64), 23).float().cpu() * size
        V[:, :block] = 0
        V[1, 10 * block:12 * block] = 0                  # and zeros again after other blocks
        c, ora, lens = _made(zb, K, V, block, fmt, 24)
        _check(zb, c, ora, lens, queries(G, n_q), G, causal, 0.125)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("G,n_q,causal", ROWS)
def test_a_block_of_large_values_under_most_of_the_weight(fmt, block, G, n_q, causal):
    # its other features are zeros: there the outputs are the many keys' of hardly any weight
    import linear_hybrid_attention_b200 as zb
    n = 6000
    for times, first in ((2.0 ** 10, 0), (2.0 ** 14, 0), (2.0 ** 14, 4096)):
        K, queries = _loaded(2, n, 10.0, 31, at=first + 3)
        V = _rand((2, n, 64), 33).float().cpu()
        V[:, first:first + block] *= times
        V[:, first:first + block, 32:] = 0
        c, ora, lens = _made(zb, K, V, block, fmt, 34)
        _check(zb, c, ora, lens, queries(G, n_q), G, causal, 0.125)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("G,n_q,causal", ROWS)
def test_scales_far_apart(fmt, G, n_q, causal):
    # scales from 2^-40 to 2^100, up and down along the keys: sums, lse and weights do not depend on them; a value
    # may be lost that is 2^-31 of the head's largest
    import linear_hybrid_attention_b200 as zb
    n, block = 2000, 64
    K = _rand((3, n, 64), 41, 0.3).float().cpu()
    V = _rand((3, n, 64), 42).float().cpu()
    step = torch.arange(n) // 256
    V[0] *= torch.exp2(-40 + 20.0 * step)[:, None]
    V[1] *= torch.exp2(100 - 20.0 * step)[:, None]
    V[2] *= torch.exp2(torch.where(step % 2 == 0, 100.0, -40.0))[:, None]
    c, ora, lens = _made(zb, K, V, block, fmt, 43)
    _check(zb, c, ora, lens, _rand((3 * G, n_q, 64), 44, 0.3), G, causal, 0.125, rel_v=2.0 ** -31)


@pytest.mark.parametrize("G,n_q,causal", ROWS)
def test_values_at_both_ends_of_their_type(G, n_q, causal):
    # bf16 goes to 3.4e38; values of 2^-110 and 30,000 keys of nearly equal weight
    import linear_hybrid_attention_b200 as zb
    K, V = _rand((1, 700, 64), 51, 0.3).float().cpu(), torch.randn((1, 700, 64), generator=torch.Generator().manual_seed(52))
    c, ora, lens = _made(zb, K, V.clamp(-3, 3) * 2.0 ** 126, 64, "int8", 53)
    _check(zb, c, ora, lens, _rand((G, n_q, 64), 54, 0.3), G, causal, 0.125)
    n = 30000
    K = torch.randn((1, n, 64), generator=torch.Generator().manual_seed(55)) * 0.1
    V = torch.rand((1, n, 64), generator=torch.Generator().manual_seed(56)) * 2.0 ** -110
    c, ora, lens = _made(zb, K, V, 64, "int8", 57)
    _check(zb, c, ora, lens, _rand((G, n_q, 64), 58, 0.3), G, causal, 0.125)


@pytest.mark.parametrize("rows", [1, 40, 150])
def test_scales_that_no_append_makes(rows):
    # a cache filled by the caller: small codes under scales up to fp32's end, and zero codes under a scale of zero
    import linear_hybrid_attention_b200 as zb
    n, block = 320, 64
    g = torch.Generator().manual_seed(59)
    c, _, lens = _made(zb, _rand((1, n, 64), 59, 0.3).float(), torch.zeros((1, n, 64)), block, "int8", 60)
    codes = torch.randint(-1, 2, (1, c.slots, block, 64), generator=g, dtype=torch.int8)
    scales = torch.tensor([2.0 ** 126 * 1.75, 2.0 ** 127 * 1.5, 0.0, 2.0 ** 120, 3.0])
    live = c.table[0, :5].long()
    c.v.copy_(codes)
    c.v_scale[0, live] = scales.cuda()
    c.v[0, live[2]] = 0
    V = (c.v[0, live].double().cpu() * scales.double()[:, None, None]).reshape(n, 64).numpy()
    Q = _rand((1, rows, 64), 61, 0.3)
    O = host(zb.zb_kv8_attn(Q, c, lens, scale=0.125))[0]
    sync_ok()
    k64 = c.k[0, live].double().cpu() * c.k_scale[0, live].double().cpu()[:, None, None]
    k64, q64 = k64.reshape(n, 64).numpy(), host(Q)
    ref = oracle.cache_attention(q64, k64, V, 0.125, False, block)[0][0]
    absO = oracle.cache_attention(q64, k64, np.abs(V), 0.125, False, block)[0][0]
    d = 64 * 2.0 ** -23 * 0.125 * np.max(np.abs(q64[0]) @ np.abs(k64).T, -1)[:, None]
    bound = 2.0 ** -8 * np.abs(ref) + (2 * d + 2.0 ** -11 + 2.0 ** -18) * absO + 2.0 ** -31 * np.abs(V).sum(0)
    assert np.all(np.abs(O - ref) <= bound), float(np.max(np.abs(O - ref) / bound))


# ------------------------------------------------------------ logits, queries ----
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("G,n_q,causal", ROWS)
def test_logits_that_keep_rising(block, G, n_q, causal):
    # the maximum moves with every tile, by little and by much; then back down
    import linear_hybrid_attention_b200 as zb
    n, q, scale = 2500, 4.0, 0.125
    K = _rand((2, n, 64), 61, 0.3).float().cpu()
    ramp = torch.arange(n).float() / n
    K[0, :, 0] = ramp * 60.0 / (q * scale)
    K[1, :, 0] = torch.where(ramp < 0.5, ramp * 200.0, 100.0 - 30.0 * ramp) / (q * scale)
    c, ora, lens = _made(zb, K, _rand((2, n, 64), 62).float(), block, "int8", 63)
    Q = _rand((2 * G, n_q, 64), 64, 0.3)
    Q[..., 0] = q
    _check(zb, c, ora, lens, Q, G, causal, scale)


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("G,n_q,causal", MANY)
def test_query_sizes_of_many_rows(block, G, n_q, causal):
    # queries far outside fp16's range, tiny ones, zeros, and all of them in one call
    import linear_hybrid_attention_b200 as zb
    K, V = _rand((1, 700, 64), 71, 0.3).float(), _rand((1, 700, 64), 72).float()
    c, ora, lens = _made(zb, K, V, block, "e4m3", 73)
    Q = _rand((G, n_q, 64), 74, 0.3)
    _check(zb, c, ora, lens, Q * 2.0 ** 40, G, causal, 2.0 ** -43)
    _check(zb, c, ora, lens, Q * 2.0 ** -60, G, causal, 2.0 ** 57)
    Q = Q * torch.exp2(-20.0 * (torch.arange(n_q, device="cuda") % 4))[:, None].bfloat16()
    Q[:, ::5] = 0
    _check(zb, c, ora, lens, Q, G, causal, 0.125)


@pytest.mark.parametrize("block", [16, 64, 128])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("G,n_q", [(1, 24), (1, 40), (2, 60), (1, 150), (2, 140)])
def test_not_finite_blocks_spoil_the_rows_that_see_them(block, which, G, n_q):
    import linear_hybrid_attention_b200 as zb
    n = 500
    K, V = _rand((2, n, 64), 81, 0.3).float().cpu(), _rand((2, n, 64), 82).float().cpu()
    bad = (n - n_q // 2) // block                        # begins within the causal rows' ends, or before
    first = bad * block
    (K if which == "k" else V)[1, first, 5] = float("inf") if block == 16 else float("nan")
    c, ora, lens = _made(zb, K, V, block, "int8", 83)
    Q = _rand((2 * G, n_q, 64), 84, 0.3)
    O, lse = zb.zb_kv8_attn(Q, c, lens, causal=True, scale=0.125, want_lse=True)
    sync_ok()
    sees = torch.arange(n_q) + n - n_q >= first          # of the rows of head 1
    O, lse = O.reshape(2, G, n_q, 64).cpu(), lse.reshape(2, G, n_q).cpu()
    assert torch.isfinite(O[0]).all() and torch.isfinite(lse[0]).all()
    assert torch.isnan(O[1][:, sees]).all()
    assert torch.isnan(lse[1][:, sees]).all() if which == "k" else torch.isfinite(lse[1]).all()
    # the others are what they are without that block's tokens
    if (~sees).any():
        ora[1].k, ora[1].v = np.nan_to_num(ora[1].k, posinf=0), np.nan_to_num(ora[1].v, posinf=0)
        rows = np.broadcast_to((~sees).numpy(), (G, n_q))
        Kr, Vr = ora[1].values()[:2]
        q64 = host(Q).reshape(2, G, n_q, 64)[1]
        refO = oracle.cache_attention(q64, Kr, Vr, 0.125, True, block)[0]
        absO = oracle.cache_attention(q64, Kr, np.abs(Vr), 0.125, True, block)[0]
        d = 64 * 2.0 ** -23 * 0.125 * np.max(np.abs(q64) @ np.abs(Kr).T, -1)[..., None]
        bound = 2.0 ** -8 * np.abs(refO) + (2 * d + 2.0 ** -11 + 2.0 ** -18) * absO + 2.0 ** -31 * np.abs(Vr).sum(0)
        assert np.all((np.abs(host(O[1]) - refO) <= bound)[rows])


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("G,n_q,causal", ROWS)
def test_queries_that_are_not_finite_spoil_their_own_rows(block, G, n_q, causal):
    import linear_hybrid_attention_b200 as zb
    c, ora, lens = _made(zb, _rand((1, 700, 64), 91, 0.3).float(), _rand((1, 700, 64), 92).float(), block, "int8", 93)
    Q = _rand((G, n_q, 64), 94, 0.3)
    bad = torch.zeros((G, n_q), dtype=torch.bool)
    bad[0, 3] = bad[-1, n_q - 1] = True
    Q[0, 3, 9], Q[-1, n_q - 1, 63] = float("inf"), float("nan")
    got, lse = zb.zb_kv8_attn(Q, c, lens, causal=causal, want_lse=True)
    assert torch.isnan(got[bad.cuda()]).all() and torch.isnan(lse[bad.cuda()]).all()
    clean = Q.clone()
    clean[0, 3, 9] = clean[-1, n_q - 1, 63] = 0
    want, wl = zb.zb_kv8_attn(clean, c, lens, causal=causal, want_lse=True)
    assert torch.equal(got[~bad.cuda()], want[~bad.cuda()]) and torch.equal(lse[~bad.cuda()], wl[~bad.cuda()])
    sync_ok()


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("rows", [1, 16, 33, 300])
def test_values_that_are_nan_under_hardly_any_weight(block, rows):
    # the weight underflows and the part that holds it is one of many: the outputs are NaN all the same
    import linear_hybrid_attention_b200 as zb
    n, q, scale = 40000, 4.0, 0.125
    K = _rand((1, n, 64), 141, 0.3).float().cpu()
    K[..., 0] = 0.0
    K[:, 30000, 0] = 250.0 / (q * scale)
    V = _rand((1, n, 64), 142).float().cpu()
    V[0, 5, 9] = float("nan")
    c, _, lens = _made(zb, K, V, block, "int8", 143)
    Q = _rand((1, rows, 64), 144, 0.3)
    Q[..., 0] = q
    O, lse = zb.zb_kv8_attn(Q, c, lens, scale=scale, want_lse=True)
    sync_ok()
    assert torch.isnan(O).all() and torch.isfinite(lse).all()


# --------------------------------------------------------------- exact rounding ----
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("low,high", [(1.0, 2.0), (2.0 ** -104, 2.0 ** -98), (2.0 ** -122, 2.0 ** -104), (2.0 ** -131, 2.0 ** -122)])
def test_ties_of_every_scale(fmt, low, high):
    # values within bf16's rounding of a tie between two codes, for scales with few and many bits, tiny ones among them
    import linear_hybrid_attention_b200 as zb
    rng = np.random.default_rng(101)
    grid = np.arange(128.0) if fmt == "int8" else oracle.E4M3_VALUES
    x = np.zeros((64, 64, 64))
    for h in range(64):
        top = float(torch.tensor(np.exp(rng.uniform(np.log(low), np.log(high)))).bfloat16())
        s = float(np.float32(top / grid[-1]))
        k = rng.integers(0, len(grid) - 2, (64, 64))
        x[h] = np.where(rng.random((64, 64)) < 0.5, 1, -1) * (grid[k] + grid[k + 1]) / 2 * s
        x[h, 0, 0] = top
    X = torch.from_numpy(x).bfloat16()
    X = torch.where(X.abs() > X[:, :1, :1], X[:, :1, :1], X).cuda()
    c = zb.KV8Cache.empty(64, 64, 64, fmt)
    zb.zb_kv8_append(c, X, X, _ints([0] * 64))
    sync_ok()
    codes = c.k[:, 0].double().cpu().numpy()
    for h in range(64):
        q, s = oracle.quantise_block(host(X[h]), fmt)
        assert float(c.k_scale[h, 0].double()) == s
        np.testing.assert_array_equal(codes[h], q)
    K, _ = zb.zb_kv8_read(c, _ints([64] * 64), 64)
    want = torch.from_numpy(np.asarray(codes * c.k_scale[:, 0].double().cpu().numpy()[:, None, None], np.float32))
    assert torch.equal(K.cpu(), want.bfloat16())


# ------------------------------------------------------ calls that write where they read ----
@pytest.mark.parametrize("N", [1, 63, 65, 700])
@pytest.mark.parametrize("H", [1, 3, 16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_in_place(N, H, layout):
    # idle lanes, rows of several groups of tokens, many times over: the same bits as into memory of its own
    import linear_hybrid_attention_b200 as zb
    X = _rand((2, H, N, 64), 111)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None, None] + 100_000
    turns = zb.zb_rope_frequencies(64).turns.cuda()
    want = zb.zb_rope(X, pos, turns, layout=layout)
    for _ in range(20):
        Y = X.clone()
        zb.zb_rope(Y, pos, turns, layout=layout, out=Y)
        assert torch.equal(Y, want)
    sync_ok()


def test_lengths_advanced_in_place():
    # by an append and an eviction, of more heads than run at once
    import linear_hybrid_attention_b200 as zb
    H, block = 3000, 16
    X = _rand((H, 5, 64), 112)
    lens = (torch.arange(H, dtype=torch.int32, device="cuda") * 7) % 200
    a, b = (zb.KV8Cache.empty(H, 256, block) for _ in range(2))
    inplace = lens.clone()
    want = zb.zb_kv8_append(a, X, X, lens)
    zb.zb_kv8_append(b, X, X, inplace, lens_out=inplace)
    assert torch.equal(inplace, want) and torch.equal(want, lens + 5) and torch.equal(a.k, b.k)
    _, less, _ = zb.zb_kv8_evict(a.table, a.mass, want, block, 3)
    zb.zb_kv8_evict(a.table, a.mass, inplace, block, 3, lens_out=inplace)
    assert torch.equal(inplace, less)
    sync_ok()


# ------------------------------------------------------------- the layer's refusals ----
def test_layer_with_full_heads():
    """A head without room: zeros for its queries, no weight added, its cache as it was; the others go on."""
    import linear_hybrid_attention_b200 as zb
    B, H, G, block = 2, 4, 2, 16
    make = lambda: zb.CachedAttention(B, H, G, 4 * block, block, "int8", norm="rms", budget=4)
    one, all_ = make(), make()
    X = _rand((B, H + 2 * G, 60, 64), 121, 0.3)
    split = lambda x: (x[:, :H], x[:, H:H + G], x[:, H + G:])
    for layer in (one, all_):
        layer.step(*split(X[:, :, :50]))
    one.lens[1] = one.lens[2] = 60                       # of sequence 0, head 1 and of sequence 1, head 0: 60 + 10 > 64
    k, mass, tail = one.cache.k.clone(), one.cache.mass.clone(), one.cache.k_tail.clone()
    O = one.step(*split(X[:, :, 50:]))
    want = all_.step(*split(X[:, :, 50:]))
    with pytest.raises(zb.ZbError, match="INDEX"):
        sync_ok()
    assert one.lens.tolist() == [60, 60, 60, 60]
    O, want = (t.reshape(B * G, -1, 10, 64) for t in (O, want))
    for h in range(B * G):
        if h in (1, 2):
            assert not O[h].any() and torch.equal(one.cache.k[h], k[h]) and torch.equal(one.cache.k_tail[h], tail[h])
            assert torch.equal(one.cache.mass[h], mass[h])
        else:
            # (runs of other lengths: each within half a bf16 step and 2^-11 + 2^-18 of the values; d <= 2^-14)
            near = 2.0 ** -7 * want[h].float().abs() + 2.0 ** -9 * X.float().abs().max()
            assert ((O[h].float() - want[h].float()).abs() <= near).all() and O[h].any()
            torch.testing.assert_close(one.cache.mass[h], all_.cache.mass[h], rtol=2.0 ** -12, atol=0)
    # all heads full: nothing changes
    lens = one.lens.clone()
    assert not one.step(*split(X[:, :, :10])).any() and torch.equal(one.lens, lens)
    with pytest.raises(zb.ZbError, match="INDEX"):
        sync_ok()


def test_layer_refuses_before_it_changes_anything():
    import linear_hybrid_attention_b200 as zb
    layer = zb.CachedAttention(1, 4, 2, 128)
    X = _rand((1, 8, 3, 64), 122, 0.3)
    Q, K, V = X[:, :4], X[:, 4:6], X[:, 6:]
    layer.step(Q, K, V)
    state = [t.clone() for t in (layer.lens, layer.cache.k, layer.cache.k_tail)]
    for bad, err in (((Q.float(), K, V), TypeError), ((Q, K.float(), V), TypeError), ((Q, K, V.float()), TypeError),
                     ((Q.cpu(), K, V), ValueError), ((Q, K, V.cpu()), ValueError)):
        with pytest.raises(err):
            layer.step(*bad)
        assert all(torch.equal(a, b) for a, b in zip(state, (layer.lens, layer.cache.k, layer.cache.k_tail)))
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError, match="scale"):
            zb.CachedAttention(1, 4, 2, 128, scale=scale)
    sync_ok()


@pytest.mark.parametrize("causal", [True, False])
def test_layer_attends_in_bands(causal, monkeypatch):
    """A step whose workspace would pass the bound attends band by band; a full head among the others."""
    import linear_hybrid_attention_b200 as zb
    from linear_hybrid_attention_b200 import cache as mod
    B, H, G, n = 1, 6, 2, 700
    make = lambda: zb.CachedAttention(B, H, G, 1024, 64, "e4m3", norm="rms", budget=16)
    whole, banded = make(), make()
    X = _rand((B, H + 2 * G, n, 64), 131, 0.3)
    parts = (X[:, :H], X[:, H:H + G], X[:, H + G:])
    for layer in (whole, banded):
        layer.step(*(p[:, :, :100].contiguous() for p in parts))
        layer.lens[1] = 400                              # 400 + 700 > 1024
    want = whole.step(*parts, causal=causal)
    sizes = []

    def attn(Q, cache, lens, **how):
        sizes.append((Q.shape[1], zb.zb_kv8_attn_workspace_bytes(cache, Q.shape[0], Q.shape[1], how["add_mass"])))
        return zb.zb_kv8_attn(Q, cache, lens, **how)
    bound = 83 << 18                                     # 350 queries need 20.76 MiB, 175 need 20.69
    monkeypatch.setattr(mod, "WORKSPACE_BOUND", bound, raising=False)
    monkeypatch.setattr(mod, "zb_kv8_attn", attn)
    O = banded.step(*parts, causal=causal)
    with pytest.raises(zb.ZbError, match="INDEX"):
        sync_ok()
    assert len(sizes) > 1 and sum(s for s, _ in sizes) == n and all(b <= bound for _, b in sizes), sizes
    assert not O[:, 3:].any() and O[:, :3].any() and banded.lens.tolist() == [800, 400]
    near = 2.0 ** -7 * want.float().abs() + 2.0 ** -9 * X.float().abs().max()
    assert ((O.float() - want.float()).abs() <= near).all()
    torch.testing.assert_close(banded.cache.mass, whole.cache.mass, rtol=2.0 ** -12, atol=1e-6)
