"""The 8-bit cache's attention where values, logits and scales are uneven, for every kernel that serves it: few query
rows of a cache head (up to 32) and many (items of 128 rows, and of 256).

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

