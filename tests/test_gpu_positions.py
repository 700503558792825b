"""Rotary positions and the norm of queries and keys on the GPU, against the fp64 oracle.

Tolerances.  Outputs are rounded to bf16 once: half a step, 2^-8 of the value.  Before that everything is
fp32 on values no larger than the row's largest M times the magnitude: sines and cosines off by 2^-20.5 at most,
two of them in a feature (2^-19.5 M), products and a sum, some ten roundings of 2^-24 and the row's statistics (a sum
of 64 squares, rsqrt): under 2^-18 M in all.  A weight
gradient is a sum of n products, at most 100 of them one after another in a thread (sizes below), then trees:
128 * 2^-24 of the sum of the products' sizes, and the products' own error (see there).
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests.gpu_helpers import host, sync_ok

pytestmark = pytest.mark.gpu
HALF_BF16, ARITH = 2.0 ** -8, 2.0 ** -18


def _rand(shape, seed, spread=0.7):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[-1], generator=g))
    return x.bfloat16().cuda()


def _pos(B, axes, N, far, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-5 if far else 0, far + 50, (B, axes, N), generator=g, dtype=torch.int32)


def _close(got, ref, size):
    """|got - ref| <= half a bf16 step of ref + fp32 arithmetic on values of `size` (per row)."""
    got = host(got) if isinstance(got, torch.Tensor) else got
    bound = HALF_BF16 * np.abs(ref) + ARITH * size + 1e-30
    assert np.all(np.abs(got - ref) <= bound), float(np.max(np.abs(got - ref) / bound))


CASES = [  # batch, heads, tokens, rotary_dim, axes, layout, scaling, far, shared positions
    (1, 1, 1, 64, 1, "half", "none", 0, False),
    (3, 5, 1, 64, 1, "interleaved", "ntk", 2_000_000_000, False),
    (1, 16, 77, 64, 1, "half", "none", 0, True),
    (2, 3, 130, 32, 1, "half", "parts", 1_000_000, True),
    (2, 4, 65, 48, 1, "half", "linear", 4000, False),
    (2, 4, 65, 16, 1, "interleaved", "linear", 4000, False),
    (1, 6, 200, 64, 2, "half", "none", 0, True),
    (2, 1, 64, 32, 2, "half", "ntk", 100, False),
    (2, 7, 63, 64, 2, "interleaved", "none", 100, False),
    (1, 2, 1500, 32, 2, "interleaved", "parts", 0, True),
]


def _freq(zb, rot, axes, scaling):
    fr = zb.zb_rope_frequencies(rot, base=10000.0 if axes == 1 else 100.0, scaling=scaling, factor=8.0,
                                original_len=4096.0, axes=axes)
    return fr, fr.turns.cuda()


@pytest.mark.parametrize("B,H,N,rot,axes,layout,scaling,far,shared", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(B, H, N, rot, axes, layout, scaling, far, shared, inverse):
    import linear_hybrid_attention_b200 as zb
    X, pos = _rand((B, H, N, 64), 1), _pos(1 if shared else B, axes, N, far, 2)
    fr, turns = _freq(zb, rot, axes, scaling)
    Y = zb.zb_rope(X, pos.cuda(), turns, axes=axes, layout=layout, magnitude=fr.magnitude, inverse=inverse)
    ref = oracle.rope(host(X), pos.numpy(), fr.radians.numpy(), axes=axes, layout=layout, magnitude=fr.magnitude,
                      inverse=inverse)
    sync_ok()
    _close(Y, ref, np.abs(host(X)).max(-1, keepdims=True) * fr.magnitude)
    assert torch.equal(Y[..., rot:], X[..., rot:])     # the rest of the head passes unchanged
    # in place, and 3-dim tensors
    Z = X.clone()
    assert zb.zb_rope(Z, pos.cuda(), turns, axes=axes, layout=layout, magnitude=fr.magnitude, inverse=inverse,
                      out=Z) is Z
    assert torch.equal(Z, Y)
    if B == 1:
        assert torch.equal(zb.zb_rope(X[0], pos.cuda(), turns, axes=axes, layout=layout, magnitude=fr.magnitude,
                                      inverse=inverse), Y[0])


def test_rope_strides():
    import linear_hybrid_attention_b200 as zb
    B, H, N = 2, 5, 70
    fr, turns = _freq(zb, 64, 1, "none")
    pos = _pos(B, 1, N, 1000, 3).cuda()
    X = _rand((B, H, N, 64), 4)
    want = zb.zb_rope(X, pos, turns)
    # token-major storage with room around the heads, in and out
    store = torch.full((B, N, H + 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    view = store[:, :, 1:1 + H].transpose(1, 2)
    view.copy_(X)
    assert torch.equal(zb.zb_rope(view, pos, turns), want)
    assert zb.zb_rope(view, pos, turns, out=view) is view
    assert torch.equal(view, want)
    assert (store[:, :, 0] == 7).all() and (store[:, :, 1 + H:] == 7).all()
    # rows wider than a head (72 features a row), and one row repeated over the heads
    wide = torch.zeros((B, H, N, 72), dtype=torch.bfloat16, device="cuda")[..., 8:]
    wide.copy_(X)
    assert torch.equal(zb.zb_rope(wide, pos, turns), want)
    assert torch.equal(zb.zb_rope(X[:, :1].expand(-1, H, -1, -1), pos, turns), want[:, :1].expand(-1, H, -1, -1))


def _norm_case(B, Hq, Hk, N, kind, rot, axes, layout, scaling, far, seed):
    import linear_hybrid_attention_b200 as zb
    qk = _rand((B, N, Hq + Hk, 64), seed).transpose(1, 2)     # both inside one projection's output
    Q, K = qk[:, :Hq], qk[:, Hq:]
    g = torch.Generator().manual_seed(seed + 1)
    wq, wk = (1 + 0.3 * torch.randn(64, generator=g) for _ in range(2))
    bq, bk = (0.2 * torch.randn(64, generator=g) if kind == "layer" else None for _ in range(2))
    pos = _pos(B, axes, N, far, seed + 2)
    fr, turns = _freq(zb, rot, axes, scaling)
    dev = lambda t: None if t is None else t.cuda()
    how = dict(norm=kind, wq=dev(wq), wk=dev(wk), eps=1e-6, axes=axes, layout=layout, magnitude=fr.magnitude)
    ora = dict(axes=axes, layout=layout, magnitude=fr.magnitude)
    return zb, Q, K, (wq, wk, bq, bk), pos, fr, turns, how, ora


NORM_CASES = [  # batch, q heads, k heads, tokens, norm, rotary_dim, axes, layout, scaling, far
    (1, 1, 1, 1, "rms", 64, 1, "half", "none", 0),
    (5, 8, 2, 1, "layer", 64, 1, "half", "ntk", 2_000_000_000),
    (1, 16, 16, 77, "rms", 32, 1, "interleaved", "parts", 100_000),
    (2, 6, 3, 129, "layer", 64, 2, "half", "none", 30),
    (2, 4, 4, 64, "none", 48, 1, "half", "none", 0),
    (1, 20, 1, 650, "rms", 64, 2, "interleaved", "linear", 30),
]


@pytest.mark.parametrize("B,Hq,Hk,N,kind,rot,axes,layout,scaling,far", NORM_CASES)
def test_qk_norm_rope(B, Hq, Hk, N, kind, rot, axes, layout, scaling, far):
    zb, Q, K, (wq, wk, bq, bk), pos, fr, turns, how, ora = _norm_case(B, Hq, Hk, N, kind, rot, axes, layout, scaling,
                                                                      far, 11)
    dev = lambda t: None if t is None else t.cuda()
    Qo, Ko = zb.zb_qk_norm_rope(Q, K, pos.cuda(), turns, bq=dev(bq), bk=dev(bk), **how)
    sync_ok()
    for got, x, w, b in ((Qo, Q, wq, bq), (Ko, K, wk, bk)):
        assert got.is_contiguous()
        n64 = lambda t: None if t is None else t.double().numpy()
        plain = oracle.qk_norm_rope(host(x), n64(w), n64(b), kind, float(np.float32(1e-6)), None, None)
        ref = oracle.qk_norm_rope(host(x), n64(w), n64(b), kind, float(np.float32(1e-6)), pos.numpy(),
                                  fr.radians.numpy(), **ora)
        # a layer norm subtracts the mean first: its error is of the size of the row's largest value
        size = np.abs(plain).max(-1, keepdims=True) * fr.magnitude * (4 if kind == "layer" else 1)
        _close(got, ref, size)
    # queries alone give the same queries
    alone, none = zb.zb_qk_norm_rope(Q, None, pos.cuda(), turns, bq=dev(bq), **how)
    assert none is None and torch.equal(alone, Qo)
    # no rotation: the norm alone
    if kind != "none":
        y, _ = zb.zb_qk_norm_rope(Q, None, None, None, bq=dev(bq), **how)
        _close(y, oracle.qk_norm_rope(host(Q), wq.double().numpy(), None if bq is None else bq.double().numpy(), kind,
                                      float(np.float32(1e-6)), None, None),
               np.abs(host(y)).max(-1, keepdims=True) * 4)


@pytest.mark.parametrize("B,Hq,Hk,N,kind,rot,axes,layout,scaling,far", NORM_CASES)
def test_qk_norm_rope_backward(B, Hq, Hk, N, kind, rot, axes, layout, scaling, far):
    zb, Q, K, (wq, wk, _, _), pos, fr, turns, how, ora = _norm_case(B, Hq, Hk, N, kind, rot, axes, layout, scaling,
                                                                    far, 21)
    gq, gk = _rand((B, Hq, N, 64), 31), _rand((B, Hk, N, 64), 32)
    store = torch.zeros((B, N, Hq + Hk, 64), dtype=torch.bfloat16, device="cuda")
    views = store.transpose(1, 2)
    out = zb.zb_qk_norm_rope_backward(gq, gk, Q, K, pos.cuda(), turns, dQ=views[:, :Hq], dK=views[:, Hq:], **how)
    sync_ok()
    for got, x, g, w, dw, db in ((out[0], Q, gq, wq, out[2], out[4]), (out[1], K, gk, wk, out[3], out[5])):
        w64 = w.double().numpy()
        eps = float(np.float32(1e-6))
        dx, rw, rb = oracle.qk_norm_rope_grad(host(g), host(x), w64, kind, eps, pos.numpy(), fr.radians.numpy(), **ora)
        xh, r = oracle.qk_norm(host(x), kind, eps)
        size = r * np.abs(host(g)).max(-1, keepdims=True) * fr.magnitude * (1 if kind == "none" else np.abs(w64).max())
        # dx subtracts xh mean(g xh): values up to max|xh| = 8 times the row's mean of products
        _close(got, dx, size * (1 + 2 * np.abs(xh).max(-1, keepdims=True) if kind != "none" else 1))
        if kind == "none":
            assert dw is None and db is None
            continue
        dy = oracle.rope(host(g), pos.numpy(), fr.radians.numpy(), inverse=True, **ora)
        # dy = a cos + b sin may cancel: its own error is ARITH of the row's largest gradient (as in _close),
        # not of dy, and enters the sums multiplied by xh
        big = np.abs(host(g)).max(-1, keepdims=True) * fr.magnitude
        tol = 128 * 2.0 ** -24 * np.abs(dy * xh).sum((0, 1, 2)) + 4 * ARITH * (big * np.abs(xh)).sum((0, 1, 2)) + 1e-30
        assert np.all(np.abs(dw.cpu().double().numpy() - rw) <= tol)
        if kind == "layer":
            tol = 128 * 2.0 ** -24 * np.abs(dy).sum((0, 1, 2)) + ARITH * (big + 0 * dy).sum((0, 1, 2)) + 1e-30
            assert np.all(np.abs(db.cpu().double().numpy() - rb) <= tol)
        else:
            assert db is None
    # the same bits again, into fresh contiguous outputs, from gradients that are not contiguous
    again = zb.zb_qk_norm_rope_backward(gq.transpose(1, 2).contiguous().transpose(1, 2), gk, Q, K, pos.cuda(), turns,
                                        **how)
    for x, y in zip(out, again):
        assert (x is None and y is None) or torch.equal(x, y)


def test_zero_rows_and_no_eps():
    # a row of zeros with eps > 0 gives zeros (and a zero gradient path through eps); rows the kernel
    # pads its last group with do not reach the weight gradients even with eps = 0
    import linear_hybrid_attention_b200 as zb
    Q = _rand((1, 3, 7, 64), 5)
    g = _rand((1, 3, 7, 64), 6)
    w = torch.ones(64, device="cuda")
    dQ, _, dw, _, _, _ = zb.zb_qk_norm_rope_backward(g, None, Q, None, None, None, norm="rms", wq=w, eps=0.0)
    dx, rw, _ = oracle.qk_norm_rope_grad(host(g), host(Q), None, "rms", 0.0, None, None)
    assert np.isfinite(host(dQ)).all() and torch.isfinite(dw).all()
    xh, _ = oracle.qk_norm(host(Q), "rms", 0.0)
    assert np.all(np.abs(dw.cpu().double().numpy() - rw)
                  <= (128 * 2.0 ** -24 + 4 * ARITH) * np.abs(host(g) * xh).sum((0, 1, 2)))
    Z = torch.zeros_like(Q)
    y, _ = zb.zb_qk_norm_rope(Z, None, None, None, norm="rms", wq=w, eps=1e-6)
    assert (y == 0).all()
    sync_ok()


def test_nan_stays_in_its_row():
    import linear_hybrid_attention_b200 as zb
    fr, turns = _freq(zb, 64, 1, "none")
    pos = _pos(1, 1, 40, 0, 1).cuda()
    X = _rand((1, 4, 40, 64), 8)
    Y = X.clone()
    Y[0, 2, 13, 5] = float("nan")
    a, _ = zb.zb_qk_norm_rope(X, None, pos, turns)
    b, _ = zb.zb_qk_norm_rope(Y, None, pos, turns)
    assert torch.isnan(b[0, 2, 13]).all()
    b[0, 2, 13] = a[0, 2, 13]
    assert torch.equal(a, b)


def test_graph_replay_and_streams():
    import linear_hybrid_attention_b200 as zb
    fr, turns = _freq(zb, 64, 1, "none")
    X = _rand((1, 4, 100, 64), 9)
    pos = _pos(1, 1, 100, 500, 1).cuda()
    zb.zb_rope(X, pos, turns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        q, _ = zb.zb_qk_norm_rope(X, None, pos, turns)
        d = zb.zb_qk_norm_rope_backward(q, None, X, None, pos, turns)
    X.copy_(_rand((1, 4, 100, 64), 10))
    pos += 3
    graph.replay()
    torch.cuda.synchronize()
    q2, _ = zb.zb_qk_norm_rope(X, None, pos, turns)
    d2 = zb.zb_qk_norm_rope_backward(q2, None, X, None, pos, turns)
    assert torch.equal(q, q2) and torch.equal(d[0], d2[0]) and torch.equal(d[2], d2[2])


def test_binding_refusals():
    import linear_hybrid_attention_b200 as zb
    fr, turns = _freq(zb, 64, 1, "none")
    X = _rand((1, 4, 10, 64), 9)
    pos = _pos(1, 1, 10, 0, 1).cuda()
    bad = [(dict(X=X.float()), TypeError), (dict(X=X[..., :32]), ValueError), (dict(X=X.transpose(2, 3)), ValueError),
           (dict(pos=pos[..., :9]), ValueError), (dict(pos=pos.long()), ValueError), (dict(pos=pos.cpu()), ValueError),
           (dict(turns=turns.cpu()), ValueError), (dict(turns=turns[::2]), ValueError), (dict(axes=2), ValueError),
           (dict(layout="both"), ValueError), (dict(turns=turns[:20].contiguous()), zb.ZbError),
           (dict(out=X[:, :3]), ValueError), (dict(out=X[:, :1].expand(-1, 4, -1, -1)), zb.ZbError),
           (dict(X=X.view(-1)[4:4 + 9 * 64].view(1, 1, 9, 64), pos=pos[..., :9].contiguous()), zb.ZbError)]
    for over, err in bad:
        with pytest.raises(err):
            zb.zb_rope(**{**dict(X=X, pos=pos, turns=turns), **over})
    w = torch.ones(64, device="cuda")
    for over, err in [(dict(norm="group"), ValueError), (dict(wq=w.cpu()), ValueError), (dict(wq=w[:32]), ValueError),
                      (dict(bq=w), zb.ZbError), (dict(K=X[:, :, :9]), ValueError), (dict(eps=-1.0), zb.ZbError),
                      (dict(out_q=X.transpose(1, 2)), ValueError)]:
        with pytest.raises(err):
            zb.zb_qk_norm_rope(**{**dict(Q=X, K=X, pos=pos, turns=turns), **over})
    with pytest.raises(ValueError):
        zb.zb_qk_norm_rope_backward(X[:, :2], None, X, None, pos, turns)
    with pytest.raises(ValueError):
        zb.zb_qk_norm_rope_backward(X, None, X, None, pos, turns, ws=torch.empty(1 << 22, dtype=torch.uint8))


@pytest.mark.parametrize("axes,layout,rot", [(1, "half", 64), (1, "interleaved", 48), (2, "half", 64), (2, "interleaved", 32)])
def test_position_zero_changes_nothing(axes, layout, rot):
    import linear_hybrid_attention_b200 as zb
    fr, turns = _freq(zb, rot, axes, "none")
    X = _rand((2, 3, 70, 64), 40)
    pos = torch.zeros((1, axes, 70), dtype=torch.int32, device="cuda")
    for inverse in (False, True):
        assert torch.equal(zb.zb_rope(X, pos, turns, axes=axes, layout=layout, inverse=inverse), X)


# more items than the GPU takes at once: a CTA's share begins and ends inside a token's heads, and groups of
# tokens cross from one sequence to the next
MANY = [(3, 7, 3, 4001, "rms", 64, 1, "half", "ntk", 100_000), (2, 5, 5, 5003, "layer", 32, 1, "interleaved", "none", 0),
        (1, 9, 1, 9000, "layer", 64, 2, "half", "none", 30)]


@pytest.mark.parametrize("B,Hq,Hk,N,kind,rot,axes,layout,scaling,far", MANY)
def test_many_items(B, Hq, Hk, N, kind, rot, axes, layout, scaling, far):
    zb, Q, K, (wq, wk, bq, bk), pos, fr, turns, how, ora = _norm_case(B, Hq, Hk, N, kind, rot, axes, layout, scaling,
                                                                      far, 51)
    dev = lambda t: None if t is None else t.cuda()
    n64 = lambda t: None if t is None else t.double().numpy()
    eps = float(np.float32(1e-6))
    pos_d = pos.cuda()
    y = zb.zb_rope(Q, pos_d, turns, axes=axes, layout=layout, magnitude=fr.magnitude)
    _close(y, oracle.rope(host(Q), pos.numpy(), fr.radians.numpy(), **ora),
           np.abs(host(Q)).max(-1, keepdims=True) * fr.magnitude)
    outs = zb.zb_qk_norm_rope(Q, K, pos_d, turns, bq=dev(bq), bk=dev(bk), **how)
    gq, gk = _rand((B, Hq, N, 64), 52), _rand((B, Hk, N, 64), 53)
    grad = zb.zb_qk_norm_rope_backward(gq, gk, Q, K, pos_d, turns, **how)
    sync_ok()
    for got, x, w, b, g, dx, dw, db in ((outs[0], Q, wq, bq, gq, grad[0], grad[2], grad[4]),
                                        (outs[1], K, wk, bk, gk, grad[1], grad[3], grad[5])):
        plain = oracle.qk_norm_rope(host(x), n64(w), n64(b), kind, eps, None, None)
        ref = oracle.qk_norm_rope(host(x), n64(w), n64(b), kind, eps, pos.numpy(), fr.radians.numpy(), **ora)
        _close(got, ref, np.abs(plain).max(-1, keepdims=True) * fr.magnitude * (4 if kind == "layer" else 1))
        rx, rw, rb = oracle.qk_norm_rope_grad(host(g), host(x), n64(w), kind, eps, pos.numpy(), fr.radians.numpy(), **ora)
        xh, r = oracle.qk_norm(host(x), kind, eps)
        big = np.abs(host(g)).max(-1, keepdims=True) * fr.magnitude
        size = r * big * np.abs(n64(w)).max()
        _close(dx, rx, size * (1 + 2 * np.abs(xh).max(-1, keepdims=True)))
        dy = oracle.rope(host(g), pos.numpy(), fr.radians.numpy(), inverse=True, **ora)
        # as in test_qk_norm_rope_backward: at most 100 products one after another in a thread
        tol = 128 * 2.0 ** -24 * np.abs(dy * xh).sum((0, 1, 2)) + 4 * ARITH * (big * np.abs(xh)).sum((0, 1, 2))
        assert np.all(np.abs(dw.cpu().double().numpy() - rw) <= tol)
        if kind == "layer":
            tol = 128 * 2.0 ** -24 * np.abs(dy).sum((0, 1, 2)) + ARITH * (big + 0 * dy).sum((0, 1, 2))
            assert np.all(np.abs(db.cpu().double().numpy() - rb) <= tol)


def test_offsets_past_32_bits():
    import linear_hybrid_attention_b200 as zb
    far = 2 ** 31 + 64                                  # elements from one head to the next
    store = torch.zeros(far + 5 * 64, dtype=torch.bfloat16, device="cuda")
    view = store.as_strided((1, 2, 5, 64), (0, far, 64, 1))
    X = _rand((1, 2, 5, 64), 60)
    view.copy_(X)
    fr, turns = _freq(zb, 64, 1, "none")
    pos = _pos(1, 1, 5, 1000, 61).cuda()
    want = zb.zb_rope(X, pos, turns)
    assert torch.equal(zb.zb_rope(view, pos, turns), want)
    q, _ = zb.zb_qk_norm_rope(view, None, pos, turns)
    q2, _ = zb.zb_qk_norm_rope(X, None, pos, turns)
    assert torch.equal(q, q2)
    d = zb.zb_qk_norm_rope_backward(want, None, X, None, pos, turns)
    zb.zb_qk_norm_rope_backward(want, None, X, None, pos, turns, dQ=view)
    assert torch.equal(view, d[0])
    assert zb.zb_rope(view, pos, turns, out=view) is view and torch.equal(view, zb.zb_rope(d[0], pos, turns))
    sync_ok()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_norm_of_rows_of_every_size(kind, eps):
    """Rows whose squares pass fp32, or are lost below it, between ordinary ones.  Forward as above: a normalised row
    is at most 8.  Backward, T the largest |w dy| of a row: dx = r (t - xh mean(t xh) - mean t) is at most 10 r T
    before its last rounding, and fp32 arithmetic and the sines take 2^-17 of that."""
    import linear_hybrid_attention_b200 as zb
    N = 150
    Q = _rand((1, 2, N, 64), 71)
    size = torch.tensor([2.0 ** e for e in (-100, 118, 0, 70, -60, 55, -45)]).repeat(N)[:N]
    Q = (Q.float() * size.cuda()[:, None]).bfloat16()
    g = torch.Generator().manual_seed(72)
    w, b = 1 + 0.3 * torch.randn(64, generator=g), 0.2 * torch.randn(64, generator=g) if kind == "layer" else None
    pos = _pos(1, 1, N, 1000, 73)
    fr, turns = _freq(zb, 64, 1, "none")
    got, _ = zb.zb_qk_norm_rope(Q, None, pos.cuda(), turns, norm=kind, wq=w.cuda(), bq=None if b is None else b.cuda(), eps=eps)
    sync_ok()
    w64, b64 = w.double().numpy(), None if b is None else b.double().numpy()
    e32 = float(np.float32(eps))
    ref = oracle.qk_norm_rope(host(Q), w64, b64, kind, e32, pos.numpy(), fr.radians.numpy())
    plain = oracle.qk_norm_rope(host(Q), w64, b64, kind, e32, None, None)
    _close(got, ref, np.abs(plain).max(-1, keepdims=True) + np.abs(w64).max() * 1.0)
    dy = _rand((1, 2, N, 64), 74, 0.3)
    dQ, _, dwq, _, dbq, _ = zb.zb_qk_norm_rope_backward(dy, None, Q, None, pos.cuda(), turns, norm=kind, wq=w.cuda(), eps=eps)
    sync_ok()
    dx, dw, db = oracle.qk_norm_rope_grad(host(dy), host(Q), w64, kind, e32, pos.numpy(), fr.radians.numpy())
    r = oracle.qk_norm(host(Q), kind, e32)[1]
    T = np.abs(oracle.rope(host(dy), pos.numpy(), fr.radians.numpy(), inverse=True) * w64).max(-1, keepdims=True)
    assert np.all(np.abs(host(dQ) - dx) <= HALF_BF16 * np.abs(dx) + 2.0 ** -17 * 10 * r * T)
    # sums of 300 products of at most 8 |dy| each, whose errors are 2^-18 of that
    assert np.all(np.abs(dwq.double().cpu().numpy() - dw) <= 300 * 2.0 ** -17 * 8 * np.abs(host(dy)).max())
    if kind == "layer":
        assert np.all(np.abs(dbq.double().cpu().numpy() - db) <= 300 * 2.0 ** -17 * np.abs(host(dy)).max())
