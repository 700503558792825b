"""Rotary positions and the norm of queries and keys, on the host: frequencies, the oracle's pins, refusals.
No call here reaches a CUDA API."""
import math

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


@pytest.mark.parametrize("how", [dict(), dict(base=100.0), dict(scaling="linear", factor=4.0),
                                 dict(scaling="ntk", factor=8.0),
                                 dict(scaling="parts", factor=16.0, original_len=4096.0),
                                 dict(scaling="parts", factor=8.0, original_len=8192.0, low=1.0, high=4.0)])
@pytest.mark.parametrize("rot,axes", [(64, 1), (16, 1), (64, 2), (32, 2)])
def test_frequencies(lib, how, rot, axes):
    import linear_hybrid_attention_b200 as zb
    f, m = oracle.rope_frequencies(rot // (2 * axes), **how)
    got = zb.zb_rope_frequencies(rot, axes=axes, **how)
    # each side takes some six fp64 roundings; the mix of ZB_ROPE_PARTS divides its result by up to the factor
    # (16 here) against terms that keep their absolute error: 2 * 6 * 16 * 2^-53
    rtol = 2 * 6 * 16 * 2.0 ** -53
    np.testing.assert_allclose(got.radians.numpy(), f, rtol=rtol)
    assert got.magnitude == pytest.approx(m, rel=1e-7)
    # turns: the same frequency in 64-bit fixed point (fp64 carries 53 bits of it)
    np.testing.assert_allclose(got.turns.numpy() / 2.0 ** 64 * 2 * np.pi, f, rtol=rtol)


def test_phases_of_far_positions_are_exact():
    # pos * turns mod 2^64 against integer arithmetic on the exact product
    import linear_hybrid_attention_b200 as zb
    fr = zb.zb_rope_frequencies(64)
    for pos in (0, 1, -7, 1_000_003, 2 ** 31 - 1, -2 ** 31):
        for t, f in zip(fr.turns.tolist(), fr.radians.tolist()):
            frac = ((pos * t) % 2 ** 64) / 2.0 ** 64
            want = math.fmod(pos * (f / (2 * math.pi)), 1.0)
            d = abs(frac - want) % 1.0
            # fp64 holds pos * f to 2^-53 of a value up to 2^31 * 0.16 turns
            assert min(d, 1 - d) <= 2.0 ** -22


def test_frequency_refusals(lib):
    import linear_hybrid_attention_b200 as zb
    buf = torch.zeros(32, dtype=torch.int64)
    t = buf.data_ptr()
    call = lambda pairs=8, base=1e4, sc=0, f=1.0, L=0.0, lo=1.0, hi=32.0, out=t: lib.zb_rope_frequencies(
        pairs, base, sc, f, L, lo, hi, out, None, None)
    assert call() == 0
    assert call(pairs=0) == 2 and call(pairs=33) == 2
    assert call(base=1.0) == 2 and call(base=float("nan")) == 2
    assert call(sc=4) == 4 and call(sc=-1) == 4
    assert call(sc=1, f=0.5) == 2 and call(sc=1, f=float("nan")) == 2
    assert call(sc=2, f=2.0, pairs=1) == 2
    assert call(sc=3, f=2.0) == 2                       # no original length
    assert call(sc=3, f=2.0, L=100.0, lo=4.0, hi=4.0) == 2
    assert call(out=None) == 1
    with pytest.raises(ValueError, match="scaling"):
        zb.zb_rope_frequencies(64, scaling="more")
    with pytest.raises(ValueError, match="rotary_dim"):
        zb.zb_rope_frequencies(18, axes=2)


def test_grid_positions():
    import linear_hybrid_attention_b200 as zb
    p = zb.grid_positions(2, grid=3, specials=2)
    assert p.shape == (1, 2, 22) and p.dtype == torch.int32
    assert p[0, 0, :11].tolist() == [0, 0, 1, 1, 1, 2, 2, 2, 3, 3, 3]
    assert p[0, 1, :11].tolist() == [0, 0, 1, 2, 3, 1, 2, 3, 1, 2, 3]
    assert torch.equal(p[..., :11], p[..., 11:])


# ------------------------------------------------------------ oracle's pins ----
def test_oracle_rotation_is_relative_and_keeps_norms():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 1, 64))
    f, _ = oracle.rope_frequencies(32)
    for layout in ("half", "interleaved"):
        turn = lambda x, p: oracle.rope(x, np.array([[[p]]]), f, layout=layout)
        dots = [(turn(q, 3 + d) * turn(k, d)).sum() for d in (0, 5, 1000)]
        np.testing.assert_allclose(dots, dots[0], rtol=1e-9)
        np.testing.assert_allclose((turn(q, 77) ** 2).sum(), (q ** 2).sum(), rtol=1e-12)
        back = oracle.rope(turn(q, 9), np.array([[[9]]]), f, layout=layout, inverse=True)
        np.testing.assert_allclose(back, q, atol=1e-12)
    # by hand: one pair, a quarter turn
    x = np.zeros((1, 1, 1, 64)); x[..., 0], x[..., 1] = 2.0, 3.0
    y = oracle.rope(x, np.array([[[1]]]), np.array([np.pi / 2]), layout="interleaved")
    np.testing.assert_allclose(y[0, 0, 0, :3], [-3.0, 2.0, 0.0], atol=1e-15)


@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("layout,axes", [("half", 1), ("interleaved", 2)])
def test_oracle_gradient_against_differences(kind, layout, axes):
    rng = np.random.default_rng(2)
    x, g = rng.standard_normal((2, 1, 2, 3, 64))
    w, b = rng.standard_normal((2, 64))
    b = b if kind == "layer" else None
    pos = rng.integers(0, 50, (1, axes, 3))
    f, _ = oracle.rope_frequencies(32 // (2 * axes), base=100.0)
    how = dict(axes=axes, layout=layout, magnitude=1.2)
    out = lambda x, w, b: (g * oracle.qk_norm_rope(x, w, b, kind, 1e-3, pos, f, **how)).sum()
    dx, dw, db = oracle.qk_norm_rope_grad(g, x, w, kind, 1e-3, pos, f, **how)
    h = 1e-6
    for at in [(0, 0, 0, 0), (0, 1, 2, 17), (0, 0, 1, 40), (0, 1, 0, 63)]:
        d = np.zeros_like(x); d[at] = h
        assert (out(x + d, w, b) - out(x - d, w, b)) / (2 * h) == pytest.approx(dx[at], rel=1e-6, abs=1e-7)
    if kind != "none":
        for e in (0, 21, 50):
            d = np.zeros(64); d[e] = h
            assert (out(x, w + d, b) - out(x, w - d, b)) / (2 * h) == pytest.approx(dw[e], rel=1e-6, abs=1e-7)
            if kind == "layer":
                assert (out(x, w, b + d) - out(x, w, b - d)) / (2 * h) == pytest.approx(db[e], rel=1e-6, abs=1e-7)


# ---------------------------------------------------------------- refusals ----
def _rows(b=1280, h=640, t=64):
    """Strides of a contiguous [B, 2, 10, 64] tensor unless told otherwise."""
    from linear_hybrid_attention_b200._lib import ZbRows
    return ZbRows(b, h, t)


def _rot(**over):
    from linear_hybrid_attention_b200._lib import ZbRotation
    d = dict(pos=FAKE, stride=0, turns=FAKE, rot=64, axes=1, layout=0, mag=1.0, inv=0)
    d.update(over)
    return ZbRotation(*d.values())


def test_rope_refusals(lib):
    call = lambda X=FAKE, xs=None, b=1, h=2, n=10, d=64, rot=None, Y=FAKE, ys=None: lib.zb_rope(
        X, xs or _rows(), b, h, n, d, rot or _rot(), Y, ys or _rows(), None)
    assert call(b=0) == 2 and call(h=0) == 2 and call(n=0) == 2
    assert call(d=128) == 4 and call(n=2 ** 31) == 4
    assert call(X=None) == 1 and call(Y=None) == 1
    assert call(X=FAKE + 8) == 3 and call(Y=FAKE + 2) == 3
    assert call(xs=_rows(t=60)) == 3 and call(xs=_rows(h=-64)) == 3 and call(ys=_rows(t=68)) == 3
    # outputs that overlap: repeated rows, heads closer than their tokens, a stride shared by two extents
    assert call(ys=_rows(t=0)) == 2 and call(ys=_rows(h=64)) == 2 and call(ys=_rows(t=32)) == 2
    assert call(b=2, ys=_rows(b=64)) == 2
    for r, want in ((_rot(rot=72), 2), (_rot(rot=-16), 2), (_rot(rot=24), 4), (_rot(rot=16, axes=2), 4),
                    (_rot(axes=3), 4), (_rot(layout=2), 4), (_rot(mag=0.0), 2), (_rot(mag=float("nan")), 2),
                    (_rot(mag=float("inf")), 2), (_rot(pos=None), 1), (_rot(turns=None), 1), (_rot(pos=FAKE + 2), 3),
                    (_rot(turns=FAKE + 4), 3), (_rot(stride=-1), 2)):
        assert call(rot=r) == want


def test_norm_rope_refusals(lib):
    from linear_hybrid_attention_b200._lib import ZbQkNorm
    nm = lambda kind=1, eps=1e-6, wq=None, wk=None, bq=None, bk=None: ZbQkNorm(kind, eps, wq, wk, bq, bk)
    fwd = lambda Q=FAKE, hq=2, K=FAKE, hk=2, n=10, d=64, norm=None, rot=None, Qo=FAKE, Ko=FAKE, ks=None: \
        lib.zb_qk_norm_rope(Q, _rows(), hq, K, ks or _rows(), hk, 1, n, d, norm or nm(), rot or _rot(), Qo, Ko, None)
    assert fwd(hq=0) == 2 and fwd(hk=-1) == 2 and fwd(d=32) == 4
    assert fwd(Q=None) == 1 and fwd(K=None) == 1 and fwd(Ko=None) == 1
    assert fwd(K=FAKE + 4) == 3 and fwd(ks=_rows(h=4)) == 3
    assert fwd(norm=nm(kind=3)) == 4 and fwd(norm=nm(eps=-1.0)) == 2 and fwd(norm=nm(eps=float("nan"))) == 2
    assert fwd(norm=nm(bq=FAKE)) == 4 and fwd(norm=nm(kind=2, bk=FAKE + 2)) == 3 and fwd(norm=nm(wq=FAKE + 1)) == 3
    assert fwd(rot=_rot(inv=1)) == 4
    need = lib.zb_qk_norm_rope_backward_workspace_bytes()
    bwd = lambda g=FAKE, Q=FAKE, K=FAKE, hk=2, norm=None, dQ=FAKE, dqs=None, dw=None, db=None, ws=FAKE, wsb=need: \
        lib.zb_qk_norm_rope_backward(g, g, Q, _rows(), 2, K, _rows(), hk, 1, 10, 64, norm or nm(), _rot(), dQ,
                                     dqs or _rows(), FAKE, _rows(), dw, dw, db, db, ws, wsb, None)
    assert bwd(g=None) == 1 and bwd(dQ=None) == 1 and bwd(dQ=FAKE + 8) == 3
    assert bwd(dqs=_rows(t=0)) == 2 and bwd(dqs=_rows(t=12)) == 3
    assert bwd(ws=None) == 5 and bwd(wsb=need - 1) == 5 and bwd(ws=FAKE + 4) == 3
    assert bwd(db=FAKE) == 4 and bwd(norm=nm(kind=0), dw=FAKE) == 4 and bwd(dw=FAKE + 2) == 3


def test_binding_refuses_cpu_tensors():
    import linear_hybrid_attention_b200 as zb
    x = torch.zeros(2, 10, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        zb.zb_rope(x, torch.zeros(1, 1, 10, dtype=torch.int32), torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        zb.zb_qk_norm_rope(x, x, None, None)
