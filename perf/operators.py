"""Cases that measure the operators around the attention calls: rotary positions, the per-head norm of
queries and keys with the rotation in the same pass (and its gradient), the 8-bit key/value cache with the
attention that reads it, and eviction from that cache by accumulated attention weight.

Heads are 64 wide and tensors bf16, as everywhere in the library.  ``run`` computes the plain form, or with
``own`` set calls the library.  Sizes come from the library's own workloads (16 heads, 1,374 tokens a view,
32 and 256 views, tiles of 64 and 128, 10,992 tiles with 660 kept) or are generic.
"""
import math

import torch

own = False

D = 64
TOP = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one new token of each of 40 sequences far into a scaled context: a decode step's latency
        dict(name="rope_step", op="rope", batch=40, heads=16, n=1, rot=64, axes=1, layout="half", scaling="ntk",
             far=1_000_000, inverse=False),
        # the gradient of a 2-D rotation over 32 views, queries as the attention's backward leaves them
        dict(name="rope_grad_views", op="rope", batch=1, heads=16, n=43_968, rot=64, axes=2, layout="half",
             scaling="none", far=0, inverse=True),
        # one view entering the layer: q and k taken out of their common projection's output
        dict(name="norm_rope_view", op="norm_rope", batch=1, heads=16, kv_heads=16, n=1_374, norm="rms", rot=64,
             axes=1, layout="half", scaling="none", far=0),
        # 32 views, layer norm and a 2-D rotation: the shape of the 32-view attention stage
        dict(name="norm_rope_views", op="norm_rope", batch=1, heads=16, kv_heads=16, n=43_968, norm="layer", rot=64,
             axes=2, layout="half", scaling="none", far=0),
        # a training step: forward and backward, grouped heads, half of the head rotated, long-context scaling
        dict(name="norm_rope_train", op="norm_rope_train", batch=2, heads=16, kv_heads=4, n=10_992, norm="rms", rot=32,
             axes=1, layout="interleaved", scaling="parts", far=500_000),
        # 32 views entering the cache at once, and read back in bf16 for the bf16 attention calls
        dict(name="append_views", op="append", heads=16, n=43_968, block=128, fmt="int8", past=0),
        # one token against two views: the smallest attention call, where latency counts
        dict(name="attend_short", op="attend", seqs=1, kv_heads=16, group=1, n_q=1, longest=2_749, ragged=False,
             block=64, fmt="int8", causal=False, add_mass=False),
        # a batch of sequences of very different lengths, grouped heads, attention weight kept for eviction
        dict(name="attend_batch", op="attend", seqs=24, kv_heads=4, group=4, n_q=1, longest=16_384, ragged=True,
             block=64, fmt="int8", causal=False, add_mass=True),
        # one token against 256 views: the bytes of the cache are all that counts
        dict(name="attend_long", op="attend", seqs=1, kv_heads=16, group=1, n_q=1, longest=351_744, ragged=False,
             block=128, fmt="e4m3", causal=False, add_mass=True),
        # a chunk of one view's tokens, causal, against 32 views: bound by arithmetic
        dict(name="attend_chunk", op="attend", seqs=1, kv_heads=16, group=1, n_q=1_374, longest=43_968, ragged=False,
             block=128, fmt="int8", causal=True, add_mass=True),
        # every head of one 1,024-view sequence down to the library's 660 kept tiles
        dict(name="evict_long", op="evict", heads=16, slots=10_992, block=128, budget=660, sinks=4, recent=12),
        # a batch of sequences in serving, each near its budget
        dict(name="evict_batch", op="evict", heads=384, slots=344, block=64, budget=256, sinks=1, recent=8),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "norm_rope_train", "append", "attend", "attend", "attend", "evict"])
    if op == "evict":
        slots = _spread(rng, 40, 10_992)
        sinks, recent = rng.randint(0, 4), rng.randint(1, 12)
        budget = rng.randint(sinks + recent, max(sinks + recent, (slots * 3) // 4))
        return dict(op=op, heads=max(1, min(_spread(rng, 4, 1_024), 400_000 // slots)), slots=slots,
                    block=rng.choice([16, 32, 64, 128]), budget=budget, sinks=sinks, recent=recent)
    block, fmt = rng.choice([16, 32, 64, 128]), rng.choice(["int8", "e4m3"])
    if op == "append":
        heads = _spread(rng, 4, 128)
        n, past = rng.choice([1, rng.randint(1, 8), _spread(rng, 1, 600_000 // heads)]), rng.randint(0, 40 * block)
        if past % block + n > block:
            # the rows of the block in progress make way for those of the last one: a pass could not be repeated
            past -= past % block
        return dict(op=op, heads=heads, n=n, block=block, fmt=fmt, past=past)
    if op == "attend":
        seqs, kv_heads, group = _spread(rng, 1, 32), rng.choice([2, 4, 8, 16]), rng.choice([1, 2, 4, 8])
        n_q = rng.choice([1, 1, 2, 5, _spread(rng, 2, 1_374)])
        longest = min(_spread(rng, 300, 351_744), 4_000_000 // (seqs * kv_heads))
        longest = max(n_q + 1, min(longest, 600_000_000 // (seqs * kv_heads * group * n_q)))
        return dict(op=op, seqs=seqs, kv_heads=kv_heads, group=group, n_q=n_q, longest=longest,
                    ragged=rng.random() < 0.7, block=block, fmt=fmt, causal=rng.random() < 0.5,
                    add_mass=rng.random() < 0.6)
    axes = rng.choice([1, 2])
    heads = rng.choice([4, 6, 8, 16, 20, 32])
    batch = _spread(rng, 1, 40)
    c = dict(op=op, batch=batch, heads=heads, n=max(1, _spread(rng, 1, 600_000) // (batch * heads)),
             rot=rng.choice([16, 32, 48, 64]) if axes == 1 else rng.choice([32, 64]), axes=axes,
             layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "parts"]),
             far=0 if axes == 2 else rng.choice([0, 4_000, 1_000_000]))
    if op == "rope":
        return dict(c, inverse=rng.random() < 0.5)
    return dict(c, kv_heads=rng.choice([h for h in (1, 2, 4, 8, 16, 32) if heads % h == 0]),
                norm=rng.choice(["rms", "layer"]))


# ----------------------------------------------------------------- inputs ----
def _frequencies(c):
    """The rotation's frequencies (radians a position) and magnitude, as Python floats."""
    n = c["rot"] // (2 * c["axes"])
    base, factor, length = (100.0 if c["axes"] == 2 else 10_000.0), 8.0, 4_096.0
    if c["scaling"] == "ntk":
        base *= factor ** (n / (n - 1))
    f = [base ** (-i / n) for i in range(n)]
    if c["scaling"] == "linear":
        f = [x / factor for x in f]
    if c["scaling"] == "parts":  # by the rotations a frequency makes over the trained length
        g = [min(1.0, max(0.0, (length * x / (2 * math.pi) - 1.0) / 31.0)) for x in f]
        return [(1 - r) * x / factor + r * x for x, r in zip(f, g)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _positions(c, gen):
    B, N = c["batch"], c["n"]
    if c["axes"] == 2:  # 37 x 37 patches after five special tokens a view, patches counted from 1
        t = torch.arange(N, device="cuda") % 1_374
        p = torch.clamp(t - 5, min=0)
        row, col = p // 37 + 1, p % 37 + 1
        return torch.stack([torch.where(t < 5, 0, row), torch.where(t < 5, 0, col)])[None].to(torch.int32).contiguous()
    first = torch.randint(0, c["far"] + 1, (B, 1, 1), device="cuda", generator=gen)
    return (first + torch.arange(N, device="cuda")).to(torch.int32).contiguous()


def _heavy(shape, gen):
    """Rows as a projection makes them: a few channels far larger than the rest."""
    x = torch.randn(shape, device="cuda", generator=gen)
    return x * torch.exp(0.7 * torch.randn(shape[-1], device="cuda", generator=gen))


def _quantised(x, fmt):
    """Codes [..., B, 64] (whole numbers of steps as fp32 values) and scales [...] of blocks x in fp32."""
    s = (x.abs().amax((-1, -2)).double() / TOP[fmt]).float()
    t = x.double() / torch.where(s > 0, s, torch.ones_like(s)).double()[..., None, None]
    if fmt == "int8":
        return t.round().float(), s
    step = torch.exp2(torch.clamp(torch.frexp(t)[1] - 1, min=-6).double() - 3)
    return (torch.round(t / step) * step).clamp(-448, 448).float(), s


def _codes(v, fmt):
    return v.to(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(c)
    if c["op"] in ("rope", "norm_rope", "norm_rope_train"):
        B, H, N = c["batch"], c["heads"], c["n"]
        f, st["magnitude"] = _frequencies(c)
        st["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        st["turns"] = torch.tensor([round(x / (2 * math.pi) * 2.0 ** 64) for x in f], dtype=torch.int64, device="cuda")
        st["pos"] = _positions(c, gen)
        if c["op"] == "rope":
            st["x"] = _heavy((B, H, N, D), gen).bfloat16()
            return st
        G = c["kv_heads"]
        # the projection's output: [batch][token][q heads | k heads][64]
        st["qk"] = _heavy((B, N, H + G, D), gen).bfloat16()
        for w in ("wq", "wk"):
            st[w] = 1 + 0.2 * torch.randn(D, device="cuda", generator=gen)
        for b in ("bq", "bk"):
            st[b] = 0.1 * torch.randn(D, device="cuda", generator=gen) if c["norm"] == "layer" else None
        if c["op"] == "norm_rope_train":
            st["gq"] = torch.randn((B, H, N, D), device="cuda", generator=gen).bfloat16()
            st["gk"] = torch.randn((B, G, N, D), device="cuda", generator=gen).bfloat16()
        return st
    if c["op"] == "evict":
        H, S = c["heads"], c["slots"]
        st["table"] = torch.rand((H, S), device="cuda", generator=gen).argsort(1).to(torch.int32)
        # most blocks get little weight, many the same little
        m = torch.exp(2.5 * torch.randn((H, S), device="cuda", generator=gen))
        st["mass"] = (m * 16).floor() / 16
        low = max(1, (S * c["block"] * 3) // 4)
        st["lens"] = torch.randint(low, S * c["block"] + 1, (H,), device="cuda", generator=gen).to(torch.int32)
        return st
    B, fmt = c["block"], c["fmt"]
    if c["op"] == "append":
        H, lens = c["heads"], torch.full((c["heads"],), c["past"], dtype=torch.int32, device="cuda")
        slots = -(-(c["past"] + c["n"]) // B) + 2
    else:
        H = c["seqs"] * c["kv_heads"]
        slots = -(-c["longest"] // B)
        each = torch.full((c["seqs"],), float(c["longest"]), device="cuda")
        if c["ragged"] and c["seqs"] > 1:  # from one token to the longest, both among them
            u = torch.rand(c["seqs"], device="cuda", generator=gen)
            u[0], u[-1] = 1.0, 0.0
            each = (1 + u * (c["longest"] - 1)).round()
        lens = each.to(torch.int32).repeat_interleave(c["kv_heads"]).contiguous()
    st["lens"] = lens
    typ = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
    for n in ("k", "v"):
        st[n] = torch.empty((H, slots, B, D), dtype=typ, device="cuda")
        st[n + "_scale"] = torch.empty((H, slots), device="cuda")
        for h in range(H):
            v, st[n + "_scale"][h] = _quantised(_heavy((slots, B, D), gen).bfloat16().float(), fmt)
            st[n][h] = _codes(v, fmt)
        st[n + "_tail"] = _heavy((H, B, D), gen).bfloat16()
    st["table"] = torch.rand((H, slots), device="cuda", generator=gen).argsort(1).to(torch.int32)
    # weight of earlier calls, of the size of this one's
    st["mass"] = torch.rand((H, slots), device="cuda", generator=gen) * (c.get("group", 1) * c.get("n_q", 1) / slots)
    st["lens_out"] = torch.empty_like(lens)
    if c["op"] == "append":
        st["K"], st["V"] = (_heavy((H, c["n"], D), gen).bfloat16() for _ in range(2))
    else:
        st["Q"] = torch.randn((H * c["group"], c["n_q"], D), device="cuda", generator=gen).bfloat16()
    if own:
        import linear_hybrid_attention_b200 as zb
        st["cache"] = zb.KV8Cache(**{n: st[n] for n in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail", "table",
                                                        "mass")})
    return st


# ------------------------------------------------------------ plain forms ----
def _angles(st):
    """cos and sin [batch or 1, 1, n, axes, pairs]: angles in 64 bits, rounded once."""
    a = st["pos"].transpose(1, 2)[:, None, :, :, None].double() * st["freq"]
    return (torch.cos(a) * st["magnitude"]).float(), (torch.sin(a) * st["magnitude"]).float()


def _rotated(x, st, back):
    """x fp32 [B, H, N, 64] with the first `rot` features rotated (backwards: by the opposite angles)."""
    r, axes = st["rot"], st["axes"]
    cos, sin = _angles(st)
    if back:
        sin = -sin
    n = r // (2 * axes)
    half = st["layout"] == "half"
    part = x[..., :r].reshape(*x.shape[:-1], axes, *((2, n) if half else (n, 2)))
    a, b = (part[..., 0, :], part[..., 1, :]) if half else (part[..., 0], part[..., 1])
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -2 if half else -1)
    return torch.cat([turned.reshape(*x.shape[:-1], r), x[..., r:]], -1)


def _normed(x, norm):
    """(normalised x, the factor 1 / sigma) over the last axis, in fp32."""
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    return x * r, r


def _norm_rope(x, w, b, st):
    y = _normed(x, st["norm"])[0] * w
    return _rotated(y if b is None else y + b, st, False).bfloat16()


def _norm_rope_grad(g, x, w, st):
    dy = _rotated(g.float(), st, True)
    xh, r = _normed(x, st["norm"])
    dw, db = (dy * xh).sum((0, 1, 2)), dy.sum((0, 1, 2))
    t = dy * w
    dx = t - xh * (t * xh).mean(-1, keepdim=True)
    if st["norm"] == "layer":
        dx = dx - t.mean(-1, keepdim=True)
    return (dx * r).bfloat16(), dw, (db if st["norm"] == "layer" else None)


def _split(st):
    H = st["heads"]
    qk = st["qk"].transpose(1, 2)
    return qk[:, :H], qk[:, H:]


def _values(st, n):
    """The cached values [H, tokens, 64] in logical order, fp32."""
    t = st["table"].long()
    c = st[n].float().gather(1, t[:, :, None, None].expand(-1, -1, *st[n].shape[2:]))
    return (c * st[n + "_scale"].gather(1, t)[:, :, None, None]).flatten(1, 2)


def _append(st):
    B, fmt, H = st["block"], st["fmt"], st["heads"]
    held = st["lens"] % B  # all heads hold whole blocks or parts of one; new rows follow them
    rows = -(-(B - 1 + st["n"]) // B) * B
    at = torch.arange(rows, device="cuda")[None]
    new = at - held[:, None]
    inside = (new >= 0) & (new < st["n"])
    first = st["lens"] // B
    blocks = (held + st["n"] + B - 1) // B
    lanes = torch.arange(rows // B, device="cuda")[None]
    live = lanes < blocks[:, None]
    slot = st["table"].long().gather(1, (first[:, None] + lanes).clamp(max=st["table"].shape[1] - 1))
    last = (held + st["n"]) // B * B  # the first row of the block left in progress
    for n, x in (("k", st["K"]), ("v", st["V"])):
        y = x.float().gather(1, new.clamp(0, st["n"] - 1)[..., None].expand(-1, -1, D)) * inside[..., None]
        y[:, :B] += st[n + "_tail"].float() * (at[:, :B] < held[:, None])[..., None]
        v, s = _quantised(y.unflatten(1, (-1, B)), fmt)
        hs = torch.arange(H, device="cuda")[:, None].expand_as(slot)[live]
        st[n][hs, slot[live]] = _codes(v, fmt)[live]
        st[n + "_scale"][hs, slot[live]] = s[live]
        i = torch.arange(B, device="cuda")[None]
        fresh = (i < ((held + st["n"]) % B)[:, None])[..., None]
        tail = y.gather(1, (last[:, None] + i).clamp(max=rows - 1)[..., None].expand(-1, -1, D))
        st[n + "_tail"].copy_(torch.where(fresh, tail.bfloat16(), st[n + "_tail"]))
    opened = live & ((lanes > 0) | (held == 0)[:, None])
    hs = torch.arange(H, device="cuda")[:, None].expand_as(slot)[opened]
    st["mass"][hs, slot[opened]] = 0.0
    st["lens_out"].copy_(st["lens"] + st["n"])
    i = torch.arange(st["n"], device="cuda")[None] + st["lens"][:, None]
    read = [_values(st, n).gather(1, i[..., None].expand(-1, -1, D)).bfloat16() for n in ("k", "v")]
    return read


def _attend(st):
    B, G, n_q = st["block"], st["group"], st["n_q"]
    K, V = _values(st, "k"), _values(st, "v")
    H, T = K.shape[:2]
    q = st["Q"].float().reshape(H, G * n_q, D)
    x = torch.matmul(q, K.transpose(1, 2)) * (1.0 / math.sqrt(D))
    j = torch.arange(T, device="cuda")
    end = st["lens"][:, None].expand(H, G * n_q)
    if st["causal"]:
        end = end - (n_q - 1) + torch.arange(n_q, device="cuda").repeat(G)[None]
    x = torch.where(j < end[..., None], x, torch.full_like(x[:1, :1, :1], -math.inf))
    top = x.amax(-1, keepdim=True)
    base = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp(x - base)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    O = torch.matmul(p, V).reshape(H * G, n_q, D).bfloat16()
    lse = (base + torch.log(total)).reshape(H * G, n_q)
    if st["add_mass"]:
        m = p.sum(1).unflatten(1, (-1, B)).sum(-1)
        st["mass"].scatter_add_(1, st["table"].long(), m)
    return O, lse


def _evict(st):
    S, H = st["slots"], st["heads"]
    t = st["table"].long()
    blocks = (st["lens"] + st["block"] - 1) // st["block"]
    over = (blocks - st["budget"]).clamp(min=0)
    b = torch.arange(S, device="cuda")[None]
    live = b < blocks[:, None]
    m = st["mass"].gather(1, t)
    m = torch.where((b < st["sinks"]) | (b >= blocks[:, None] - st["recent"]), torch.full_like(m, math.inf), m)
    m = torch.where(live, m, torch.full_like(m, -math.inf))
    order = torch.sort(m, dim=1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(1, order, b.expand_as(order))
    kept = live & (rank < st["budget"])
    to = torch.sort((~kept).to(torch.int8), dim=1, stable=True)[1]
    index = torch.where(b < kept.sum(1)[:, None], to, torch.full_like(to, -1))[:, :st["budget"]]
    return (t.gather(1, to).to(torch.int32), (st["lens"] - over * st["block"]).to(torch.int32),
            index.to(torch.int32))


def _plain(st):
    if st["op"] == "rope":
        return {"y": _rotated(st["x"].float(), st, st["inverse"]).bfloat16()}
    if st["op"] in ("norm_rope", "norm_rope_train"):
        q, k = _split(st)
        out = {"q": _norm_rope(q.float(), st["wq"], st["bq"], st), "k": _norm_rope(k.float(), st["wk"], st["bk"], st)}
        if st["op"] == "norm_rope_train":
            out["dq"], out["dwq"], out["dbq"] = _norm_rope_grad(st["gq"], q.float(), st["wq"], st)
            out["dk"], out["dwk"], out["dbk"] = _norm_rope_grad(st["gk"], k.float(), st["wk"], st)
        return out
    if st["op"] == "append":
        k, v = _append(st)
        return _cache_state(st, k, v)
    if st["op"] == "attend":
        O, lse = _attend(st)
        return {"O": O, "lse": lse, "mass": st["mass"]}
    table, lens, kept = _evict(st)
    return {"table": table, "lens": lens, "kept": kept}


def _cache_state(st, k, v):
    return {"K": k, "V": v, "lens": st["lens_out"], "k_scale": st["k_scale"], "v_scale": st["v_scale"],
            "k_tail": st["k_tail"], "v_tail": st["v_tail"], "mass": st["mass"]}


# -------------------------------------------------------------- own calls ----
def _own(st):
    import linear_hybrid_attention_b200 as zb
    if st["op"] == "rope":
        return {"y": zb.zb_rope(st["x"], st["pos"], st["turns"], axes=st["axes"], layout=st["layout"],
                                magnitude=st["magnitude"], inverse=st["inverse"])}
    if st["op"] in ("norm_rope", "norm_rope_train"):
        q, k = _split(st)
        how = dict(norm=st["norm"], wq=st["wq"], wk=st["wk"], bq=st["bq"], bk=st["bk"], eps=1e-6, axes=st["axes"],
                   layout=st["layout"], magnitude=st["magnitude"])
        out = {}
        out["q"], out["k"] = zb.zb_qk_norm_rope(q, k, st["pos"], st["turns"], **how)
        if st["op"] == "norm_rope_train":
            for n in ("bq", "bk"):
                del how[n]  # the gradient does not depend on them
            g = zb.zb_qk_norm_rope_backward(st["gq"], st["gk"], q, k, st["pos"], st["turns"], **how)
            out["dq"], out["dk"], out["dwq"], out["dwk"], out["dbq"], out["dbk"] = g
        return out
    if st["op"] == "append":
        zb.zb_kv8_append(st["cache"], st["K"], st["V"], st["lens"], lens_out=st["lens_out"])
        k, v = zb.zb_kv8_read(st["cache"], st["lens_out"], st["n"])
        return _cache_state(st, k, v)
    if st["op"] == "attend":
        O, lse = zb.zb_kv8_attn(st["Q"], st["cache"], st["lens"], causal=st["causal"], want_lse=True,
                                add_mass=st["add_mass"])
        return {"O": O, "lse": lse, "mass": st["mass"]}
    table, lens, kept = zb.zb_kv8_evict(st["table"], st["mass"], st["lens"], st["block"], st["budget"],
                                        sinks=st["sinks"], recent=st["recent"])
    return {"table": table, "lens": lens, "kept": kept}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work ----
def work(case):
    c = case
    if c["op"] == "rope":
        rows = c["batch"] * c["heads"] * c["n"]
        return {"bytes": rows * 4 * D, "flops": rows * 3 * c["rot"]}
    if c["op"] in ("norm_rope", "norm_rope_train"):
        rows = c["batch"] * (c["heads"] + c["kv_heads"]) * c["n"]
        train = c["op"] == "norm_rope_train"
        # forward: a row in, a row out; backward: the row and its gradient in, a gradient out (the row counts once)
        return {"bytes": rows * (8 if train else 4) * D, "flops": rows * D * (20 if train else 7)}
    if c["op"] == "append":
        rows = c["heads"] * c["n"]
        # K and V in, codes out, values out of them again in bf16
        return {"bytes": rows * 2 * D * (2 + 1 + 2), "flops": rows * 2 * D * 4}
    if c["op"] == "evict":
        n = c["heads"] * c["slots"]
        return {"bytes": n * (4 + 4 + 4) + c["heads"] * (8 + 4 * c["budget"]), "flops": n}
    heads, rows = c["seqs"] * c["kv_heads"], c["group"] * c["n_q"]
    longest = float(c["longest"])
    mean = (longest + 1) / 2 if c["ragged"] and c["seqs"] > 1 else longest
    blocks = heads * mean / c["block"]
    return {"bytes": heads * mean * 2 * D + blocks * (8 + 4 + (8 if c["add_mass"] else 0)) + heads * rows * (4 * D + 4),
            "flops": heads * rows * mean * 4 * D * (1 - 0.5 * c["n_q"] / longest if c["causal"] else 1)}


# ------------------------------------------------------------------ exact ----
def _exact_rotation(x, st, sign):
    """Rotation as a product with unit complex numbers, in 64 bits; x [B, H, N, 64]."""
    y = x.clone()
    width = st["rot"] // st["axes"]
    n = width // 2
    for a in range(st["axes"]):
        theta = sign * st["pos"][:, a].double()[:, None, :, None] * st["freq"]
        unit = torch.polar(torch.full_like(theta, st["magnitude"]), theta)
        first = torch.arange(n, device="cuda")
        one = a * width + (first if st["layout"] == "half" else 2 * first)
        two = one + (n if st["layout"] == "half" else 1)
        z = torch.complex(x[..., one], x[..., two]) * unit
        y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_norm(x, norm):
    mean = x.mean(-1, keepdim=True) if norm == "layer" else torch.zeros_like(x[..., :1])
    sigma = torch.sqrt(((x - mean) ** 2).sum(-1, keepdim=True) / D + 1e-6)
    return (x - mean) / sigma, sigma


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "rope":
        return {"y": _exact_rotation(st["x"].double(), st, -1.0 if st["inverse"] else 1.0)}
    if st["op"] in ("norm_rope", "norm_rope_train"):
        q, k = _split(st)
        out = {}
        for n, x in (("q", q), ("k", k)):
            xh, sigma = _exact_norm(x.double(), st["norm"])
            w, b = st["w" + n].double(), st["b" + n]
            out[n] = _exact_rotation(xh * w + (0 if b is None else b.double()), st, 1.0)
            if st["op"] == "norm_rope_train":
                dy = _exact_rotation(st["g" + n].double(), st, -1.0)
                out["dw" + n] = torch.einsum("bhnd,bhnd->d", dy, xh)
                out["db" + n] = torch.einsum("bhnd->d", dy) if st["norm"] == "layer" else None
                g = dy * w
                # the norm's Jacobian: (I - xh xh^T / d, less the mean's direction) / sigma
                g = g - xh * (g * xh).sum(-1, keepdim=True) / D - (g.mean(-1, keepdim=True) if b is not None else 0)
                out["d" + n] = g / sigma
        return out
    if st["op"] == "append":
        B, fmt, first, held = st["block"], st["fmt"], st["past"] // st["block"], st["past"] % st["block"]
        out, rows = {}, held + st["n"]
        for n, x in (("k", st["K"]), ("v", st["V"])):
            x = torch.cat([st[n + "_tail"][:, :held], x], 1).double()
            y = torch.nn.functional.pad(x, (0, 0, 0, -rows % B)).unflatten(1, (-1, B))
            s = (y.abs().amax((2, 3)) / TOP[fmt]).float().double()
            t = y / torch.where(s > 0, s, 1.0)[..., None, None]
            if fmt == "int8":
                c = torch.round(t)
            else:  # the nearest of the format's values, the even code where two are as near
                grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
                hi = torch.searchsorted(grid, t.abs().contiguous()).clamp(1, 126)
                lo = hi - 1
                d = (t.abs() - grid[lo]) - (grid[hi] - t.abs())
                c = torch.where((d > 0) | ((d == 0) & (hi % 2 == 0)), grid[hi], grid[lo]) * torch.sign(t)
            out[n.upper()] = (c * s[..., None, None]).flatten(1, 2)[:, held:rows]
            scale = st[n + "_scale"].double()
            at = st["table"].long()[:, first:first + s.shape[1]]
            out[n + "_scale"] = scale.scatter(1, at, s)
            tail = st[n + "_tail"].double()
            left = rows % B
            tail[:, :left] = x[:, rows - left:]
            out[n + "_tail"] = tail
        out["mass"] = st["mass"].double().scatter(1, at[:, 1 if held else 0:], 0.0)
        return {**out, "lens": None}
    if st["op"] == "evict":
        return None  # whole numbers alone
    H, G, n_q, B = st["seqs"] * st["kv_heads"], st["group"], st["n_q"], st["block"]
    Q = st["Q"].double().reshape(H, G * n_q, D)
    O, lse = torch.zeros_like(Q), torch.full((H, G * n_q), -math.inf, dtype=torch.float64, device="cuda")
    mass = st["mass"].double()
    for h, L in enumerate(st["lens"].tolist()):
        blocks = st["table"][h, :-(-L // B)].long()
        K, V = ((st[n][h, blocks].double() * st[n + "_scale"][h, blocks].double()[:, None, None]).flatten(0, 1)[:L]
                for n in ("k", "v"))
        seen = torch.ones(n_q, L, dtype=torch.bool, device="cuda")
        if st["causal"]:
            seen = torch.tril(seen, diagonal=L - n_q)
        for g in range(G):
            rows = slice(g * n_q, (g + 1) * n_q)
            x = (Q[h, rows] @ K.T / 8.0).masked_fill(~seen, -math.inf)
            lse[h, rows] = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(torch.isfinite(lse[h, rows]), lse[h, rows], 0.0)[:, None])
            O[h, rows] = p @ V
            if st["add_mass"]:
                w = torch.nn.functional.pad(p.sum(0), (0, -L % B)).reshape(-1, B).sum(1)
                mass[h, blocks] += w
    return {"O": O.reshape(H * G, n_q, D), "lse": lse.reshape(H * G, n_q), "mass": mass}
