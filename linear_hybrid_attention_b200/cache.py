"""The 8-bit key/value cache (bindings of ``csrc/kv8_cache.cu`` and ``csrc/kv8_attn.cu``).

``KV8Cache`` holds a cache's tensors, the ``zb_kv8_*`` functions carry the C
names, and ``CachedAttention`` chains them for one layer that serves tokens (or
views) one group after another: norm and rotation of the new queries and keys,
append, attention over everything cached, eviction down to a budget.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import HEAD_DIM, _call, _lib, _lib_handle, _need, _out, _ptr, _ws
from .positions import RopeFrequencies, zb_qk_norm_rope

__all__ = ["KV8Cache", "zb_kv8_append", "zb_kv8_read", "zb_kv8_attn", "zb_kv8_attn_workspace_bytes", "zb_kv8_evict",
           "CachedAttention"]

# what a step's attention may take of workspace before it attends band by band (bytes)
WORKSPACE_BOUND = 1 << 30
FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


class KV8Cache:
    """The tensors of an 8-bit key/value cache (see zb.h, zb_kv8); the lengths live outside.

    k, v: int8 or float8_e4m3fn [heads, slots, block, 64]; k_scale, v_scale: fp32 [heads, slots];
    k_tail, v_tail: bf16 [heads, block, 64]; table: int32 [heads, slots]; mass: fp32 [heads, slots] or
    None.  The object keeps the tensors alive and their addresses, so they must not be reassigned.
    """

    def __init__(self, k, v, k_scale, v_scale, k_tail, v_tail, table, mass=None):
        if not isinstance(k, torch.Tensor) or k.dtype not in (torch.int8, torch.float8_e4m3fn):
            raise TypeError("k must be an int8 or float8_e4m3fn torch.Tensor")
        _need(k, k.dtype, "k", 4)
        heads, slots, block, d = k.shape
        for t, dt, shape, name in ((v, k.dtype, (heads, slots, block, d), "v"),
                                   (k_scale, torch.float32, (heads, slots), "k_scale"),
                                   (v_scale, torch.float32, (heads, slots), "v_scale"),
                                   (k_tail, torch.bfloat16, (heads, block, d), "k_tail"),
                                   (v_tail, torch.bfloat16, (heads, block, d), "v_tail"),
                                   (table, torch.int32, (heads, slots), "table"),
                                   (mass, torch.float32, (heads, slots), "mass")):
            if t is None and name == "mass":
                continue
            _need(t, dt, name, len(shape))
            if tuple(t.shape) != shape or t.device != k.device:
                raise ValueError(f"{name} must be {shape} on {k.device}, got {tuple(t.shape)} on {t.device}")
        if d != HEAD_DIM or block not in (16, 32, 64, 128):
            raise ValueError(f"a cache has blocks of 16, 32, 64 or 128 tokens of {HEAD_DIM}, got {block} of {d}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.k_tail, self.v_tail, self.table, self.mass = k_tail, v_tail, table, mass
        self.heads, self.slots, self.block, self.device = heads, slots, block, k.device
        self.struct = _lib.ZbKv8(heads, slots, d, block, 0 if k.dtype == torch.int8 else 1, k.data_ptr(), v.data_ptr(),
                                 k_scale.data_ptr(), v_scale.data_ptr(), k_tail.data_ptr(), v_tail.data_ptr(),
                                 table.data_ptr(), _ptr(mass))
        self._ws_bytes = {}

    @classmethod
    def empty(cls, heads: int, capacity: int, block: int = 64, format: str = "int8", mass: bool = True,
              device="cuda") -> "KV8Cache":
        """A cache for `capacity` tokens a head (rounded up to whole blocks), its slots in order."""
        if format not in FORMATS:
            raise ValueError(f"format must be one of {sorted(FORMATS)}, got {format!r}")
        if heads < 1 or capacity < 1:
            raise ValueError(f"heads and capacity must be at least 1, got {heads} and {capacity}")
        if block not in (16, 32, 64, 128):
            raise ValueError(f"block must be 16, 32, 64 or 128, got {block}")
        slots = -(-capacity // block)
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
        codes = [z((heads, slots, block, HEAD_DIM), torch.uint8).view(FORMATS[format]) for _ in range(2)]
        table = torch.arange(slots, dtype=torch.int32, device=device).repeat(heads, 1)
        return cls(*codes, z((heads, slots), torch.float32), z((heads, slots), torch.float32),
                   z((heads, block, HEAD_DIM), torch.bfloat16), z((heads, block, HEAD_DIM), torch.bfloat16), table,
                   z((heads, slots), torch.float32) if mass else None)

    @property
    def capacity(self) -> int:
        """Tokens a head can hold."""
        return self.slots * self.block


def _lens(lens, cache: KV8Cache, name: str = "lens") -> int:
    if not isinstance(lens, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if lens.dtype != torch.int32 or lens.shape != (cache.heads,) or lens.device != cache.device or \
            not lens.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 [{cache.heads}] tensor on {cache.device}, "
                         f"got {lens.dtype} {tuple(lens.shape)} on {lens.device}")
    return lens.data_ptr()


def _rows(x, name: str, device) -> None:
    _need(x, torch.bfloat16, name, 3)
    if x.shape[2] != HEAD_DIM or x.device != device:
        raise ValueError(f"{name} must be [heads, tokens, {HEAD_DIM}] on {device}, got {tuple(x.shape)} on {x.device}")


def zb_kv8_append(cache: KV8Cache, K, V, lens, lens_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Append K, V (bf16 [heads, n, 64]) after each head's first ``lens`` tokens; returns the new lengths.

    lens: int32 [heads] on the device.  lens_out: where the new lengths go (``lens`` itself advances it in
    place; a fresh tensor if not given).  A head without room keeps its contents and length, and the device
    status says ZB_ERR_INDEX."""
    _rows(K, "K", cache.device)
    _rows(V, "V", cache.device)
    if K.shape != V.shape or K.shape[0] != cache.heads:
        raise ValueError(f"K and V must both be [{cache.heads}, n, {HEAD_DIM}], got {tuple(K.shape)}, {tuple(V.shape)}")
    lp = _lens(lens, cache)
    if lens_out is None:
        lens_out = torch.empty_like(lens)
    _call(cache.device, "zb_kv8_append", cache.struct, K.data_ptr(), V.data_ptr(), K.shape[1], lp,
          _lens(lens_out, cache, "lens_out"))
    return lens_out


def zb_kv8_read(cache: KV8Cache, lens, n: int, out_k: Optional[torch.Tensor] = None,
                out_v: Optional[torch.Tensor] = None):
    """(K, V) bf16 [heads, n, 64]: the newest n tokens of every head as the cache holds them."""
    n = int(n)
    lp = _lens(lens, cache)
    if n < 1:
        raise ValueError(f"n must be at least 1, got {n}")
    K = _out((cache.heads, n, HEAD_DIM), torch.bfloat16, cache.device, out_k, "out_k")
    V = _out((cache.heads, n, HEAD_DIM), torch.bfloat16, cache.device, out_v, "out_v")
    if K.device != cache.device or V.device != cache.device:
        raise ValueError(f"out_k and out_v must be on {cache.device}")
    _call(cache.device, "zb_kv8_read", cache.struct, lp, n, K.data_ptr(), V.data_ptr())
    return K, V


def zb_kv8_attn_workspace_bytes(cache: KV8Cache, heads_q: int, n_q: int, add_mass: bool = False) -> int:
    return int(_lib_handle().zb_kv8_attn_workspace_bytes(cache.struct, heads_q, n_q, 1 if add_mass else 0))


def _ws_bytes(cache: KV8Cache, heads_q: int, n_q: int, add_mass: bool) -> int:
    key = (heads_q, n_q, add_mass)
    need = cache._ws_bytes.get(key)
    if need is None:
        need = cache._ws_bytes[key] = zb_kv8_attn_workspace_bytes(cache, heads_q, n_q, add_mass)
    return need


def zb_kv8_attn(Q, cache: KV8Cache, lens, causal: bool = False, scale: Optional[float] = None,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, want_lse: bool = False,
                add_mass: bool = False, ws: Optional[torch.Tensor] = None):
    """Softmax attention of Q (bf16 [heads_q, n_q, 64]) over the cache; returns O (and lse if asked).

    heads_q is a multiple of the cache's heads (shared keys and values).  causal: the queries are the newest
    n_q of the lens tokens.  add_mass: add each block's softmax weight to cache.mass."""
    _rows(Q, "Q", cache.device)
    heads_q, n_q, d = Q.shape
    lp = _lens(lens, cache)
    if add_mass and cache.mass is None:
        raise ValueError("add_mass needs a cache with mass")
    O = torch.empty_like(Q) if out is None else _out((heads_q, n_q, d), torch.bfloat16, Q.device, out, "O")
    if want_lse or lse is not None:
        lse = torch.empty_strided((heads_q, n_q), (n_q, 1), dtype=torch.float32, device=cache.device) if lse is None \
            else _out((heads_q, n_q), torch.float32, Q.device, lse, "lse")
    ws = _ws(_ws_bytes(cache, heads_q, n_q, add_mass), cache.device, ws)
    for t, name in ((O, "O"), (lse, "lse"), (ws, "ws")):
        if t is not None and t.device != cache.device:
            raise ValueError(f"{name} must be on {cache.device}, is on {t.device}")
    _call(cache.device, "zb_kv8_attn", Q.data_ptr(), heads_q, n_q, cache.struct, lp, 1 if causal else 0,
          1.0 / math.sqrt(d) if scale is None else float(scale), O.data_ptr(), _ptr(lse), 1 if add_mass else 0,
          ws.data_ptr(), ws.numel() * ws.element_size())
    return (O, lse) if lse is not None else O


def zb_kv8_evict(table, mass, lens, block: int, budget: int, sinks: int = 0, recent: int = 1,
                 table_out: Optional[torch.Tensor] = None, lens_out: Optional[torch.Tensor] = None,
                 kept: Optional[torch.Tensor] = None):
    """Keep at most `budget` blocks of every head by their weight (see zb.h): (table, lens, kept).

    table int32, mass fp32 [heads, slots], lens int32 [heads].  kept: int32 [heads, budget], the kept
    logical blocks of the old order, then -1.  table_out must be another tensor than table."""
    _need(table, torch.int32, "table", 2)
    _need(mass, torch.float32, "mass", 2)
    _need(lens, torch.int32, "lens", 1)
    heads, slots = table.shape
    dev = table.device
    if mass.shape != table.shape or lens.shape[0] != heads or mass.device != dev or lens.device != dev:
        raise ValueError(f"mass must be {(heads, slots)} and lens ({heads},) on {dev}, got {tuple(mass.shape)} on "
                         f"{mass.device} and {tuple(lens.shape)} on {lens.device}")
    budget = int(budget)
    if budget < 1:
        raise ValueError(f"budget must be at least 1, got {budget}")
    table_out = torch.empty_like(table) if table_out is None else \
        _out((heads, slots), torch.int32, dev, table_out, "table_out")
    lens_out = torch.empty_like(lens) if lens_out is None else _out((heads,), torch.int32, dev, lens_out, "lens_out")
    kept = torch.empty_strided((heads, budget), (budget, 1), dtype=torch.int32, device=dev) if kept is None else \
        _out((heads, budget), torch.int32, dev, kept, "kept")
    for t, name in ((table_out, "table_out"), (lens_out, "lens_out"), (kept, "kept")):
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}, is on {t.device}")
    _call(dev, "zb_kv8_evict", table.data_ptr(), mass.data_ptr(), lens.data_ptr(), heads, slots, block, budget, sinks,
          recent, table_out.data_ptr(), lens_out.data_ptr(), kept.data_ptr())
    return table_out, lens_out, kept


class CachedAttention:
    """One attention layer that serves tokens group after group from an 8-bit cache.

    ``step(Q, K, V, pos)`` takes the new tokens' queries, keys and values ([B, heads, n, 64], any strides
    for Q and K), normalises and rotates Q and K, appends K and V, and returns the queries' attention over
    everything cached (``causal`` by default).  With ``budget`` (blocks a head) each step that attends adds
    its softmax weight to the blocks', and ``evict()`` keeps the heaviest; its workspace (one fp32 a query
    row and 64 tokens of capacity) is held to 1 GiB by attending in bands of queries.  The lengths live on the device
    (``lens``, int32 [B * kv_heads]) and no call waits for the GPU, so a step can be captured in a graph and
    replayed.  Not for use from two streams at once: a step changes the cache.
    """

    def __init__(self, batch: int, heads: int, kv_heads: int, capacity: int, block: int = 64, format: str = "int8",
                 freqs: Optional[RopeFrequencies] = None, axes: int = 1, layout: str = "half", norm: str = "none",
                 wq=None, wk=None, bq=None, bk=None, eps: float = 1e-6, budget: Optional[int] = None, sinks: int = 1,
                 recent: int = 2, scale: Optional[float] = None, device="cuda"):
        if kv_heads < 1 or heads % kv_heads:
            raise ValueError(f"heads must be a multiple of kv_heads, got {heads} and {kv_heads}")
        if scale is not None and not 0.0 < scale <= 3.4e38:
            raise ValueError(f"scale must be a positive number, got {scale}")
        self.batch, self.heads, self.kv_heads = batch, heads, kv_heads
        self.cache = KV8Cache.empty(batch * kv_heads, capacity, block, format, mass=budget is not None, device=device)
        dev = self.cache.device
        self.lens = torch.zeros(batch * kv_heads, dtype=torch.int32, device=dev)
        self.turns = None if freqs is None else freqs.turns.to(dev)
        self.how = dict(norm=norm, wq=wq, wk=wk, bq=bq, bk=bk, eps=eps, axes=axes, layout=layout,
                        magnitude=1.0 if freqs is None else freqs.magnitude)
        self.budget, self.sinks, self.recent, self.scale = budget, sinks, recent, scale
        if budget is not None:
            if not 1 <= recent <= sinks + recent <= budget <= self.cache.slots:
                raise ValueError(f"a budget holds the sinks and at least one recent block and fits the cache: got "
                                 f"budget {budget}, sinks {sinks}, recent {recent}, {self.cache.slots} slots")
            self._table = torch.empty_like(self.cache.table)
            self._kept = torch.empty((batch * kv_heads, budget), dtype=torch.int32, device=dev)

    def step(self, Q, K, V, pos=None, causal: bool = True) -> torch.Tensor:
        """O [B, heads, n, 64] of the new tokens; they are in the cache afterwards.

        A head without room for them (lens + n above the cache's capacity) stays as it is and its queries get
        zeros and add no weight; ``lens`` does not grow there, and the device status says ZB_ERR_INDEX."""
        B, H, G = self.batch, self.heads, self.kv_heads
        n = Q.shape[2] if isinstance(Q, torch.Tensor) and Q.dim() == 4 else -1
        for t, shape, name in ((Q, (B, H, n, HEAD_DIM), "Q"), (K, (B, G, n, HEAD_DIM), "K"), (V, (B, G, n, HEAD_DIM), "V")):
            if not isinstance(t, torch.Tensor) or tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {shape}, got {tuple(getattr(t, 'shape', ()))}")
            # (all of it before the append: a call that is refused changes nothing)
            if t.dtype != torch.bfloat16:
                raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
            if t.device != self.cache.device:
                raise ValueError(f"{name} must be on {self.cache.device}, is on {t.device}")
        if self.turns is not None or self.how["norm"] != "none":
            Q, K = zb_qk_norm_rope(Q, K, pos, self.turns, **self.how)
        K, V, Q = (t.reshape(-1, n, HEAD_DIM).contiguous() for t in (K, V, Q))
        room = self.lens <= self.cache.capacity - n
        zb_kv8_append(self.cache, K, V, self.lens, lens_out=self.lens)
        how = dict(causal=causal, scale=self.scale, add_mass=self.budget is not None)
        lens, band = self.lens * room, self._band(n)
        if band >= n:
            O = zb_kv8_attn(Q, self.cache, lens, **how)
        else:
            O = torch.empty_like(Q)
            for end in range(band, n + band, band):
                first, end = end - band, min(end, n)
                # a causal band's queries are the newest of the tokens before its end
                seen = lens - (n - end) if causal else lens
                O[:, first:end] = zb_kv8_attn(Q[:, first:end].contiguous(), self.cache, seen, **how)
        return O.view(B, H, n, HEAD_DIM)

    def _band(self, n: int) -> int:
        """How many of n queries attend at once: with a budget the workspace grows with queries times capacity."""
        if self.budget is None:
            return n
        while n > 1 and _ws_bytes(self.cache, self.batch * self.heads, n, True) > WORKSPACE_BOUND:
            n = -(-n // 2)
        return n

    def evict(self) -> torch.Tensor:
        """Keep at most ``budget`` blocks a head; returns the kept logical blocks (int32 [heads, budget], then -1).

        The tensor is the layer's own, and the next call writes it again."""
        if self.budget is None:
            raise ValueError("evict() needs a layer made with a budget")
        c = self.cache
        zb_kv8_evict(c.table, c.mass, self.lens, c.block, self.budget, self.sinks, self.recent, table_out=self._table,
                     lens_out=self.lens, kept=self._kept)
        c.table.copy_(self._table)
        return self._kept
