"""Serving from the paged 4-bit key/value cache: torch-facing handles and calls over
the C ABI.  A KVCache holds the six arrays, a KVSequences says which of its
tokens belong to the sequences of a batch; both keep the pointers that the calls pass,
so that a decode step pays for its launches and little else.  The values of kv_lens, cu_q and
block_table may change between calls (and under a captured graph); their tensors
may not be replaced."""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _lib as L
from .layer import _need_cuda


def _stream_of(index: int) -> int:
    """The current stream of device `index` as an address."""
    return torch.cuda.current_stream(index).cuda_stream


# (without the Stream object, which costs a tenth of a small call)
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def _need(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str, device=None) -> None:
    _need_cuda(t, dtype, name)
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {shape}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


class KVCache:
    """A 4-bit key/value cache: (codes uint8 [slots, W/2], scales float32 [slots, W/group],
    zeros int32 [slots, W/group]) for keys and for values, as kv_quantize returns
    them, W = heads * head_dim.  Slots are pages of page_size (by default one page)."""

    def __init__(self, keys, values, head_dim: int, group: int = 128,
                 page_size: Optional[int] = None):
        codes = keys[0]
        _need_cuda(codes, torch.uint8, "codes")
        if codes.dim() != 2:
            raise ValueError("codes must be [slots, heads*head_dim/2]")
        slots, width = codes.shape[0], 2 * codes.shape[1]
        if head_dim <= 0 or group <= 0 or width % head_dim or width % group:
            raise ValueError("the row width must be a multiple of head_dim and of group")
        for name, (c, s, z) in (("key", keys), ("value", values)):
            _need(c, torch.uint8, (slots, width // 2), f"{name} codes", codes.device)
            _need(s, torch.float32, (slots, width // group), f"{name} scales", codes.device)
            _need(z, torch.int32, (slots, width // group), f"{name} zeros", codes.device)
        self.keys, self.values = tuple(keys), tuple(values)
        self.slots, self.width, self.head_dim, self.group = slots, width, head_dim, group
        self.heads, self.groups = width // head_dim, width // group
        self.page_size = max(1, slots) if page_size is None else page_size
        if self.page_size < 1:
            raise ValueError("page_size must be at least 1")
        self.pages = slots // self.page_size
        self.device = codes.device
        self._c = L.QrKvCache(*(t.data_ptr() for t in self.keys + self.values), slots, self.heads,
                              head_dim, group, self.page_size)

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, head_dim: int, group: int = 128,
              device="cuda") -> "KVCache":
        """A cache of zeros."""
        rows, width = pages * page_size, heads * head_dim

        def side():
            return (torch.zeros((rows, width // 2), dtype=torch.uint8, device=device),
                    torch.zeros((rows, width // group), dtype=torch.float32, device=device),
                    torch.zeros((rows, width // group), dtype=torch.int32, device=device))
        return cls(side(), side(), head_dim, group, page_size)


class KVSequences:
    """The sequences of a batch on a cache.  kv_lens int32 [batch]: tokens each
    holds, those of the coming call included.  cu_q int32 [batch + 1]: the rows of the
    call that are its newest tokens.  block_table int32 [batch, pages]: its pages; without
    one sequence b has pages [b n, (b + 1) n), n = cache.pages // batch."""

    def __init__(self, cache: KVCache, kv_lens: torch.Tensor, cu_q: Optional[torch.Tensor] = None,
                 block_table: Optional[torch.Tensor] = None):
        _need_cuda(kv_lens, torch.int32, "kv_lens")
        if kv_lens.dim() != 1:
            raise ValueError("kv_lens must be [batch]")
        batch = kv_lens.shape[0]
        _need(kv_lens, torch.int32, (batch,), "kv_lens", cache.device)
        if cu_q is not None:
            _need(cu_q, torch.int32, (batch + 1,), "cu_q", cache.device)
        if block_table is not None:
            if block_table.dim() != 2:
                raise ValueError("block_table must be [batch, pages]")
            _need(block_table, torch.int32, (batch, block_table.shape[1]), "block_table", cache.device)
            self.max_pages = block_table.shape[1]
        else:
            self.max_pages = cache.pages // max(1, batch)
        self.cache, self.kv_lens, self.cu_q, self.block_table = cache, kv_lens, cu_q, block_table
        self.batch, self.capacity = batch, self.max_pages * cache.page_size
        self.device = cache.device
        self._index = cache.device.index if cache.device.index is not None else torch.cuda.current_device()
        self._c = L.QrKvSeqs(batch, self.max_pages,
                             None if block_table is None else block_table.data_ptr(),
                             kv_lens.data_ptr(), None if cu_q is None else cu_q.data_ptr())
        self._args = (ctypes.byref(cache._c), ctypes.byref(self._c))
        self._workspace = None                  # (tokens, q_heads) of the last kv_attention, and its workspace's bytes

    def _call(self, fn, *args):
        """fn(cache, seqs, *args, stream) on the cache's device and its current stream."""
        i = self._index
        if torch.cuda.current_device() != i:
            with torch.cuda.device(i):
                return fn(*self._args, *args, _stream_of(i))
        return fn(*self._args, *args, _stream_of(i))

    def _workspace_bytes(self, tokens: int, q_heads: int) -> int:
        """Bytes of kv_attention's workspace: the cut of its work, and so they, depend on the cache's device."""
        last = self._workspace
        if last is not None and last[0] == (tokens, q_heads):
            return last[1]
        need = self._call(lambda c, s, *a: L.qr_kv_attention_workspace(c, s, *a[:-1]), tokens, q_heads)
        if need < 0:
            raise ValueError("sizes outside what the kernels handle")
        self._workspace = (tokens, q_heads), need
        return need

    def _rows(self, t: torch.Tensor, name: str, unit: int) -> None:
        """t: fp16 rows on the cache's device, a multiple of unit wide, at any stride between rows."""
        if t.dtype != torch.float16 or t.device != self.device:
            raise ValueError(f"{name} must be a torch.float16 tensor on {self.device}, "
                             f"got {t.dtype} on {t.device}")
        if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] != 1):
            raise ValueError(f"{name} must be a 2-D row-major tensor")
        if t.shape[1] % unit or t.shape[1] == 0:
            raise ValueError(f"the width of {name} must be a multiple of {unit}")

    def _need_cu(self) -> None:
        if self.cu_q is None:
            raise ValueError("the sequences have no cu_q")


def _ld(t: torch.Tensor) -> int:
    rows, width = t.shape
    return t.stride(0) if rows > 1 else max(t.stride(0), width)


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors of rows share an element (or may: rows of unlike pitch that lie between each other)."""
    def span(t):
        first = t.data_ptr()
        return first, first + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))
    if a.numel() == 0 or b.numel() == 0:
        return False
    (a0, a1), (b0, b1) = span(a), span(b)
    if not (a0 < b1 and b0 < a1):
        return False
    pitch = a.stride(0)
    if a.dtype != b.dtype or pitch != b.stride(0) or (b0 - a0) % a.element_size():
        return True
    # columns of the same rows: b's begin `at` elements behind a's, or behind those of some other row
    at = (b0 - a0) // a.element_size() % pitch if pitch > 0 else 0
    return at < a.shape[1] or at + b.shape[1] > pitch


class Rope:
    """Rotary embedding over one or several position axes: pair i of every head turns by
    position[axis[i]] * inv_freq[i].  inv_freq float32 [pairs]; axis int32 [pairs] (None: one
    axis); pairs are elements (i, i + pairs), or (2 i, 2 i + 1) when interleaved."""

    def __init__(self, inv_freq: torch.Tensor, axis: Optional[torch.Tensor] = None,
                 interleaved: bool = False):
        _need_cuda(inv_freq, torch.float32, "inv_freq")
        if inv_freq.dim() != 1 or inv_freq.shape[0] == 0:
            raise ValueError("inv_freq must be [pairs]")
        _need(inv_freq, torch.float32, (inv_freq.shape[0],), "inv_freq")
        if axis is not None:
            _need(axis, torch.int32, (inv_freq.shape[0],), "axis", inv_freq.device)
        self.inv_freq, self.axis, self.interleaved = inv_freq, axis, interleaved

    def _c(self, positions: torch.Tensor, tokens: int) -> L.QrKvRope:
        if positions is None:
            raise ValueError("a rope needs positions")
        if positions.dim() == 1:
            positions = positions.unsqueeze(0)
        if (positions.dtype != torch.int32 or positions.device != self.inv_freq.device
                or positions.dim() != 2 or positions.shape[1] != tokens
                or (tokens > 1 and positions.stride(1) != 1)):
            raise ValueError(f"positions must be int32 [axes, {tokens}] rows on {self.inv_freq.device}")
        axes = positions.shape[0]
        if axes == 0:
            raise ValueError("positions must have at least one axis")
        if axes > 1 and positions.stride(0) < tokens:      # one row expanded over the axes, or rows that overlap
            positions = positions.contiguous()
        ld = max(positions.stride(0), tokens) if axes == 1 else positions.stride(0)
        c = L.QrKvRope(self.inv_freq.data_ptr(), None if self.axis is None else self.axis.data_ptr(),
                       positions.data_ptr(), ld, self.inv_freq.shape[0], axes, 1 if self.interleaved else 0)
        c.rows = positions                                 # lives until the launch
        return c


def kv_append(seqs: KVSequences, q: Optional[torch.Tensor], k: Optional[torch.Tensor],
              v: Optional[torch.Tensor], rope: Optional[Rope] = None,
              positions: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Rope and R3 on q and k, and 4-bit codes of k and v into the cache at the newest
    places of the sequences.  q, k, v fp16 [tokens, heads*head_dim] (rows at any stride that is
    a multiple of 8; any may be None); positions int32 [axes, tokens], or [tokens], with a
    rope (one row expanded over the axes is copied).  Returns q with rope and R3 (None without q), the queries of kv_attention.  Rows
    outside cu_q's range are left unwritten."""
    given = [t for t in (q, k, v) if t is not None]
    if not given:
        raise ValueError("nothing to do")
    seqs._need_cu()
    cache = seqs.cache
    tokens = given[0].shape[0]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is None:
            continue
        seqs._rows(t, name, cache.head_dim)
        if t.shape[0] != tokens or (name != "q" and t.shape[1] != cache.width):
            raise ValueError("q, k, v must have the same rows, k and v the cache's width")
    if rope is None and positions is not None:
        raise ValueError("positions without a rope")
    if rope is not None and rope.inv_freq.device != seqs.device:
        raise ValueError(f"the rope must be on {seqs.device}")
    if q is not None:
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            _need(out, torch.float16, tuple(q.shape), "out", seqs.device)
            if any(_overlap(out, t) for t in given):
                raise ValueError("out must not overlap the inputs")
    elif out is not None:
        raise ValueError("out without q")
    c = None if rope is None else rope._c(positions, tokens)
    seqs._call(L.qr_kv_append, None if c is None else ctypes.byref(c),
               None if q is None else q.data_ptr(), 0 if q is None else _ld(q),
               None if k is None else k.data_ptr(), 0 if k is None else _ld(k),
               None if v is None else v.data_ptr(), 0 if v is None else _ld(v), tokens,
               0 if q is None else q.shape[1] // cache.head_dim,
               None if out is None else out.data_ptr())
    return out


def kv_dequantize(seqs: KVSequences, tokens: int) -> tuple[torch.Tensor, torch.Tensor]:
    """The values that the codes of the sequences' newest tokens stand for, fp16 [tokens,
    heads*head_dim] each: keys (in R3's basis, as the cache holds them) and values.  Rows outside
    cu_q's range are left unwritten."""
    seqs._need_cu()
    cache = seqs.cache
    k = seqs.kv_lens.new_empty((tokens, cache.width), dtype=torch.float16)
    v = torch.empty_like(k)
    seqs._call(L.qr_kv_dequantize, tokens, k.data_ptr(), v.data_ptr())
    return k, v


def kv_attention(seqs: KVSequences, q: torch.Tensor, causal: bool = True,
                 scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                 return_lse: bool = False):
    """softmax(scale q K^T) V over the cache for the rows of q (fp16 [tokens, q_heads*head_dim],
    with R3 applied, as kv_append and kv_quantize return it); q_heads a multiple of the
    cache's heads.  causal: the rows of a sequence are its newest tokens and see no
    later ones; otherwise every row sees all kv_lens tokens (cross attention).  scale
    defaults to 1/sqrt(head_dim).  Returns out fp16 like q, and with return_lse the
    log of the softmax's sum, float32 [tokens, q_heads] (-inf, and 0 out, for a row that sees
    no key).  Rows outside cu_q's range are left unwritten.  Prompts and single tokens of one step
    are better called apart: the kernel is chosen for the call as a whole."""
    seqs._need_cu()
    cache = seqs.cache
    seqs._rows(q, "q", cache.width)
    tokens, q_heads = q.shape[0], q.shape[1] // cache.head_dim
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        seqs._rows(out, "out", cache.width)
        if out.shape != q.shape:
            raise ValueError(f"out must have q's shape {tuple(q.shape)}")
        if _overlap(out, q):
            raise ValueError("out must not overlap q")
    lse = q.new_empty((tokens, q_heads), dtype=torch.float32) if return_lse else None
    need = seqs._workspace_bytes(tokens, q_heads)
    ws = q.new_empty(need, dtype=torch.uint8) if need else None
    seqs._call(L.qr_kv_attention, q.data_ptr(), _ld(q), tokens, q_heads,
               1.0 / math.sqrt(cache.head_dim) if scale is None else scale, 1 if causal else 0,
               out.data_ptr(), _ld(out), None if lse is None else lse.data_ptr(),
               None if ws is None else ws.data_ptr(), need)
    return (out, lse) if return_lse else out


def kv_attention_mass(seqs: KVSequences, q: torch.Tensor, lse: torch.Tensor, mass: torch.Tensor,
                      causal: bool = True, scale: Optional[float] = None) -> torch.Tensor:
    """Adds to mass (float32 [batch, groups, >= capacity], in place) the attention weight that
    each cached token receives from the rows of q, summed over the rows and the heads of each
    quantization group; lse as kv_attention returned it for the same rows.  Prompts and single tokens
    of one step are better called apart.  Returns mass."""
    seqs._need_cu()
    cache = seqs.cache
    seqs._rows(q, "q", cache.width)
    tokens, q_heads = q.shape[0], q.shape[1] // cache.head_dim
    _need(lse, torch.float32, (tokens, q_heads), "lse", seqs.device)
    _need_mass(seqs, mass, "mass")
    seqs._call(L.qr_kv_attention_mass, q.data_ptr(), _ld(q), tokens, q_heads,
               1.0 / math.sqrt(cache.head_dim) if scale is None else scale, 1 if causal else 0,
               lse.data_ptr(), mass.data_ptr(), mass.shape[2])
    return mass


def _need_mass(seqs: KVSequences, mass: torch.Tensor, name: str) -> None:
    if mass.dim() != 3 or mass.shape[2] < seqs.capacity:
        raise ValueError(f"{name} must be [batch, groups, at least {seqs.capacity}]")
    _need(mass, torch.float32, (seqs.batch, seqs.cache.groups, mass.shape[2]), name, seqs.device)


def kv_evict(seqs: KVSequences, mass: torch.Tensor, keep: int, recent: int,
             table_out: Optional[torch.Tensor] = None):
    """Eviction by accumulated mass: of a sequence that holds more than keep tokens the newest
    `recent` stay and the keep - recent others with the largest mass (per quantization group;
    equal masses: the lower place), moved in order to the first keep places.  In place,
    mass along with them, or, with table_out (int32 like block_table, other pages than
    those being read), into those pages and a mass of their own.  Returns (kept int32 [batch, groups,
    keep]: the place each kept token had, -1 behind the last; lens int32 [batch]:
    what each sequence holds now; mass).  kv_lens is left as it is.  Tokens without a page in the cache
    hold nothing that could move: give them a mass of -inf, and keep no more than are there (the
    place that one moves to keeps what it held)."""
    cache = seqs.cache
    _need_mass(seqs, mass, "mass")
    if not 1 <= keep or not 0 <= recent <= keep:
        raise ValueError("keep must be at least 1 and recent in [0, keep]")
    if table_out is not None:
        _need(table_out, torch.int32, (seqs.batch, seqs.max_pages), "table_out", seqs.device)
    kept = seqs.kv_lens.new_empty((seqs.batch, cache.groups, keep))
    lens = torch.empty_like(seqs.kv_lens)
    mass_out = mass if table_out is None else torch.empty_like(mass)
    seqs._call(L.qr_kv_evict, mass.data_ptr(), mass.shape[2], keep, recent,
               None if table_out is None else table_out.data_ptr(), mass_out.data_ptr(),
               kept.data_ptr(), lens.data_ptr())
    return kept, lens, mass_out
