"""Plain float64 numpy restatement of the calls on the paged 4-bit KV cache, for the
tests: page tables are followed token by token and softmax is written out."""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Optional

import numpy as np


@dataclass
class Cache:
    """Host copy of a cache: codes uint8 [slots, W/2], scales, zeros [slots, W/group] per side."""
    keys: tuple
    values: tuple
    heads: int
    head_dim: int
    group: int
    page_size: int

    @property
    def groups(self):
        return self.heads * self.head_dim // self.group

    @property
    def pages(self):
        return self.keys[0].shape[0] // self.page_size


def random_cache(rng, pages, page_size, heads, head_dim, group) -> Cache:
    slots, w = pages * page_size, heads * head_dim

    def side():
        return (rng.integers(0, 256, (slots, w // 2)).astype(np.uint8),
                rng.uniform(0.02, 0.3, (slots, w // group)).astype(np.float32),
                rng.integers(-12, 4, (slots, w // group)).astype(np.int32))
    return Cache(side(), side(), heads, head_dim, group, page_size)


def values(c: Cache, side: int, slots) -> np.ndarray:
    """scale * (code - zero) of some slots: float64 [n, heads, head_dim]."""
    codes, scales, zeros = (a[slots] for a in (c.values if side else c.keys))
    n = np.empty((codes.shape[0], 2 * codes.shape[1]), np.int64)
    n[:, 0::2], n[:, 1::2] = codes & 15, codes >> 4
    n = np.where(n > 7, n - 16, n).reshape(codes.shape[0], c.groups, c.group)
    v = scales.astype(np.float64)[..., None] * (n - zeros.astype(np.int64)[..., None])
    return v.reshape(codes.shape[0], c.heads, c.head_dim)


def slots_of(c: Cache, table: Optional[np.ndarray], max_pages: int, b: int, n: int) -> np.ndarray:
    """Slot of each of the first n tokens of sequence b, -1 where the page is not there."""
    out = np.full(n, -1, np.int64)
    for t in range(n):
        p = t // c.page_size
        page = int(table[b, p]) if table is not None else b * max_pages + p
        if 0 <= page < c.pages:
            out[t] = page * c.page_size + t % c.page_size
    return out


@dataclass
class Attended:
    out: np.ndarray          # [tokens, heads * head_dim]
    lse: np.ndarray          # [tokens, q_heads]
    weight: np.ndarray       # [tokens, heads * head_dim]: sum of p |v|
    reach: np.ndarray        # [tokens, q_heads]: largest scale * sum |q k| over the keys
    mass: np.ndarray         # [batch, groups, capacity]
    mass_err: np.ndarray     # sum of p * reach, for the mass's tolerance


def attention(c: Cache, q: np.ndarray, lens, cu, table, max_pages, causal=True, scale=None) -> Attended:
    d, tokens = c.head_dim, q.shape[0]
    hq = q.shape[1] // d
    g = hq // c.heads
    scale = 1 / math.sqrt(d) if scale is None else scale
    q = q.astype(np.float64).reshape(tokens, hq, d)
    cap = max_pages * c.page_size
    r = Attended(np.zeros((tokens, hq, d)), np.full((tokens, hq), -np.inf), np.zeros((tokens, hq, d)),
                 np.zeros((tokens, hq)), np.zeros((len(lens), c.groups, cap)),
                 np.zeros((len(lens), c.groups, cap)))
    for b in range(len(lens)):
        n, new = min(max(int(lens[b]), 0), cap), int(cu[b + 1] - cu[b])
        slots = slots_of(c, table, max_pages, b, n)
        there = slots >= 0
        k, v = values(c, 0, slots[there]), values(c, 1, slots[there])
        t = np.arange(n)[there]
        for i in range(new):
            limit = n - new + i + 1 if causal else n
            see = t < limit
            if not see.any():
                continue
            for h in range(hq):
                kk, vv, row = k[see, h // g], v[see, h // g], cu[b] + i
                x = scale * (kk @ q[row, h])
                m = x.max()
                p = np.exp(x - m)
                r.lse[row, h] = m + math.log(p.sum())
                p /= p.sum()
                r.out[row, h] = p @ vv
                r.weight[row, h] = p @ np.abs(vv)
                r.reach[row, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[row, h]))).max()
                j = (h // g) * d // c.group
                r.mass[b, j, t[see]] += p
                r.mass_err[b, j, t[see]] += p * r.reach[row, h]
    r.out, r.weight = r.out.reshape(tokens, -1), r.weight.reshape(tokens, -1)
    return r


def evict(mass: np.ndarray, n: int, keep: int, recent: int) -> np.ndarray:
    """Places that stay, ascending, of one sequence and group."""
    if n <= keep:
        return np.arange(n)
    old = n - recent
    key = np.where(np.isnan(mass[:old]), -np.inf, mass[:old].astype(np.float64))
    best = np.argsort(-key, kind="stable")[:keep - recent]
    return np.concatenate([np.sort(best), np.arange(old, n)])


def hadamard(d: int) -> np.ndarray:
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return h


def rope(x: np.ndarray, head_dim: int, inv_freq: np.ndarray, axis, positions: np.ndarray,
         interleaved: bool) -> np.ndarray:
    """The rotary embedding with sine and cosine rounded to float32 and every product and sum
    in float32, as the call documents it; x fp16 [tokens, heads * head_dim]."""
    pairs = inv_freq.shape[0]
    axis = np.zeros(pairs, int) if axis is None else axis
    ok = (axis >= 0) & (axis < positions.shape[0])
    angle = positions[np.where(ok, axis, 0)].T.astype(np.float64) * inv_freq.astype(np.float64)
    angle = np.where(ok, angle, 0.0)
    cos, sin = np.cos(angle).astype(np.float32)[:, None], np.sin(angle).astype(np.float32)[:, None]
    y = x.astype(np.float32).reshape(x.shape[0], -1, head_dim).copy()
    i = np.arange(pairs)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    xa, xb = y[:, :, a].copy(), y[:, :, b].copy()
    y[:, :, a] = xa * cos - xb * sin
    y[:, :, b] = xb * cos + xa * sin
    return y.reshape(x.shape)
