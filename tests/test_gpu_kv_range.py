"""Attention over the paged 4-bit KV cache at the ends of its range.  Against a float64 restatement, under the
tolerances of test_gpu_kv_attention."""
import math

import numpy as np
import pytest
import torch

import w4a4_rotation_quantized_b200 as Q
from tests import kv_reference as R
from tests.gpu_helpers import host, require_gpu
from tests.test_gpu_kv_attention import check, gpu_cache, make_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert Q._lib.qr_device_status() == 0


@pytest.mark.parametrize("d,rows", [(128, 40), (64, 40), (32, 40), (256, 40), (128, 1)])
@pytest.mark.parametrize("lag", [14.5, 9.0])
@pytest.mark.parametrize("up", [15.5, 17.0, 23.5, 24.5, 25.5, 27.0])
def test_a_maximum_that_jumps(d, rows, lag, up):
    """Scores of 0, one of `lag` (in powers of two) that does not raise the running maximum yet, and 32 tokens behind it,
    in every place of a block of keys, one of `up` that does: the first weighs 2^(lag - up) of the other and can be read off
    the output, because each token's value is 1 in an element of its own."""
    n, page = 256, 256
    rng = np.random.default_rng(0)
    for first in (6, 40, 70, 100, 134, 170, 198):
        c = R.random_cache(rng, 1, page, 256 // d, d, 256)
        nib = np.zeros((n, 256), np.int64)
        where = {first: 0, first + 32: d // 2 - 1}
        for h in range(256 // d):
            for t, e in where.items():
                nib[t, h * d + e] = 1
        c.values[0][:] = (nib[:, 0::2] | (nib[:, 1::2] << 4)).astype(np.uint8)
        c.values[1][:], c.values[2][:] = 1.0, 0
        c.keys[0][:], c.keys[2][:] = 0x11, 0                 # every key s_t (1, 1, ..)
        c.keys[1][:] = 0.0
        c.keys[1][first], c.keys[1][first + 32] = lag, up
        q = np.ones((rows, 256), np.float16)
        check(c, q, [n], [0, rows], None, 1, causal=False, scale=math.log(2) / d)


@pytest.mark.parametrize("new,lens", [([1], [1]), ([1, 1], [17, 1]), ([2], [33]), ([1], [300]), ([3, 1], [65, 300]),
                                      ([40], [300])])
@pytest.mark.parametrize("spare", [0, 40])                  # a wide table: items are cut instead of taken whole
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 128), (8, 1, 128), (4, 4, 128), (10, 10, 128), (20, 10, 128), (4, 4, 64),
                                     (2, 1, 256)])
@pytest.mark.parametrize("size", [10.0, 30.0, -30.0])
def test_scores_far_from_zero(hq, hk, d, new, lens, spare, size):
    """Keys of one sign and queries of one sign: every score is some -100, -300 or +300, and a head's warps that hold
    none of the tokens, or none that a row sees, must not count with a maximum of 0."""
    rng = np.random.default_rng(hq * 100 + d + sum(lens))
    page = 64
    mp = -(-max(lens) // page) + spare
    c = R.random_cache(rng, len(new) * mp, page, hk, d, 256 if d == 256 else 128)
    c.keys[1][:] = rng.uniform(0.08, 0.12, c.keys[1].shape)
    c.keys[2][:] = 8                                        # c - z in [-16, -1]
    cu = np.concatenate([[0], np.cumsum(new)])
    q = (size * np.sqrt(128 / d) * rng.uniform(0.9, 1.1, (cu[-1], hq * d))).astype(np.float16)
    check(c, q, lens, cu, make_table(rng, len(new), mp, c.pages), mp)


class Wide:
    """A cache made on the device, and float64 attention of some of its rows there."""

    def __init__(self, seqs, n, hk, d, page, seed, key_zero=0, value_zero=-9):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.hk, self.d, self.page = n, hk, d, page
        per, w = -(-n // page), hk * d
        rows = seqs * per * page

        def side(zero):
            return (torch.randint(0, 256, (rows, w // 2), generator=self.gen, device="cuda", dtype=torch.uint8),
                    0.05 + 0.1 * torch.rand((rows, w // 128), generator=self.gen, device="cuda"),
                    torch.full((rows, w // 128), zero, dtype=torch.int32, device="cuda"))
        self.keys, self.values = side(key_zero), side(value_zero)
        order = torch.randperm(seqs * per, generator=self.gen, device="cuda").to(torch.int32)
        self.table = order.reshape(seqs, per).contiguous()

    def sequences(self, lens, cu):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        cache = Q.KVCache(self.keys, self.values, self.d, 128, self.page)
        return Q.KVSequences(cache, i32(lens), i32(cu), self.table)

    def wide(self, side, b, n, head):
        """Values of the first n tokens of a sequence and head: float64 [n, d]."""
        t = torch.arange(n, device="cuda")
        slots = self.table[b].long()[t // self.page] * self.page + t % self.page
        codes, scales, zeros = side
        d, j = self.d, head * self.d // 128
        c = codes[slots, head * d // 2:(head + 1) * d // 2]
        x = torch.stack([c & 15, c >> 4], -1).flatten(1).double()
        x = torch.where(x > 7, x - 16, x)
        return (x - zeros[slots, j].double()[:, None]) * scales[slots, j].double()[:, None]

    def attend(self, q, b, head, limits):
        """out [rows, d], lse [rows], sum of p |v|, largest sum |q k| of rows q [rows, d] that see limits[i] tokens."""
        n = int(max(limits))
        k, v = self.wide(self.keys, b, n, head), self.wide(self.values, b, n, head)
        x = q.double() @ k.T / math.sqrt(self.d)
        x.masked_fill_(torch.arange(n, device="cuda") >= torch.tensor(limits, device="cuda")[:, None], -math.inf)
        p = torch.softmax(x, 1)
        reach = (q.double().abs() @ k.abs().T).amax(1) / math.sqrt(self.d)
        return p @ v, torch.logsumexp(x, 1), p @ v.abs(), reach


@pytest.mark.parametrize("n,causal", [(32768, False), (131072, True)])
@pytest.mark.parametrize("size", [0.0, 0.02, 1.0])
def test_prompt_behind_a_long_context(n, causal, size):
    """A prompt of 2048 behind n tokens, values of one sign, even weights: every block sums tens of thousands of keys, and
    what such sums lose must stay below what the output's own rounding does.

    Tensor memory sums at most 8192 keys in a row, 512 instructions; one that cuts up to 2^-22 of a sum that grows
    evenly loses up to 512 2^-22 / 2 = 2^-14 of it, always towards zero.  The output's rounding, up to 2^-11 and of
    either sign, leaves 2^-11 / sqrt(3 N) of the mean of N outputs, of which four are allowed; so do the weights'
    roundings, of which there are n more.  l adds 4096 weights in a row in fp32: 4096 / 2 half steps of 2^-24."""
    hq, hk, d, new = 64, 8, 128, 2048
    c = Wide(1, n, hk, d, 256, n)
    q = (size * torch.randn((new, hq * d), generator=c.gen, device="cuda")).half()
    out, lse = Q.kv_attention(c.sequences([n], [0, new]), q, causal=causal, return_lse=True)
    rows = [0, 1, 700, 1500, 2047]
    off, heads = [], [0, 13, 37, 63]
    for h in heads:
        at = slice(h * d, (h + 1) * d)
        want, want_lse, weight, reach = c.attend(q[rows, at], 0, h // 8, [n - new + r + 1 if causal else n for r in rows])
        got = out[rows, at].double()
        tol = 2.0 ** -11 * want.abs() + (2.0 ** -11 + 2.0 ** -14 + 4 * (d + 8) * 2.0 ** -24 * reach[:, None]) * weight + 2.0 ** -24
        assert bool(((got - want).abs() <= tol).all())
        off.append((got - want) / want)
        assert bool(((lse[rows, h].double() - want_lse).abs()
                     <= 2.0 ** -13 + (d + 8) * 2.0 ** -24 * reach + 2.0 ** -22 * want_lse.abs()).all())
    off = torch.cat(off).flatten()
    mean = off.mean().item()
    assert abs(mean) <= 2.0 ** -14 + 4 * 2.0 ** -11 / math.sqrt(3 * off.numel()), f"off by {mean:.3g} on average"


@pytest.mark.parametrize("d,hk,gq", [(128, 16, 1), (64, 32, 2), (256, 8, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_items_of_several_sums(d, hk, gq, causal):
    """Sequences somewhat longer than what is summed in a row, in ranges that hold whole ones and parts: with scores of
    all sizes, with sequences and rows that see only the first sum's keys, or none."""
    seqs, n, new = 19, 9000, 40
    group = 128 if d <= 128 else 256
    c = Wide(seqs, n, hk, d, 64, d)
    if d == 256:
        c.keys, c.values = (tuple(a if i == 0 else a[:, ::2].contiguous() for i, a in enumerate(s)) for s in (c.keys, c.values))
        c.wide = lambda side, b, m, head, f=c.wide: f((side[0],) + tuple(a.repeat_interleave(2, 1) for a in side[1:]), b, m, head)
    lens = [n - 37 * b for b in range(seqs)]
    lens[3], lens[4], lens[5], lens[6] = 8192, 8193, 0, 8200
    q = 3 * torch.randn((seqs * new, hk * gq * d), generator=c.gen, device="cuda").half()
    q[::7] *= 0
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    s = Q.KVSequences(Q.KVCache(c.keys, c.values, d, group, c.page), i32(lens), i32(list(range(0, seqs * new + 1, new))), c.table)
    out, lse = Q.kv_attention(s, q, causal=causal, return_lse=True)
    again = Q.kv_attention(s, q, causal=causal, return_lse=True)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    for b in range(seqs):
        rows = slice(b * new, (b + 1) * new)
        limits = [lens[b] - new + i + 1 if causal else lens[b] for i in range(new)]
        if lens[b] == 0:
            assert bool((out[rows] == 0).all()) and bool(torch.isneginf(lse[rows]).all())
            continue
        for h in range(0, hk * gq, 3):
            at = slice(h * d, (h + 1) * d)
            want, want_lse, weight, reach = c.attend(q[rows, at], b, h // gq, limits)
            xe = (d + 8) * 2.0 ** -24 * reach
            tol = 2.0 ** -11 * want.abs() + (2.0 ** -11 + 2.0 ** -14 + 4 * xe[:, None]) * weight + n * 2.0 ** -25 * 3 + 2.0 ** -24
            assert bool(((out[rows, at].double() - want).abs() <= tol).all()), (b, h)
            assert bool(((lse[rows, h].double() - want_lse).abs() <= xe + 2.0 ** -13 + 2.0 ** -22 * want_lse.abs()).all())


@pytest.mark.parametrize("new", [1, 40])
def test_a_table_of_no_pages(new):
    """max_pages = 0 with a table, as the C ABI allows it: nothing is held, whatever the lengths say, and the table has no
    element to read."""
    rng = np.random.default_rng(new)
    c = R.random_cache(rng, 2, 16, 2, 128, 128)
    cache = gpu_cache(c)
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([new, 30], [0, new, 2 * new]))
    seqs = Q.KVSequences(cache, lens, cu, torch.zeros((2, 0), dtype=torch.int32, device="cuda"))
    table = torch.zeros(1, dtype=torch.int32, device="cuda")           # the address of an empty table
    seqs._c.block_table = table.data_ptr()
    assert seqs.max_pages == 0 and seqs.capacity == 0
    q = torch.randn((2 * new, 4 * 128), device="cuda").half()
    out, lse = Q.kv_attention(seqs, q, return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    mass = torch.ones((2, 2, 3), device="cuda")
    assert bool((Q.kv_attention_mass(seqs, q, lse, mass) == 1).all())
    before = [a.clone() for a in cache.keys + cache.values]
    k = torch.randn((2 * new, 2 * 128), device="cuda").half()
    assert bool(torch.isfinite(Q.kv_append(seqs, q, k, k)).all())
    assert all(torch.equal(a, b) for a, b in zip(before, cache.keys + cache.values))
    assert all(bool((a == 0).all()) for a in Q.kv_dequantize(seqs, 2 * new))
    kept, now, _ = Q.kv_evict(seqs, mass, 2, 1)
    assert bool((kept == -1).all()) and host(now).tolist() == [0, 0]


@pytest.mark.parametrize("in_place", [True, False])
def test_eviction_with_pages_that_were_given_up(in_place):
    """Tokens whose page is not in the cache, with a mass of -inf: none stays while others are there, and what stays
    is moved as if they had never been.  One that stays all the same leaves its place as it was."""
    rng = np.random.default_rng(1)
    hk, d, page, mp, n, keep, recent = 2, 128, 16, 6, 90, 40, 10
    c = R.random_cache(rng, 2 * mp + 1, page, hk, d, 128)
    table = np.array([[0, -1, 2, 2 * mp + 1, 4, 5]], np.int32)       # pages 1 and 3 are gone: 90 - 32 tokens are there
    to = np.arange(mp, 2 * mp, dtype=np.int32)[None]
    if in_place:
        to = table
    mass = np.exp(rng.standard_normal((1, hk, mp * page))).astype(np.float32)
    src = R.slots_of(c, table, mp, 0, mp * page)
    dst = R.slots_of(c, to, mp, 0, mp * page)
    mass[:, :, src < 0] = -np.inf
    for budget in (keep, 70):                                        # 70: twelve that are not there stay too
        cache = gpu_cache(c)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        seqs = Q.KVSequences(cache, i32([n]), None, i32(table.tolist()))
        kept, now, _ = Q.kv_evict(seqs, torch.tensor(mass, device="cuda"), budget, recent,
                                  None if in_place else i32(to.tolist()))
        assert host(now).tolist() == [budget]
        want = [[a.copy() for a in side] for side in (c.keys, c.values)]
        for j in range(hk):
            stay = R.evict(mass[0, j], n, budget, recent)
            assert (src[stay] < 0).sum() == (0 if budget == keep else 12)
            np.testing.assert_array_equal(host(kept)[0, j], stay)
            ok = (src[stay] >= 0) & (dst[:budget] >= 0)
            for side, old in zip(want, (c.keys, c.values)):
                for a, o, w in zip(side, old, (64, 1, 1)):
                    a[dst[:budget][ok], j * w:(j + 1) * w] = o[src[stay][ok], j * w:(j + 1) * w]
        for side, w in zip((cache.keys, cache.values), want):
            for a, b in zip(side, w):
                np.testing.assert_array_equal(host(a), b)


@pytest.mark.parametrize("batch,rows,hq,hk", [(4096, 1, 2, 2), (2100, 40, 1, 1), (2048, 40, 1, 1)])
def test_the_largest_batches(batch, rows, hq, hk):
    """As many sequences as a call takes, and more than the kernel for many rows takes (2048)."""
    rng = np.random.default_rng(batch)
    page, mp, d = 16, 3, 128
    c = R.random_cache(rng, batch * mp, page, hk, d, 128)
    table = make_table(rng, batch, mp, c.pages)
    lens = rng.integers(0, 49, batch)
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")
    cu = np.arange(batch + 1) * rows
    q = rng.standard_normal((batch * rows, hq * d)).astype(np.float16)
    few = np.concatenate([np.arange(5), [batch // 2, batch - 2, batch - 1]])
    seqs = Q.KVSequences(gpu_cache(c), i32(lens), i32(cu), i32(table))
    out, lse = Q.kv_attention(seqs, torch.tensor(q, device="cuda"), return_lse=True)
    out, lse = host(out).astype(np.float64).reshape(batch, rows, -1)[few], host(lse).reshape(batch, rows, -1)[few]
    ref = R.attention(c, q.reshape(batch, rows, -1)[few].reshape(-1, hq * d), lens[few], np.arange(9) * rows, table[few], mp)
    xe = np.repeat((d + 8) * 2.0 ** -24 * ref.reach, d, axis=1)
    tol = 2.0 ** -11 * np.abs(ref.out) + (2.0 ** -11 + 2.0 ** -16 + 4 * xe) * ref.weight + 2.0 ** -20
    assert np.all(np.abs(out.reshape(-1, hq * d) - ref.out) <= tol)
    gone = np.isneginf(ref.lse)
    lse = lse.reshape(-1, hq)
    assert np.array_equal(np.isneginf(lse), gone)
    xe = (d + 8) * 2.0 ** -24 * ref.reach[~gone]
    assert np.all(np.abs(lse[~gone] - ref.lse[~gone]) <= xe + 2.0 ** -16 + 2.0 ** -22 * np.abs(ref.lse[~gone]))


@pytest.mark.parametrize("batch,hk,rows,n", [(300, 8, 1, 131072), (300, 1, 1, 131072), (3, 8, 4, 131072), (40, 8, 40, 20000)])
@pytest.mark.parametrize("at", [5, -3])
@pytest.mark.parametrize("gap", [22.4, 25.4])
def test_one_heavy_token_before_a_long_even_rest(batch, hk, rows, n, at, gap):
    """One token outweighs each of the others by 2^gap, and these by their number still count: what the weights' rounding
    leaves of the rest must not show in fp16.  (All sequences share the same pages.)"""
    d, page = 128, 1024
    pages = -(-n // page)
    full = lambda x, dtype, w: torch.full((pages * page, w), x, dtype=dtype, device="cuda")
    # every key s_t (1, 1, ..), every value +-1: -1 for the heavy one
    keys = [full(0x11, torch.uint8, hk * 64), full(0.0, torch.float32, hk), full(0, torch.int32, hk)]
    values = [full(0x11, torch.uint8, hk * 64), full(1.0, torch.float32, hk), full(0, torch.int32, hk)]
    keys[1][at % n] = gap
    values[0][at % n] = 0xff
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(batch, -1).contiguous()
    seqs = Q.KVSequences(Q.KVCache(keys, values, d, 128, page), i32([n] * batch),
                         i32(np.arange(batch + 1) * rows), table)
    q = torch.ones((batch * rows, hk * d), device="cuda").half()
    out, lse = Q.kv_attention(seqs, q, causal=False, scale=math.log(2) / d, return_lse=True)
    rest = (n - 1) * 2.0 ** -gap
    want = (rest - 1) / (rest + 1)
    # one rounding of the output, one of the weights, and 2^-12 of the sum for weights too small for fp16
    assert (out.double() - want).abs().max().item() <= 2.0 ** -11 * abs(want) + 2.0 ** -11 + 2.0 ** -12
    # a score of gap ln 2, off by (d + 8) 2^-24 of itself.  l next to the heavy weight, 1 to 2 of it, adds in a row no more
    # than n / 32 <= 4096 sums of a piece (few rows), or 4096 weights (many rows); each rounds to half a step, 2^-24 of
    # the heavy weight, which is no less than 2^-24 of l: 2^-12 in all
    assert (lse.double() - (gap * math.log(2) + math.log1p(rest))).abs().max().item() \
        <= (d + 8) * 2.0 ** -24 * gap + 2.0 ** -12 + 2.0 ** -18
