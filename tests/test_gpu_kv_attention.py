"""Attention over the paged 4-bit KV cache, and the attention weight of its tokens, against
a float64 restatement.

Tolerances.  With eps = 2^-11 (half a step of fp16, relative), p the softmax weights and
A = sum p |v|: the output's rounding gives eps |o|; a weight rounded to fp16 is off by at most
eps of itself, which gives eps A, or by half the smallest step, 2^-25 of the largest weight, which
over n keys of values up to V gives n 2^-25 V; a score formed in fp32 from d products
is off by at most (d + 8) 2^-24 of scale sum |q k| =: x_err, and so is the log of the
sum, so that a weight is off by a factor of at most e^(2 x_err) and the output by 2 x_err A
(4 x_err A is allowed, with 2^-16 A for exp, log and the running sums of up to 2^12 keys).
The log of the sum is off by x_err and a few steps of its own size.  The mass
of a token is off by 2 x_err of its weights and 2^-16 of the sum."""
import numpy as np
import pytest
import torch

import w4a4_rotation_quantized_b200 as Q
from tests import kv_reference as R
from tests.gpu_helpers import dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert Q._lib.qr_device_status() == 0


def gpu_cache(c: R.Cache) -> Q.KVCache:
    return Q.KVCache(tuple(dev(a) for a in c.keys), tuple(dev(a) for a in c.values), c.head_dim,
                     c.group, c.page_size)


def make_table(rng, batch, max_pages, pages):
    return rng.permutation(pages)[:batch * max_pages].reshape(batch, max_pages).astype(np.int32)


def check(c, q, lens, cu, table, max_pages, causal=True, scale=None, q_dev=None, seqs=None):
    """Runs both calls and compares them with the restatement; returns (out, lse)."""
    ref = R.attention(c, q, lens, cu, table, max_pages, causal, scale)
    if seqs is None:
        seqs = Q.KVSequences(gpu_cache(c), dev(np.asarray(lens, np.int32)), dev(np.asarray(cu, np.int32)),
                             None if table is None else dev(table))
    assert seqs.max_pages == max_pages
    q_dev = dev(q) if q_dev is None else q_dev
    out, lse = Q.kv_attention(seqs, q_dev, causal=causal, scale=scale, return_lse=True)
    first, last = int(cu[0]), int(cu[-1])
    got, want = host(out).astype(np.float64)[first:last], ref.out[first:last]
    d, hq = c.head_dim, q.shape[1] // c.head_dim
    xe = ((d + 8) * 2.0 ** -24 * ref.reach)[first:last]
    per = lambda a: np.repeat(a, d, axis=1)
    big = max(np.abs(R.values(c, 1, np.arange(c.values[0].shape[0]))).max(initial=0.0, where=np.isfinite(
        R.values(c, 1, np.arange(c.values[0].shape[0])))), 0.0)
    n = max(1, int(np.max(lens, initial=0)))
    tol = 2.0 ** -11 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16 + 4 * per(xe)) * ref.weight[first:last] \
        + n * 2.0 ** -25 * min(big, 1e4) + 2.0 ** -24
    err = np.abs(got - want)
    assert np.all(err <= tol), f"out off by {err.max():.3g}, {(err / tol).max():.3g} of the tolerance"
    gl, wl = host(lse).astype(np.float64)[first:last], ref.lse[first:last]
    empty = np.isinf(wl)
    assert np.array_equal(np.isneginf(gl), empty) and not np.isnan(gl).any()
    assert np.all(got[per(empty)] == 0)
    assert np.all(np.abs(gl - wl)[~empty] <= (xe + 2.0 ** -16 + 2.0 ** -22 * np.abs(wl))[~empty])
    mass = np.random.default_rng(3).uniform(0, 1, (len(lens), c.groups, max_pages * c.page_size + 5)).astype(np.float32)
    lse_in = np.where(np.isnan(ref.lse), -np.inf, ref.lse).astype(np.float32)
    gm = host(Q.kv_attention_mass(seqs, q_dev, dev(lse_in), dev(mass), causal=causal, scale=scale))
    cap = max_pages * c.page_size
    np.testing.assert_array_equal(gm[:, :, cap:], mass[:, :, cap:])
    wm = mass[:, :, :cap].astype(np.float64) + ref.mass
    mt = 2.0 ** -23 * wm + 2.0 ** -16 * ref.mass + 4 * (d + 8) * 2.0 ** -24 * ref.mass_err \
        + ref.mass * 2.0 ** -23 * np.abs(np.where(np.isinf(ref.lse), 0, ref.lse)).max(initial=0)
    em = np.abs(gm[:, :, :cap] - wm)
    assert np.all(em <= mt), f"mass off by {em.max():.3g}, {(em / np.maximum(mt, 1e-30)).max():.3g} of the tolerance"
    untouched = ref.mass == 0
    np.testing.assert_array_equal(gm[:, :, :cap][untouched & (mass[:, :, :cap] == wm)],
                                  mass[:, :, :cap][untouched & (mass[:, :, :cap] == wm)])
    return out, lse


SHAPES = [
    # q_heads, heads, head_dim, group
    (4, 4, 128, 128),
    (8, 1, 128, 128),
    (16, 8, 128, 128),
    (7, 1, 128, 128),
    (6, 2, 64, 128),
    (12, 12, 32, 128),
    (8, 8, 32, 256),
    (5, 1, 256, 256),
    (6, 2, 128, 256),
    (20, 1, 128, 128),
    (10, 10, 128, 128),
]
BATCHES = [
    # new, lens, page_size, causal
    ([1], [1], 16, True),
    ([1], [300], 64, True),
    ([1, 1, 1, 1], [1, 17, 64, 259], 16, True),
    ([1, 1, 1], [33, 0, 100], 33, True),                  # a sequence that holds nothing
    ([3, 1, 2], [3, 40, 131], 100, True),                  # drafts; a whole sequence in one call
    ([5, 9], [3, 200], 7, True),                           # more rows than tokens: rows that see none
    ([40, 0, 70], [130, 50, 70], 48, True),
    ([37, 20], [129, 65], 129, False),                     # cross attention
    ([4, 3], [0, 50], 16, False),                          # ... to nothing
]


@pytest.mark.parametrize("new,lens,page,causal", BATCHES)
@pytest.mark.parametrize("hq,hk,d,group", SHAPES)
def test_attention_and_mass(hq, hk, d, group, new, lens, page, causal):
    if group // d > 1 and hk * d % group:
        pytest.skip("no such cache")
    rng = np.random.default_rng(hq * 1000 + d + len(new) + page)
    mp = -(-max(lens) // page) + 1
    c = R.random_cache(rng, len(new) * mp + 2, page, hk, d, group)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((cu[-1], hq * d)).astype(np.float16)
    check(c, q, lens, cu, make_table(rng, len(new), mp, c.pages), mp, causal)


@pytest.mark.parametrize("new,lens", [([1], [5000]), ([2, 1], [4097, 2300]), ([150], [700]), ([300], [300]),
                                      ([129, 1, 64], [1000, 900, 64])])
@pytest.mark.parametrize("hq,hk,d,group", [(8, 2, 128, 128), (4, 4, 64, 128), (2, 1, 256, 256)])
def test_long(hq, hk, d, group, new, lens):
    rng = np.random.default_rng(sum(lens) + d)
    page = 64
    mp = -(-max(lens) // page)
    c = R.random_cache(rng, len(new) * mp, page, hk, d, group)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = (2 * rng.standard_normal((cu[-1], hq * d))).astype(np.float16)
    check(c, q, lens, cu, make_table(rng, len(new), mp, c.pages), mp)


def test_without_a_table_and_one_page():
    rng = np.random.default_rng(5)
    c = R.random_cache(rng, 3, 90, 2, 128, 128)
    q = rng.standard_normal((6, 4 * 128)).astype(np.float16)
    check(c, q, [90, 11, 64], [0, 2, 3, 6], None, 1)


@pytest.mark.parametrize("new", [1, 70])
def test_what_lies_behind_the_mask_is_not_seen(new):
    """NaN and infinite scales in slots past the end, in pages of nobody, and in causally hidden
    tokens; page numbers outside the cache."""
    rng = np.random.default_rng(new)
    page, mp, hk, d = 16, 12, 2, 128
    c = R.random_cache(rng, 40, page, hk, d, 128)
    table = make_table(rng, 2, mp, c.pages)
    lens, cu = [150, 75], [0, new, 2 * new]
    used = np.concatenate([R.slots_of(c, table, mp, b, n) for b, n in enumerate(lens)])
    free = np.setdiff1d(np.arange(c.pages * page), used)
    for side in (c.keys, c.values):
        side[1][free] = np.where(rng.random((free.size, 2)) < 0.5, np.nan, np.inf)
        side[2][free] = -2 ** 31
    table[0, 4], table[1, 2], table[1, 3] = -1, 40, 2 ** 31 - 1      # holes
    q = rng.standard_normal((2 * new, 4 * d)).astype(np.float16)
    check(c, q, lens, cu, table, mp)
    # a hidden token: the newest one is NaN, and only the last row sees it
    if new > 1:
        slot = R.slots_of(c, table, mp, 0, 150)[-1]
        c.keys[1][slot], c.values[1][slot] = np.nan, np.nan
        seqs = Q.KVSequences(gpu_cache(c), dev(np.asarray(lens, np.int32)), dev(np.asarray(cu, np.int32)), dev(table))
        out = host(Q.kv_attention(seqs, dev(q)))
        assert np.isfinite(out[:new - 1]).all() and np.isnan(out[new - 1]).all() and np.isfinite(out[new:]).all()


@pytest.mark.parametrize("new", [1, 66])
def test_extreme_scales_and_zeros(new):
    """Groups of scale 0, zeros far outside the codes' range, values that differ by 2^24 in
    size with the weight on the small ones."""
    rng = np.random.default_rng(20 + new)
    page, mp, hk, d, n = 32, 8, 2, 128, 200
    c = R.random_cache(rng, mp, page, hk, d, 128)
    table = make_table(rng, 1, mp, c.pages)
    c.keys[1][::7] = 0.0
    c.values[1][::5] = 0.0
    c.values[2][3::11] = -30705                            # values with a large offset ...
    c.values[1][3::11] = 1e-4                              # ... of which the step is small
    c.keys[2][2::13] = 2_000_000
    c.keys[1][2::13] = 1e-7
    q = rng.standard_normal((new, 4 * d)).astype(np.float16)
    check(c, q, [n], [0, new], table, mp)
    # one token with huge values and almost no weight: the others must keep their bits
    c = R.random_cache(rng, mp, page, hk, d, 128)
    c.values[1][:] = 1e-4
    slot = R.slots_of(c, table, mp, 0, n)[10]
    c.values[1][slot] = 100.0
    c.keys[0][slot] = 0x88                                 # codes -8 ...
    c.keys[2][slot] = -8                                   # ... of value 0
    q = (4 * rng.standard_normal((new, 4 * d))).astype(np.float16)
    ref = R.attention(c, q, [n], [0, new], table, mp)
    seqs = Q.KVSequences(gpu_cache(c), dev(np.asarray([n], np.int32)), dev(np.asarray([0, new], np.int32)), dev(table))
    got = host(Q.kv_attention(seqs, dev(q))).astype(np.float64)
    xe = np.repeat((d + 8) * 2.0 ** -24 * ref.reach, d, axis=1)
    tol = 2.0 ** -11 * np.abs(ref.out) + (2.0 ** -11 + 2.0 ** -16 + 4 * xe) * ref.weight + 2.0 ** -25
    assert np.all(np.abs(got - ref.out) <= tol)


def test_strided_rows_other_streams_and_rows_of_nobody():
    rng = np.random.default_rng(8)
    page, mp, hk, d = 64, 3, 2, 128
    c = R.random_cache(rng, 2 * mp, page, hk, d, 128)
    table = make_table(rng, 2, mp, c.pages)
    wide = dev(rng.standard_normal((12, 4 * d + 3 * hk * d)).astype(np.float16))
    q = wide[:, 8:8 + 4 * d]                               # queries inside a wider projection
    lens, cu = [100, 170], [2, 3, 10]                      # rows 0, 1, 10, 11 belong to no sequence
    seqs = Q.KVSequences(gpu_cache(c), dev(np.asarray(lens, np.int32)), dev(np.asarray(cu, np.int32)), dev(table))
    check(c, host(q), lens, cu, table, mp, q_dev=q, seqs=seqs)
    base = torch.full((12, 6 * d), 7.0, dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = Q.kv_attention(seqs, q, out=base[:, d:5 * d])
    torch.cuda.current_stream().wait_stream(s)
    want = Q.kv_attention(seqs, q)
    assert torch.equal(out[2:10], want[2:10])
    assert bool((base[:, :d] == 7).all() and (base[:, 5 * d:] == 7).all())
    assert bool((base[:2] == 7).all() and (base[10:] == 7).all())


@pytest.mark.parametrize("new", [1, 4, 100])
def test_graph_sees_new_lengths_and_equal_calls_give_equal_bits(new):
    rng = np.random.default_rng(30 + new)
    page, mp, hk, d = 16, 40, 2, 128
    c = R.random_cache(rng, 2 * mp, page, hk, d, 128)
    table = make_table(rng, 2, mp, c.pages)
    cu = [0, new, 2 * new]
    lens = dev(np.asarray([600, 130], np.int32))
    seqs = Q.KVSequences(gpu_cache(c), lens, dev(np.asarray(cu, np.int32)), dev(table))
    qh = rng.standard_normal((2 * new, 8 * d)).astype(np.float16)
    q = dev(qh)
    mass = torch.zeros((2, hk, mp * page), device="cuda")
    first = Q.kv_attention(seqs, q, return_lse=True)
    again = Q.kv_attention(seqs, q, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                     # two graphs, alive together
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            out, lse = Q.kv_attention(seqs, q, return_lse=True)
            m = Q.kv_attention_mass(seqs, q, lse, mass)
        graphs.append((g, out, lse))
    for ln in ([600, 130], [new, 640], [311, 312]):
        lens.copy_(torch.tensor(ln, dtype=torch.int32))
        ref = R.attention(c, qh, ln, cu, table, mp)
        mass.zero_()
        for g, out, lse in graphs:
            out.fill_(9)
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], graphs[1][1]) and torch.equal(graphs[0][2], graphs[1][2])
        eager = Q.kv_attention(seqs, q)
        assert torch.equal(eager, graphs[0][1])
        np.testing.assert_allclose(host(mass), 2 * ref.mass, rtol=1e-3, atol=1e-5)


def test_two_streams_at_once():
    rng = np.random.default_rng(77)
    page, mp, hk, d = 64, 32, 8, 128
    c = R.random_cache(rng, 4 * mp, page, hk, d, 128)
    table = make_table(rng, 4, mp, c.pages)
    cache = gpu_cache(c)
    mk = lambda lens: Q.KVSequences(cache, dev(np.asarray(lens, np.int32)), dev(np.arange(5, dtype=np.int32)), dev(table))
    a, b = mk([2000, 100, 700, 1]), mk([5, 2048, 900, 33])
    qa, qb = (dev(rng.standard_normal((4, 16 * d)).astype(np.float16)) for _ in range(2))
    wa, wb = Q.kv_attention(a, qa), Q.kv_attention(b, qb)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(sa):
            xa = Q.kv_attention(a, qa)
        with torch.cuda.stream(sb):
            xb = Q.kv_attention(b, qb)
        got.append((xa, xb))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in got)


def test_large_batch_and_slots_past_32_bits():
    """A batch of 300 short sequences, and slots whose byte offset passes 2^32."""
    rng = np.random.default_rng(9)
    page, hk, d = 16, 2, 128
    c = R.random_cache(rng, 600, page, hk, d, 128)
    table = make_table(rng, 300, 2, c.pages)
    lens = rng.integers(0, 33, 300)
    cu = np.arange(301)
    q = rng.standard_normal((300, 4 * d)).astype(np.float16)
    check(c, q, lens, cu, table, 2)
    hk, page = 64, 64                                      # 4096 bytes of codes a slot
    pages = (1 << 32) // 4096 // page + 4
    slots = pages * page
    side = lambda: (torch.zeros((slots, hk * d // 2), dtype=torch.uint8, device="cuda"),
                    torch.zeros((slots, hk), dtype=torch.float32, device="cuda"),
                    torch.zeros((slots, hk), dtype=torch.int32, device="cuda"))
    keys, vals = side(), side()
    small = R.random_cache(rng, 2, page, hk, d, 128)
    far = [pages - 1, pages - 3]
    for p, at in enumerate(far):
        for big, little in zip(keys + vals, small.keys + small.values):
            big[at * page:(at + 1) * page] = dev(little[p * page:(p + 1) * page])
    cache = Q.KVCache(keys, vals, d, 128, page)
    seqs = Q.KVSequences(cache, dev(np.asarray([100], np.int32)), dev(np.asarray([0, 2], np.int32)),
                         dev(np.asarray([far], np.int32)))
    q = rng.standard_normal((2, hk * d)).astype(np.float16)
    check(small, q, [100], [0, 2], np.asarray([[0, 1]], np.int32), 2, seqs=seqs)
