"""Append (rope over several axes, R3, 4-bit write), read back and eviction on the paged KV cache,
and a run of all its calls as a serving loop makes them."""
import numpy as np
import pytest
import torch

import oracle as O
import w4a4_rotation_quantized_b200 as Q
from tests import kv_reference as R
from tests.gpu_helpers import ROT_TOL, dev, host, require_gpu
from tests.test_gpu_kv import _check_group_side
from tests.test_gpu_kv_attention import gpu_cache, make_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert Q._lib.qr_device_status() == 0


def sequences(cache, lens, cu, table):
    i32 = lambda a: None if a is None else dev(np.asarray(a, np.int32))
    return Q.KVSequences(cache, i32(lens), i32(cu), i32(table))


def side_rows(side, slots):
    return [host(a)[slots] for a in side]


@pytest.mark.parametrize("hq,hk,d,group", [(8, 4, 128, 128), (4, 2, 64, 128), (16, 8, 32, 256), (3, 1, 256, 256),
                                           (4, 2, 128, 256)])
def test_append_without_rope_equals_kv_quantize(hq, hk, d, group):
    """The same bits as qr_kv_quantize, at the tokens' slots, from rows of a wider projection."""
    rng = np.random.default_rng(d + group)
    page, mp = 7, 5
    new, lens = [1, 9, 0, 13], [30, 9, 4, 20]
    cu = np.concatenate([[0], np.cumsum(new)])
    cache = Q.KVCache.empty(4 * mp, page, hk, d, group)
    ref = R.Cache(None, None, hk, d, group, page)
    wide = dev((rng.standard_normal((cu[-1], (hq + 2 * hk) * d)) * 3).astype(np.float16))
    q, k, v = wide[:, :hq * d], wide[:, hq * d:(hq + hk) * d], wide[:, (hq + hk) * d:]
    table = make_table(rng, 4, mp, 4 * mp)
    seqs = sequences(cache, lens, cu, table)
    q_rot = Q.kv_append(seqs, q, k, v)
    want_q = Q.kv_quantize(q.contiguous(), None, None, d, group)[0]
    _, ks, vs = Q.kv_quantize(None, k.contiguous(), v.contiguous(), d, group)
    assert torch.equal(q_rot, want_q)
    pages = R.Cache((host(cache.keys[0]),), None, hk, d, group, page)
    slots = np.concatenate([R.slots_of(pages, table, mp, b, n)[n - m:] for b, (n, m) in enumerate(zip(lens, new))])
    for got, want in ((cache.keys, ks), (cache.values, vs)):
        for a, b in zip(got, want):
            np.testing.assert_array_equal(host(a)[slots], host(b))
        rest = np.setdiff1d(np.arange(cache.slots), slots)
        assert all((host(a)[rest] == 0).all() for a in got)          # nothing else is written
    # the read back: the values, rounded to fp16
    kd, vd = Q.kv_dequantize(seqs, int(cu[-1]))
    c = R.Cache(tuple(host(a) for a in cache.keys), tuple(host(a) for a in cache.values), hk, d, group, page)
    for got, side in ((kd, 0), (vd, 1)):
        want = R.values(c, side, slots).reshape(len(slots), -1)
        # one rounding to fp32, one to fp16
        assert np.all(np.abs(host(got).astype(np.float64) - want) <= (2.0 ** -11 + 2.0 ** -23) * np.abs(want) + 2.0 ** -25)


ROPES = [
    # head_dim, group, pairs, axes, interleaved, far
    (128, 128, 64, 1, False, False),
    (128, 128, 64, 3, False, False),
    (128, 128, 64, 3, True, False),
    (128, 128, 32, 2, False, False),           # the first half of the head turns
    (128, 128, 10, 1, False, False),           # pairs that fill no vector
    (64, 128, 32, 3, False, False),
    (64, 128, 15, 2, True, False),
    (32, 256, 16, 1, False, False),
    (256, 256, 128, 3, False, False),
    (256, 256, 20, 3, False, False),
    (128, 128, 64, 1, False, True),             # positions up to 2^31
]


@pytest.mark.parametrize("d,group,pairs,axes,interleaved,far", ROPES)
def test_append_with_rope(d, group, pairs, axes, interleaved, far):
    rng = np.random.default_rng(pairs * 7 + axes)
    hk = 4 * group // d if d < group else 2
    hq = 2 * hk
    tokens, page = 23, 8
    q, k, v = (rng.standard_normal((tokens, h * d)).astype(np.float16) for h in (hq, hk, hk))
    k[:, 5] *= 15
    inv = (10000.0 ** (-np.arange(pairs) / pairs)).astype(np.float32)
    axis = rng.integers(0, axes, pairs).astype(np.int32)
    if axes > 1:
        axis[0] = axes                                            # no such axis: the pair stays as it is
    pos = rng.integers(0, 2 ** 31 - 1 if far else 5000, (axes, tokens)).astype(np.int32)
    cache = Q.KVCache.empty(4, page, hk, d, group)
    seqs = sequences(cache, [tokens], [0, tokens], None)
    rope = Q.Rope(dev(inv), dev(axis) if axes > 1 else None, interleaved)
    q_rot = Q.kv_append(seqs, dev(q), dev(k), dev(v), rope, dev(pos))
    turned = [R.rope(x, d, inv, axis if axes > 1 else None, pos, interleaved).astype(np.float64) for x in (q, k)]
    # the oracle's R3 and group quantizer on the turned rows, under the tests' rules for them
    ref_q = O.rotate_heads(turned[0], d)
    hn = np.repeat(np.linalg.norm(ref_q.reshape(tokens, hq, d), axis=2), d, axis=1)
    assert np.all(np.abs(host(q_rot).astype(np.float64) - ref_q) <= 2.0 ** -11 * np.abs(ref_q) + ROT_TOL * hn + 1e-7)
    rot_k = O.rotate_heads(turned[1], d)
    rows = lambda side: tuple(a[:tokens].contiguous() for a in side)
    _check_group_side(rows(cache.keys), O.quantize_groups_asym(rot_k, group), rot_k, group, "keys")
    v64 = v.astype(np.float64)
    _check_group_side(rows(cache.values), O.quantize_groups_asym(v64, group), v64, group, "values")


def test_rope_angles_are_exact_at_far_positions():
    """q with one element set: rope without R3 can be read off after undoing R3 exactly."""
    d = 32
    pos = np.array([[0, 1, 131071, 1 << 20, 2 ** 31 - 1]], np.int32)
    q = np.zeros((5, 4 * d), np.float16)
    q[:, 0::d] = 1.0
    inv = np.array([1.0] + [0.5] * 15, np.float32)
    cache = Q.KVCache.empty(1, 8, 4, d, 128)
    seqs = sequences(cache, [5], [0, 5], None)
    out = host(Q.kv_append(seqs, dev(q), None, None, Q.Rope(dev(inv)), dev(pos))).astype(np.float64)
    # element 0 becomes cos, element 16 sin; R3 spreads them: rows 0 and 16 of H / sqrt(d)
    back = out.reshape(5, 4, d) @ R.hadamard(d) / np.sqrt(d)
    a = pos[0].astype(np.float64)
    # each of the 32 summed entries is off by half a step of fp16 of at most 2 / sqrt(32)
    tol = np.sqrt(d) * 2.0 ** -11 * 2 / np.sqrt(d) + 1e-6
    assert np.all(np.abs(back[:, 0, 0] - np.cos(a)) <= tol) and np.all(np.abs(back[:, 0, 16] - np.sin(a)) <= tol)


def test_append_parts_places_and_rows_of_nobody():
    rng = np.random.default_rng(4)
    hk, d, page = 2, 128, 16
    cache = Q.KVCache.empty(6, page, hk, d)
    table = np.array([[0, 1], [2, 9], [-1, 4]], np.int32)          # pages that are not there
    lens, cu = [20, 20, 20], [1, 6, 11, 16]
    k, v = (dev(rng.standard_normal((18, hk * d)).astype(np.float16)) for _ in range(2))
    q = dev(rng.standard_normal((18, 4 * d)).astype(np.float16))
    seqs = sequences(cache, lens, cu, table)
    out = torch.full((18, 4 * d), 5.0, dtype=torch.float16, device="cuda")
    Q.kv_append(seqs, q, k, None, out=out)
    assert bool((out[:1] == 5).all() and (out[16:] == 5).all() and (out[1:16] != 5).any(1).all())
    assert all(bool((a == 0).all()) for a in cache.values)          # no v: the side stays
    written = np.nonzero(host(cache.keys[1]).any(1))[0]
    want = [15, 16 + 0, 16 + 1, 16 + 2, 16 + 3] + [2 * 16 + 15] + [4 * 16 + t for t in range(4)]
    assert sorted(written) == sorted(want)
    kd, _ = Q.kv_dequantize(seqs, 18)
    gone = [1 + 5 + t for t in range(1, 5)] + [11]                  # tokens without a page read as 0
    assert bool((kd[gone] == 0).all())
    # lengths beyond what the pages hold, and below zero
    for bad in ([100, -5, 2], [0, 0, 0]):
        cache2 = Q.KVCache.empty(6, page, hk, d)
        Q.kv_append(sequences(cache2, bad, cu, table), q, k, v)
        assert (host(cache2.keys[1]).any(1).sum()) <= 10
    # queries alone
    assert torch.equal(Q.kv_append(seqs, q, None, None)[1:16], out[1:16])


def test_offsets_that_do_not_ascend_are_not_followed():
    """Row offsets of a broken batch: nothing outside the sequences' tokens is read or written."""
    rng = np.random.default_rng(6)
    hk, d, page = 2, 128, 16
    x = [dev(rng.standard_normal((8, h * d)).astype(np.float16)) for h in (4, hk, hk)]
    for cu in ([0, 7, 2, 4], [3, 3, -5, 8], [0, 100, 2, 9], [-4, 2, 5, 8]):
        cache = Q.KVCache.empty(3, page, hk, d)
        seqs = sequences(cache, [9, 16, 3], cu, None)
        q = Q.kv_append(seqs, *x)
        Q.kv_dequantize(seqs, 8)
        q = torch.where(torch.isfinite(q), q, torch.zeros_like(q))        # rows of nobody are not written
        out, lse = Q.kv_attention(seqs, q, return_lse=True)
        lse = torch.where(torch.isfinite(lse), lse, torch.full_like(lse, 50.0))
        Q.kv_attention_mass(seqs, q, lse, torch.zeros((3, hk, page), device="cuda"))
        torch.cuda.synchronize()
        written = np.nonzero(host(cache.keys[1]).any(1))[0]
        assert all(r % page < n for r, n in zip(written, np.array([9, 16, 3])[written // page]))


EVICTS = [
    # heads, head_dim, group, page, lens, keep, recent
    (2, 128, 128, 16, [100, 40, 0, 64], 40, 8),
    (4, 64, 128, 7, [200, 199], 150, 0),
    (1, 256, 256, 64, [3000], 1500, 1500),                 # only the newest
    (8, 32, 256, 33, [77, 500, 78], 77, 1),
    (2, 128, 128, 64, [9000, 5000], 4111, 300),
    (3, 128, 128, 16, [50, 60], 1, 0),
    (2, 128, 256, 50, [400], 399, 200),
]


@pytest.mark.parametrize("hk,d,group,page,lens,keep,recent", EVICTS)
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(hk, d, group, page, lens, keep, recent, in_place):
    rng = np.random.default_rng(keep + hk)
    batch, mp = len(lens), -(-max(max(lens), 1) // page)
    c = R.random_cache(rng, 2 * batch * mp, page, hk, d, group)
    tables = rng.permutation(2 * batch * mp).reshape(2, batch, mp).astype(np.int32)
    mass = np.exp(rng.standard_normal((batch, c.groups, mp * page + 3)) * 2).astype(np.float32)
    mass[rng.random(mass.shape) < 0.2] = 1.5                        # many equal ones
    mass[rng.random(mass.shape) < 0.1] = 0.0
    mass[:, :, 5::50], mass[:, :, 6::70], mass[:, :, 9::90], mass[:, :, 11::60] = np.nan, np.inf, -np.inf, -0.0
    cache = gpu_cache(c)
    seqs = sequences(cache, lens, None, tables[0])
    m = dev(mass)
    kept, now, m2 = Q.kv_evict(seqs, m, keep, recent, None if in_place else dev(tables[1]))
    assert (m2 is m) == in_place
    np.testing.assert_array_equal(host(now), np.minimum(lens, keep))
    to = tables[0] if in_place else tables[1]
    want = [[a.copy() for a in side] for side in (c.keys, c.values)]
    per = [group // 2, 1, 1]
    for b, n in enumerate(lens):
        src, dst = R.slots_of(c, tables[0], mp, b, mp * page), R.slots_of(c, to, mp, b, mp * page)
        for j in range(c.groups):
            stay = R.evict(mass[b, j], n, keep, recent)
            row = np.full(keep, -1)
            row[:len(stay)] = stay
            np.testing.assert_array_equal(host(kept)[b, j], row)
            wm = np.zeros(mass.shape[2], np.float32)
            wm[:len(stay)] = mass[b, j, stay]
            np.testing.assert_array_equal(host(m2)[b, j], wm)
            for s, old in enumerate((c.keys, c.values)):
                for a, o, w in zip(want[s], old, per):
                    a[dst[:len(stay)], j * w:(j + 1) * w] = o[src[stay], j * w:(j + 1) * w]
    for side, w in zip((cache.keys, cache.values), want):
        for a, b in zip(side, w):
            np.testing.assert_array_equal(host(a), b)


def test_evict_without_a_table_and_twice():
    """In place on the default pages; evicting again with nothing above the budget changes nothing."""
    rng = np.random.default_rng(12)
    c = R.random_cache(rng, 2, 200, 2, 128, 128)
    cache = gpu_cache(c)
    mass = dev(rng.random((2, 2, 200)).astype(np.float32))
    lens = dev(np.asarray([200, 90], np.int32))
    seqs = Q.KVSequences(cache, lens, None, None)
    _, now, _ = Q.kv_evict(seqs, mass, 100, 10)
    before = [a.clone() for a in cache.keys + cache.values] + [mass.clone()]
    kept, again, _ = Q.kv_evict(Q.KVSequences(cache, now, None, None), mass, 100, 10)
    assert torch.equal(now, again) and host(now).tolist() == [100, 90]
    assert all(torch.equal(a, b) for a, b in zip(before, list(cache.keys + cache.values) + [mass]))
    assert host(kept)[1, 0].tolist() == list(range(90)) + [-1] * 10


def test_a_serving_loop():
    """A prompt, then decode steps with the running mass, an eviction in between, and more steps: the
    output follows a float64 model that keeps, per head, exactly the tokens the cache should hold."""
    rng = np.random.default_rng(99)
    hq, hk, d, page, keep, recent = 4, 2, 128, 16, 48, 12
    batch, mp = 2, 8
    cache = Q.KVCache.empty(batch * mp, page, hk, d)
    table = make_table(rng, batch, mp, batch * mp)
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    cu = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    seqs = Q.KVSequences(cache, lens, cu, dev(table))
    rope = Q.Rope(dev((10000.0 ** (-np.arange(64) / 64)).astype(np.float32)))
    mass = torch.zeros((batch, hk, seqs.capacity), device="cuda")
    arrived = [0, 0]

    def host_cache():
        return R.Cache(tuple(host(a) for a in cache.keys), tuple(host(a) for a in cache.values), hk, d, 128, page)

    for step, new in enumerate([(60, 37), (1, 1), (1, 1), (9, 1), "evict", (1, 1), (3, 2), "evict", (1, 1)]):
        if new == "evict":
            before, m0, n0 = host_cache(), host(mass).copy(), host(lens).copy()
            kept, now, _ = Q.kv_evict(seqs, mass, keep, recent)
            after = host_cache()
            for b in range(batch):
                slots = R.slots_of(before, table, mp, b, seqs.capacity)
                for j in range(hk):
                    stay = R.evict(m0[b, j], int(n0[b]), keep, recent)
                    assert host(kept)[b, j, :len(stay)].tolist() == stay.tolist()
                    for side in (0, 1):
                        old, got = (R.values(x, side, slots) for x in (before, after))
                        np.testing.assert_array_equal(got[:len(stay), j], old[stay, j])
            lens.copy_(now)
            continue
        t = sum(new)
        q, k, v = (dev(rng.standard_normal((t, h * d)).astype(np.float16)) for h in (hq, hk, hk))
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(arrived, new)]).astype(np.int32)
        arrived = [a + n for a, n in zip(arrived, new)]
        lens.add_(torch.tensor(new, dtype=torch.int32, device="cuda"))
        cu.copy_(torch.tensor([0, new[0], t], dtype=torch.int32))
        m0 = host(mass).astype(np.float64)
        q_rot = Q.kv_append(seqs, q, k, v, rope, dev(pos))
        out, lse = Q.kv_attention(seqs, q_rot, return_lse=True)
        Q.kv_attention_mass(seqs, q_rot, lse, mass)
        ref = R.attention(host_cache(), host(q_rot), host(lens), host(cu), table, mp)
        # one rounding of the weights and one of the output (2^-11 each), scores of |x| < 40 in fp32
        tol = 2.0 ** -11 * np.abs(ref.out) + (2.0 ** -11 + 1e-3) * ref.weight + 2.0 ** -20
        assert np.all(np.abs(host(out) - ref.out) <= tol), step
        np.testing.assert_allclose(host(mass), m0 + ref.mass, rtol=1e-3, atol=1e-6)
    assert host(lens).tolist() == [49, 44]
