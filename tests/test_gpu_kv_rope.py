"""The rotary embedding of kv_append: positions of any stride, and its results bit for bit (each product and sum
rounded to float32 on its own, then the butterflies of R3 in float32, stage by stage, and one rounding to fp16)."""
import numpy as np
import pytest
import torch

import w4a4_rotation_quantized_b200 as Q
from tests import kv_reference as R
from tests.gpu_helpers import dev, host, require_gpu, unpack
from tests.test_gpu_kv_cache import sequences

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert Q._lib.qr_device_status() == 0


@pytest.mark.parametrize("tokens", [1, 5, 300])
def test_positions_expanded_over_the_axes_equal_their_copy(tokens):
    """Text in a model with time, height and width positions: one row of positions for all three axes."""
    rng = np.random.default_rng(tokens)
    d, hk = 128, 2
    q, k, v = (dev(rng.standard_normal((tokens, h * d)).astype(np.float16)) for h in (2 * hk, hk, hk))
    inv = dev((10000.0 ** (-np.arange(64) / 64)).astype(np.float32))
    rope = Q.Rope(inv, dev(rng.integers(0, 3, 64).astype(np.int32)))
    row = dev(rng.integers(1, 5000, tokens + 2).astype(np.int32))
    for pos in (row[:tokens].unsqueeze(0).expand(3, -1), row.as_strided((3, tokens), (1, 1))):
        got = []
        for p in (pos, dev(host(pos))):
            cache = Q.KVCache.empty(1, tokens, hk, d)
            q_rot = Q.kv_append(sequences(cache, [tokens], [0, tokens], None), q, k, v, rope, p)
            got.append([q_rot, *cache.keys, *cache.values])
        assert all(torch.equal(a, b) for a, b in zip(*got))


def butterflies(x: np.ndarray, d: int) -> np.ndarray:
    """The unnormalised Hadamard transform of each head in float32, index bits from the lowest."""
    x = x.astype(np.float32).reshape(x.shape[0], -1, d)
    h = 1
    while h < d:
        y = x.reshape(*x.shape[:2], d // (2 * h), 2, h)
        x = np.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(x.shape)
        h *= 2
    return x.reshape(x.shape[0], -1)


def rotated(x, d, inv, axis, pos, interleaved):
    """Rope and unnormalised butterflies, float32."""
    return butterflies(R.rope(x, d, inv, axis, pos, interleaved), d)


def code_bits(y: np.ndarray, group: int, unit: np.float32):
    """Asymmetric 4-bit codes of the groups of y, of which unit is left out: (codes in [-8, 7], scales, zeros).  A code is
    the whole number next to y r + z, which 64 bits hold exactly."""
    y = y.reshape(y.shape[0], -1, group)
    lo, hi = y.min(2), y.max(2)
    span = hi - lo
    r = np.float32(15) / span
    z = np.rint(-lo * r)
    codes = np.rint(y.astype(np.float64) * r.astype(np.float64)[..., None] + (z.astype(np.float64) - 8)[..., None])
    return np.clip(codes, -8, 7).astype(int).reshape(y.shape[0], -1), span * unit / np.float32(15), z.astype(np.int32) - 8


SHAPES = [
    # head_dim, group, pairs, axes, interleaved
    (128, 128, 64, 1, False),
    (128, 128, 64, 3, False),
    (128, 128, 64, 2, True),
    (128, 128, 16, 2, False),
    (128, 128, 10, 1, False),
    (64, 128, 32, 3, False),
    (64, 128, 15, 2, True),
    (32, 256, 16, 1, False),
    (256, 256, 128, 3, False),
    (256, 256, 20, 3, False),
]


@pytest.mark.parametrize("d,group,pairs,axes,interleaved", SHAPES)
@pytest.mark.parametrize("tokens", [5, 700])                # one token a block, and four
def test_each_operation_is_rounded(d, group, pairs, axes, interleaved, tokens):
    rng = np.random.default_rng(pairs + 10 * axes + tokens)
    hq, hk = 2 * group // d, group // d
    q, k = ((rng.standard_normal((tokens, h * d)) * 3).astype(np.float16) for h in (hq, hk))
    inv = (10000.0 ** (-np.arange(pairs) / pairs)).astype(np.float32)
    axis = rng.integers(0, axes, pairs).astype(np.int32)
    pos = rng.integers(0, 5000, (axes, tokens)).astype(np.int32)
    cache = Q.KVCache.empty(1, tokens, hk, d, group)
    seqs = sequences(cache, [tokens], [0, tokens], None)
    got = host(Q.kv_append(seqs, dev(q), dev(k), None, Q.Rope(dev(inv), dev(axis), interleaved), dev(pos)))
    unit = np.float32(1 / np.sqrt(np.float64(d)))
    want = (rotated(q, d, inv, axis, pos, interleaved) * unit).astype(np.float16)
    off = got.view(np.uint16) != want.view(np.uint16)
    assert not off.any(), f"{off.sum()} of {off.size} queries differ from the formula's bits"
    codes, scales, zeros = code_bits(rotated(k, d, inv, axis, pos, interleaved), group, unit)
    np.testing.assert_array_equal(host(cache.keys[1]), scales)
    np.testing.assert_array_equal(host(cache.keys[2]), zeros)
    np.testing.assert_array_equal(unpack(cache.keys[0]), codes)
