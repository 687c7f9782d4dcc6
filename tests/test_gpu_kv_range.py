"""Attention over the paged 4-bit KV cache at the ends of its range.  Against a float64 restatement, under the
tolerances of test_gpu_kv_attention."""
import math

import numpy as np
import pytest

import w4a4_rotation_quantized_b200 as Q
from tests import kv_reference as R
from tests.gpu_helpers import require_gpu
from tests.test_gpu_kv_attention import check, make_table

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
