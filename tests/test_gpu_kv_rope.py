"""The rotary embedding of kv_append: positions of any stride."""
import numpy as np
import pytest
import torch

import w4a4_rotation_quantized_b200 as Q
from tests.gpu_helpers import dev, host, require_gpu
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
