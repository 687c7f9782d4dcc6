"""What the wrappers of the calls on the paged KV cache hand to the C ABI, without a GPU: host tensors stand in for
the device's, and the entry points are replaced by ones that note their arguments."""
import ctypes

import numpy as np
import pytest
import torch

import w4a4_rotation_quantized_b200 as Q
from w4a4_rotation_quantized_b200 import _lib as L
from w4a4_rotation_quantized_b200 import kv


class Calls(list):
    """The calls made: (name, arguments)."""

    def take(self, name):
        def call(*args, **kw):
            self.append((name, args))
            return 256
        return call


@pytest.fixture
def calls(monkeypatch):
    made = Calls()
    monkeypatch.setattr(kv, "_need_cuda", lambda t, dtype, name: None)
    monkeypatch.setattr(kv, "_stream_of", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for name in ("qr_kv_append", "qr_kv_dequantize", "qr_kv_attention", "qr_kv_attention_workspace",
                 "qr_kv_attention_mass", "qr_kv_evict"):
        monkeypatch.setattr(L, name, made.take(name))
    return made


def sequences(tokens=5):
    cache = Q.KVCache.empty(4, 16, 2, 128, device="cpu")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    return Q.KVSequences(cache, i32([tokens]), i32([0, tokens]), None)


def positions_read(c: L.QrKvRope, tokens: int) -> np.ndarray:
    """The positions that the kernel reads: row of `tokens` at every multiple of ld_pos, one an axis."""
    got = np.empty((c.axes, tokens), np.int32)
    for a in range(c.axes):
        got[a] = np.ctypeslib.as_array((ctypes.c_int32 * tokens).from_address(c.positions + 4 * a * c.ld_pos))
    return got


POSITIONS = {
    "contiguous": lambda n: torch.arange(3 * n, dtype=torch.int32).reshape(3, n),
    "expanded": lambda n: torch.arange(n, dtype=torch.int32).unsqueeze(0).expand(3, -1),
    "expanded rows of two": lambda n: torch.arange(2 * n, dtype=torch.int32).reshape(2, n)[1:].expand(3, -1),
    "overlapping": lambda n: torch.arange(n + 2, dtype=torch.int32).as_strided((3, n), (1, 1)),
    "part of wider rows": lambda n: torch.arange(3 * (n + 7), dtype=torch.int32).reshape(3, n + 7)[:, 4:4 + n],
    "every second row": lambda n: torch.arange(6 * n, dtype=torch.int32).reshape(6, n)[::2],
    "one axis": lambda n: torch.arange(n, dtype=torch.int32).unsqueeze(0),
    "one axis, one dimension": lambda n: torch.arange(n, dtype=torch.int32),
    "one axis of an expanded row": lambda n: torch.arange(n, dtype=torch.int32).expand(1, n),
}


@pytest.mark.parametrize("kind", POSITIONS)
@pytest.mark.parametrize("tokens", [1, 5])
def test_positions_of_any_stride_are_read_within_their_storage(calls, kind, tokens):
    pos = POSITIONS[kind](tokens)
    want = np.atleast_2d(pos.numpy())
    rope = Q.Rope(torch.ones(64), torch.zeros(64, dtype=torch.int32))
    c = rope._c(pos, tokens)
    assert c.axes == want.shape[0]
    if c.axes > 1:
        assert c.ld_pos >= tokens
        # the last element read lies in the tensor that the struct keeps
        store = getattr(c, "rows", pos).untyped_storage()
        end = store.data_ptr() + store.nbytes()
        assert c.positions + 4 * ((c.axes - 1) * c.ld_pos + tokens) <= end
    np.testing.assert_array_equal(positions_read(c, tokens), want)
    # ... and so through the call
    k = torch.zeros((tokens, 256), dtype=torch.float16)
    Q.kv_append(sequences(tokens), None, k, k.clone(), rope, pos)
    (name, args), = calls
    assert name == "qr_kv_append"
    assert args[2]._obj.ld_pos == c.ld_pos and args[2]._obj.axes == c.axes
    np.testing.assert_array_equal(positions_read(args[2]._obj, tokens), want)


def test_positions_without_a_rope_are_refused(calls):
    k = torch.zeros((5, 256), dtype=torch.float16)
    with pytest.raises(ValueError, match="rope"):
        Q.kv_append(sequences(), None, k, k.clone(), positions=torch.arange(5, dtype=torch.int32))
    assert not calls
    Q.kv_append(sequences(), None, k, k.clone())
    assert len(calls) == 1


def test_the_workspace_is_asked_for_on_the_caches_device(calls, monkeypatch):
    """The current device is another one: both the size and the launch belong to the cache's.  One size is kept."""
    inside = []

    class Device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            inside.append(self.i)

        def __exit__(self, *error):
            inside.append(None)

    seqs = sequences(5)
    seqs._index = 1
    monkeypatch.setattr(torch.cuda, "device", Device)
    seen = []
    for name in ("qr_kv_attention_workspace", "qr_kv_attention"):
        monkeypatch.setattr(L, name, lambda *a, name=name: seen.append((name, a, inside[-1] if inside else None)) or 64)
    for tokens in (5, 5, 3, 5):
        q = torch.zeros((tokens, 512), dtype=torch.float16)
        Q.kv_attention(seqs, q)
    assert [n for n, _, _ in seen] == ["qr_kv_attention_workspace", "qr_kv_attention", "qr_kv_attention"] \
        + ["qr_kv_attention_workspace", "qr_kv_attention"] * 2
    assert all(at == 1 for _, _, at in seen)
    assert all(a[2:] == (tokens, 4) for (n, a, _), tokens in zip([x for x in seen if x[0].endswith("workspace")], (5, 3, 5)))
    assert seqs._workspace == ((5, 4), 64)


def test_overlap_is_that_of_elements():
    """Columns of one buffer do not overlap; everything that shares an element does.  Against the elements' addresses."""
    buf = torch.zeros(4096, dtype=torch.float16)

    def elements(t):
        rows, cols = t.shape
        return {t.storage_offset() + i * t.stride(0) + j * t.stride(1) for i in range(rows) for j in range(cols)}

    rng = np.random.default_rng(0)
    views = [buf.as_strided((int(rng.integers(0, 5)), w), (int(rng.choice([p for p in (16, 24, 40) if p >= w])), 1),
                            int(rng.integers(0, 100))) for w in rng.choice([8, 16, 24], 60)]
    for a in views:
        for b in views:
            shared = bool(elements(a) & elements(b))
            assert kv._overlap(a, b) or not shared
            columns = lambda t: {(t.storage_offset() + j) % t.stride(0) for j in range(t.shape[1])}
            if a.stride(0) == b.stride(0) and not columns(a) & columns(b):
                assert not kv._overlap(a, b)


def test_outputs_beside_the_queries_in_one_buffer(calls):
    """A wide buffer of rows: queries in some columns, outputs in others."""
    rows = torch.zeros((5, 1024), dtype=torch.float16)
    Q.kv_attention(sequences(), rows[:, :512], out=rows[:, 512:])
    Q.kv_attention(sequences(), rows[:, 512:], out=rows[:, :512])
    assert sum(n == "qr_kv_attention" for n, _ in calls) == 2
    for out in (rows[:, :512], rows[:, 256:768], rows[:, 504:1016]):
        with pytest.raises(ValueError, match="overlap"):
            Q.kv_attention(sequences(), rows[:, :512], out=out)
