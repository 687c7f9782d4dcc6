"""Refusals of the calls on the paged KV cache: the C ABI's argument errors (nothing is launched, the
pointers are never followed) and the wrappers' checks, without a GPU."""
import ctypes
import math

import pytest
import torch

import w4a4_rotation_quantized_b200 as Q
from w4a4_rotation_quantized_b200 import _lib as L
from w4a4_rotation_quantized_b200 import build as B

FAKE = 0x10000


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return L.load()


def cache(**kw):
    d = dict(k_codes=FAKE, k_scales=FAKE, k_zeros=FAKE, v_codes=FAKE, v_scales=FAKE, v_zeros=FAKE,
             slots=1024, heads=4, head_dim=128, group=128, page_size=16)
    d.update(kw)
    return L.QrKvCache(**d)


def seqs(**kw):
    d = dict(batch=2, max_pages=8, block_table=FAKE, kv_lens=FAKE, cu_q=FAKE)
    d.update(kw)
    return L.QrKvSeqs(**d)


def ref(x):
    return None if x is None else ctypes.byref(x)


def attend(c=None, s=None, Q_=FAKE, ldq=1024, tokens=3, hq=8, scale=0.1, causal=1, out=FAKE, ldo=1024,
           lse=FAKE, ws=FAKE, wsb=1 << 40):
    return L.qr_kv_attention(ref(c or cache()), ref(s or seqs()), Q_, ldq, tokens, hq, scale, causal, out,
                             ldo, lse, ws, wsb, None, check=False)


CACHE_ERRORS = [
    (dict(heads=0), L.QR_ERR_INVALID_ARG),
    (dict(page_size=0), L.QR_ERR_INVALID_ARG),
    (dict(slots=-1), L.QR_ERR_INVALID_ARG),
    (dict(k_codes=None), L.QR_ERR_INVALID_ARG),
    (dict(v_zeros=None), L.QR_ERR_INVALID_ARG),
    (dict(head_dim=96), L.QR_ERR_UNSUPPORTED),
    (dict(group=64), L.QR_ERR_UNSUPPORTED),
    (dict(head_dim=256), L.QR_ERR_UNSUPPORTED),              # a group holds whole heads
    (dict(heads=3, group=256), L.QR_ERR_UNSUPPORTED),
    (dict(heads=1024), L.QR_ERR_UNSUPPORTED),
    (dict(k_codes=FAKE + 8), L.QR_ERR_ALIGNMENT),
    (dict(v_scales=FAKE + 2), L.QR_ERR_ALIGNMENT),
]
SEQ_ERRORS = [
    (dict(batch=-1), L.QR_ERR_INVALID_ARG),
    (dict(max_pages=-1), L.QR_ERR_INVALID_ARG),
    (dict(kv_lens=None), L.QR_ERR_INVALID_ARG),
    (dict(batch=5000), L.QR_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 28), L.QR_ERR_UNSUPPORTED),
    (dict(cu_q=FAKE + 2), L.QR_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,want", CACHE_ERRORS)
def test_cache_errors(kw, want):
    c, s = cache(**kw), seqs()
    assert attend(c=c) == want
    assert L.qr_kv_dequantize(ref(c), ref(s), 3, FAKE, FAKE, None, check=False) == want
    assert L.qr_kv_append(ref(c), ref(s), None, FAKE, 512, FAKE, 512, FAKE, 512, 3, 4, 2 * FAKE, None,
                          check=False) == want
    assert L.qr_kv_evict(ref(c), ref(s), FAKE, 1 << 20, 4, 1, None, FAKE, FAKE, 2 * FAKE, None, check=False) == want
    assert L.qr_kv_attention_workspace(ref(c), ref(s), 3, 8) == -1


@pytest.mark.parametrize("kw,want", SEQ_ERRORS)
def test_sequence_errors(kw, want):
    assert attend(s=seqs(**kw)) == want
    assert L.qr_kv_evict(ref(cache()), ref(seqs(**kw)), FAKE, 1 << 20, 4, 1, None, FAKE, FAKE, 2 * FAKE, None,
                         check=False) == want


def test_attention_errors():
    assert attend(tokens=-1) == L.QR_ERR_INVALID_ARG
    assert attend(hq=6) == L.QR_ERR_INVALID_ARG              # not a multiple of the cache's heads
    assert attend(hq=0) == L.QR_ERR_INVALID_ARG
    assert attend(scale=math.inf) == L.QR_ERR_INVALID_ARG
    assert attend(scale=math.nan) == L.QR_ERR_INVALID_ARG
    assert attend(Q_=None) == L.QR_ERR_INVALID_ARG
    assert attend(ldq=1000) == L.QR_ERR_INVALID_ARG
    assert attend(out=None) == L.QR_ERR_INVALID_ARG
    assert attend(ldo=8) == L.QR_ERR_INVALID_ARG
    assert attend(hq=1024, ldq=1 << 20, ldo=1 << 20) == L.QR_ERR_UNSUPPORTED
    assert attend(Q_=FAKE + 2) == L.QR_ERR_ALIGNMENT
    assert attend(ldq=1028) == L.QR_ERR_ALIGNMENT
    assert attend(ldo=1025) == L.QR_ERR_ALIGNMENT
    assert attend(lse=FAKE + 1) == L.QR_ERR_ALIGNMENT
    assert attend(ws=FAKE + 4) == L.QR_ERR_ALIGNMENT
    assert attend(s=seqs(cu_q=None)) == L.QR_ERR_INVALID_ARG
    assert L.qr_kv_attention(None, ref(seqs()), FAKE, 1024, 3, 8, 0.1, 1, FAKE, 1024, None, None, 0, None,
                             check=False) == L.QR_ERR_INVALID_ARG
    need = L.qr_kv_attention_workspace(ref(cache()), ref(seqs()), 3, 8)
    if need > 0:
        assert attend(wsb=need - 1) == L.QR_ERR_INVALID_ARG
        assert attend(ws=None) == L.QR_ERR_INVALID_ARG
    assert attend(tokens=0) == L.QR_OK
    assert attend(s=seqs(batch=0, kv_lens=None, cu_q=None)) == L.QR_OK


def test_mass_errors():
    def mass(c=None, s=None, Q_=FAKE, ldq=1024, tokens=3, hq=8, lse=FAKE, m=FAKE, ld=128):
        return L.qr_kv_attention_mass(ref(c or cache()), ref(s or seqs()), Q_, ldq, tokens, hq, 0.1, 1, lse, m,
                                      ld, None, check=False)
    assert mass(lse=None) == L.QR_ERR_INVALID_ARG
    assert mass(m=None) == L.QR_ERR_INVALID_ARG
    assert mass(ld=127) == L.QR_ERR_INVALID_ARG
    assert mass(hq=5) == L.QR_ERR_INVALID_ARG
    assert mass(m=FAKE + 2) == L.QR_ERR_ALIGNMENT
    assert mass(tokens=0) == L.QR_OK


def test_append_errors():
    def app(c=None, s=None, rope=None, Q_=FAKE, ldq=1024, K=FAKE, ldk=512, V=FAKE, ldv=512, tokens=3, hq=8,
            out=2 * FAKE):
        return L.qr_kv_append(ref(c or cache()), ref(s or seqs()), ref(rope), Q_, ldq, K, ldk, V, ldv, tokens,
                              hq, out, None, check=False)

    def rope(**kw):
        d = dict(inv_freq=FAKE, axis=FAKE, positions=FAKE, ld_pos=3, pairs=64, axes=3, interleaved=0)
        d.update(kw)
        return L.QrKvRope(**d)
    assert app(out=None) == L.QR_ERR_INVALID_ARG
    assert app(Q_=None) == L.QR_ERR_INVALID_ARG
    assert app(out=FAKE) == L.QR_ERR_INVALID_ARG             # partners are read again: not in place
    assert app(hq=0) == L.QR_ERR_INVALID_ARG
    assert app(ldq=512) == L.QR_ERR_INVALID_ARG
    assert app(ldk=504) == L.QR_ERR_INVALID_ARG
    assert app(ldv=516) == L.QR_ERR_ALIGNMENT
    assert app(K=FAKE + 8) == L.QR_ERR_ALIGNMENT
    assert app(c=cache(head_dim=64, heads=4), hq=5, ldk=256, ldv=256) == L.QR_ERR_UNSUPPORTED   # half a group of queries
    for bad in (dict(pairs=0), dict(pairs=65), dict(axes=0), dict(inv_freq=None), dict(positions=None), dict(ld_pos=2)):
        assert app(rope=rope(**bad)) == L.QR_ERR_INVALID_ARG, bad
    assert app(rope=rope(axis=FAKE + 2)) == L.QR_ERR_ALIGNMENT
    assert app(tokens=0, rope=rope(positions=None, ld_pos=0)) == L.QR_OK
    assert app(tokens=-2) == L.QR_ERR_INVALID_ARG


def test_evict_errors():
    def ev(c=None, s=None, mass=FAKE, ld=128, keep=10, recent=2, to=None, mo=FAKE, kept=FAKE, lo=2 * FAKE):
        return L.qr_kv_evict(ref(c or cache()), ref(s or seqs()), mass, ld, keep, recent, to, mo, kept, lo, None,
                             check=False)
    assert ev(keep=0) == L.QR_ERR_INVALID_ARG
    assert ev(recent=-1) == L.QR_ERR_INVALID_ARG
    assert ev(recent=11) == L.QR_ERR_INVALID_ARG
    assert ev(keep=1 << 30) == L.QR_ERR_UNSUPPORTED
    assert ev(ld=100) == L.QR_ERR_INVALID_ARG
    for name in ("mass", "mo", "kept", "lo"):
        assert ev(**{name: None}) == L.QR_ERR_INVALID_ARG
    assert ev(lo=FAKE) == L.QR_ERR_INVALID_ARG                # kv_lens itself
    assert ev(to=FAKE) == L.QR_ERR_INVALID_ARG                # the table being read
    assert ev(to=FAKE + 2) == L.QR_ERR_ALIGNMENT
    assert ev(s=seqs(batch=0, kv_lens=None, cu_q=None)) == L.QR_OK


def test_wrappers_refuse_host_tensors():
    side = (torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 1)), torch.zeros((4, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        Q.KVCache(side, side, 128)
    with pytest.raises(ValueError, match="CUDA"):
        Q.Rope(torch.ones(64))
