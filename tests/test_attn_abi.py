"""Refusals of the attention-side entry points (no GPU: every call returns from the
host checks), and the oracle's byte layout against hand-computed positions."""

import ctypes

import numpy as np
import pytest

import oracle
from w4a16_decode_amd import _lib

FAKE = 0x100000  # a 16-byte-aligned non-NULL address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _cache(codes=FAKE, scales=FAKE, pages=4, page_size=32, kv_heads=2, head_dim=128, group=128):
    return ctypes.byref(_lib.PagedKV(codes, scales, codes, scales, pages, page_size, kv_heads, head_dim, group))


def test_paged_sizes(lib):
    assert lib.q4_paged_codes_bytes(4, 32, 2, 128) == 4 * 32 * 2 * 64
    assert lib.q4_paged_scales_count(4, 32, 2, 128, 64) == 4 * 32 * 2 * 2
    assert lib.q4_paged_codes_bytes(0, 32, 2, 128) == 0
    assert lib.q4_paged_codes_bytes(4, 24, 2, 128) == 0                  # page_size % 16
    assert lib.q4_paged_codes_bytes(4, 32, 2, 96) == 0                   # head_dim
    assert lib.q4_paged_scales_count(4, 32, 2, 64, 128) == 0             # head_dim % group
    assert lib.q4_paged_codes_bytes(1 << 27, 16, 2, 128) == 0            # 2^31 slots
    assert b"2^31" in lib.q4_last_error()


def test_cache_refusals(lib):
    def f(cache, slots=FAKE, n=3, k=FAKE, ks=256):
        return lib.q4_paged_kv_append(k, ks, FAKE, 256, n, cache, slots, None)

    assert f(None) == 1
    assert f(_cache(codes=None)) == 1
    assert f(_cache(), slots=None) == 1
    assert f(_cache(), k=None) == 1
    assert f(_cache(page_size=8)) == 2
    assert f(_cache(pages=0)) == 2
    assert f(_cache(kv_heads=0)) == 2
    assert f(_cache(head_dim=80)) == 5
    assert f(_cache(group=16)) == 3
    assert f(_cache(head_dim=64, group=128)) == 3
    assert f(_cache(codes=FAKE + 8)) == 4
    assert f(_cache(scales=FAKE + 2)) == 4
    assert f(_cache(), n=-1) == 2
    assert f(_cache(), ks=255) == 2                                       # rows would overlap
    assert f(_cache(), ks=260) == 4                                       # not a multiple of 8
    assert f(_cache(), k=FAKE + 2) == 4
    assert f(_cache(), slots=FAKE + 2) == 4
    assert f(_cache(), n=0) == 0
    d = lib.q4_paged_kv_dequant
    assert d(_cache(), FAKE, -1, FAKE, FAKE, None) == 2
    assert d(_cache(), FAKE, 0, None, None, None) == 0
    assert d(_cache(), None, 1, FAKE, FAKE, None) == 1
    assert d(_cache(), FAKE, 1, FAKE + 8, FAKE, None) == 4


def test_norm_rope_refusals(lib):
    def f(q=FAKE, qs=512, k=FAKE, ks=256, n=3, hq=4, hk=2, d=128, qw=None, eps=1e-6, pos=FAKE, table=FAKE, rows=10,
          rot=128, qo=FAKE, qos=512, ko=FAKE, kos=256):
        return lib.q4_qk_norm_rope(q, qs, k, ks, n, hq, hk, d, qw, None, eps, pos, table, rows, rot, 0, qo, qos, ko, kos,
                                   None)

    assert f(q=None) == 1 and f(ko=None) == 1 and f(pos=None) == 1
    assert f(d=96) == 5
    assert f(rot=24) == 5 and f(rot=144) == 5 and f(rot=-16) == 5
    assert f(rows=0) == 2 and f(n=-1) == 2 and f(hq=-1) == 2
    assert f(qs=504) == 2 and f(kos=255) == 2
    assert f(qs=516) == 4 and f(qo=FAKE + 8) == 4 and f(qw=FAKE + 8) == 4 and f(table=FAKE + 8) == 4
    assert f(qw=FAKE, eps=-1.0) == 2 and f(qw=FAKE, eps=float("nan")) == 2
    assert f(n=0, q=None) == 0 and f(hq=0, hk=0, q=None) == 0
    t = lib.q4_rope_table
    assert t(-1, 64, 1e4, FAKE, None) == 2
    assert t(4, 24, 1e4, FAKE, None) == 5
    assert t(4, 64, 0.0, FAKE, None) == 2 and t(4, 64, float("nan"), FAKE, None) == 2
    assert t(4, 64, 1e4, None, None) == 1
    assert t(4, 64, 1e4, FAKE + 8, None) == 4
    assert t(0, 64, 1e4, None, None) == 0


def test_oracle_tile_positions():
    """Single codes at byte positions worked out from the written layout by hand."""
    for d, tok, ch, is_v, byte, shift in [
        (128, 0, 0, False, 0, 0),              # first dword, nibble 0
        (128, 5, 41, False, 4 * ((5 + 16) * 4 + 1) + 2, 0),      # m = 1, c = 1, e = 1 -> nibble 4
        (64, 3, 63, False, 4 * ((3 + 48) * 2 + 1) + 3, 4),       # m = 1, c = 3, e = 7 -> nibble 7
        (256, 1, 130, False, 4 * ((64 + 1) * 4) + 0, 4),         # m = 4: second half, e = 2 -> nibble 1
        (128, 0, 0, True, 0, 0),
        (128, 6, 53, True, 4 * ((5 + 16) * 4 + 1) + 1, 4),       # t % 4 = 2 -> byte 1, n = 1
        (64, 13, 40, True, 4 * ((8 + 48) * 2 + 1) + 2, 0),       # t % 4 = 1 -> byte 2
    ]:
        codes = np.full((16, d), -8)
        codes[tok, ch] = 5                                        # 13 = 0xD; all others 0
        got = oracle.paged.tile_bytes(codes, is_v)
        assert got.size == 8 * d and np.count_nonzero(got) == 1
        assert got[byte] == 0xD << shift, (d, tok, ch, is_v)


def test_oracle_norm_rope_closed_forms():
    """A quarter turn swaps a pair with a sign; a unit weight gives unit mean square."""
    x = np.arange(1, 17, dtype=np.float16).reshape(1, 1, 16)
    zero, one = np.zeros((1, 4)), np.ones((1, 4))
    y = oracle.paged.norm_rope(x, cos=zero, sin=one)
    assert np.array_equal(y[0, 0], [-5, -6, -7, -8, 1, 2, 3, 4, *range(9, 17)])
    y = oracle.paged.norm_rope(x, cos=zero, sin=one, interleaved=True)
    assert np.array_equal(y[0, 0, :8], [-2, 1, -4, 3, -6, 5, -8, 7])
    y = oracle.paged.norm_rope(x, np.ones(16, np.float16), 0.0)
    assert abs(np.mean(y * y) - 1) < 1e-12


def test_oracle_attention_closed_forms():
    """Equal scores average the values that are seen; a window of one returns its value."""
    k = [np.zeros((5, 1, 16))]
    v = [np.arange(5.0)[:, None, None] * np.ones((1, 1, 16))]
    q = np.ones((3, 2, 16))
    y = oracle.paged.attention(q, k, v, [5], [0, 2], 1.0)
    assert np.allclose(y[0], 1.5) and np.allclose(y[1], 2.0) and np.all(np.isnan(y[2]))
    y = oracle.paged.attention(q, k, v, [5], [0, 2], 1.0, window=1)
    assert np.allclose(y[0], 3) and np.allclose(y[1], 4)
    y = oracle.paged.attention(q, [k[0][:1]], [v[0][:1]], [1], [0, 2], 1.0)
    assert np.all(y[0] == 0) and np.allclose(y[1], 0)


def test_attention_refusals(lib):
    def f(q=FAKE, qs=1024, cache=None, tab=FAKE, mb=4, off=FAKE, lens=FAKE, seqs=2, n=3, mq=2, mkv=100, hq=8, scale=0.1,
          window=0, out=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.q4_paged_attention(q, qs, cache or _cache(), tab, mb, off, lens, seqs, n, mq, mkv, hq, scale, window,
                                      out, ws, wsb, None)

    assert f(q=None) == 1 and f(tab=None) == 1 and f(off=None) == 1 and f(lens=None) == 1 and f(out=None) == 1
    assert f(hq=7) == 2 and f(hq=0) == 2 and f(seqs=-1) == 2 and f(n=-1) == 2 and f(mq=-1) == 2 and f(mkv=-1) == 2
    assert f(window=-1) == 2 and f(scale=float("inf")) == 2 and f(mb=-1) == 2
    assert f(seqs=1 << 25, n=1 << 28, mq=1 << 20) == 2
    assert f(qs=1000) == 2 and f(qs=1028) == 4 and f(q=FAKE + 8) == 4 and f(out=FAKE + 4) == 4 and f(off=FAKE + 2) == 4
    assert f(cache=_cache(page_size=20)) == 2 and f(cache=_cache(codes=None)) == 1
    assert f(seqs=0, q=None) == 0 and f(n=0, q=None) == 0 and f(mq=0, q=None) == 0


def test_rows_beyond_a_launch(lib):
    """A launch of 2^24 workgroups or more is refused: 4 tokens each of the norm and rotation, 16 rows
    or one sequence's head of an attention over short contexts."""
    f = lib.q4_qk_norm_rope
    for n, st in ((1 << 26) - 3, 2), ((1 << 26) - 4, 1):
        assert f(None, 512, None, 256, n, 4, 2, 128, None, None, 0.0, FAKE, FAKE, 10, 128, 0, FAKE, 512, FAKE, 256,
                 None) == st
    w = lib.q4_paged_attention_workspace_bytes
    for seqs, st in (1 << 21, 2), ((1 << 21) - 1, 1):
        assert w(seqs, seqs, 1, 512, 8, 8, 128, 128, 0) == 0
        assert lib.q4_paged_attention(None if st == 1 else FAKE, 1024, _cache(kv_heads=8), FAKE, 4, FAKE, FAKE, seqs, seqs,
                                      1, 512, 8, 0.1, 0, FAKE, None, 0, None) == st


def test_scale_limits(lib):
    f = lambda scale: lib.q4_paged_attention(None, 1024, _cache(), FAKE, 4, FAKE, FAKE, 2, 3, 2, 100, 8, scale, 0, FAKE,
                                             None, 0, None)
    assert f(2.5e38) == 2 and f(-2.5e38) == 2 and f(float("nan")) == 2
    assert f(1.9e38) == 1 and f(-1.9e38) == 1 and f(0.0) == 1                          # q is NULL


def test_rope_table_needs_a_gpu():
    """A table is filled on a GPU: a host device is refused before any launch."""
    from w4a16_decode_amd import rope_table

    for device in ("cpu", "meta"):
        with pytest.raises(ValueError, match="GPU"):
            rope_table(4, 64, device=device)


def test_copies_of_a_cache_drop_what_calls_keep(monkeypatch):
    """What a cache keeps for its calls (addresses in a C structure) stays behind in copies and pickles."""
    import copy
    import pickle

    import torch

    from w4a16_decode_amd import PagedKVCache4

    monkeypatch.setattr(PagedKVCache4, "_check", lambda self: None)
    codes, scales = torch.zeros((2, 1, 1024), dtype=torch.uint8), torch.zeros((2, 1, 16), dtype=torch.float16)
    cache = PagedKVCache4(codes, scales, codes.clone(), scales.clone(), 16, 128, 128)
    cache._c()
    assert cache._struct is not None
    for other in (copy.copy(cache), copy.deepcopy(cache), pickle.loads(pickle.dumps(cache))):
        assert other._struct is None and other.pages == 2 and other.page_size == 16
        assert torch.equal(other.k_codes, codes) and other._c()[0][0] == other.k_codes.data_ptr()
    assert cache._struct is not None
