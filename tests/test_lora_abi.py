"""Refusals of the product with adapters (no GPU: every call returns from the host checks)."""

import pytest

from w4a16_decode_amd import _lib

FAKE = 0x100000  # a 16-byte-aligned non-NULL address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_refusals(lib):
    def f(x=FAKE, B=3, packed=FAKE, zeros=None, out=64, in_=256, g=128, a=FAKE, b=FAKE, s=FAKE, n=2, rank=16, ids=FAKE,
          y=FAKE, ws=FAKE, wsb=1 << 20):
        return lib.q4_gemm_lora(x, B, packed, FAKE, zeros, out, in_, g, a, b, s, n, rank, ids, y, ws, wsb, None)

    assert f(x=None) == 1 and f(a=None) == 1 and f(b=None) == 1 and f(s=None) == 1 and f(ids=None) == 1 and f(y=None) == 1
    assert f(B=-1) == 2 and f(out=0) == 2 and f(n=-1) == 2 and f(n=1 << 30) == 2
    assert f(g=96) == 3 and f(in_=200) == 3
    assert f(rank=0) == 5 and f(rank=12) == 5 and f(rank=136) == 5
    assert f(x=FAKE + 8) == 4 and f(a=FAKE + 8) == 4 and f(b=FAKE + 2) == 4 and f(ids=FAKE + 2) == 4 and f(ws=FAKE + 8) == 4
    assert f(ws=None) == 6
    assert f(wsb=lib.q4_workspace_bytes_lora(3, 64, 256, 128, 16) - 1) == 6
    assert f(B=0, x=None, ws=None) == 0


def test_workspace_sizes(lib):
    w = lib.q4_workspace_bytes_lora
    assert w(3, 64, 256, 128, 16) > 0
    assert w(0, 64, 256, 128, 16) == 0 and w(3, 64, 256, 96, 16) == 0 and w(3, 64, 256, 128, 12) == 0
    assert w(3, 64, 200, 128, 16) == 0


def test_rows_beyond_a_launch(lib):
    """2^24 workgroups and more are refused (16 rows, 16 adapters, 4 slices of 4096 channels each)."""
    most = ((1 << 24) - 1) // (16 * 4) * 16
    w = lib.q4_workspace_bytes_lora
    assert w(most, 64, 4096, 128, 16) > 0 and w(most + 1, 64, 4096, 128, 16) == 0
    f = lambda B: lib.q4_gemm_lora(FAKE, B, FAKE, FAKE, None, 64, 4096, 128, FAKE, FAKE, FAKE, 2, 16, FAKE, FAKE, None,
                                   0, None)
    assert f(most) == 6 and f(most + 1) == 2
