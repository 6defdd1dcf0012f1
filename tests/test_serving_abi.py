"""Refusals of the serving loop's entry points (no GPU: every call returns from the host
checks), and the oracle's plan and choice of tokens against hand-computed ones."""

import math

import numpy as np
import pytest

import oracle
from w4a16_decode_amd import _lib

FAKE = 0x100000  # a 16-byte-aligned non-NULL address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_plan_refusals(lib):
    def f(lens=FAKE, new=FAKE, reset=None, starts=None, seqs=3, tokens=5, page=16, pages=9, table=FAKE, blocks=4,
          free=FAKE, count=FAKE, off=FAKE, pos=FAKE, slots=FAKE, lens_out=FAKE, count_out=FAKE, lacking=FAKE, ws=None,
          size=0):
        return lib.q4_paged_plan(lens, new, reset, starts, seqs, tokens, page, pages, table, blocks, free, count, off, pos,
                                 slots, lens_out, count_out, lacking, ws, size, None)

    assert f(seqs=-1) == 2 and f(seqs=65537) == 2 and f(tokens=-1) == 2 and f(tokens=1 << 30) == 2
    assert f(page=8) == 2 and f(page=0) == 2 and f(page=-16) == 2
    assert f(pages=0) == 2 and f(pages=1 << 27) == 2                      # 2^31 slots
    assert f(blocks=-1) == 2 and f(blocks=(1 << 26) + 1) == 2             # above 2^30 tokens a sequence
    for name in ("lens", "table", "off", "pos", "slots", "lens_out", "lacking", "count", "count_out"):
        assert f(**{name: None}) == 1, name
        assert f(**{name: FAKE + 2}) == 4, name
    for name in ("new", "reset", "starts", "free"):
        assert f(**{name: FAKE + 1}) == 4, name
    need = lib.q4_paged_plan_workspace_bytes(3, 100000)
    assert need > 0 and lib.q4_paged_plan_workspace_bytes(3, 5) == 0
    assert f(tokens=100000) == 6 and f(tokens=100000, ws=FAKE, size=need - 1) == 6
    assert f(tokens=100000, ws=FAKE + 4, size=need) == 4
    assert lib.q4_paged_plan_workspace_bytes(-1, 5) == 0 and lib.q4_paged_plan_workspace_bytes(3, -5) == 0


def test_sample_refusals(lib):
    def f(x=FAKE, dtype=0, stride=100, rows=3, vocab=100, u=FAKE, t=None, k=None, p=None, m=None, out=FAKE, probs=None):
        need = lib.q4_sample_workspace_bytes(rows, vocab)
        return lib.q4_sample(x, dtype, stride, rows, vocab, u, t, k, p, m, out, probs, FAKE, need, None)

    assert f(dtype=3) == 5 and f(dtype=-1) == 5
    assert f(rows=-1) == 2 and f(rows=1 << 22) == 2 and f(vocab=0) == 2 and f(vocab=(1 << 20) + 1) == 2
    assert f(stride=-1) == 2 and f(stride=1 << 40) == 2
    assert f(rows=0, x=None, u=None, out=None) == 0
    assert f(x=None) == 1 and f(u=None) == 1 and f(out=None) == 1
    assert f(x=FAKE + 1) == 4 and f(x=FAKE + 2, dtype=2) == 4
    for name in ("u", "t", "k", "p", "m", "out", "probs"):
        assert f(**{name: FAKE + 2}) == 4, name
    for vocab in (16384, 16385, 32768, 32769, 128256):     # a workspace serves fewer rows
        sizes = [lib.q4_sample_workspace_bytes(rows, vocab) for rows in (0, 1, 31, 32, 33, 34, 500)]
        assert sizes == sorted(sizes) and (sizes[-1] > 0) == (vocab > 16384), (vocab, sizes)
    assert lib.q4_sample_workspace_bytes(-1, 5) == 0 and lib.q4_sample_workspace_bytes(5, 0) == 0


def test_wrappers_refuse_host_tensors():
    import torch

    import w4a16_decode_amd as q4

    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        q4.paged_plan(i, None, torch.zeros(2, 3, dtype=torch.int32), 16, 2, pages=4)
    with pytest.raises(ValueError):
        q4.paged_plan(i, None, i, 16, 2, pages=4)
    with pytest.raises(ValueError):
        q4.sample(torch.zeros(2, 10), torch.zeros(2))
    with pytest.raises(TypeError):
        q4.sample(np.zeros((2, 10)), torch.zeros(2))
    with pytest.raises(ValueError):
        q4.page_pool(0)


def test_oracle_plan():
    """Two sequences of 3 and 16 tokens on pages 5 and 6; the second needs a page, the stack's top is 7."""
    table = np.array([[5, -1, -1], [6, -1, -1]])
    free = np.array([9, 8, 7, 0])
    off, pos, slots, lens, tab, stack, count, lacking = oracle.serving.plan([3, 16], [2, 1], table, 16, 4, 10, free, 3,
                                                                           starts=[0, 100])
    assert off.tolist() == [0, 2, 3] and pos.tolist() == [3, 4, 116, 0]
    assert slots.tolist() == [5 * 16 + 3, 5 * 16 + 4, 7 * 16, -1]
    assert lens.tolist() == [5, 17] and tab.tolist() == [[5, -1, -1], [6, 7, -1]]
    assert count == 2 and lacking == 0 and stack.tolist() == free.tolist()
    # the first ends: its page 5 is pushed behind 7 and is the next one popped
    off, pos, slots, lens, tab, stack, count, lacking = oracle.serving.plan([3, 16], [0, 1], table, 16, 1, 10, free, 3,
                                                                           reset=[1, 0])
    assert stack.tolist() == [9, 8, 7, 5] and tab[1].tolist() == [6, 5, -1] and lens.tolist() == [0, 17] and count == 3
    # one page for 40 tokens: 16 are stored, two pages lack
    off, pos, slots, lens, tab, stack, count, lacking = oracle.serving.plan([0], [40], np.array([[-1, -1]]), 16, 40, 10,
                                                                           free, 1)
    assert lens.tolist() == [16] and lacking == 2 and count == 0 and (slots[16:] == -1).all() and slots[15] == 159


def test_oracle_sample():
    """w = 1, 2, 4, 1 (logits ln 1, ln 2, ln 4, ln 1)."""
    x = np.log([1.0, 2.0, 4.0, 1.0])
    f = oracle.serving.sample
    assert [f(x, u)[0] for u in (0.0, 0.124, 0.126, 0.374, 0.376, 0.874, 0.876, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert math.isclose(f(x, 0.5)[1], 0.5) and f(x, 0.5, temperature=0.0) == (2, 1.0)
    assert [f(x, u, top_k=3)[0] for u in (0.0, 0.15, 0.99)] == [0, 1, 2]       # of the equal ones the first stays
    assert [f(x, u, top_p=0.5)[0] for u in (0.0, 0.99)] == [2, 2]              # 4 of 8 is enough
    assert [f(x, u, top_p=0.51)[0] for u in (0.3, 0.4)] == [1, 2]
    assert [f(x, u, min_p=0.4)[0] for u in (0.3, 0.4)] == [1, 2]
    assert math.isclose(f(x, 0.9, temperature=0.5)[1], 16 / 22)
    assert f(np.array([-np.inf, np.nan]), 0.5) == (-1, 0.0)
    assert f(np.array([1.0, np.inf, 2.0, np.inf]), 0.6) == (3, 0.5)


def test_shared_attention_refusals(lib):
    import ctypes

    def cache(**kw):
        d = dict(codes=FAKE, scales=FAKE, pages=4, page_size=32, kv_heads=2, head_dim=128, group=128)
        d.update(kw)
        return ctypes.byref(_lib.PagedKV(d["codes"], d["scales"], d["codes"], d["scales"], d["pages"], d["page_size"],
                                         d["kv_heads"], d["head_dim"], d["group"]))

    def f(q=FAKE, qs=512, c=None, ptab=FAKE, pblocks=4, plens=FAKE, goff=FAKE, groups=2, tab=FAKE, blocks=4, off=FAKE,
          lens=FAKE, seqs=3, tokens=3, max_q=1, max_kv=100, max_gq=3, max_prefix=100, hq=4, scale=0.1, out=FAKE, ws=FAKE,
          size=1 << 40):
        return lib.q4_paged_attention_shared(q, qs, cache() if c is None else c, ptab, pblocks, plens, goff, groups, tab,
                                             blocks, off, lens, seqs, tokens, max_q, max_kv, max_gq, max_prefix, hq, scale,
                                             out, ws, size, None)

    for name in ("q", "ptab", "plens", "goff", "tab", "off", "lens", "out"):
        assert f(**{name: None}) == 1, name
        assert f(**{name: FAKE + 2}) == 4, name
    assert f(c=cache(codes=None)) == 1 and f(c=cache(page_size=8)) == 2 and f(c=cache(group=16)) == 3
    for name in ("pblocks", "groups", "blocks", "seqs", "tokens", "max_q", "max_kv", "max_gq", "max_prefix"):
        assert f(**{name: -1}) == 2 and f(**{name: 1 << 30}) == 2, name
    assert f(hq=3) == 2 and f(hq=0) == 2 and f(qs=504) == 2 and f(qs=516) == 4
    assert f(scale=2.1e38) == 2 and f(scale=float("nan")) == 2
    assert f(groups=1 << 22, max_gq=1 << 12, tokens=1 << 12) == 2          # too many jobs
    assert f(ws=None) == 6 and f(size=16) == 6 and f(ws=FAKE + 8) == 4
    assert f(seqs=0) == 0 and f(tokens=0) == 0 and f(max_q=0) == 0
    w = lib.q4_paged_attention_shared_workspace_bytes
    assert w(3, 2, 3, 1, 100, 3, 100, 4, 2, 128, 128) >= 3 * 4 * 130 * 4
    assert w(3, 0, 3, 1, 100, 3, 100, 4, 2, 128, 128) == 0 and w(3, -1, 3, 1, 100, 3, 100, 4, 2, 128, 128) == 0
    assert w(3, 2, 3, 1, 100, 3, 100, 4, 2, 96, 32) == 0 and w(3, 2, 3, 1, 100, 3, 100, 3, 2, 128, 128) == 0


def test_shared_attention_own_keys_grid(lib):
    """More than 256 rows of a group, own keys of 513 to 4096: a workgroup a sequence, tile and head over those, which
    are refused from 2^24 on (2^32 threads) before anything is launched."""
    import ctypes

    w = lib.q4_paged_attention_shared_workspace_bytes
    cache = ctypes.byref(_lib.PagedKV(FAKE, FAKE, FAKE, FAKE, 4, 32, 8, 128, 128))
    for seqs, max_q, max_kv, fits in ((1 << 21, 1, 1000, False), (1 << 21, 2, 4096, False), ((1 << 21) - 1, 2, 4096, True),
                                      (1 << 20, 3, 1000, True), (1 << 22, 1, 513, False), (1 << 21, 1, 4097, True)):
        need = w(seqs, 1, seqs, max_q, max_kv, 64, 100, 64, 8, 128, 128)
        assert (need > 0) == fits, (seqs, max_q, max_kv, need)
        # without a workspace no call gets as far as a launch: its sizes are refused (2), or its workspace (6)
        st = lib.q4_paged_attention_shared(FAKE, 8192, cache, FAKE, 4, FAKE, FAKE, 1, FAKE, 4, FAKE, FAKE, seqs, seqs, max_q,
                                           max_kv, 64, 100, 64, 0.1, FAKE, None, 0, None)
        assert st == (6 if fits else 2), (seqs, max_q, max_kv, st)


def test_shared_attention_line_grid(lib):
    """Whole jobs and the pieces of the cut ones together are one grid: 419430 sequences of up to 80 rows of 8 heads a KV
    head are 16777200 jobs, so that any cut among them (a tenth of a round's jobs at least, into two pieces or more)
    makes 2^24 workgroups or more, which are refused: no workspace. Without a cut none is needed."""
    w = lib.q4_paged_attention_shared_workspace_bytes
    seqs = 419430
    for tokens in range(1 << 24, (1 << 24) + 20000, 97):
        assert w(seqs, 1, tokens, 80, 2000, 90, 6000, 64, 8, 128, 128) == 0, tokens
    few = [w(1000, 1, tokens, 80, 2000, 90, 6000, 64, 8, 128, 128) for tokens in range(40000, 60000, 97)]
    assert any(n > 0 for n in few)


def test_shared_attention_mixed_batch(lib):
    """A chunk beside single tokens behind one prefix: the workspace holds what the group's rows have seen of the prefix,
    which is read once for all of them (and not cut jobs of sequences that read it each by itself)."""
    w = lib.q4_paged_attention_shared_workspace_bytes
    for chunks, new in ((1, 80), (1, 512), (4, 512), (8, 100)):
        tokens = chunks * new + 64 - chunks
        rows = 8 * 8 * tokens * 130 * 4
        need = w(64, 1, tokens, new, new + 300, tokens, 8190, 64, 8, 128, 128)
        assert rows <= need <= 3 * rows + (16 << 20), (chunks, new, need, rows)


def test_shared_attention_prompt_beside_a_group(lib):
    """A prompt in no group beside a few rows behind a prefix: no partial results of the prompt's rows for each piece of
    its keys (133 MB a piece here), only of what the last round of the chip is cut into."""
    w = lib.q4_paged_attention_shared_workspace_bytes
    need = w(9, 1, 4008, 4000, 4000, 8, 8190, 64, 8, 128, 128)
    assert 8 * 64 * 130 * 4 <= need < 4008 * 64 * 130 * 4


def test_shared_attention_loose_bounds(lib):
    """Long chunks of like sizes under a loose max_q stay lines of keys: at most a round's jobs are cut, and no partial
    results of all rows over the prefix are left. Long prompts outside the groups make no lines."""
    w = lib.q4_paged_attention_shared_workspace_bytes
    for new, max_q in ((300, 300), (300, 2400), (1500, 6000)):
        rows = 8 * 8 * 7 * new * 130 * 4
        assert w(7, 1, 7 * new, max_q, 100, 7 * new, 300, 64, 8, 128, 128) < rows, (new, max_q)
    rows = 8 * 8 * 40 * 130 * 4
    assert w(6, 1, 4 * 4000 + 40, 4000, 4000, 40, 300, 64, 8, 128, 128) >= rows


def test_oracle_shared_attention():
    """One row, prefix of one key, one key of its own: equal scores average the two; no key is zero."""
    q = np.zeros((3, 1, 2))
    pk, pv = [np.ones((1, 1, 2))], [np.full((1, 1, 2), 4.0)]
    k, v = [np.ones((1, 1, 2)), np.ones((0, 1, 2))], [np.full((1, 1, 2), 2.0), np.ones((0, 1, 2))]
    out = oracle.paged.attention_shared(q, pk, pv, [0, 1], k, v, [1, 0], [0, 2, 3], 1.0)
    assert out[:, 0].tolist() == [[4, 4], [3, 3], [0, 0]]                   # row 0 lies ahead of its sequence's start
