"""Attention over the paged INT4 cache against the oracle in float64.

Bound of an output's error, from the arithmetic. With A = sum_t p_t |v_t| (p the exact
softmax), Z = max_t sum_c |q_c k_tc| * scale:
 - each weight, times its V scale, is rounded to float16: 2^-11 A;
 - a score is a float32 dot product of D / 32 matrix steps plus the scaling, the
   subtraction of the maximum and the exponential: (D / 32 + 8) roundings of 2^-23
   relative to Z + 1, which changes a weight by that much of itself, and the sum of
   the weights by no more: 2 (D / 32 + 8) 2^-23 (Z + 1) A;
 - float32 sums over n keys in steps of 32 and up to a few hundred joins: (n / 32 + 32)
   2^-24 A twice;
 - the result is rounded to float16: 2^-11 |o| (subnormal: 2^-25).
"""

import numpy as np
import pytest

import oracle
from gpu_util import say, to_gpu, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import w4a16_decode_amd as q4mod

    say("libq4", q4mod.version())
    return q4mod


class Batch:
    """Sequences with their keys in a paged cache; every slot that no length covers, and
    every unused page, holds random codes and NaN scales."""

    def __init__(self, q4, lens, news, hq, hkv, d, g, page, seed=0, spread=1.0, extra_rows=0, v_scale=1.0):
        import torch

        r = np.random.default_rng(seed)
        self.q4, self.lens, self.page, self.d = q4, list(lens), page, d
        self.offsets = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        blocks = max(1, max(-(-n // page) for n in lens))
        pages = len(lens) * blocks + 3
        self.table = r.permutation(pages)[:len(lens) * blocks].reshape(len(lens), blocks).astype(np.int32)
        rows = int(self.offsets[-1]) + extra_rows
        self.q = (spread * r.standard_normal((rows, hq, d))).astype(np.float16)
        self.cache = q4.paged_kv_alloc(pages, page, hkv, d, g)
        for t in (self.cache.k_codes, self.cache.v_codes):
            t.copy_(torch.randint(0, 256, t.shape, dtype=torch.uint8))
        for t in (self.cache.k_scales, self.cache.v_scales):
            t.fill_(float("nan"))
        self.k, self.v, self.k16, self.v16 = [], [], [], []
        for n, length in enumerate(lens):
            k16 = (r.standard_normal((length, hkv, d)) * np.exp(0.4 * r.standard_normal((1, hkv, d)))).astype(np.float16)
            v16 = (v_scale * r.standard_normal((length, hkv, d))).astype(np.float16)
            self.k16.append(k16), self.v16.append(v16)
            self.k.append(oracle.paged.store(k16, g)[2] if length else np.zeros((0, hkv, d)))
            self.v.append(oracle.paged.store(v16, g)[2] if length else np.zeros((0, hkv, d)))
            if length:
                self.put(n, k16, v16)

    def slots(self, n, length):
        t = np.arange(length)
        return (self.table[n][t // self.page] * self.page + t % self.page).astype(np.int32)

    def put(self, n, k16, v16):
        self.q4.paged_kv_append(to_gpu(k16), to_gpu(v16), self.cache, to_gpu(self.slots(n, len(k16))))

    def run(self, window=0, scale=None, table=None, **kw):
        news = np.diff(self.offsets)
        args = dict(max_q=int(news.max()), max_kv=max(self.lens))
        args.update(kw)
        q = args.pop("q", None)
        out = self.q4.paged_attention(to_gpu(self.q) if q is None else q, self.cache,
                                      to_gpu(self.table if table is None else table), to_gpu(self.offsets),
                                      to_gpu(np.array(self.lens, np.int32)), window=window, scale=scale, **args)
        return out

    def check(self, got, window=0, scale=None, what="", heads=None):
        """`heads`: the query heads to look at (all by default)."""
        if heads is not None:
            worst, share = 0.0, self.q.shape[1] // self.k[0].shape[1]
            for h in heads:
                one = Batch.__new__(Batch)
                one.lens, one.offsets, one.d, one.q = self.lens, self.offsets, self.d, self.q[:, h:h + 1]
                one.k, one.v = ([t[:, h // share:h // share + 1] for t in kv] for kv in (self.k, self.v))
                worst = max(worst, one.check(got[:, h:h + 1], window, scale, (what, h)))
            return worst
        s = self.d ** -0.5 if scale is None else scale
        got = to_np(got).astype(np.float64)
        worst = 0.0
        for n, length in enumerate(self.lens):
            a, b = self.offsets[n], self.offsets[n + 1]
            if a == b:
                continue
            share = self.q.shape[1] // self.k[n].shape[1]
            off = [0, b - a]
            ref = oracle.paged.attention(self.q[a:b], [self.k[n]], [self.v[n]], [length], off, s, window)
            mag = oracle.paged.attention(self.q[a:b], [self.k[n]], [np.abs(self.v[n])], [length], off, s, window)
            z = 1.0
            if length:
                kk = np.abs(self.k[n]).max(axis=0)
                z += np.abs(s) * (np.abs(self.q[a:b].astype(np.float64)) * np.repeat(kk, share, axis=0)).sum(-1).max()
            rel = 2.0 ** -11 + 2 * (self.d / 32 + 8) * 2.0 ** -23 * z + 2 * (length / 32 + 32) * 2.0 ** -24
            bound = rel * mag + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
            err = np.abs(got[a:b] - ref)
            assert np.all(np.isfinite(got[a:b])), (what, n)
            assert np.all(err <= bound), (what, n, length, (err / bound).max())
            worst = max(worst, (err / bound).max())
        return worst


SHAPES = [  # hq, hkv, d, g, page
    (8, 1, 128, 128, 16),
    (4, 4, 64, 64, 16),
    (14, 2, 128, 64, 48),
    (6, 2, 256, 128, 32),
    (16, 2, 64, 32, 64),
    (8, 1, 128, 32, 32),
    (3, 1, 256, 32, 16),
    (20, 1, 256, 64, 16),
]


@pytest.mark.parametrize("hq,hkv,d,g,page", SHAPES)
def test_decode(q4, hq, hkv, d, g, page):
    """One row a sequence, lengths around every tile, step and page border."""
    say("decode", hq, hkv, d, g, page)
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 200, 1000]
    b = Batch(q4, lens, [1] * len(lens), hq, hkv, d, g, page, seed=d + g)
    say("  worst share of the bound", b.check(b.run()))
    say("  window 16", b.check(b.run(window=16), window=16))


@pytest.mark.parametrize("hq,hkv,d,g,page", SHAPES)
def test_chunks(q4, hq, hkv, d, g, page):
    """Prompts, chunks over a context, single rows, and sequences without rows, in one call."""
    say("chunks", hq, hkv, d, g, page)
    lens, news = [40, 300, 77, 5, 130, 64, 97], [40, 33, 1, 0, 129, 2, 64]
    b = Batch(q4, lens, news, hq, hkv, d, g, page, seed=d + g + 1)
    say("  worst share of the bound", b.check(b.run()))
    say("  window 33", b.check(b.run(window=33), window=33))
    say("  window 1", b.check(b.run(window=1), window=1))


@pytest.mark.parametrize("new", [1, 3, 70])
def test_long_context(q4, new):
    b = Batch(q4, [9001, 4500], [new, new], 8, 2, 128, 128, 32, seed=new)
    say("long context", new, b.check(b.run()))
    say("  bounds larger than the lengths", b.check(b.run(max_q=new + 5, max_kv=20000)))


def test_large_scores_and_small_values(q4):
    """A softmax close to one-hot, and V scales among float16's subnormals: the weights
    keep their precision."""
    b = Batch(q4, [500, 70], [4, 4], 8, 2, 128, 64, 16, seed=5, spread=30.0)
    say("sharp", b.check(b.run()))
    b = Batch(q4, [700], [3], 8, 2, 128, 128, 16, seed=6, v_scale=2.0 ** -13)
    say("small v", b.check(b.run()))
    b = Batch(q4, [700], [3], 8, 2, 128, 128, 16, seed=6, v_scale=4000.0)
    say("large v", b.check(b.run()))
    b = Batch(q4, [300], [3], 8, 2, 128, 128, 16, seed=7)
    say("negative scale", b.check(b.run(scale=-0.3), scale=-0.3))
    b.check(b.run(scale=0.0), scale=0.0)


def test_rows_that_see_nothing_and_rows_of_no_sequence(q4):
    """Empty sequences and rows ahead of a sequence's start are zero; rows behind the last
    sequence keep their contents."""
    import torch

    b = Batch(q4, [0, 3, 20], [2, 8, 1], 8, 2, 128, 128, 16, seed=8, extra_rows=5)
    out = torch.full((16, 8, 128), 3.0, dtype=torch.float16, device="cuda")
    b.run(out=out)
    b.check(out)
    got = to_np(out)
    assert not got[:2].any() and not got[2:7].any()          # length 0; rows ahead of a length of 3
    assert np.all(got[11:] == 3.0)
    b = Batch(q4, [0, 0], [1, 1], 8, 2, 128, 128, 16, seed=9)
    assert not to_np(b.run()).any()
    assert not to_np(b.run(max_kv=64)).any()


def test_hidden_infinities(q4):
    """A new token's K and V hold infinities (their groups' scales are infinite): rows that do not
    see it are as without it, in the same tile too."""
    b = Batch(q4, [40], [10], 8, 2, 128, 128, 16, seed=10)
    clean = to_np(b.run())
    k16, v16 = b.k16[0].copy(), b.v16[0].copy()
    k16[36:, :, 3] = np.inf
    v16[36:, :, 5] = -np.inf
    b.put(0, k16, v16)
    got = to_np(b.run())
    assert np.array_equal(got[:6].view(np.uint16), clean[:6].view(np.uint16))
    assert not np.isfinite(got[6:]).any()


def test_pages_outside_the_cache(q4):
    """Keys of a bad page number are hidden; entries behind the length may hold anything."""
    b = Batch(q4, [100, 40], [2, 1], 8, 2, 128, 64, 16, seed=11)
    table = b.table.copy()
    table[1, 3:] = [-7, 2 ** 31 - 1, b.cache.pages, -1][:table.shape[1] - 3]
    assert np.array_equal(to_np(b.run(table=table)), to_np(b.run()))
    table[0, 2] = b.cache.pages
    table[0, 4] = -1
    got = b.run(table=table)
    keep = np.array([t for t in range(100) if t // 16 not in (2, 4)])
    c = Batch(q4, [100], [2], 8, 2, 128, 64, 16, seed=11)
    for i in range(2):          # row i of the two newest tokens: neither sits on a bad page
        seen = keep[keep <= 98 + i]
        c.lens, c.offsets, c.q = [len(seen)], np.array([0, 1]), b.q[i:i + 1]
        c.k, c.v = [b.k[0][seen]], [b.v[0][seen]]
        c.check(got[i:i + 1], what="bad page")


def test_lengths_cut_to_the_bounds(q4):
    """Lengths beyond max_kv or the table, offsets beyond the rows: cut, in bounds."""
    import torch

    b = Batch(q4, [48, 48], [1, 1], 8, 2, 128, 128, 16, seed=12)
    lens = to_gpu(np.array([48, 2 ** 31 - 1], np.int32))
    args = (to_gpu(b.q), b.cache, to_gpu(b.table))
    got = q4.paged_attention(*args, to_gpu(b.offsets), lens, 1, 48)
    assert torch.equal(got, b.run())
    got = q4.paged_attention(*args, to_gpu(b.offsets), to_gpu(np.array([48, -3], np.int32)), 1, 48)
    assert torch.equal(got[0], b.run()[0]) and not got[1].any()
    out = torch.full((2, 8, 128), 5.0, dtype=torch.float16, device="cuda")
    q4.paged_attention(*args, to_gpu(np.array([0, 2 ** 31 - 1, -4], np.int32)), lens, 2, 48, out=out)
    torch.cuda.synchronize()


def test_shared_pages_strided_queries_and_order(q4):
    """Two sequences on the same pages; q as slices of fused rows; batch order does not matter."""
    import torch

    b = Batch(q4, [150, 90], [1, 30], 8, 2, 128, 128, 16, seed=13)
    ref = b.run()
    wide = torch.zeros((31, 12, 128), dtype=torch.float16, device="cuda")
    wide[:, :8] = to_gpu(b.q)
    assert torch.equal(b.run(q=wide[:, :8]), ref)
    twice = q4.paged_attention(to_gpu(np.concatenate([b.q[:1], b.q[:1]])), b.cache, to_gpu(b.table[[0, 0]]),
                               to_gpu(np.array([0, 1, 2], np.int32)), to_gpu(np.array([150, 150], np.int32)), 1, 150)
    assert torch.equal(twice[0], twice[1])
    assert torch.equal(b.run(), ref)                          # the same bits again


def test_empty_calls(q4):
    import torch

    b = Batch(q4, [20], [1], 8, 2, 128, 128, 16, seed=14)
    e = torch.zeros((0, 8, 128), dtype=torch.float16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    assert q4.paged_attention(e, b.cache, torch.zeros((0, 4), **i32), torch.zeros(1, **i32), torch.zeros(0, **i32), 1,
                              8).shape == (0, 8, 128)
    out = torch.full((1, 8, 128), 2.0, dtype=torch.float16, device="cuda")
    q4.paged_attention(to_gpu(b.q), b.cache, torch.zeros((1, 0), **i32), to_gpu(b.offsets), torch.zeros(1, **i32), 1, 0,
                       out=out)
    assert not out.any()


def test_refusals(q4):
    import torch

    b = Batch(q4, [20], [1], 8, 2, 128, 128, 16, seed=15)
    q, tab, off, lens = to_gpu(b.q), to_gpu(b.table), to_gpu(b.offsets), to_gpu(np.array([20], np.int32))
    with pytest.raises(TypeError):
        q4.paged_attention(q.float(), b.cache, tab, off, lens, 1, 20)
    with pytest.raises(ValueError):
        q4.paged_attention(q[..., :64], b.cache, tab, off, lens, 1, 20)
    with pytest.raises(TypeError):
        q4.paged_attention(q, b.cache, tab.long(), off, lens, 1, 20)
    with pytest.raises(ValueError):
        q4.paged_attention(q, b.cache, tab, off[:1], lens, 1, 20)
    with pytest.raises(q4.Q4Error):
        q4.paged_attention(q[:, :7], b.cache, tab, off, lens, 1, 20)          # 7 heads over 2
    with pytest.raises(q4.Q4Error):
        q4.paged_attention(q, b.cache, tab, off, lens, 1, 20, window=-1)
    with pytest.raises(q4.Q4Error):
        q4.paged_attention(q, b.cache, tab, off, lens, 1, 20, scale=float("nan"))
    with pytest.raises(ValueError):
        q4.paged_attention(q, b.cache, tab, off, lens, 1, 20, out=torch.empty_like(q)[:, :4])


@pytest.mark.parametrize("d,g,page", [(64, 32, 16), (64, 64, 48), (128, 128, 32), (128, 64, 16), (128, 32, 64),
                                      (256, 128, 16), (256, 64, 32), (256, 32, 48)])
def test_many_rows(q4, d, g, page):
    """Enough rows and heads that tiles of 128 rows fill the chip: chunks over contexts, a prompt, a
    ragged last tile, a sequence without rows, windows."""
    say("many rows", d, g, page)
    lens, news = [193, 700, 260, 9, 450], [193, 150, 199, 0, 1]
    b = Batch(q4, lens, news, 64, 32, d, g, page, seed=d + 3 * g, extra_rows=3)
    heads = [0, 1, 33, 63]
    say("  worst share of the bound", b.check(b.run(), heads=heads))
    say("  window 70", b.check(b.run(window=70), window=70, heads=heads))
    say("  window 1", b.check(b.run(window=1), window=1, heads=[5]))


def test_many_rows_hidden(q4):
    """Hidden infinities, bad pages and rows that see nothing, in tiles of 128 rows."""
    lens, news = [220, 30, 300, 210, 0], [200, 60, 250, 199, 5]
    b = Batch(q4, lens, news, 64, 32, 128, 128, 16, seed=31)
    clean = to_np(b.run())
    b.check(clean_t := b.run(), heads=[2, 40])
    assert np.array_equal(to_np(clean_t).view(np.uint16), clean.view(np.uint16))
    assert not clean[200:230].any() and not clean[-5:].any()
    k16, v16 = b.k16[0].copy(), b.v16[0].copy()
    k16[150:, :, 3], v16[150:, :, 5] = np.inf, -np.inf
    b.put(0, k16, v16)
    got = to_np(b.run())
    assert np.array_equal(got[:130].view(np.uint16), clean[:130].view(np.uint16))     # positions 20 .. 149
    assert not np.isfinite(got[130:200]).any()
    assert np.array_equal(got[200:].view(np.uint16), clean[200:].view(np.uint16))
    b.put(0, b.k16[0], b.v16[0])
    table = b.table.copy()
    table[3, 2] = b.cache.pages + 5
    got = to_np(b.run(table=table)).astype(np.float64)
    keep = np.array([t for t in range(210) if t // 16 != 2])
    first = int(b.offsets[3])
    for i in (0, 60, 120, 198):
        pos = 210 - 199 + i
        if pos // 16 == 2:
            continue
        seen = keep[keep <= pos]
        ref = oracle.paged.attention(b.q[first + i:first + i + 1, :1], [b.k[3][seen][:, :1]], [b.v[3][seen][:, :1]],
                                     [len(seen)], [0, 1], 128 ** -0.5)
        assert np.abs(got[first + i, 0] - ref[0, 0]).max() <= 2.0 ** -9 * max(1.0, np.abs(ref).max())


def test_many_rows_sharp(q4):
    b = Batch(q4, [400, 300], [200, 200], 128, 64, 64, 32, 16, seed=33, spread=20.0, v_scale=2.0 ** -12)
    say("sharp, small v", b.check(b.run(), heads=[0, 77]))


@pytest.mark.parametrize("d,g,page", [(64, 32, 16), (64, 64, 48), (128, 128, 32), (128, 64, 16), (128, 32, 64),
                                      (256, 128, 16), (256, 32, 48)])
def test_many_rows_cut(q4, d, g, page):
    """Jobs of 128 rows left over after whole rounds of the chip, their keys cut into pieces: long and
    short sequences, pieces without keys, a window, hidden infinities, a workspace of garbage."""
    import torch

    say("many rows, cut", d, g, page)
    lens, news = [193, 9, 0, 450, 3900], [193, 3, 0, 140, 199]
    b = Batch(q4, lens, news, 64, 32, d, g, page, seed=d + 5 * g, extra_rows=1000)
    rows = b.q.shape[0]
    heads = [0, 33, 62, 63]

    def bound(window):
        """max_q with which the launch is cut (the bounds may exceed the lengths), and its workspace."""
        for mq in range(199, rows, 32):
            need = q4.paged_attention_workspace_bytes(5, rows, mq, 8190, 64, 32, d, g, window)
            if need:
                return mq, need
        raise AssertionError("no bound cuts a job")

    for window in (0, 3300):
        mq, need = bound(window)
        ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        got = b.run(window=window, max_q=mq, max_kv=8190, workspace=ws)
        say("  window", window, "max_q", mq, "worst share of the bound", b.check(got, window=window, heads=heads))
        assert bool((ws[need:] == 0xFF).all())
        again = b.run(window=window, max_q=mq, max_kv=8190)
        assert torch.equal(got[:int(b.offsets[-1])], again[:int(b.offsets[-1])])
    mq, need = bound(0)
    with pytest.raises(q4.Q4Error):
        b.run(max_q=mq, max_kv=8190, workspace=ws[:need - 16])
    first = int(b.offsets[4])
    before = to_np(b.run(max_q=mq, max_kv=8190))[first:first + 199]
    k16, v16 = b.k16[4].copy(), b.v16[4].copy()
    k16[3800:, :, 3], v16[3800:, :, 5] = np.inf, -np.inf
    b.put(4, k16, v16)
    after = to_np(b.run(max_q=mq, max_kv=8190))[first:first + 199]
    # Positions 3701 .. 3799 see none of it. Hidden V scales may still move the power of two that a
    # workgroup's weights carry, and the exponents x - base (below 2^6 in size) round to 2^-24 of
    # themselves: a weight moves by 2^-18 at most, and so by a whole float16 step, 2^-10, where that
    # crosses a border. The weighted mean then moves by 2^-10 of the largest |v|, its rounding
    # by another 2^-10.
    top = np.repeat(np.abs(b.v[4]).max(axis=0), 2, axis=0)
    assert np.all(np.abs(after[:99].astype(np.float64) - before[:99]) <= 2.0 ** -9 * top)
    assert not np.isfinite(after[99:]).all(axis=-1).any()


@pytest.mark.parametrize("scale", [0.0, -0.11, 1e-30])
def test_scales_of_any_sign(q4, scale):
    """Zero (the mean of what is seen), negative and tiny scales, in 16-, 32- and 128-row tiles."""
    for lens, news, hq, hkv in (([700, 40], [1, 1], 8, 2), ([600, 90], [5, 9], 16, 2), ([400, 150], [260, 129], 64, 64)):
        b = Batch(q4, lens, news, hq, hkv, 128, 128, 32, seed=41)
        say("scale", scale, news, "worst share of the bound", b.check(b.run(scale=scale), scale=scale, heads=[0, hq - 1]))


def test_many_rows_cut_captured(q4):
    """Cut jobs in a graph, replayed with other queries and lengths beside eager work."""
    import torch

    b = Batch(q4, [193, 9, 0, 450, 2100], [193, 3, 0, 140, 199], 64, 32, 128, 128, 32, seed=51, extra_rows=1000)
    rows = b.q.shape[0]
    mq = next(m for m in range(199, rows, 32)
              if q4.paged_attention_workspace_bytes(5, rows, m, 8190, 64, 32, 128, 128, 0))
    ws = torch.empty(q4.paged_attention_workspace_bytes(5, rows, mq, 8190, 64, 32, 128, 128, 0), dtype=torch.uint8,
                     device="cuda")
    q, lens = to_gpu(b.q), to_gpu(np.array(b.lens, np.int32))
    table, offsets, out = to_gpu(b.table), to_gpu(b.offsets), torch.zeros_like(to_gpu(b.q))

    def call(out, ws=None):
        return q4.paged_attention(q, b.cache, table, offsets, lens, mq, 8190, out=out, workspace=ws)

    call(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for i in range(4):
        q.copy_(to_gpu(np.roll(b.q, i, axis=0)))
        lens[4] = 2100 - 300 * i
        want = call(torch.zeros_like(out))
        out.zero_()
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def _quiet_channels(b, g, large):
    """K with codes of zero in half the channels, where q is large and of one sign: the scores come from the
    other half, small next to what q adds up to."""
    r = np.random.default_rng(61)
    loud = np.arange(b.d) % 4 < 2
    b.q = np.where(loud, large + r.standard_normal(b.q.shape), 0.5 * r.standard_normal(b.q.shape)).astype(np.float16)
    for n, k16 in enumerate(b.k16):
        k16[:, :, loud] *= np.float16(2.0 ** -12)
        b.k[n] = oracle.paged.store(k16, g)[2]
        assert not b.k[n][:, :, loud].any()
        b.put(n, k16, b.v16[n])


@pytest.mark.parametrize("d,g", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 128), (256, 32)])
@pytest.mark.parametrize("form", [16, 32, 128])
def test_scores_small_next_to_q(q4, form, d, g):
    """Scores that are small next to the sum of q, in tiles of 16, 32 and 128 rows: codes must enter the
    products exactly, without an offset that is taken off again."""
    hq, hkv, lens, news = {16: (8, 1, [4, 64, 2000], [1, 1, 1]), 32: (8, 1, [4, 64, 2000], [3, 3, 3]),
                           128: (64, 32, [200, 264, 2000, 199], [200, 200, 160, 199])}[form]
    for large in (3.0, 60.0, 1000.0):
        b = Batch(q4, lens, news, hq, hkv, d, g, 32, seed=d + g)
        _quiet_channels(b, g, large)
        say("quiet channels", form, d, g, large, "worst share of the bound", b.check(b.run(), heads=[0, 7]))


@pytest.mark.parametrize("d,g", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 128), (256, 32)])
@pytest.mark.parametrize("sign", [-1, 1])
def test_infinite_scores(q4, sign, d, g):
    """Every key of a row at a score of -infinity (or +infinity): the softmax is NaN, not the zero of a
    row that sees nothing, and the other rows are as without it; a finite score outweighs -infinity."""
    for hq, hkv, lens, news in ((8, 1, [40, 900, 3], [1, 1, 1]), (8, 1, [40, 900, 4], [3, 3, 4]),
                                (64, 32, [200, 264, 900, 199], [200, 200, 160, 199])):
        b = Batch(q4, lens, news, hq, hkv, d, g, 16, seed=d + g)
        for n, k16 in enumerate(b.k16):
            k16[:, :, 5] = np.float16(8.0)                    # codes above zero there
            b.put(n, k16, b.v16[n])
            b.k[n] = oracle.paged.store(k16, g)[2]
            assert (b.k[n][:, :, 5] > 0).all()
        clean = to_np(b.run())
        hit = np.array([int(b.offsets[1]) - 1, int(b.offsets[2]) - 1])
        b.q[hit, 1, 5] = sign * np.inf
        got = to_np(b.run())
        assert np.isnan(got[hit, 1]).all(), (hq, lens, got[hit, 1])
        got[hit, 1] = clean[hit, 1] = 0
        # rows of one tile raise their maxima together, so another row's may be raised elsewhere: its weights
        # move by a float16 step, 2^-10, at most, and the rounding of the mean by another
        assert np.abs(got.astype(np.float64) - clean).max() <= 2.0 ** -9 * max(np.abs(v).max() for v in b.v)
    if sign < 0:
        b = Batch(q4, [900], [1], 8, 1, d, g, 16, seed=3)
        scale = -1e38
        b.q[:] = 1.0
        k16 = np.full(b.k16[0].shape, 8.0, np.float16)        # q . k = 8 d: the scores overflow to -infinity
        k16[700:] = 0                                        # and 0 here
        b.put(0, k16, b.v16[0])
        got = to_np(b.run(scale=scale)).astype(np.float64)
        want = b.v[0][700:, 0].mean(axis=0)
        assert np.abs(got[0] - want).max() <= 2.0 ** -9 * np.abs(b.v[0]).max()
        k16[:] = 8.0
        b.put(0, k16, b.v16[0])
        assert np.isnan(to_np(b.run(scale=scale))).all()


def test_offsets_cut_to_the_bounds(q4):
    """Descending offsets, offsets outside the rows and more rows than max_q: the rows that the cut bounds
    leave, with every form of the launch; rows of no sequence and what lies behind `out` keep their contents."""
    import torch

    for hq, hkv, tokens, max_q, max_kv in ((8, 2, 200, 2, 48), (8, 2, 200, 2, 900), (16, 2, 200, 9, 900), (64, 32, 420, 200, 900)):
        mid, last = (3, 5) if tokens == 200 else (20, 150)
        mid, last = min(mid, max_q), min(mid, max_q) + min(last - mid, max_q)
        lens = [70, 600, 333, 900, 10]
        news = [0, mid, last - mid, max_q, 0]
        b = Batch(q4, lens, news, hq, hkv, 128, 128, 16, seed=71, extra_rows=tokens - last - max_q)
        raw = to_gpu(np.array([50, -3, mid, last, 2 ** 31 - 1, 7], np.int32))
        big = torch.full((tokens + 40, hq, 128), 5.0, dtype=torch.float16, device="cuda")
        q4.paged_attention(to_gpu(b.q), b.cache, to_gpu(b.table), raw, to_gpu(np.array(lens, np.int32)), max_q, max_kv,
                           out=big[:tokens])
        b.lens = [min(n, max_kv) for n in lens]
        b.k, b.v = ([t[:max_kv] for t in kv] for kv in (b.k, b.v))
        say("offsets", hq, max_q, max_kv, "worst share of the bound", b.check(big[:tokens], heads=[0, hq - 1]))
        assert bool((big[last + max_q:] == 5.0).all())


def test_subnormal_queries(q4):
    """Queries among float16's subnormals keep their value in the matrix products."""
    for hq, hkv, lens, news in ((8, 2, [300, 33], [1, 1]), (16, 2, [300, 33], [5, 3]),
                                (64, 32, [264, 200, 199, 193], [199, 200, 199, 193])):
        b = Batch(q4, lens, news, hq, hkv, 128, 128, 16, seed=81, spread=2.0 ** -17)
        b.check(b.run(scale=2.0 ** 13), scale=2.0 ** 13, heads=[0, hq - 1])
