"""Attention behind shared prefixes over the paged INT4 cache against the oracle in float64
(needs an MI355X).

Bound of an output's error, from the arithmetic. With A = sum_t p_t |v_t| (p the exact softmax over
prefix and own keys), Z = max_t sum_c |q_c k_tc| * scale:
 - weights, scores, sums and the last rounding as in attention without a prefix: 2^-11 A,
   2 (D / 32 + 8) 2^-23 (Z + 1) A, 2 (n / 32 + 32) 2^-24 A, 2^-11 |o|;
 - the parts of a row's keys (the prefix's pieces, the own keys') hold the reference m of their exponents in
   float32, |m| <= 1.45 Z + 64 (at most 14 + 12 + 15 binades from the largest score, and there are below 2^20
   keys), and are added up with 2^(difference): two references and their difference, rounded once each,
   3 * 2^-24 (1.45 Z + 64) of a weight, and 4 products of 2^-24.

Groups of up to 256 rows a KV head, most of the cases here, go through tiles of 16 rows; test_gpu_shared_forms.py has
the other forms.
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


def i32(a):
    return to_gpu(np.asarray(a, dtype=np.int32))


class Shared:
    """Groups of sequences with prefixes of `prefix` tokens; sequence n has lens[n] keys of its own and
    news[n] rows. Every slot that no length covers holds random codes and NaN scales."""

    def __init__(self, q4, sizes, prefix, lens, news, hq, hkv, d, g, page, seed=0, spread=1.0, extra_rows=0, lead=0,
                 pages=None, v_scale=1.0):
        import torch

        r = np.random.default_rng(seed)
        self.q4, self.page, self.d, self.g = q4, page, d, g
        self.prefix, self.lens = list(prefix), list(lens)
        self.groups = lead + np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        wide = max(1, max([-(-n // page) for n in prefix] + [0]))
        narrow = max(1, max(-(-n // page) for n in lens))
        need = len(prefix) * wide + len(lens) * narrow
        self.pages = need + 3 if pages is None else pages
        order = r.permutation(self.pages)[:need] if pages is None else self.pages - 1 - r.permutation(need)
        self.ptable = order[:len(prefix) * wide].reshape(len(prefix), wide).astype(np.int32)
        self.table = order[len(prefix) * wide:].reshape(len(lens), narrow).astype(np.int32)
        rows = int(self.offsets[-1]) + extra_rows
        self.q = (spread * r.standard_normal((rows, hq, d))).astype(np.float16)
        self.cache = q4.paged_kv_alloc(self.pages, page, hkv, d, g)
        if pages is None:
            for t in (self.cache.k_codes, self.cache.v_codes):
                t.copy_(torch.randint(0, 256, t.shape, dtype=torch.uint8))
        for t in (self.cache.k_scales, self.cache.v_scales):
            t.fill_(float("nan"))
        self.pk, self.pv, self.k, self.v = [], [], [], []
        for table, counts, ks, vs in ((self.ptable, prefix, self.pk, self.pv), (self.table, lens, self.k, self.v)):
            for n, length in enumerate(counts):
                k16 = (r.standard_normal((length, hkv, d)) * np.exp(0.4 * r.standard_normal((1, hkv, d)))).astype(np.float16)
                v16 = (v_scale * r.standard_normal((length, hkv, d))).astype(np.float16)
                ks.append(np.zeros((0, hkv, d))), vs.append(np.zeros((0, hkv, d)))
                if length:
                    self.put(table[n], k16, v16, ks, vs, n)

    def put(self, table, k16, v16, ks, vs, n):
        t = np.arange(len(k16))
        slots = table[t // self.page] * self.page + t % self.page
        self.q4.paged_kv_append(to_gpu(k16), to_gpu(v16), self.cache, i32(slots))
        ks[n], vs[n] = oracle.paged.store(k16, self.g)[2], oracle.paged.store(v16, self.g)[2]

    def args(self):
        news = np.diff(self.offsets)
        rows = [self.offsets[b] - self.offsets[a] for a, b in zip(self.groups, self.groups[1:])]
        return dict(max_q=int(news.max()), max_kv=max(self.lens), max_group_q=int(max(rows + [0])),
                    max_prefix=max(self.prefix + [0]))

    def run(self, scale=None, **kw):
        args = self.args()
        t = dict(q=self.q, prefix_table=self.ptable, prefix_lens=np.array(self.prefix, np.int32), group_offsets=self.groups,
                 block_table=self.table, q_offsets=self.offsets, kv_lens=np.array(self.lens, np.int32))
        t = {k: kw.pop(k) if k in kw else to_gpu(v) for k, v in t.items()}
        args.update(kw)
        return self.q4.paged_attention_shared(t.pop("q"), self.cache, **t, **args, scale=scale)

    def view(self, **fields):
        """The same tensors with other groups, prefixes or values to compare with."""
        other = Shared.__new__(Shared)
        other.__dict__.update(self.__dict__, **fields)
        return other

    def check(self, got, scale=None, what="", only=None):
        """`only`: a slice of the rows to look at."""
        s = self.d ** -0.5 if scale is None else scale
        got = to_np(got).astype(np.float64)
        rows = self.offsets[-1]
        ref, mag = (oracle.paged.attention_shared(self.q, self.pk, f(self.pv), self.groups, self.k, f(self.v), self.lens,
                                                  self.offsets, s)[:rows]
                    for f in (list, lambda v: [np.abs(t) for t in v]))
        keys = np.concatenate(self.pk + self.k)
        share = self.q.shape[1] // keys.shape[1]
        z = 1.0 + np.abs(s) * (np.abs(self.q[:rows].astype(np.float64)) *
                               np.repeat(np.abs(keys).max(axis=0), share, axis=0)).sum(-1).max() if len(keys) else 1.0
        n = max(self.prefix + [0]) + max(self.lens)
        rel = 2.0 ** -11 + 2 * (self.d / 32 + 8) * 2.0 ** -23 * z + 2 * (n / 32 + 32) * 2.0 ** -24
        rel += (4 + 3 * (1.45 * z + 64)) * 2.0 ** -24
        bound = rel * mag + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
        got = got[:rows]
        if only is not None:
            got, ref, bound = got[only], ref[only], bound[only]
        err = np.abs(got - ref)
        assert np.all(np.isfinite(got)), what
        assert np.all(err <= bound), (what, (err / bound).max(), np.argwhere(err > bound)[:4])
        return (err / bound).max()


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
    """One row a sequence behind prefixes and own lengths around every tile, step and page border, groups
    of one and of many, and one without sequences."""
    say("shared decode", hq, hkv, d, g, page)
    sizes = [1, 3, 1, 2, 0, 4, 1, 5]
    prefix = [1, 15, 16, 17, 40, 64, 129, 1000]
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 1, 48, 49, 63, 64, 65, 130, 1, 200]
    b = Shared(q4, sizes, prefix, lens, [1] * len(lens), hq, hkv, d, g, page, seed=d + g)
    say("  worst share of the bound", b.check(b.run()))
    say("  long bounds", b.check(b.run(max_kv=5000, max_prefix=9000, max_group_q=300)))


@pytest.mark.parametrize("hq,hkv,d,g,page", SHAPES)
def test_chunks(q4, hq, hkv, d, g, page):
    """Questions of several tokens, single rows and sequences without rows, prefixes of 0 and more tokens."""
    say("shared chunks", hq, hkv, d, g, page)
    sizes, prefix = [2, 3, 1], [77, 0, 300]
    lens, news = [40, 9, 70, 1, 0, 130], [33, 9, 70, 1, 0, 18]
    b = Shared(q4, sizes, prefix, lens, news, hq, hkv, d, g, page, seed=d + g + 1)
    say("  worst share of the bound", b.check(b.run()))
    say("  long bounds", b.check(b.run(max_kv=4000, max_prefix=4000)))


@pytest.mark.parametrize("d,g", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 128), (256, 64), (256, 32)])
@pytest.mark.parametrize("bound", [200, 9000])
def test_many_rows(q4, d, g, bound):
    """128-row workgroups behind the prefix too, whole and (a long bound) cut."""
    say("shared many rows", d, g, bound)
    seqs = 35
    r = np.random.default_rng(d)
    lens = r.integers(40, 60, seqs)
    lens[0] = 200
    b = Shared(q4, [20, 15], [100, 33], lens, np.minimum(lens, 40), 16, 16, d, g, 16, seed=2)
    say("  worst share of the bound", b.check(b.run(max_kv=bound)))


def test_spread_scores(q4):
    """Softmaxes with few winners, in the prefix or behind it, and V scales far from 1."""
    for seed, spread, v in ((3, 8.0, 1.0), (4, 30.0, 1e-4), (5, 1.0, 3000.0), (6, 0.01, 1e-6)):
        b = Shared(q4, [4, 2], [500, 31], [90, 3, 1, 17, 200, 5], [1, 3, 1, 2, 40, 5], 8, 2, 128, 64, 32, seed=seed,
                   spread=spread, v_scale=v)
        say("  spread", spread, v, b.check(b.run(), what=seed))
        say("  scale", b.check(b.run(scale=-0.3 / spread), scale=-0.3 / spread, what=seed))
        say("  scale 0", b.check(b.run(scale=0.0), scale=0.0, what=seed))


def test_without_prefix_is_paged_attention(q4):
    """No group, no prefix token, no group row: the bits of paged_attention."""
    import torch

    b = Shared(q4, [3], [64], [90, 30, 700], [1, 1, 1], 8, 2, 128, 128, 16, seed=7)
    plain = q4.paged_attention(to_gpu(b.q), b.cache, to_gpu(b.table), to_gpu(b.offsets), i32(b.lens), 1, 700)
    assert torch.equal(b.run(max_prefix=0), plain) and torch.equal(b.run(max_group_q=0), plain)
    got = b.run(prefix_table=i32(np.zeros((0, 2))), prefix_lens=i32([]), group_offsets=i32([0]))
    assert torch.equal(got, plain)
    none = np.zeros((0, 2, 128))
    b.view(pk=[none], pv=[none]).check(b.run(prefix_lens=i32([0])))
    out = torch.full_like(plain, 3.0)
    assert b.run(q=to_gpu(b.q[:0]), out=out[:0]).numel() == 0 and bool((out == 3.0).all())


def test_same_as_plain_block_tables(q4):
    """A prefix of whole pages read through each sequence's own table, by paged_attention."""
    page = 32
    b = Shared(q4, [2, 3], [5 * page, 2 * page], [40, 1, 33, 64, 100], [1] * 5, 16, 2, 128, 128, page, seed=8)
    of = [0, 0, 1, 1, 1]
    blocks = 5 + 4
    table = np.zeros((5, blocks), np.int32)
    lens = []
    for n, g in enumerate(of):
        p = b.prefix[g] // page
        row = np.concatenate([b.ptable[g][:p], b.table[n]])[:blocks]
        table[n, :len(row)] = row
        lens.append(b.prefix[g] + b.lens[n])
    plain = q4.paged_attention(to_gpu(b.q), b.cache, to_gpu(table), to_gpu(b.offsets), i32(lens), 1, max(lens))
    got = b.run()
    b.check(got)
    b.check(plain)


def test_sequences_outside_groups_and_rows_behind(q4):
    """Sequences before the first group and behind the last have no prefix; rows of no sequence stay."""
    import torch

    b = Shared(q4, [2, 1], [50, 20], [9, 40, 3, 17, 60], [1, 2, 3, 1, 20], 8, 2, 64, 64, 16, seed=9, extra_rows=4, lead=1)
    out = torch.full((len(b.q), 8, 64), 7.0, dtype=torch.float16, device="cuda")
    got = b.run(out=out)
    assert got is out and bool((out[b.offsets[-1]:] == 7.0).all())
    b.check(out)


def test_rows_ahead_of_their_sequence(q4):
    """More rows than own keys: the first rows see the prefix alone, or nothing (zero)."""
    b = Shared(q4, [2, 1], [50, 0], [2, 0, 1], [4, 3, 4], 8, 2, 64, 64, 16, seed=10)
    got = b.run()
    b.check(got)
    assert np.all(to_np(got)[7:10] == 0) and np.any(to_np(got)[4:7] != 0)


@pytest.mark.parametrize("d,g", [(64, 32), (128, 128), (128, 64), (256, 64)])
@pytest.mark.parametrize("page", [16, 48])
def test_rows_that_fill_tiles(q4, d, g, page):
    """Sequences of 640 and more rows a KV head walk prefix and own keys as one line: lengths around its borders,
    sequences outside groups, rows ahead of their start, rows beyond max_group_q, jobs whole and cut."""
    import torch

    prefix = [1, 63, 64, 65, 200, 0, 130]
    sizes = [1, 1, 2, 1, 1, 1, 1]
    lens = [30, 40, 17, 64, 100, 5, 3, 0, 70, 33]
    news = [20, 40, 17, 9, 33, 16, 20, 4, 1, 12]
    b = Shared(q4, sizes, prefix, lens, news, 32, 2, d, g, page, seed=d + page, lead=1, extra_rows=3)
    out = torch.full((len(b.q), 32, d), 7.0, dtype=torch.float16, device="cuda")
    say("  line", d, g, page, b.check(b.run(out=out)))
    assert bool((out[b.offsets[-1]:] == 7.0).all())
    say("  long bounds", b.check(b.run(max_kv=3000, max_prefix=3000, max_group_q=90, max_q=50)))
    # rows of a group beyond the bound have no prefix: of group 2's, 9 and 33, those from the second's 17 - 9th on
    none = np.zeros((0, 2, d))
    alone = b.view(groups=np.arange(1, 10), prefix=prefix[:3] + [0] + prefix[3:], pk=b.pk[:3] + [none] + b.pk[3:],
                   pv=b.pv[:3] + [none] + b.pv[3:])
    got = b.run(max_group_q=17)
    alone.check(got, only=slice(b.offsets[4] + 8, b.offsets[5]))
    b.check(got, only=slice(b.offsets[3], b.offsets[4] + 8))
    # a page of prefix and one of own keys outside the cache: their keys are hidden
    ptable, table = b.ptable.copy(), b.table.copy()
    ptable[4, 1], table[5, 0] = b.pages, -5
    hole = b.view(pk=list(b.pk), pv=list(b.pv))
    keep = np.array([t for t in range(200) if t // page != 1])
    hole.pk[4], hole.pv[4] = b.pk[4][keep], b.pv[4][keep]
    hole.check(b.run(prefix_table=i32(ptable)))
    b.run(block_table=i32(table))
    for groups in ([5, 0, 5, 1, 2, 3, 4, 9], [-3, 900, 2, 7, 7, 7, 8, 2 ** 31 - 1]):
        b.run(group_offsets=i32(groups), prefix_lens=i32([2 ** 31 - 1, -1, 5, 900, 3, 2, 1]))
    torch.cuda.synchronize()


def test_bounds_and_bad_entries(q4):
    """Lengths cut to their bounds, rows beyond max_group_q without a prefix, pages outside the cache hidden,
    offsets that descend or lie outside."""
    import torch

    b = Shared(q4, [3, 2], [100, 64], [20, 30, 40, 50, 60], [1, 1, 1, 1, 1], 8, 2, 128, 128, 16, seed=11)
    full = to_np(b.run())
    # prefixes cut
    b.view(prefix=[48, 48], pk=[t[:48] for t in b.pk], pv=[t[:48] for t in b.pv]).check(b.run(max_prefix=48))
    # the third member's row of group 0 lies beyond the bound
    none = np.zeros((0, 2, 128))
    got = b.run(max_group_q=2)
    b.view(groups=np.array([0, 2, 3, 5]), prefix=[100, 0, 64], pk=[b.pk[0], none, b.pk[1]],
           pv=[b.pv[0], none, b.pv[1]]).check(got)
    # pages outside the cache: the keys of blocks 2 and 5 of the first prefix hidden, then all of them
    ptable = b.ptable.copy()
    ptable[0, 2], ptable[0, 5] = b.pages, -1
    keep = np.array([t for t in range(100) if t // 16 not in (2, 5)])
    b.view(pk=[b.pk[0][keep], b.pk[1]], pv=[b.pv[0][keep], b.pv[1]]).check(b.run(prefix_table=i32(ptable)))
    ptable[0] = -7
    b.view(pk=[none, b.pk[1]], pv=[none, b.pv[1]]).check(b.run(prefix_table=i32(ptable)))
    # garbage in the small arrays stays inside the buffers
    for groups in ([5, 0, 5], [-3, 900, 2], [0, 5, 3], [2 ** 31 - 1, -2 ** 31, 0]):
        for lens in ([100, 64], [-1, 2 ** 31 - 1], [2 ** 31 - 1, 7]):
            b.run(group_offsets=i32(groups), prefix_lens=i32(lens))
    b.run(q_offsets=i32([0, 900, -5, 3, 2, 5]), kv_lens=i32([-1, 2 ** 31 - 1, 0, 4, 5]))
    torch.cuda.synchronize()
    assert np.array_equal(to_np(b.run()), full)


def test_infinite_scores(q4):
    """Scores beyond float32: -infinity all over the prefix leaves the own keys, all over the own keys the
    prefix, everywhere NaN; +infinity anywhere NaN."""
    hq, hkv, d, page = 4, 1, 64, 16
    one, zero = np.ones((40, hkv, d), np.float16), np.zeros((40, hkv, d), np.float16)
    r = np.random.default_rng(12)
    for at_prefix, at_own in ((one, zero), (zero, one), (one, one), (zero, zero)):
        for sign in (-1.0, 1.0):
            for new in (1, 9):                                    # one tile of 16 rows and several
                b = Shared(q4, [2], [40], [40, 40], [new, new], hq, hkv, d, 64, page, seed=13)
                b.q[:] = 60000.0
                v = [r.standard_normal((40, hkv, d)).astype(np.float16) for _ in range(3)]
                b.put(b.ptable[0], at_prefix, v[0], b.pk, b.pv, 0)
                b.put(b.table[0], at_own, v[1], b.k, b.v, 0)
                b.put(b.table[1], at_own, v[2], b.k, b.v, 1)
                got = to_np(b.run(scale=sign * 1e36))
                lost = at_prefix is one and at_own is one if sign < 0 else at_prefix is one or at_own is one
                if lost:
                    assert np.all(np.isnan(got)), (sign, new)
                    continue
                rows = b.offsets
                for n in range(2):
                    for i in range(new):
                        own = v[1 + n][:40 - new + i + 1] if at_own is zero else v[0][:0]
                        seen = np.concatenate([v[0] if at_prefix is zero else v[0][:0], own])
                        want = np.mean(oracle.paged.store(np.ascontiguousarray(seen), 64)[2], axis=0)
                        # equal weights, one half step of float16 in them and one in the result
                        bound = 2.0 ** -10 * np.mean(np.abs(oracle.paged.store(np.ascontiguousarray(seen), 64)[2]), axis=0)
                        assert np.all(np.abs(got[rows[n] + i] - want) <= bound + 2.0 ** -18), (sign, new, n, i)


def test_not_finite_values(q4):
    """A NaN or infinite V group in the prefix reaches the rows of its group, and those alone; one behind a
    prefix's length nobody."""
    b = Shared(q4, [2, 2], [40, 40], [20, 20, 20, 20], [1, 1, 1, 1], 8, 2, 128, 64, 16, seed=14)
    bad = np.zeros((40, 2, 128), np.float16)
    bad[3, 1, 70] = np.nan
    at = np.arange(40)
    q4.paged_kv_append(to_gpu(np.zeros_like(bad)), to_gpu(bad), b.cache, i32(b.ptable[1][at // 16] * 16 + at % 16))
    got = to_np(b.run())
    assert np.all(np.isfinite(got[:2])) and np.all(np.isnan(got[2:, 4:, 64:])) and np.all(np.isfinite(got[2:, :4]))
    assert np.all(np.isfinite(got[2:, 4:, :64]))
    got = to_np(b.run(prefix_lens=i32([40, 3])))
    assert np.all(np.isfinite(got))
    b.q[0, 0, 0] = np.inf
    got = to_np(b.run())
    assert np.all(np.isnan(got[0, 0])) and np.all(np.isfinite(got[0, 1:])) and np.all(np.isfinite(got[1]))


def test_strided_q_and_workspace(q4):
    import torch

    b = Shared(q4, [5], [200], [700, 3, 1, 50, 9], [1] * 5, 8, 2, 128, 128, 16, seed=15)
    wide = torch.zeros((5, 14, 128), dtype=torch.float16, device="cuda")
    wide[:, 3:11] = to_gpu(b.q)
    want = b.run()
    assert torch.equal(b.run(q=wide[:, 3:11]), want)
    a = b.args()
    need = q4.paged_attention_shared_workspace_bytes(5, 1, 5, a["max_q"], a["max_kv"], a["max_group_q"], a["max_prefix"],
                                                     8, 2, 128, 128)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")  # NaNs as float32
    assert torch.equal(b.run(workspace=ws[:need]), want) and bool((ws[need:] == 255).all())
    with pytest.raises(q4.Q4Error):
        b.run(workspace=ws[:need - 16])


def test_captured_and_streams(q4):
    """Captured once, replayed with other lengths, groups and queries; two streams at once; as eager."""
    import torch

    b = Shared(q4, [3, 2], [900, 500], [700, 30, 40, 600, 60], [1] * 5, 8, 2, 128, 128, 16, seed=16)
    t = dict(q=to_gpu(b.q), prefix_lens=i32(b.prefix), group_offsets=i32(b.groups), kv_lens=i32(b.lens))
    bounds = dict(max_group_q=5, max_kv=700, max_prefix=900)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.run(**t, **bounds)
    torch.cuda.synchronize()
    fixed = dict(prefix_table=to_gpu(b.ptable), block_table=to_gpu(b.table), q_offsets=to_gpu(b.offsets))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.run(**t, **fixed, **bounds)
    r = np.random.default_rng(17)
    for i in range(6):
        t["q"].copy_(to_gpu(r.standard_normal(b.q.shape).astype(np.float16)))
        t["prefix_lens"].copy_(i32([r.integers(0, 901), r.integers(0, 501)]))
        t["group_offsets"].copy_(i32([0, r.integers(0, 6), 5]))
        t["kv_lens"].copy_(i32([r.integers(1, n + 1) for n in b.lens]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, b.run(**t, **fixed, **bounds)), i
    two = [Shared(q4, [3], [300 + 77 * s], [100, 20, 640], [1, 7, 1], 8, 2, 128, 64, 32, seed=18 + s) for s in range(2)]
    want = [s.run() for s in two]
    ready = [{k: to_gpu(v) for k, v in dict(q=s.q, prefix_table=s.ptable, prefix_lens=np.array(s.prefix, np.int32),
                                            group_offsets=s.groups, block_table=s.table, q_offsets=s.offsets,
                                            kv_lens=np.array(s.lens, np.int32)).items()} for s in two]
    torch.cuda.synchronize()
    streams, res = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(10):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                res[s].append(two[s].run(**ready[s]))
    torch.cuda.synchronize()
    for s in range(2):
        assert all(torch.equal(r, want[s]) for r in res[s])


def test_offsets_beyond_32_bits(q4):
    """Pages whose codes lie 4 GiB and more into the cache."""
    b = Shared(q4, [2], [100], [40, 5], [1, 3], 16, 8, 128, 128, 16, seed=20, pages=560000)
    assert b.cache.k_codes.numel() > 2 ** 32 and int(b.ptable.min()) * 8 * 16 * 64 > 2 ** 32
    b.check(b.run())
