"""Attention behind shared prefixes in the forms for more than 256 rows of a group and KV head, against the oracle's
formula in float64 (needs an MI355X): the prefix first and the rows behind it from there, in tiles of 16, 32 and
128 rows whose own keys a workgroup takes whole or in pieces, and prefix and own keys as one line.

Bound of an output's error, from the arithmetic. With A = sum_t p_t |v_t| (p the exact softmax over
prefix and own keys), Z = max_t sum_c |q_c k_tc| * scale:
 - weights, scores, sums and the last rounding as in attention without a prefix: 2^-11 A,
   2 (D / 32 + 8) 2^-23 (Z + 1) A, 2 (n / 32 + 32) 2^-24 A, 2^-11 |o|;
 - the parts of a row's keys (pieces, halves, wavefronts, what lies behind the prefix) each hold the float32
   reference m + E of their exponents, |m + E| <= 1.45 Z + 64 (E within 12 + 14 + 4 binades of 0, sums below
   2^34), and enter with 2^(difference). Between the weights of two keys at most 8 roundings of such numbers
   count: both parts' last reference, the difference, and a reference's rises for a larger V scale, of
   which a test's scales (a few binades) cause up to 5 (a rise of m shrinks what came before it by 2^3 and more):
   8 * 2^-24 (1.45 Z + 64), and 4 products of 2^-24;
 - P = 2^(s - m - E) vs (vs the key's V scale) as float16 is off by 2^-25 at least where it is subnormal, however small
   the key's own part. In the output that is 2^-25 |code| / l with l >= 2^(max s - m - E) and m <= max s (the held
   maximum of scores seen, while scales stay below 2^11), so 2^-25 2^E |code| at most; E is the binade above the largest
   scale among the sequence's and its prefix's keys, seen or not, less 12: 2^E |code| <= 2 * 2^-12 max |v|. Over
   n keys: n 2^-36 max |v|.
"""

import numpy as np
import pytest

import oracle
from gpu_util import say, to_gpu, to_np
from test_gpu_shared_attention import Shared, i32, q4  # noqa: F401  (q4: the fixture)

pytestmark = pytest.mark.gpu


def reference(b, s):
    """oracle.paged.attention_shared in float64 on the GPU, a sequence at a time (rows that see no key are 0), and the
    same of |v|."""
    import torch

    rows, hq, d = b.q.shape
    share = hq // b.k[0].shape[1]
    out, mag = (torch.zeros((rows, hq, d), dtype=torch.float64, device="cuda") for _ in range(2))

    def by_head(t):
        return to_gpu(t).double().transpose(0, 1)

    pk, pv = [by_head(t) for t in b.pk], [by_head(t) for t in b.pv]
    queries = to_gpu(b.q).double()
    for n, length in enumerate(b.lens):
        first, last = int(b.offsets[n]), int(b.offsets[n + 1])
        if first == last:
            continue
        of = [g for g in range(len(pk)) if b.groups[g] <= n < b.groups[g + 1]]
        k = torch.cat([pk[g] for g in of] + [by_head(b.k[n])], 1)                    # [KV heads, keys, d]
        v = torch.cat([pv[g] for g in of] + [by_head(b.v[n])], 1).contiguous()
        q = queries[first:last].view(last - first, -1, share, d).permute(1, 0, 2, 3).reshape(len(k), -1, d)
        own = length - (last - first) + torch.arange(last - first, device="cuda") + 1
        seen = torch.arange(k.shape[1], device="cuda")[None] < (k.shape[1] - length) + own.clamp(min=0)[:, None]
        some = seen.any(1)
        if not bool(some.any()):
            continue
        z = torch.matmul(q.contiguous(), k.transpose(1, 2).contiguous()) * s
        z = z.view(len(k), last - first, share, -1).masked_fill(~seen[None, :, None], -np.inf)[:, some]
        p = torch.softmax(z, -1).reshape(len(k), -1, z.shape[-1])
        for to, x in ((out, v), (mag, v.abs())):
            o = torch.matmul(p, x).view(len(k), -1, share, d).permute(1, 0, 2, 3).reshape(-1, hq, d)
            to[first:last][some] = o
    return to_np(out), to_np(mag)


def largest(b):
    """[rows, q heads, 1]: the largest |v| among a row's own keys and its prefix's, seen or not."""
    out = np.zeros((len(b.q), b.q.shape[1], 1))
    for n in range(len(b.lens)):
        vs = [b.v[n]] + [b.pv[g] for g in range(len(b.pk)) if b.groups[g] <= n < b.groups[g + 1]]
        top = np.max([np.abs(t).max(axis=(0, 2), initial=0.0) for t in vs], axis=0)     # [KV heads]
        out[b.offsets[n]:b.offsets[n + 1], :, 0] = np.repeat(top, b.q.shape[1] // len(top))
    return out


def check(b, got, scale=None, what="", only=None):
    s = b.d ** -0.5 if scale is None else scale
    got, rows = to_np(got).astype(np.float64), int(b.offsets[-1])
    ref, mag = (t[:rows] for t in reference(b, s))
    keys = np.concatenate(b.pk + b.k)
    share = b.q.shape[1] // keys.shape[1]
    z = 1.0 + np.abs(s) * (np.abs(b.q[:rows].astype(np.float64)) *
                           np.repeat(np.abs(keys).max(axis=0), share, axis=0)).sum(-1).max()
    n = max(b.prefix + [0]) + max(b.lens)
    rel = 2.0 ** -11 + 2 * (b.d / 32 + 8) * 2.0 ** -23 * z + 2 * (n / 32 + 32) * 2.0 ** -24
    rel += (4 + 8 * (1.45 * z + 64)) * 2.0 ** -24
    bound = rel * mag + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + n * 2.0 ** -36 * largest(b)[:rows]
    got = got[:rows]
    if only is not None:
        got, ref, bound = got[only], ref[only], bound[only]
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), what
    assert np.all(err <= bound), (what, (err / bound).max(), np.argwhere(err > bound)[:4])
    return (err / bound).max()


# rows of a sequence, q heads and KV heads, and a bound of the own keys that has them cut, for each form
FORMS = {
    "16 rows": dict(new=1, hq=16, hkv=2), "16 rows, cut": dict(new=1, hq=16, hkv=2, max_kv=5000, own=700),
    "32 rows": dict(new=4, hq=16, hkv=2), "32 rows, cut": dict(new=4, hq=16, hkv=2, max_kv=5000, own=700),
    "128 rows": dict(new=40, hq=16, hkv=16), "128 rows, cut": dict(new=40, hq=30, hkv=30, max_kv=9000),
    "line": dict(new=40, hq=32, hkv=2), "line, cut": dict(new=40, hq=32, hkv=2, max_kv=9000),
}
ALL = list(FORMS)


def make(q4, form, d=128, g=128, page=16, prefix=(300, 5, 40, 0), seed=0, own=None, pages=None, ragged=True, lead=1, **kw):
    """Sequences of a form: most of them in the first group, one without rows, `lead` in no group."""
    f = FORMS[form]
    r = np.random.default_rng(seed + 1000)
    own = own or f.get("own", 70)
    seqs = 39 if f["new"] < 40 else 35 if f["hkv"] > 2 else 9
    first = 37 if f["new"] == 1 else 24 if seqs > 9 else 5
    sizes = [first] + [1 if n + 1 < len(prefix) else seqs - first - (len(prefix) - 2) for n in range(1, len(prefix))]
    if ragged:
        news = [f["new"]] + list(r.integers((3 * f["new"] + 3) // 4, f["new"] + 1, seqs + lead - 1))
        news[3] = 0
    else:
        news = [f["new"]] * (seqs + lead)
    lens = [max(1, int(n)) for n in np.maximum(news, r.integers(1, own + 1, seqs + lead))]
    b = Shared(q4, sizes, prefix, lens, news, f["hq"], f["hkv"], d, g, page, seed=seed, lead=lead, pages=pages, **kw)
    b.bounds = {k: v for k, v in f.items() if k == "max_kv"}
    share, tokens = f["hq"] // f["hkv"], [int(b.offsets[e] - b.offsets[s]) for s, e in zip(b.groups, b.groups[1:])]
    assert max(tokens) * share > 256 and len(sizes) == len(prefix)
    line = f["new"] * share >= 640 and 3 * int(b.offsets[-1]) >= len(news) * f["new"]
    assert line == form.startswith("line")
    return b


def run(b, **kw):
    return b.run(**{**b.bounds, **kw})


def test_reference(q4):
    b = Shared(q4, [2, 1], [5, 0], [3, 2, 4, 7], [2, 3, 0, 1], 4, 2, 64, 64, 16, seed=1, lead=1)
    want = oracle.paged.attention_shared(b.q, b.pk, b.pv, b.groups, b.k, b.v, b.lens, b.offsets, 0.125)
    assert np.allclose(reference(b, 0.125)[0], want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("form", ALL)
@pytest.mark.parametrize("d,g", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 128), (256, 64)])
def test_sizes(q4, form, d, g):
    """All heads and scale groups, prefixes of pages that end inside tiles, rows behind the last sequence left alone."""
    import torch

    say("shared,", form, d, g)
    b = make(q4, form, d, g, page=48 if g == 64 else 16, seed=d + g, extra_rows=3)
    out = torch.full((len(b.q), b.q.shape[1], d), 7.0, dtype=torch.float16, device="cuda")
    say("  worst share of the bound", check(b, run(b, out=out)))
    assert bool((out[b.offsets[-1]:] == 7.0).all())


@pytest.mark.parametrize("form", ALL)
@pytest.mark.parametrize("d,g", [(64, 64), (128, 128), (128, 64), (256, 128)])
@pytest.mark.parametrize("groups", [2, 200])
def test_long_prefixes(q4, form, d, g, groups):
    """Prefixes of thousands of keys: in many pieces, and (200 groups, all but two of them without rows) in one, which
    an eight-wavefront workgroup walks in dozens of rounds through its two buffers."""
    say("shared, long prefix,", form, d, g, groups)
    b = make(q4, form, d, g, page=64, prefix=(5037, 1000), seed=d, own=200, lead=0)
    more = {}
    if groups > 2:
        none = b.groups[-1]
        more = dict(prefix_table=i32(np.concatenate([b.ptable, np.zeros((groups - 2, b.ptable.shape[1]))])),
                    prefix_lens=i32(b.prefix + [900] * (groups - 2)),
                    group_offsets=i32(np.concatenate([b.groups, [none] * (groups - 2)])))
    say("  worst share of the bound", check(b, run(b, **more)))


@pytest.mark.parametrize("form", ALL)
def test_own_keys_beyond_their_rule(q4, form):
    """Own keys of more than 4096, which 16- and 32-row workgroups share out, beside short ones."""
    b = make(q4, form, 128, 128, page=32, prefix=(130, 70), seed=3)
    lens = list(b.lens)
    lens[1], lens[5] = 4500, 300
    news = np.diff(b.offsets)
    long = Shared(q4, np.diff(b.groups), b.prefix, lens, news, b.q.shape[1], b.cache.kv_heads, 128, 128, 32, seed=3, lead=1)
    say("shared, long own keys,", form, check(long, long.run()))


@pytest.mark.parametrize("form", ALL)
@pytest.mark.parametrize("d,g", [(64, 32), (128, 128), (256, 128)])
def test_spread_scores(q4, form, d, g):
    """Softmaxes with few winners, in the prefix or behind it, and V scales far from 1, of prefix and own keys alike or
    a million apart."""
    for seed, spread, v, own_v in ((3, 8.0, 1.0, 1.0), (4, 30.0, 1e-4, 1e-4), (5, 1.0, 3000.0, 3000.0),
                                   (6, 0.01, 1e-6, 1e-6), (7, 2.0, 3000.0, 1e-3), (8, 2.0, 1e-3, 3000.0)):
        b = make(q4, form, d, g, prefix=(500, 31, 64), seed=seed, spread=spread, v_scale=v)
        if own_v != v:
            r = np.random.default_rng(seed)
            for n, length in enumerate(b.lens):
                shape = (length, b.cache.kv_heads, d)
                k16 = r.standard_normal(shape).astype(np.float16)
                b.put(b.table[n], k16, (own_v * r.standard_normal(shape)).astype(np.float16), b.k, b.v, n)
        say("  shared, spread,", form, d, spread, v, own_v, check(b, run(b), what=seed))
        check(b, run(b, scale=-0.3 / spread), scale=-0.3 / spread, what=seed)
        check(b, run(b, scale=0.0), scale=0.0, what=seed)


@pytest.mark.parametrize("form", ALL)
def test_infinite_scores(q4, form):
    """Scores beyond float32: -infinity all over the prefix leaves the own keys, all over the own keys the
    prefix, everywhere NaN; +infinity anywhere NaN."""
    hkv, d = FORMS[form]["hkv"], 64
    r = np.random.default_rng(12)
    for far_prefix, far_own in ((True, False), (False, True), (True, True), (False, False)):
        b = make(q4, form, d, 64, prefix=(200, 40), seed=13, lead=0, ragged=False, own=60)
        b.q[:] = 60000.0
        for tables, far, ks, vs, counts in ((b.ptable, far_prefix, b.pk, b.pv, b.prefix), (b.table, far_own, b.k, b.v, b.lens)):
            for n, length in enumerate(counts):
                k16 = np.full((length, hkv, d), 1.0 if far else 0.0, np.float16)
                b.put(tables[n], k16, r.standard_normal((length, hkv, d)).astype(np.float16), ks, vs, n)
        for sign in (-1.0, 1.0):
            got = to_np(run(b, scale=sign * 1e36))
            if far_prefix and far_own if sign < 0 else far_prefix or far_own:
                assert np.all(np.isnan(got)), (form, sign, far_prefix, far_own)
                continue
            # what is left has equal weights: the same as with what is far away left out
            keep = b.view(pk=[t[:0] if far_prefix else t for t in b.pk], pv=[t[:0] if far_prefix else t for t in b.pv])
            if far_own:
                keep.lens, keep.k, keep.v = [0] * len(b.lens), [t[:0] for t in b.k], [t[:0] for t in b.v]
            elif far_prefix:
                keep.prefix = [0] * len(b.prefix)
            want, mag = reference(keep, 0.0)
            # equal weights: half a step of float16 in them, one in the result, sums of up to 300 in float32
            bound = (2.0 ** -11 + 2.0 ** -15) * mag + 2.0 ** -11 * np.abs(want) + 2.0 ** -24
            assert np.all(np.abs(got - want) <= bound), (form, sign, far_prefix, far_own)


@pytest.mark.parametrize("form", ALL)
def test_not_finite_values(q4, form):
    """A NaN V group of the prefix reaches the rows of its group, one of an own key the rows that see it, one behind a
    length nobody; an infinite q its own row and head."""
    hq, hkv = FORMS[form]["hq"], FORMS[form]["hkv"]
    share = hq // hkv
    b = make(q4, form, 128, 64, prefix=(300, 40, 90), seed=14, lead=0)
    rows = [slice(int(b.offsets[s]), int(b.offsets[e])) for s, e in zip(b.groups, b.groups[1:])]
    at = np.arange(40)
    bad = np.zeros((40, hkv, 128), np.float16)
    bad[3, 1, 70] = np.nan
    q4.paged_kv_append(to_gpu(np.zeros_like(bad)), to_gpu(bad), b.cache, i32(b.ptable[1][at // 16] * 16 + at % 16))
    got = to_np(run(b))
    lost = np.zeros(got.shape, bool)
    lost[rows[1], share:2 * share, 64:] = True
    assert np.array_equal(np.isnan(got), lost)
    assert np.all(np.isfinite(to_np(run(b, prefix_lens=i32([300, 3, 90])))))
    # the last own key of sequence 2: its last row alone sees it
    n = 2
    length = b.lens[n]
    bad = np.zeros((1, hkv, 128), np.float16)
    bad[0, 0, 5] = np.inf
    q4.paged_kv_append(to_gpu(np.zeros_like(bad)), to_gpu(bad), b.cache,
                       i32([b.table[n][(length - 1) // 16] * 16 + (length - 1) % 16]))
    got = to_np(run(b, prefix_lens=i32([300, 3, 90])))
    lost[:] = False
    lost[b.offsets[n + 1] - 1, :share, :64] = True
    assert np.array_equal(~np.isfinite(got), lost)
    b.q[1, 0, 0] = np.inf
    got = to_np(run(b, prefix_lens=i32([300, 3, 90])))
    assert np.all(np.isnan(got[1, 0])) and np.all(np.isfinite(got[1, 1:])) and np.all(np.isfinite(got[0]))


@pytest.mark.parametrize("form", ALL)
@pytest.mark.parametrize("d,g", [(64, 64), (128, 64), (256, 64)])
def test_bounds_and_bad_entries(q4, form, d, g):
    """Prefixes cut to their bound, rows of a group beyond its bound without a prefix, pages outside the cache hidden,
    rows ahead of their sequence's start, contents that lead nowhere."""
    import torch

    b = make(q4, form, d, g, prefix=(300, 40, 64), seed=15)
    hkv = b.cache.kv_heads
    none = np.zeros((0, hkv, d))
    full = to_np(run(b))
    cut = [min(n, 48) for n in b.prefix]
    check(b.view(prefix=cut, pk=[t[:48] for t in b.pk], pv=[t[:48] for t in b.pv]), run(b, max_prefix=48))
    # rows beyond max_group_q: of the first group's all but the last two
    first, last = int(b.offsets[b.groups[0]]), int(b.offsets[b.groups[1]])
    share = b.q.shape[1] // hkv
    assert (last - first - 2) * share > 256
    got = run(b, max_group_q=last - first - 2)
    check(b, got, only=slice(0, last - 2))
    check(b.view(pk=[none] + b.pk[1:], pv=[none] + b.pv[1:]), got, only=slice(last - 2, last))
    # pages outside the cache: blocks 2 and 5 of the first prefix hidden, then all of it
    ptable = b.ptable.copy()
    ptable[0, 2], ptable[0, 5] = b.pages, -1
    keep = np.array([t for t in range(300) if t // 16 not in (2, 5)])
    check(b.view(pk=[b.pk[0][keep]] + b.pk[1:], pv=[b.pv[0][keep]] + b.pv[1:]), run(b, prefix_table=i32(ptable)))
    ptable[0] = -7
    check(b.view(pk=[none] + b.pk[1:], pv=[none] + b.pv[1:]), run(b, prefix_table=i32(ptable)))
    # fewer keys than rows: the first rows see the prefix alone, those of no group nothing
    news = np.diff(b.offsets)
    short = [max(0, int(n) - 2) for n in news]
    v = b.view(lens=short, k=[t[:n] for t, n in zip(b.k, short)], v=[t[:n] for t, n in zip(b.v, short)])
    got = run(v, kv_lens=i32(short), max_kv=b.bounds.get("max_kv", max(b.lens)))
    check(v, got)
    assert np.all(to_np(got)[:min(2, int(news[0]))] == 0)
    # garbage in the small arrays stays inside the buffers
    for groups in ([len(b.lens), 0, 5, 0], [-3, 900, 2, 9], [0, 5, 3, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31, 0, 7]):
        for lens in ([300, 40, 64], [-1, 2 ** 31 - 1, 7], [2 ** 31 - 1, 7, -2 ** 31]):
            run(b, group_offsets=i32(groups), prefix_lens=i32(lens))
    offsets = b.offsets.copy()
    offsets[[1, 4, 7]] = [900, -5, 3]
    lens = np.array(b.lens)
    lens[[0, 2, 6]] = [-1, 2 ** 31 - 1, -2 ** 31]
    table = b.table.copy()
    table[::2, 0] = [(-5, b.pages, 2 ** 31 - 1)[i % 3] for i in range(len(table[::2]))]
    run(b, q_offsets=i32(offsets), kv_lens=i32(lens), block_table=i32(table))
    torch.cuda.synchronize()
    assert np.array_equal(to_np(run(b)), full)


@pytest.mark.parametrize("form", ALL)
def test_workspace(q4, form):
    """A workspace of the size that is asked for, of any contents, nothing behind it written; too small: refused."""
    import torch

    b = make(q4, form, seed=16)
    a = {**b.args(), **b.bounds}
    need = q4.paged_attention_shared_workspace_bytes(len(b.lens), len(b.prefix), len(b.q), a["max_q"], a["max_kv"],
                                                     a["max_group_q"], a["max_prefix"], b.q.shape[1], b.cache.kv_heads, 128, 128)
    want = run(b)
    for fill in (255, 0x7F, 0):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(run(b, workspace=ws[:need]), want) and bool((ws[need:] == fill).all())
    if need > 0:
        with pytest.raises(q4.Q4Error):
            run(b, workspace=ws[:need - 16])
    else:
        assert form.startswith("line")


@pytest.mark.parametrize("form", ALL)
def test_captured_and_streams(q4, form):
    """Captured once, replayed with other lengths, groups and queries; two streams at once; as eager."""
    import torch

    b = make(q4, form, seed=17)
    t = dict(q=to_gpu(b.q), prefix_lens=i32(b.prefix), group_offsets=i32(b.groups), kv_lens=i32(b.lens))
    fixed = dict(prefix_table=to_gpu(b.ptable), block_table=to_gpu(b.table), q_offsets=to_gpu(b.offsets))
    bounds = {**b.args(), **b.bounds}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.run(**t, **fixed, **bounds)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.run(**t, **fixed, **bounds)
    r = np.random.default_rng(18)
    for i in range(6):
        t["q"].copy_(to_gpu(r.standard_normal(b.q.shape).astype(np.float16)))
        t["prefix_lens"].copy_(i32([r.integers(0, n + 1) for n in b.prefix]))
        t["group_offsets"].copy_(i32(np.sort(r.integers(0, len(b.lens) + 1, len(b.groups))) if i else b.groups))
        t["kv_lens"].copy_(i32([r.integers(0, n + 1) for n in b.lens]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, b.run(**t, **fixed, **bounds)), i
    two = [make(q4, form, seed=19 + s) for s in range(2)]
    want = [run(s) for s in two]
    ready = [{k: to_gpu(v) for k, v in dict(q=s.q, prefix_table=s.ptable, prefix_lens=np.array(s.prefix, np.int32),
                                            group_offsets=s.groups, block_table=s.table, q_offsets=s.offsets,
                                            kv_lens=np.array(s.lens, np.int32)).items()} for s in two]
    torch.cuda.synchronize()
    streams, res = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(10):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                res[s].append(run(two[s], **ready[s]))
    torch.cuda.synchronize()
    for s in range(2):
        assert all(torch.equal(x, want[s]) for x in res[s])


@pytest.mark.parametrize("form", ["16 rows", "16 rows, cut", "32 rows", "128 rows", "line"])
def test_offsets_beyond_32_bits(q4, form):
    """Pages whose codes lie 4 GiB and more into the cache."""
    hkv = FORMS[form]["hkv"]
    b = make(q4, form, seed=20, pages=560000 * 8 // hkv)
    assert b.cache.k_codes.numel() > 2 ** 32 and int(b.ptable.min()) * hkv * 16 * 64 > 2 ** 32
    check(b, run(b))


def test_mixed_batches(q4):
    """Chunks beside single tokens behind one prefix, and behind none."""
    for news in ([200] + [1] * 40, [1] * 20 + [90, 100, 3] + [1] * 20, [41, 41] + [1] * 33):
        lens = [n + 7 * (i % 5) for i, n in enumerate(news)]
        for lead, sizes in ((0, [len(news)]), (1, [len(news) - 3]), (2, [20, len(news) - 22])):
            b = Shared(q4, sizes, [777, 130][:len(sizes)], lens, news, 16, 2, 128, 64, 32, seed=21 + lead, lead=lead)
            say("shared, mixed", len(news), lead, check(b, b.run()))


@pytest.mark.parametrize("prompts", [[1100], [200], [300, 1, 40, 800], [17, 1100]])
def test_prompts_beside_a_group(q4, prompts):
    """Prompts in no group beside few rows behind a prefix, long and short ones."""
    news = prompts + [1] * 8
    lens = [n + 3 * i for i, n in enumerate(news)]
    for sizes, prefix in (([8], [900]), ([3, 5], [70, 411])):
        b = Shared(q4, sizes, prefix, lens, news, 32, 2, 128, 128, 16, seed=30, lead=len(prompts))
        say("shared, prompts beside a group", prompts, sizes, check(b, b.run()))
