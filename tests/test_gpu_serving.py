"""The plan of a batch and the choice of the next tokens against the oracle (needs an MI355X).

Plans and tokens are whole numbers and have to be equal. A token's share is a float64 quotient
of weights that are off by 2^-45 of the largest at most (sums: 2^-45 a token), rounded once to
float32: 2^-24 relative, and 2^20 * 2^-42 = 2^-22 for the sum of the largest vocabulary.
"""

import numpy as np
import pytest

import oracle
from gpu_util import say, to_gpu, to_np

pytestmark = pytest.mark.gpu

SHARE_TOL = 2.0 ** -24 + 2.0 ** -22


@pytest.fixture(scope="module")
def q4():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import w4a16_decode_amd as q4mod

    say("libq4", q4mod.version())
    return q4mod


def i32(a):
    return to_gpu(np.asarray(a, dtype=np.int32))


# ---- the plan -------------------------------------------------------------------------


class State:
    """Sequences with pages of a pool, entries behind their lengths -7."""

    def __init__(self, seed, lens, blocks, page, spare, pages=None):
        r = np.random.default_rng(seed)
        self.page, self.lens = page, np.array(lens, np.int32)
        held = -(-self.lens // page)
        self.pages = int(held.sum()) + spare if pages is None else pages
        order = r.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(lens), blocks), -7, np.int32)
        at = 0
        for s, n in enumerate(held):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.free = np.full(self.pages, -9, np.int32)
        self.free[:self.pages - at] = order[at:]
        self.count = self.pages - at

    def check(self, q4, new, tokens, starts=None, reset=None, pool=True, what=""):
        want = oracle.serving.plan(self.lens, new, self.table, self.page, tokens, self.pages,
                                   self.free if pool else None, self.count, starts, reset)
        table = i32(self.table)
        p = q4.PagePool(i32(self.free), i32([self.count])) if pool else None
        lens = i32(self.lens)
        got = q4.paged_plan(lens, None if new is None else i32(new), table, self.page, tokens, p,
                            None if starts is None else i32(starts), None if reset is None else i32(reset),
                            pages=None if pool else self.pages)
        out = (got.q_offsets, got.positions, got.slots, got.kv_lens, table, p.pages if pool else None,
               got.free_count if pool else None, got.lacking)
        for name, g, w in zip(("q_offsets", "positions", "slots", "kv_lens", "table", "free", "count", "lacking"), out, want):
            if g is not None:
                assert np.array_equal(to_np(g).reshape(np.shape(w)), w), (what, name, to_np(g), w)
        assert np.array_equal(to_np(lens), self.lens)
        if pool:
            assert int(p.count[0]) == self.count
        self.lens, self.table = want[3].astype(np.int32), want[4]
        if pool:
            self.free, self.count = want[5], want[6]
        return want


def test_plan_steps(q4):
    """A prompt step, decode steps, requests that end and others that take their places; every page of
    the pool is held once or free once throughout."""
    r = np.random.default_rng(5)
    s = State(1, [0, 5, 16, 31, 32, 33, 100], 12, 16, 40)
    starts = r.integers(0, 5000, 7)
    for step in range(30):
        new = [40, 0, 1, 17, 5, 64, 2] if step == 0 else (r.random(7) < 0.8).astype(int)
        reset = (r.random(7) < 0.15).astype(int) if step else None
        if reset is not None:
            new = np.where(reset, r.integers(0, 60, 7), new)
        new = np.minimum(new, 12 * 16 - np.where(reset is not None and reset, 0, s.lens))
        want = s.check(q4, new, int(np.sum(new)) + step % 3, starts, reset, what=step)
        if want[7] == 0:
            held = [s.table[i, b] for i, n in enumerate(s.lens) for b in range(-(-n // 16))]
            assert sorted(held + list(s.free[:s.count])) == list(range(s.pages)), step


@pytest.mark.parametrize("seqs,new,extra", [
    (1, 1, 0), (1, 1, 5), (1, 4000, 0), (3, 0, 4), (64, 1, 0), (255, 1, 1), (256, 1, 0), (257, 1, 0), (1024, 1, 7),
    (1025, 1, 0), (2500, 2, 3), (61, 700, 0), (2, 2049, 1), (1000, 3, 0)])
@pytest.mark.parametrize("page", [16, 48])
def test_plan_sizes(q4, seqs, new, extra, page):
    say("plan", seqs, new, extra, page)
    r = np.random.default_rng(seqs + new)
    lens = r.integers(0, 200, seqs)
    news = r.integers(0, new + 1, seqs)
    news[0] = new
    blocks = (200 + new) // page + 2
    need = int((-(-(lens + news) // page)).sum())
    s = State(seqs, lens, blocks, page, need, None)
    reset = (r.random(seqs) < 0.2).astype(int)
    s.check(q4, news, int(news.sum()) + extra, r.integers(0, 9, seqs), reset)
    s.check(q4, None, seqs + extra)
    s.check(q4, news, max(int(news.sum()) - 3, 0))                # rows that do not fit are dropped


def test_plan_lacking(q4):
    """A pool that runs dry, a table that ends, counts out of range, lengths and page numbers out of range."""
    s = State(2, [16, 30, 0, 16], 4, 16, 3)
    want = s.check(q4, [20, 40, 10, 1], 71)
    assert want[7] > 0 and (want[2] == -1).any()
    s = State(3, [60, 64, 1], 4, 16, 9)
    want = s.check(q4, [10, 1, 2], 13)
    assert want[7] == 2
    s = State(4, [60, 64, 1], 4, 16, 9)
    s.lens = np.array([-5, 1000, 2 ** 31 - 1], np.int32)
    s.table[1:] = [[3, 99, -1, 2], [10 ** 9, 0, 1, 5]]
    s.check(q4, [1, 1, 1], 3, pool=False)
    s.lens = np.array([-5, 1000, 1], np.int32)
    s.check(q4, [2 ** 31 - 1, -4, 2 ** 31 - 1], 9)
    for count in (-3, 0, 10 ** 6):
        s = State(6, [16, 1], 4, 16, 5)
        s.free[:] = np.arange(s.pages)
        s.count = count
        p = q4.PagePool(i32(s.free), i32([count]))
        got = q4.paged_plan(i32(s.lens), i32([1, 1]), i32(s.table), 16, 2, p)
        held = min(max(count, 0), s.pages)
        assert int(got.free_count[0]) == max(held - 1, 0) and int(got.lacking[0]) == (held == 0)


def test_plan_without_pool_and_empty(q4):
    import torch

    s = State(7, [3, 16, 47], 4, 16, 0)
    s.table[s.table < 0] = 1
    s.check(q4, [30, 1, 2], 40, [5, 6, 7], [0, 1, 0], pool=False)
    got = q4.paged_plan(i32([]), None, i32(np.zeros((0, 3))), 16, 5, q4.page_pool(4))
    assert to_np(got.q_offsets).tolist() == [0] and to_np(got.slots).tolist() == [-1] * 5
    assert int(got.free_count[0]) == 4 and int(got.lacking[0]) == 0
    got = q4.paged_plan(i32([1]), i32([0]), i32([[0]]), 16, 0, q4.page_pool(4))
    assert to_np(got.q_offsets).tolist() == [0, 0] and got.slots.numel() == 0
    pool = q4.page_pool(3)
    assert to_np(pool.pages).tolist() == [2, 1, 0] and int(pool.count[0]) == 3
    assert isinstance(pool.pages, torch.Tensor)


@pytest.mark.parametrize("seqs,tokens", [(6, 6), (1100, 1200)])
def test_plan_captured_in_place(q4, seqs, tokens):
    """A decode step's plan captured with its state in place: each replay goes a step on."""
    import torch

    r = np.random.default_rng(8)
    s = State(9, r.integers(0, 40, seqs), 8, 16, 8 * seqs)
    lens, table, free, count = i32(s.lens), i32(s.table), i32(s.free), i32([s.count])
    pool = q4.PagePool(free, count)
    reset, starts = i32(np.zeros(seqs)), i32(r.integers(0, 90, seqs))

    def step():
        return q4.paged_plan(lens, None, table, 16, tokens, pool, starts, reset, kv_lens_out=lens, free_count_out=count)

    kept = [t.clone() for t in (lens, table, free, count)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t, k in zip((lens, table, free, count), kept):
        t.copy_(k)
    for i in range(20):
        ended = (r.random(seqs) < 0.1).astype(np.int32)
        reset.copy_(i32(ended))
        graph.replay()
        want = oracle.serving.plan(s.lens, None, s.table, 16, tokens, s.pages, s.free, s.count, to_np(starts), ended)
        torch.cuda.synchronize()
        for g, w in zip((got.q_offsets, got.positions, got.slots, lens, table, free, count, got.lacking), want):
            assert np.array_equal(to_np(g).reshape(np.shape(w)), w), i
        s.lens, s.table, s.free, s.count = want[3], want[4], want[5], want[6]
        lens.add_(0)                                                      # eager work between


# ---- the next tokens --------------------------------------------------------------------


def check_sample(q4, x, u, what="", **settings):
    """x: float32 numpy [rows, vocab] of values that the type holds, or a GPU tensor."""
    import torch

    gpu = x if isinstance(x, torch.Tensor) else to_gpu(x)
    x = gpu.float().cpu().numpy()
    dev = {k: None if v is None else to_gpu(np.asarray(v, np.int32 if k == "top_k" else np.float32))
           for k, v in settings.items()}
    tokens, probs = q4.sample(gpu, to_gpu(np.asarray(u, np.float32)), **dev)
    tokens, probs = to_np(tokens), to_np(probs)
    for r in range(len(x)):
        own = {k: float(np.float32(v[r])) if k != "top_k" else int(v[r]) for k, v in settings.items() if v is not None}
        token, share = oracle.serving.sample(x[r].astype(np.float64), float(np.float32(u[r])), **own)
        assert tokens[r] == token, (what, r, own, u[r], tokens[r], token)
        assert abs(probs[r] - share) <= SHARE_TOL * share, (what, r, probs[r], share)
    return tokens, probs


DTYPES = ["float16", "bfloat16", "float32"]


def random_settings(r, rows, vocab):
    def some(x, off):
        return np.where(r.random(rows) < 0.6, x, off)

    return dict(temperature=some(r.uniform(0.2, 2.0, rows), 1.0) * (r.random(rows) < 0.9),
                top_k=some(r.integers(1, max(2, vocab // 3), rows), 0), top_p=some(r.uniform(0.05, 1.0, rows), 1.0),
                min_p=some(r.uniform(0.001, 0.5, rows), 0.0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 3, 63, 64, 65, 255, 1000, 1023, 1024, 1025, 4097, 16384, 16385, 50257])
def test_sample_sizes(q4, dtype, vocab):
    import torch

    say("sample", dtype, vocab)
    r = np.random.default_rng(vocab)
    rows = 12
    x = to_gpu((r.standard_normal((rows, vocab)) * r.uniform(0.1, 6.0, (rows, 1))).astype(np.float32))
    x = x.to(getattr(torch, dtype))
    check_sample(q4, x, r.random(rows), **random_settings(r, rows, vocab))
    check_sample(q4, x, r.random(rows))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [4096, 16385, 32000, 32767, 32768, 32769])
def test_sample_many_rows(q4, dtype, vocab):
    import torch

    say("sample", dtype, vocab)
    r = np.random.default_rng(vocab + 1)
    rows = 33                                              # more than those that are split from 16385 logits on
    x = to_gpu((r.standard_normal((rows, vocab)) * r.uniform(0.1, 6.0, (rows, 1))).astype(np.float32))
    x = x.to(getattr(torch, dtype))
    check_sample(q4, x, r.random(rows), **random_settings(r, rows, vocab))


def test_sample_large(q4):
    """The largest vocabulary, and 128256 logits with every kind of cut."""
    import torch

    r = np.random.default_rng(1)
    x = torch.randn(2, 1 << 20, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    check_sample(q4, x, [0.3, 0.999], top_p=[0.8, 1.0])
    x = 3 * torch.randn(6, 128256, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    check_sample(q4, x, r.random(6), temperature=[0.7, 1.0, 1.3, 0.0, 5.0, 0.1], top_k=[50, 0, 100000, 0, 20, 0],
                 top_p=[0.9, 0.95, 0.5, 1.0, 1.0, 0.99], min_p=[0.0, 0.0, 0.0, 0.0, 0.1, 0.05])


@pytest.mark.parametrize("dtype", DTYPES)
def test_sample_ties(q4, dtype):
    """Few distinct logits: the cuts go through runs of equal ones, which stay in the order of indexes."""
    import torch

    r = np.random.default_rng(2)
    rows, vocab = 40, 3001
    x = to_gpu(r.integers(-3, 3, (rows, vocab)).astype(np.float32)).to(getattr(torch, dtype))
    check_sample(q4, x, r.random(rows), **random_settings(r, rows, vocab))
    x = torch.zeros(8, 20000, device="cuda", dtype=getattr(torch, dtype))
    x[1::2] = -0.0
    x[:, ::2] = 0.0
    check_sample(q4, x, r.random(8), top_k=[0, 1, 7, 19999, 20000, 0, 5000, 3], top_p=[1, 1, 1, 1, 1, 0.25, 0.5, 0.9],
                 temperature=[1, 0, 1, 2, 1, 1, 1, 1])


def test_sample_masked_and_not_finite(q4):
    inf, nan = np.inf, np.nan
    low = np.finfo(np.float32).min
    x = np.full((14, 300), -inf, np.float32)
    x[1, 7] = -5.0
    x[2, [3, 250]] = [1.0, 2.0]
    x[3] = nan
    x[4, 100:] = nan
    x[4, :100] = np.linspace(-1, 1, 100)
    x[5, [4, 9, 200]] = inf
    x[5, 10:20] = 3.0
    x[6] = low
    x[7] = low
    x[7, 33] = 0.0
    x[8] = inf
    x[9, :10] = low
    x[9, 5] = nan
    x[10, 299] = 1e38
    x[10, 0] = -1e38
    x[11, :] = 1e-42
    x[12, :] = np.finfo(np.float32).max
    x[13, ::2] = low
    u = np.linspace(0.05, 0.95, 14)
    for settings in ({}, dict(top_k=[3] * 14), dict(top_p=[0.5] * 14), dict(min_p=[0.3] * 14),
                     dict(temperature=[0.0] * 14), dict(temperature=[inf] * 14), dict(temperature=[1e-30] * 14),
                     dict(temperature=[1e38] * 14, top_k=[200] * 14, top_p=[0.7] * 14, min_p=[0.9] * 14)):
        tokens, _ = check_sample(q4, x, u, settings, **settings)
        assert tokens[0] == -1 and tokens[3] == -1 and tokens[1] == 7
    h = np.full((2, 4096), np.finfo(np.float16).min, np.float16)          # a mask of the type's lowest value
    h[1, 17] = 1.0
    check_sample(q4, to_gpu(h), [0.5, 0.5])


@pytest.mark.parametrize("vocab", [4096, 32000, 50257, 131072, 1 << 20])
@pytest.mark.parametrize("steps", [0.49, 1.49, 77.3, 1e6])
def test_sample_flat_tails(q4, vocab, steps):
    """One peak and a flat tail of `steps` weight steps each, all rounded the same way: the worst that the fixed point
    does to a sum. The token drawn holds u * total up to vocab * 2^-(s + 1) of the peak's weight and 2^-47 of the total."""
    say("sample, flat tail", vocab, steps)
    s = min(50, 62 - int(np.ceil(np.log2(vocab))))
    x = np.full(vocab, np.log(steps * 2.0 ** -s), np.float32)
    x[5] = 0.0
    w = np.exp(x.astype(np.longdouble))
    upto, n = np.cumsum(w), 400
    total = upto[-1]
    r = np.random.default_rng(vocab)
    # draws at the tail: one u in 2^-24 of the range reaches it where it is light
    reach = min(1.0, 1.5 * float(total - 1) + 2.0 ** -23)
    u = np.concatenate([1 - 2.0 ** -24 * np.arange(1, 5), 1 - r.random(n - 4) * reach]).astype(np.float32)
    u = np.minimum(u, np.float32(1 - 2.0 ** -24))
    tokens, _ = q4.sample(to_gpu(x[None]).expand(n, vocab), to_gpu(u))
    tokens = to_np(tokens)
    want = u.astype(np.longdouble) * total
    bound = vocab * 2.0 ** -(s + 1) + 2.0 ** -47 * total
    assert np.all((tokens >= 0) & (tokens < vocab))
    over, under = want - upto[tokens], upto[tokens] - w[tokens] - want
    say("  worst share of the bound", max(over.max(), under.max()) / bound, "tokens off the peak", int((tokens != 5).sum()))
    assert np.all(over <= bound) and np.all(under <= bound), (over.max(), under.max(), bound)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("vocab", [300, 17000])
def test_sample_spreads_beyond_float32(q4, dtype, vocab):
    """Finite logits that lie further apart than float32 reaches have weight where the temperature is as large, or
    infinite: every cut counts them."""
    import torch

    say("sample, spread logits", dtype, vocab)
    inf = np.inf
    r = np.random.default_rng(12)
    top = float(torch.finfo(getattr(torch, dtype)).max)
    x = np.full((10, vocab), -inf, np.float32)
    x[0, [1, vocab - 1]] = [top, -top]
    x[1, [1, vocab - 1]] = [-top, top]
    x[2, ::3], x[2, 1::3] = top, -top
    x[3, 5:9] = [top, -top, -top, 0.0]
    x[4] = top * r.uniform(-1, 1, vocab)
    x[5] = top * r.choice([-1.0, -0.5, 0.0, 0.5, 1.0], vocab)
    x[6] = -top
    x[6, 77] = top
    x[7, 200:] = top * r.uniform(-1, 0, vocab - 200)
    x[7, 3] = top
    x[8] = 1e31 * r.standard_normal(vocab)
    x[8, 9] = top
    x[9, [2, 4]] = [inf, top]
    x = to_gpu(x).to(getattr(torch, dtype))
    u = np.array([0.95, 0.03, 0.61, 0.7, 0.33, 0.88, 0.52, 0.47, 0.99, 0.2])
    for t in (inf, 3e38, 1e38, 2e37):
        for settings in ({}, dict(top_k=[3] * 10), dict(top_k=[200] * 10), dict(top_p=[0.99] * 10), dict(top_p=[0.3] * 10),
                         dict(min_p=[0.05] * 10), dict(top_k=[150] * 10, top_p=[0.8] * 10, min_p=[0.01] * 10)):
            check_sample(q4, x, u, (t, settings), temperature=[t] * 10, **settings)
    tokens, _ = check_sample(q4, x[:1], [0.95], temperature=[3e38], top_p=[0.99])
    assert tokens[0] == vocab - 1


def test_sample_settings_out_of_range(q4):
    r = np.random.default_rng(3)
    inf, nan = np.inf, np.nan
    x = np.tile(r.standard_normal((1, 500)).astype(np.float32), (30, 1))
    t = [1, -1, nan, inf, 1e-45, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 0.5, 0.5, 0.5]
    k = [0, 0, 0, 0, 0, -5, 500, 501, 2 ** 31 - 1, 1, 499, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 7, 7, 7]
    p = [1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 0, -1, nan, 2, 1e-30, inf, -inf, 1, 1, 1, 1, 1, 1, 1, 1, 1, 0.5, 0.5, 0]
    m = [0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 2, nan, -1, inf, 1e-40, 0, 0, 0, 0.2, 0, 0]
    u = r.random(30)
    u[24:27] = [nan, -0.5, 1.5]
    u[0], u[1], u[2] = 0.0, 1.0, 1 - 2.0 ** -24
    u[27:] = [0.0, 1 - 2.0 ** -24, 1.0]
    with np.errstate(all="ignore"):
        check_sample(q4, x, u, temperature=t, top_k=k, top_p=p, min_p=m)


def test_sample_strided_and_in_place_outputs(q4):
    import torch

    r = np.random.default_rng(4)
    wide = torch.randn(9, 1301, device="cuda").to(torch.float16)
    for first, n in ((0, 1300), (1, 1300), (3, 777)):                      # rows at odd addresses
        check_sample(q4, wide[:, first:first + n], r.random(9), top_p=[0.9] * 9)
    check_sample(q4, wide[::3], r.random(3), top_k=[5] * 3)
    out = torch.full((9,), 77, dtype=torch.int32, device="cuda")
    probs = torch.full((9,), 77.0, device="cuda")
    a, b = q4.sample(wide, torch.rand(9, device="cuda"), out=out, probs_out=probs)
    assert a is out and b is probs and int((out == 77).sum()) < 9
    a, b = q4.sample(wide[:0], torch.rand(0, device="cuda"))
    assert a.shape == (0,) and b.shape == (0,)
    for n in (1000, 40001):
        one = torch.randn(1, n, device="cuda").expand(5, n)                # several draws from the same logits
        check_sample(q4, one, r.random(5), top_k=[0, 0, 9, 0, 3], top_p=[1.0, 0.9, 0.8, 0.1, 1.0])
    over = torch.randn(5 * 900, device="cuda").as_strided((5, 1500), (700, 1))   # rows that overlap
    check_sample(q4, over, r.random(5), top_p=[0.95] * 5)


def test_sample_rows_far_apart(q4):
    """Rows whose offsets pass 32 bits, in bytes and in elements."""
    import torch

    r = np.random.default_rng(11)
    apart = (1 << 31) + 17
    for n in (3000, 40001):
        memory = torch.empty(2 * apart + n, dtype=torch.float16, device="cuda")
        x = memory.as_strided((3, n), (apart, 1))
        x.copy_(2 * torch.randn(3, n, device="cuda"))
        check_sample(q4, x, r.random(3), top_k=[0, 30, 0], top_p=[1.0, 0.9, 0.8])
        del memory, x


def test_workspaces(q4):
    """A workspace holds anything on entry; more rows' serves fewer; one too small is refused."""
    import torch

    x, u = 2 * torch.randn(50, 20000, device="cuda"), torch.rand(50, device="cuda")
    p, k = torch.full((50,), 0.9, device="cuda"), torch.full((50,), 300, dtype=torch.int32, device="cuda")
    ws = torch.full((q4.sample_workspace_bytes(50, 20000),), 0xA5, dtype=torch.uint8, device="cuda")
    want = q4.sample(x, u, None, k, p)
    for rows in (50, 33, 32, 7):
        for fill in (0xFF, 0x7F, 0):
            ws.fill_(fill)
            got = q4.sample(x[:rows], u[:rows], None, k[:rows], p[:rows], workspace=ws)
            assert torch.equal(got[0], want[0][:rows]) and torch.equal(got[1], want[1][:rows])
    with pytest.raises(q4.Q4Error):
        q4.sample(x[:32], u[:32], workspace=ws[:1024])
    seqs, new = 5, 500
    lens = torch.tensor([0, 40, 16, 5, 300], dtype=torch.int32, device="cuda")
    news = torch.full((seqs,), new, dtype=torch.int32, device="cuda")

    def plan(**kw):
        table = torch.arange(seqs * 60, dtype=torch.int32, device="cuda").view(seqs, 60)
        return q4.paged_plan(lens, news, table, 16, seqs * new, pages=seqs * 60, **kw)

    want = plan()
    for fill in (-1, 2 ** 31 - 1, 0):
        got = plan(workspace=torch.full((2 * seqs + 2,), fill, dtype=torch.int32, device="cuda"))
        assert all(torch.equal(getattr(got, f), getattr(want, f)) for f in ("q_offsets", "positions", "slots", "kv_lens"))
    with pytest.raises(q4.Q4Error):
        plan(workspace=torch.zeros(2 * seqs + 1, dtype=torch.int32, device="cuda"))


def test_sample_distribution(q4):
    """Equally spaced uniforms meet each token as often as its share says, to one draw."""
    import torch

    n = 4096
    x = torch.tensor([0.3, -1.0, 2.0, 0.0, -np.inf, 1.5, -2.0], device="cuda").expand(n, 7).contiguous()
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    tokens, probs = q4.sample(x, u, temperature=torch.full((n,), 0.7, device="cuda"))
    want = torch.softmax(x[0].double() / 0.7, 0).cpu().numpy()
    seen = np.bincount(to_np(tokens), minlength=7)
    assert np.all(np.abs(seen - want * n) <= 1), (seen, want * n)
    assert np.allclose(to_np(probs), want[to_np(tokens)], rtol=1e-6)


def test_sample_captured_and_streams(q4):
    """Captured once, replayed with other logits and settings; two streams at once; each as eager."""
    import torch

    rows, vocab = 5, 40000
    x = torch.zeros(rows, vocab, device="cuda", dtype=torch.float16)
    u = torch.zeros(rows, device="cuda")
    t, p = torch.ones(rows, device="cuda"), torch.ones(rows, device="cuda")
    k = torch.zeros(rows, device="cuda", dtype=torch.int32)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q4.sample(x, u, t, k, p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = q4.sample(x, u, t, k, p)
    gen = torch.Generator("cuda").manual_seed(5)
    for i in range(6):
        x.copy_(2 * torch.randn(rows, vocab, device="cuda", generator=gen))
        u.copy_(torch.rand(rows, device="cuda", generator=gen))
        t.copy_(torch.rand(rows, device="cuda", generator=gen) * (i != 2))
        p.fill_(1.0 if i % 2 else 0.8)
        k.fill_(0 if i < 3 else 40 * i)
        graph.replay()
        torch.cuda.synchronize()
        want = q4.sample(x, u, t, k, p)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [2 * torch.randn(7, vocab, device="cuda", generator=gen) for _ in range(2)]
    us = [torch.rand(7, device="cuda", generator=gen) for _ in range(2)]
    want = [q4.sample(a, b) for a, b in zip(xs, us)]
    torch.cuda.synchronize()
    res = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                res[i].append(q4.sample(xs[i], us[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in res[i]:
            assert torch.equal(r[0], want[i][0]) and torch.equal(r[1], want[i][1])
