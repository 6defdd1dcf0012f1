"""A serving loop on the GPU (needs an MI355X): plan, append, attention behind shared prefixes and the choice
of tokens, around one layer's products: shared prompts, questions, decode steps with requests that end and
others that take their places; eager and captured.

Every stage is checked against the float64 oracle on the GPU's own inputs to it.
"""

import numpy as np
import pytest

import oracle
import synth
from gpu_util import say, to_gpu, to_np

pytestmark = pytest.mark.gpu

HQ, HKV, D, G, PAGE, HID, VOCAB = 8, 2, 64, 64, 16, 512, 1000
QKV = (HQ + 2 * HKV) * D


@pytest.fixture(scope="module")
def q4():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import w4a16_decode_amd as q4mod

    say("libq4", q4mod.version())
    return q4mod


def i32(a):
    return to_gpu(np.asarray(a, dtype=np.int32))


class Model:
    """One layer between an embedding and a head, and the state of a batch of places."""

    def __init__(self, q4, seqs, prefix, group_offsets, blocks, pages, seed):
        import torch

        r = np.random.default_rng(seed)
        self.q4, self.seqs, self.blocks, self.pages = q4, seqs, blocks, pages
        self.w = {n: q4.quantize_pack(to_gpu(synth.weight(o, i, seed=seed + o)), 128)
                  for n, o, i in (("qkv", QKV, HID), ("o", HID, HQ * D), ("head", VOCAB, HID))}
        self.embed = to_gpu(r.standard_normal((VOCAB, HID)).astype(np.float16))
        self.rope = q4.rope_table(1024, D)
        self.cache = q4.paged_kv_alloc(pages, PAGE, HKV, D, G)
        self.pool = q4.page_pool(pages)
        self.table = torch.full((seqs, blocks), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        # the prefixes: sequences of a plan of their own, whose table is then the prefix table
        self.prefix, self.groups = np.array(prefix), np.array(group_offsets)
        of = np.searchsorted(self.groups, np.arange(seqs), side="right") - 1
        self.starts = i32(self.prefix[of])
        self.ptable = torch.full((len(prefix), max(prefix) // PAGE + 1), -1, dtype=torch.int32, device="cuda")
        plan = q4.paged_plan(torch.zeros(len(prefix), dtype=torch.int32, device="cuda"), i32(prefix), self.ptable, PAGE,
                             int(sum(prefix)), self.pool, free_count_out=self.pool.count)
        ids = i32(r.integers(0, VOCAB, int(sum(prefix))))
        self.heads(self.embed.index_select(0, ids), plan)
        self.plens, self.goff = i32(prefix), i32(group_offsets)

    def heads(self, x, plan):
        q4 = self.q4
        qkv = q4.gemm(x, self.w["qkv"]).view(-1, HQ + 2 * HKV, D)
        return q4.qk_norm_rope_append(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], plan.positions, self.rope,
                                      self.cache, plan.slots)

    def step(self, ids, new, reset, u, settings, rows, max_q, max_group_q, last=None, keep=None):
        """ids: the rows' tokens; last: rows whose logits are needed (all). The state moves on in place."""
        q4 = self.q4
        plan = q4.paged_plan(self.lens, new, self.table, PAGE, rows, self.pool, starts=self.starts, reset=reset,
                             kv_lens_out=self.lens, free_count_out=self.pool.count)
        q = self.heads(self.embed.index_select(0, ids), plan)
        o = q4.paged_attention_shared(q, self.cache, self.ptable, self.plens, self.goff, self.table, plan.q_offsets,
                                      self.lens, max_q, self.blocks * PAGE, max_group_q, int(self.prefix.max()))
        h = o.view(rows, HQ * D)
        if last is not None:
            h = h.index_select(0, last)
        logits = q4.gemm(q4.gemm(h, self.w["o"]), self.w["head"])
        tokens, probs = q4.sample(logits, u, **settings)
        if keep is not None:
            keep.update(plan=plan, q=q, o=o, logits=logits, tokens=tokens, probs=probs)
        return tokens

    def state(self):
        return [to_np(t).copy() for t in (self.lens, self.table, self.pool.pages, self.pool.count)]

    def values(self, table, length):
        t = np.arange(length)
        slots = (table[t // PAGE] * PAGE + t % PAGE).astype(np.int32)
        return [to_np(t).astype(np.float64) for t in self.q4.paged_kv_dequant(self.cache, to_gpu(slots))]

    def check(self, before, new, reset, u, settings, rows, keep):
        lens, table, free, count = before
        want = oracle.serving.plan(lens, new, table, PAGE, rows, self.pages, free, int(count[0]), to_np(self.starts), reset)
        p = keep["plan"]
        got = (p.q_offsets, p.positions, p.slots, self.lens, self.table, self.pool.pages, self.pool.count, p.lacking)
        for g, w in zip(got, want):
            assert np.array_equal(to_np(g).reshape(np.shape(w)), w)
        assert want[7] == 0
        off, lens, table = want[0], want[3], want[4]
        pk, pv = zip(*(self.values(t, n) for t, n in zip(to_np(self.ptable), self.prefix)))
        k, v = zip(*(self.values(table[s], lens[s]) if lens[s] else [np.zeros((0, HKV, D))] * 2 for s in range(self.seqs)))
        q = to_np(keep["q"])
        ref = oracle.paged.attention_shared(q, pk, pv, self.groups, k, v, lens, off, D ** -0.5)
        mag = oracle.paged.attention_shared(q, pk, [np.abs(t) for t in pv], self.groups, k, [np.abs(t) for t in v], lens,
                                            off, D ** -0.5)
        top = max(np.abs(t).max() for t in pk + k if t.size)
        z = 1 + np.abs(q.astype(np.float64)).sum(-1).max() * top * D ** -0.5
        # weights, V values, output 2^-11 each; keys: each score off by 2^-11 z at most, twice
        err = np.abs(to_np(keep["o"]) - ref)[:off[-1]]
        assert np.all(err <= ((3 + 2 * z) * 2.0 ** -11 * mag)[:off[-1]])
        logits = to_np(keep["logits"]).astype(np.float64)
        for r, x in enumerate(logits):
            own = {n: t[r].item() for n, t in settings.items()}
            token, share = oracle.serving.sample(x, u[r].item(), **own)
            assert token == int(keep["tokens"][r])
            assert abs(share - float(keep["probs"][r])) <= 2.0 ** -22 * share


def settings_of(seqs, seed):
    import torch

    r = np.random.default_rng(seed)
    return dict(temperature=to_gpu(r.uniform(0.5, 1.5, seqs).astype(np.float32)), top_k=i32(r.integers(0, 60, seqs)),
                top_p=to_gpu(r.uniform(0.6, 1.0, seqs).astype(np.float32)), min_p=torch.zeros(seqs, device="cuda"))


def test_loop(q4):
    """Questions behind two prompts, then decode steps; requests end, others begin in their places."""
    import torch

    seqs = 5
    m = Model(q4, seqs, [50, 33], [0, 3, 5], 6, 60, seed=3)
    r = np.random.default_rng(4)
    settings = settings_of(seqs, 5)
    ids = None
    for step in range(8):
        reset = np.zeros(seqs, np.int32) if step == 0 else (r.random(seqs) < 0.2).astype(np.int32)
        new = np.array([7, 1, 20, 16, 3]) if step == 0 else np.where(reset, r.integers(1, 12, seqs), 1)
        rows = int(new.sum())
        fresh = r.integers(0, VOCAB, rows)
        off = np.concatenate([[0], np.cumsum(new)])
        if ids is not None:
            for s in range(seqs):
                if not reset[s]:
                    fresh[off[s]] = int(ids[s])
        u = torch.rand(seqs, device="cuda")
        before, keep = m.state(), {}
        groups = [off[3], rows - off[3]]
        ids = m.step(i32(fresh), i32(new), i32(reset), u, settings, rows, int(new.max()), int(max(groups)),
                     last=to_gpu(off[1:] - 1), keep=keep)
        say("loop step", step, new, reset)
        m.check(before, new, reset, u, settings, rows, keep)


def test_loop_captured(q4):
    """Decode steps captured as a loop that feeds itself: tokens, lengths, tables and pool as the eager loop's,
    with its own eager work between the replays."""
    import torch

    seqs = 6
    models = [Model(q4, seqs, [70, 20, 5], [0, 2, 4, 6], 8, 80, seed=7) for _ in range(2)]  # eager, captured
    settings = settings_of(seqs, 8)
    new = np.array([5, 9, 1, 17, 2, 30])
    off = np.concatenate([[0], np.cumsum(new)])
    first = i32(np.random.default_rng(9).integers(0, VOCAB, off[-1]))
    u0 = torch.rand(seqs, device="cuda")
    ids = [m.step(first, i32(new), None, u0, settings, int(off[-1]), 30, 32, last=to_gpu(off[1:] - 1)) for m in models]
    assert torch.equal(*ids)
    reset, u = torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.zeros(seqs, device="cuda")
    loop = ids[1].clone()
    cap = models[1]
    kept = [t.clone() for t in (cap.lens, cap.table, cap.pool.pages, cap.pool.count, loop)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cap.step(loop, None, reset, u, settings, seqs, 1, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.copy_(cap.step(loop, None, reset, u, settings, seqs, 1, 2))
    for t, k in zip((cap.lens, cap.table, cap.pool.pages, cap.pool.count, loop), kept):
        t.copy_(k)
    r = np.random.default_rng(10)
    eager = ids[0]
    for step in range(12):
        reset.copy_(i32((r.random(seqs) < 0.15).astype(np.int32)))
        u.copy_(torch.rand(seqs, device="cuda"))
        graph.replay()
        eager = models[0].step(eager, None, reset, u, settings, seqs, 1, 2)
        torch.cuda.synchronize()
        assert torch.equal(eager, loop), step
        for a, b in zip(models[0].state(), cap.state()):
            assert np.array_equal(a, b), step
    # what the lengths cover (the step before the capture left its codes behind them)
    lens, table = models[0].state()[:2]
    for s in range(seqs):
        for a, b in zip(models[0].values(table[s], lens[s]), cap.values(table[s], lens[s])):
            assert np.array_equal(a, b), s
