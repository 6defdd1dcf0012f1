"""The attention side of a decoder layer as a serving program runs it (needs an MI355X):
the q/k/v product with the requests' adapters, norm and rotation with the append into
the paged INT4 cache, attention over it, the output product with adapters -- a prompt
chunk of several sequences, then decode steps, eager, on another stream and captured.

Every stage is checked against the float64 oracle on the GPU's own inputs to it, with the
bounds of the stages' own tests.
"""

import numpy as np
import pytest

import oracle
import synth
from gpu_util import assert_close, say, to_gpu, to_np

pytestmark = pytest.mark.gpu

HQ, HKV, D, G, PAGE, HID, RANK, N_ADAPT = 8, 2, 128, 64, 32, 1024, 16, 3
QKV = (HQ + 2 * HKV) * D


@pytest.fixture(scope="module")
def q4():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import w4a16_decode_amd as q4mod

    say("libq4", q4mod.version())
    return q4mod


class Layer:
    def __init__(self, q4, seqs, blocks, seed):
        import torch

        r = np.random.default_rng(seed)
        self.q4, self.seqs = q4, seqs
        self.w = {n: synth.weight(o, i, seed=seed + o) for n, o, i in (("qkv", QKV, HID), ("o", HID, HQ * D))}
        self.qw = {n: q4.quantize_pack(to_gpu(w), 128) for n, w in self.w.items()}
        self.lora = {}
        for n, (o, i) in (("qkv", (QKV, HID)), ("o", (HID, HQ * D))):
            self.lora[n] = ((r.standard_normal((N_ADAPT, RANK, i)) / np.sqrt(i)).astype(np.float16),
                            (0.1 * r.standard_normal((N_ADAPT, o, RANK))).astype(np.float16),
                            (0.5 + r.random(N_ADAPT)).astype(np.float32))
        self.adapters = {n: q4.LoraAdapters(*(to_gpu(t) for t in v)) for n, v in self.lora.items()}
        self.norm = [(1 + 0.2 * r.standard_normal(D)).astype(np.float16) for _ in range(2)]
        self.g_norm = [to_gpu(t) for t in self.norm]
        self.table = q4.rope_table(blocks * PAGE, D)
        self.cos_sin = to_np(self.table)
        pages = seqs * blocks + 2
        self.cache = q4.paged_kv_alloc(pages, PAGE, HKV, D, G)
        self.block_table = r.permutation(pages)[:seqs * blocks].reshape(seqs, blocks).astype(np.int32)
        self.g_block_table = to_gpu(self.block_table)
        self.max_kv = blocks * PAGE

    def slots(self, seq, positions):
        p = np.asarray(positions)
        return self.block_table[seq][p // PAGE] * PAGE + p % PAGE

    def step(self, x, ids, positions, slots, offsets, lens, max_q, keep=None):
        """One layer step; everything between the products stays on the GPU."""
        q4 = self.q4
        qkv = q4.gemm_lora(x, self.qw["qkv"], self.adapters["qkv"], ids).view(-1, HQ + 2 * HKV, D)
        q = q4.qk_norm_rope_append(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], positions, self.table, self.cache,
                                   slots, *self.g_norm)
        o = q4.paged_attention(q, self.cache, self.g_block_table, offsets, lens, max_q, self.max_kv)
        y = q4.gemm_lora(o.view(-1, HQ * D), self.qw["o"], self.adapters["o"], ids)
        if keep is not None:
            keep.update(qkv=qkv, q=q, o=o, y=y)
        return y

    def product(self, name, x, ids):
        codes, scales = oracle.quantize_sym(self.w[name], 128)
        return oracle.gemm_ref(x, oracle.dequant_sym(codes, scales, 128)) + oracle.lora.lora_delta(x, *self.lora[name], ids)

    def check(self, x, ids, positions, offsets, lens, keep):
        """Each stage of a step against the oracle, given the GPU's inputs to the stage."""
        qkv, q, o, y = (to_np(keep[n]) for n in ("qkv", "q", "o", "y"))
        assert_close(qkv.reshape(-1, QKV), self.product("qkv", x, ids), "q/k/v product")
        cs = self.cos_sin[positions]
        ref_q = oracle.paged.norm_rope(qkv[:, :HQ], self.norm[0], 1e-6, cs[..., 0], cs[..., 1])
        assert np.abs(q - ref_q).max() <= 2.0 ** -10 * np.abs(ref_q).max()
        ref_k = oracle.paged.norm_rope(qkv[:, HQ:HQ + HKV], self.norm[1], 1e-6, cs[..., 0], cs[..., 1])
        ref_k = ref_k.astype(np.float32).astype(np.float16)
        # what the cache holds of the new tokens, and of everything before
        k_all, v_all = [], []
        for n, length in enumerate(lens):
            k, v = (to_np(t) for t in self.q4.paged_kv_dequant(self.cache, to_gpu(
                self.slots(n, np.arange(length)).astype(np.int32))))
            a, b = offsets[n], offsets[n + 1]
            new = slice(length - (b - a), length)
            for got, rows in ((k, ref_k[a:b]), (v, qkv[a:b, HQ + HKV:])):
                want = oracle.paged.store(np.ascontiguousarray(rows), G)[2].astype(np.float16)
                assert np.array_equal(got[new], want)
            k_all.append(k.astype(np.float64)), v_all.append(v.astype(np.float64))
        # float16 values of code * scale are within 2^-11 of the products attention uses
        ref_o = oracle.paged.attention(q, k_all, v_all, lens, offsets, D ** -0.5)
        mag = oracle.paged.attention(q, k_all, [np.abs(v) for v in v_all], lens, offsets, D ** -0.5)
        z = 1 + max(np.abs(q.astype(np.float64)).sum(-1).max() * max(np.abs(k).max() for k in k_all) * D ** -0.5, 0)
        # weights (2^-11), V values (2^-11), output (2^-11), keys: each score off by 2^-11 Z at most, twice
        assert np.all(np.abs(o - ref_o) <= (3 + 2 * z) * 2.0 ** -11 * mag)
        assert_close(y, self.product("o", o.reshape(-1, HQ * D), ids), "output product")


def _i32(a):
    return to_gpu(np.asarray(a, dtype=np.int32))


def _plan(layer, lens, news, ids):
    """Host plan of a step: the newest `news` tokens of sequences of `lens`."""
    offsets = np.concatenate([[0], np.cumsum(news)])
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, news)])
    slots = np.concatenate([layer.slots(i, np.arange(n - m, n)) for i, (n, m) in enumerate(zip(lens, news))])
    return offsets, pos, slots, np.repeat(ids, news)


def test_chunk_then_decode(q4):
    layer = Layer(q4, 3, 4, seed=1)
    ids = np.array([2, -1, 0])
    lens = np.array([37, 5, 64])
    news = lens.copy()
    for step in range(5):
        say("layer step", step, lens)
        offsets, pos, slots, row_ids = _plan(layer, lens, news, ids)
        x = synth.activation(int(offsets[-1]), HID, seed=100 + step)
        keep = {}
        layer.step(to_gpu(x), _i32(row_ids), _i32(pos), _i32(slots), _i32(offsets), _i32(lens), int(news.max()), keep)
        layer.check(x, row_ids, pos, offsets, lens, keep)
        news = np.array([20, 1, 1]) if step == 0 else np.ones(3, np.int64)      # a second chunk, then decode
        lens = lens + news


def test_decode_step_captured(q4):
    """A decode step captured once and replayed with other tokens, positions, slots and lengths,
    eager work in between: each replay gives the eager step's bits, in output and cache."""
    import torch

    layers = [Layer(q4, 4, 4, seed=2) for _ in range(2)]                    # eager, captured
    assert np.array_equal(layers[0].block_table, layers[1].block_table)
    lens = np.array([20, 33, 64, 100])
    ids = np.array([0, 1, -1, 2])
    for layer in layers:                                                    # the prompts
        offsets, pos, slots, row_ids = _plan(layer, lens, lens, ids)
        layer.step(to_gpu(synth.activation(int(offsets[-1]), HID, seed=7)), _i32(row_ids), _i32(pos), _i32(slots),
                   _i32(offsets), _i32(lens), int(lens.max()))
    buf = dict(x=torch.zeros((4, HID), dtype=torch.float16, device="cuda"), ids=_i32(ids), pos=_i32([0] * 4),
               slots=_i32([-1] * 4), off=_i32(range(5)), lens=_i32([1] * 4))
    cap = layers[1]

    def run():
        return cap.step(buf["x"], buf["ids"], buf["pos"], buf["slots"], buf["off"], buf["lens"], 1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for step in range(6):
        lens = lens + 1
        offsets, pos, slots, row_ids = _plan(layers[0], lens, np.ones(4, np.int64), ids)
        x = to_gpu(synth.activation(4, HID, seed=50 + step))
        want = layers[0].step(x, _i32(row_ids), _i32(pos), _i32(slots), _i32(offsets), _i32(lens), 1)
        for name, value in (("x", x), ("pos", _i32(pos)), ("slots", _i32(slots)), ("lens", _i32(lens))):
            buf[name].copy_(value)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), step
        for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(layers[0].cache, name), getattr(cap.cache, name)), (step, name)


def test_two_graphs_and_streams(q4):
    """Two captured attention calls replayed on two streams at once, each with its own workspace,
    and the same calls on a side stream: the eager bits every time."""
    import torch

    r = np.random.default_rng(3)
    calls = []
    for lens in ([900, 40, 333], [1500]):
        pages = sum(-(-n // PAGE) for n in lens) + 1
        cache = q4.paged_kv_alloc(pages, PAGE, HKV, D, G)
        kv = [to_gpu(r.standard_normal((pages * PAGE, HKV, D)).astype(np.float16)) for _ in range(2)]
        q4.paged_kv_append(*kv, cache, _i32(np.arange(pages * PAGE)))
        blocks = max(-(-n // PAGE) for n in lens)
        table = np.zeros((len(lens), blocks), np.int32)
        at = 0
        for i, n in enumerate(lens):
            need = -(-n // PAGE)
            table[i, :need] = np.arange(at, at + need)
            at += need
        q = to_gpu(r.standard_normal((len(lens), HQ, D)).astype(np.float16))
        calls.append((q, cache, _i32(table), _i32(np.arange(len(lens) + 1)), _i32(lens), 1, max(lens)))
    want = [q4.paged_attention(*c) for c in calls]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(q4.paged_attention(*c))
        graphs.append(g)
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    for s, c, w in zip(streams, calls, want):
        with torch.cuda.stream(s):
            got = q4.paged_attention(*c)
        s.synchronize()
        assert torch.equal(got, w)


def test_workspace_bounds(q4):
    """paged_attention writes its workspace and nothing behind it; a smaller one is refused."""
    import torch

    cache = q4.paged_kv_alloc(40, 16, 1, 128)
    q = torch.randn((1, 8, 128), device="cuda").half()
    table, off, lens = _i32([np.arange(40)]), _i32([0, 1]), _i32([640])
    need = q4.paged_attention_workspace_bytes(1, 1, 1, 640, 8, 1, 128, 128)
    assert need > 0
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    got = q4.paged_attention(q, cache, table, off, lens, 1, 640, workspace=ws)
    assert torch.equal(got, q4.paged_attention(q, cache, table, off, lens, 1, 640))
    assert bool((ws[need:] == 0x5A).all())
    with pytest.raises(q4.Q4Error):
        q4.paged_attention(q, cache, table, off, lens, 1, 640, workspace=ws[:need - 16])


def test_many_sequences_and_long_lines_of_work(q4):
    """More sequences than a wavefront has lanes, ragged, some empty: the shares of the work
    still give every row its keys (against the same rows one sequence at a time)."""
    import torch

    r = np.random.default_rng(4)
    lens = np.concatenate([r.integers(0, 1200, 150), [0, 4000, 1, 513]])
    pages = 300
    cache = q4.paged_kv_alloc(pages, 16, 1, 64, 32)
    kv = [to_gpu(r.standard_normal((pages * 16, 1, 64)).astype(np.float16)) for _ in range(2)]
    q4.paged_kv_append(*kv, cache, _i32(np.arange(pages * 16)))
    table = r.integers(0, pages, (len(lens), 250)).astype(np.int32)             # pages shared at random
    for new in (1, 3):
        rows = len(lens) * new
        q = to_gpu(r.standard_normal((rows, 6, 64)).astype(np.float16))
        off = np.arange(0, rows + 1, new)
        got = q4.paged_attention(q, cache, _i32(table), _i32(off), _i32(lens), new, 4000)
        for n in [0, 63, 64, 65, 100, 150, 151, 152, 153]:
            one = q4.paged_attention(q[n * new:(n + 1) * new], cache, _i32(table[n:n + 1]), _i32([0, new]),
                                     _i32(lens[n:n + 1]), new, 4000)
            a, b = to_np(got[n * new:(n + 1) * new]).astype(np.float64), to_np(one).astype(np.float64)
            # the two differ in where the keys are cut: float32 sums and two float16 roundings apart
            assert np.abs(a - b).max() <= 2.0 ** -9 * max(np.abs(b).max(), 2.0 ** -14), n
