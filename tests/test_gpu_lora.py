"""The product with adapters on the GPU against the oracle (float64).

With all-zero weights the result is the adapters' part alone. Its bound: A x is a float32 sum
of in / 32 matrix steps and up to 32 joins, B t one of rank terms after a product with
the scaling: (in / 32 + 32 + rank + 2) 2^-23 relative to scaling * sum_r |B| sum_k |A| |x|,
then half a float16 step 2^-11 (subnormal: 2^-25). With real weights the suite's
tolerance of a product holds (gpu_util), and a row without an adapter has gemm's bits.
"""

import numpy as np
import pytest

import oracle
import synth
from gpu_util import assert_close, say, to_gpu, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import w4a16_decode_amd as q4mod

    say("libq4", q4mod.version())
    return q4mod


def _adapters(n, rank, N, K, seed):
    r = np.random.default_rng(seed)
    a = (r.standard_normal((n, rank, K)) / np.sqrt(K)).astype(np.float16)
    b = (0.3 * r.standard_normal((n, N, rank))).astype(np.float16)
    return a, b, (0.5 + r.random(n)).astype(np.float32)


def _ids(B, n, kind, seed):
    r = np.random.default_rng(seed)
    if kind == "same":
        return np.zeros(B, np.int32)
    if kind == "runs":
        return np.repeat(r.integers(-1, n, B), 5)[:B].astype(np.int32)
    ids = r.integers(-1, n, B).astype(np.int32)
    if B > 3:
        ids[1], ids[3] = n, 2 ** 31 - 1                # outside the adapters
    return ids


SHAPES = [  # B, N, K, g, rank, adapters, ids
    (1, 256, 256, 128, 8, 1, "same"),
    (1, 4096, 4096, 128, 16, 3, "mixed"),
    (2, 17, 96, 32, 16, 2, "mixed"),
    (3, 8192, 8192, 128, 24, 4, "mixed"),
    (4, 1000, 1024, 64, 32, 5, "mixed"),
    (13, 515, 2048, 128, 64, 20, "mixed"),
    (16, 300, 7168, 128, 128, 16, "mixed"),
    (17, 1037, 512, 128, 16, 3, "runs"),
    (50, 640, 1152, 128, 40, 7, "mixed"),
    (100, 2048, 4096, 128, 16, 30, "mixed"),
    (200, 515, 1024, 32, 64, 4, "runs"),
]


@pytest.mark.parametrize("B,N,K,g,rank,n,kind", SHAPES)
def test_adapters_alone(q4, B, N, K, g, rank, n, kind):
    import torch

    say("adapters alone", B, N, K, g, rank, n, kind)
    a, b, s = _adapters(n, rank, N, K, seed=B + N)
    ids = _ids(B, n, kind, seed=B)
    x = synth.activation(B, K, seed=B)
    qw = q4.quantize_pack(torch.zeros((N, K), dtype=torch.float16, device="cuda"), g)
    y = to_np(q4.gemm_lora(to_gpu(x), qw, q4.LoraAdapters(to_gpu(a), to_gpu(b), to_gpu(s)), to_gpu(ids)))
    ref = oracle.lora.lora_delta(x, a, b, s, ids)
    mag = oracle.lora.lora_delta(np.abs(x), np.abs(a), np.abs(b), s, ids)
    bound = (K / 32 + 32 + rank + 2) * 2.0 ** -23 * mag + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    err = np.abs(y.astype(np.float64) - ref)
    assert np.all(err <= bound), (err / bound).max()
    say("  worst share of the bound", (err / bound).max())


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("B,N,K,g,rank,n,kind", SHAPES)
def test_beside_the_product(q4, B, N, K, g, rank, n, kind, asym):
    import torch

    say("beside the product", B, N, K, g, rank, n, kind, asym)
    W = synth.weight(N, K, seed=N)
    a, b, s = _adapters(n, rank, N, K, seed=B + N)
    ids = _ids(B, n, kind, seed=B)
    x = to_gpu(synth.activation(B, K, seed=B + 1))
    qw = q4.quantize_pack(to_gpu(W), g, asym)
    y = q4.gemm_lora(x, qw, q4.LoraAdapters(to_gpu(a), to_gpu(b), to_gpu(s)), to_gpu(ids))
    plain = q4.gemm(x, qw)
    without = torch.from_numpy((ids < 0) | (ids >= n)).cuda()
    assert torch.equal(y[without], plain[without])
    if asym:
        w_hat = oracle.dequant_asym(*oracle.quantize_asym(W, g), g)
    else:
        w_hat = oracle.dequant_sym(*oracle.quantize_sym(W, g), g)
    ref = oracle.gemm_ref(to_np(x), w_hat) + oracle.lora.lora_delta(to_np(x), a, b, s, ids)
    assert_close(to_np(y), ref, "beside the product")
    again = q4.gemm_lora(x, qw, q4.LoraAdapters(to_gpu(a), to_gpu(b), to_gpu(s)), to_gpu(ids))
    assert torch.equal(y, again)


def test_no_adapters_and_no_rows(q4):
    import torch

    x = to_gpu(synth.activation(5, 256, seed=1))
    qw = q4.quantize_pack(to_gpu(synth.weight(64, 256, seed=2)), 128)
    e = q4.LoraAdapters(torch.empty((0, 8, 256), dtype=torch.float16, device="cuda"),
                        torch.empty((0, 64, 8), dtype=torch.float16, device="cuda"),
                        torch.empty(0, dtype=torch.float32, device="cuda"))
    ids = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert torch.equal(q4.gemm_lora(x, qw, e, ids), q4.gemm(x, qw))
    a = q4.LoraAdapters(*(to_gpu(t) for t in _adapters(2, 8, 64, 256, 0)))
    assert q4.gemm_lora(x[:0], qw, a, ids[:0]).shape == (0, 64)


def test_workspace_and_refusals(q4):
    import torch

    x = to_gpu(synth.activation(5, 256, seed=1))
    qw = q4.quantize_pack(to_gpu(synth.weight(64, 256, seed=2)), 128)
    a = q4.LoraAdapters(*(to_gpu(t) for t in _adapters(2, 8, 64, 256, 0)))
    ids = torch.tensor([0, 1, -1, 1, 0], dtype=torch.int32, device="cuda")
    need = q4.workspace_bytes_lora(5, 64, 256, 128, 8)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    y = q4.gemm_lora(x, qw, a, ids, workspace=ws)
    assert torch.equal(y, q4.gemm_lora(x, qw, a, ids))
    assert bool((ws[need:] == 0xFF).all())
    with pytest.raises(q4.Q4Error):
        q4.gemm_lora(x, qw, a, ids, workspace=ws[:need - 16])
    with pytest.raises(ValueError):
        q4.gemm_lora(x, qw, a, ids[:4])
    with pytest.raises(TypeError):
        q4.gemm_lora(x, qw, a, ids.long())
    with pytest.raises(ValueError):
        q4.gemm_lora(x, qw, q4.LoraAdapters(a.a, a.b[:, :32].contiguous(), a.scaling), ids)
    bad = [to_gpu(t) for t in _adapters(2, 12, 64, 256, 0)]
    with pytest.raises(q4.Q4Error):
        q4.gemm_lora(x, qw, q4.LoraAdapters(*bad), ids)                  # rank 12


@pytest.mark.parametrize("rank", [8, 16, 24, 40])
def test_infinite_adapter_values(q4, rank):
    """An infinity in B or A reaches the outputs that the formula gives it to, as an infinity,
    also where the rank does not fill the kernel's registers."""
    import torch

    N, K = 300, 256
    a, b, s = _adapters(3, rank, N, K, seed=rank)
    x = np.abs(synth.activation(5, K, seed=rank))
    a, s = np.abs(a), np.abs(s)
    b[1, 7, rank - 1] = np.inf
    b[1, 9, 0] = -np.inf
    a[2, rank - 1, 3] = np.inf
    x[:, 3] = 1.0
    b[2] = np.abs(b[2]) + np.float16(2.0 ** -10)
    ids = np.array([0, 1, 2, -1, 1], dtype=np.int32)
    qw = q4.quantize_pack(torch.zeros((N, K), dtype=torch.float16, device="cuda"), 128)
    y = to_np(q4.gemm_lora(to_gpu(x), qw, q4.LoraAdapters(to_gpu(a), to_gpu(b), to_gpu(s)), to_gpu(ids)))
    assert np.isfinite(y[[0, 3]]).all() and not y[3].any()
    for r in (1, 4):
        assert y[r, 7] == np.inf and y[r, 9] == -np.inf
        assert np.isfinite(np.delete(y[r], [7, 9])).all()
    assert (y[2] == np.inf).all()


def test_two_calls_at_once(q4):
    """Calls on two streams at the same time, eager and captured, each with its own workspace: the bits
    that each gives alone."""
    import torch

    calls = []
    for B, N, K, rank, seed in ((3, 2048, 2048, 16, 1), (40, 1037, 1024, 32, 2)):
        qw = q4.quantize_pack(to_gpu(synth.weight(N, K, seed=seed)), 128)
        adapters = q4.LoraAdapters(*(to_gpu(t) for t in _adapters(4, rank, N, K, seed)))
        calls.append((to_gpu(synth.activation(B, K, seed=seed)), qw, adapters, to_gpu(_ids(B, 4, "mixed", seed))))
    want = [q4.gemm_lora(*c) for c in calls]
    streams, graphs, outs = [torch.cuda.Stream() for _ in calls], [], []
    torch.cuda.synchronize()
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(q4.gemm_lora(*c))
        graphs.append(graph)
    for i in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), i
        got = []
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(q4.gemm_lora(*c))
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(got, want)), i


def test_adapters_far_apart(q4):
    """Adapters whose offsets pass 32 bits (8.6 GB of A and of B): the same bits as from a short list."""
    import torch

    n, rank, N, K = 2050, 128, 8192, 8192
    say("adapters far apart")
    a = torch.zeros((n, rank, K), dtype=torch.float16, device="cuda")
    b = torch.zeros((n, N, rank), dtype=torch.float16, device="cuda")
    s = torch.ones(n, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    used = [0, 1030, n - 1]
    for i in used:
        a[i] = torch.randn((rank, K), generator=g, device="cuda") / 90
        b[i] = torch.randn((N, rank), generator=g, device="cuda") / 10
    qw = q4.quantize_pack(to_gpu(synth.weight(N, K, seed=3)), 128)
    x = to_gpu(synth.activation(5, K, seed=4))
    far = q4.gemm_lora(x, qw, q4.LoraAdapters(a, b, s), torch.tensor([n - 1, 0, 1030, -1, n - 1], dtype=torch.int32, device="cuda"))
    near = q4.gemm_lora(x, qw, q4.LoraAdapters(a[used].contiguous(), b[used].contiguous(), s[:3].contiguous()),
                        torch.tensor([2, 0, 1, -1, 2], dtype=torch.int32, device="cuda"))
    assert torch.equal(far, near) and not torch.equal(far, q4.gemm(x, qw))
