"""torch-facing wrappers of include/q4_serve.h: the plan of a batch on the paged cache and
the choice of the next tokens.

As in attention.py, these functions check tensors, allocate outputs on the tensors'
device and pass raw pointers and torch's current HIP stream of that device to libq4.
"""

from __future__ import annotations

from dataclasses import dataclass

from . import _lib
from ._tensors import array, call, device, torch_
from .ops import _workspace


@dataclass
class PagePool:
    """The free pages of a paged cache: a stack, count[0] pages deep, its top at
    pages[count[0] - 1]."""

    pages: object   # int32 [pages of the cache]
    count: object   # int32 [1]


def page_pool(pages: int, device="cuda") -> PagePool:
    """All pages of a cache free; the first ones are popped first."""
    import torch

    if pages <= 0:
        raise ValueError("pages must be positive")
    return PagePool(torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device),
                    torch.full((1,), pages, dtype=torch.int32, device=device))


@dataclass(slots=True)
class BatchPlan:
    """What q4_paged_plan writes, all int32 on the GPU."""

    q_offsets: object   # [seqs + 1]
    positions: object   # [tokens]
    slots: object       # [tokens]
    kv_lens: object     # [seqs], with the new tokens
    free_count: object  # [1], the pool's count afterwards; None without a pool
    lacking: object     # [1], pages that were needed and not there


def paged_plan(kv_lens, new_lens, block_table, page_size: int, tokens: int, pool: PagePool | None = None, starts=None,
               reset=None, pages: int | None = None, kv_lens_out=None, free_count_out=None, workspace=None) -> BatchPlan:
    """q4_paged_plan: the arguments of qk_norm_rope_append and paged_attention for new_lens
    (None: one each) more tokens of sequences that hold kv_lens, with pages for them popped
    from `pool` into block_table (int32 [seqs, max_blocks], written in place). Sequences with
    reset != 0 give their pages back first and start at length 0. Rows behind the last
    sequence's, up to `tokens`, get slot -1.

    kv_lens, new_lens, starts, reset: int32 [seqs]. pool=None: the block table holds all pages
    already, of a cache of `pages` pages. The lengths and the pool's count are left as they
    were, the new ones are the plan's; kv_lens_out=kv_lens and free_count_out=pool.count keep
    them in place (the pages of reset sequences are pushed on pool.pages either way)."""
    torch = torch_()
    if block_table.dim() != 2:
        raise ValueError("block_table must be [seqs, max_blocks]")
    dev = block_table.get_device()
    seqs, blocks = shape = block_table.shape
    i32 = torch.int32
    tab = array(block_table, "block_table", i32, shape, dev)
    lens = array(kv_lens, "kv_lens", i32, (seqs,), dev)
    new = 0 if new_lens is None else array(new_lens, "new_lens", i32, (seqs,), dev)
    start = 0 if starts is None else array(starts, "starts", i32, (seqs,), dev)
    rst = 0 if reset is None else array(reset, "reset", i32, (seqs,), dev)
    stack = count = count_to = 0
    if pool is not None:
        if pages is not None:
            raise ValueError("pages goes without a pool, which has its own")
        pages = pool.pages.shape[0]
        stack = array(pool.pages, "pool.pages", i32, (pages,), dev)
        count = array(pool.count, "pool.count", i32, (1,), dev)
        if free_count_out is not None:
            count_to = array(free_count_out, "free_count_out", i32, (1,), dev)
    elif pages is None:
        raise ValueError("without a pool, pages (of the cache) must be given")
    elif free_count_out is not None:
        raise ValueError("free_count_out goes with a pool")
    lens_to = 0 if kv_lens_out is None else array(kv_lens_out, "kv_lens_out", i32, (seqs,), dev)
    if tokens < 0:
        raise ValueError("tokens must be >= 0")
    # one allocation for what is made here
    buf = torch.empty(3 + 2 * (seqs + tokens), dtype=i32, device=device(dev))
    lacking, count_new, lens_new, q_offsets, positions, slots = buf.split_with_sizes(
        (1, 1, seqs, seqs + 1, tokens, tokens))
    at = buf.data_ptr()
    if kv_lens_out is None:
        kv_lens_out, lens_to = lens_new, at + 8
    if pool is not None and free_count_out is None:
        free_count_out, count_to = count_new, at + 4
    offsets_to = at + 8 + 4 * seqs
    positions_to = offsets_to + 4 + 4 * seqs
    lib = _lib.load()
    need = lib.q4_paged_plan_workspace_bytes(seqs, tokens)
    ws, size = (None, 0) if need == 0 and workspace is None else _workspace(block_table, need, workspace)
    call(lib.q4_paged_plan, dev, lens, new, rst, start, seqs, tokens, page_size, pages, tab, blocks, stack, count,
         offsets_to, positions_to, positions_to + 4 * tokens, lens_to, count_to, at, ws, size)
    return BatchPlan(q_offsets, positions, slots, kv_lens_out, free_count_out, lacking)


def sample_workspace_bytes(rows: int, vocab: int) -> int:
    return int(_lib.load().q4_sample_workspace_bytes(rows, vocab))


_DTYPES: dict = {}


def sample(logits, uniforms, temperature=None, top_k=None, top_p=None, min_p=None, out=None, probs_out=None,
           workspace=None):
    """q4_sample: one token a row, (tokens int32 [rows], probs float32 [rows]).

    logits: float16, bfloat16 or float32 [rows, vocab], a row's elements contiguous, rows any
    stride apart (expanded ones too: several draws from the same logits); uniforms: float32 [rows], random numbers in [0, 1); temperature, top_p,
    min_p: float32 [rows], top_k: int32 [rows], each None where no row is to be cut by it
    (temperature: 1). A temperature <= 0 takes the largest logit. probs: the token's share
    of the tokens that the cuts left."""
    torch = torch_()
    if not _DTYPES:
        _DTYPES.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if not logits.is_cuda:
        raise ValueError(f"logits must live on a GPU (got {logits.device}); libq4 has no CPU path")
    dtype = _DTYPES.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"logits must be float16, bfloat16 or float32 (got {logits.dtype})")
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = logits.shape
    stride, inner = logits.stride()
    if vocab > 1 and inner != 1:
        raise ValueError("the logits of a row must be contiguous")
    dev = logits.get_device()
    f32 = torch.float32
    u = array(uniforms, "uniforms", f32, (rows,), dev)
    t = 0 if temperature is None else array(temperature, "temperature", f32, (rows,), dev)
    k = 0 if top_k is None else array(top_k, "top_k", torch.int32, (rows,), dev)
    p = 0 if top_p is None else array(top_p, "top_p", f32, (rows,), dev)
    m = 0 if min_p is None else array(min_p, "min_p", f32, (rows,), dev)
    if out is None:
        out = torch.empty(rows, dtype=torch.int32, device=device(dev))
    to = array(out, "out", torch.int32, (rows,), dev)
    if probs_out is None:
        probs_out = torch.empty(rows, dtype=f32, device=device(dev))
    pr = array(probs_out, "probs_out", f32, (rows,), dev)
    lib = _lib.load()
    ws, size = _workspace(logits, lib.q4_sample_workspace_bytes(rows, vocab), workspace)
    call(lib.q4_sample, dev, logits.data_ptr(), dtype, stride, rows, vocab, u, t, k, p, m, to, pr, ws, size)
    return out, probs_out
