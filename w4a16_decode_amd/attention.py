"""torch-facing wrappers of include/q4_attn.h (same names as the C calls): norm and
rotation of q and k, the paged INT4 KV cache and the attention over it.

As in ops.py, these functions check tensors, allocate outputs on the tensors' device
and pass raw pointers and torch's current HIP stream of that device to libq4; they
do no arithmetic of their own.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass, field
from functools import lru_cache

from . import _lib
from ._tensors import array, call, complain, device, enter, on_device, torch_
from .ops import Q4Error, _workspace


def _rows(t, name: str):
    """(tokens, heads, head_dim, stride, device) of a float16 [tokens, heads, head_dim] GPU
    tensor whose heads are contiguous and whose tokens lie a fixed stride apart."""
    torch = torch_()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not torch.float16:
        complain(t, name, torch.float16)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return n, h, d, s0 if n > 1 else h * d, t.get_device()


@dataclass(frozen=True)
class PagedKVCache4:
    """Paged INT4 KV cache: `pages` pages of page_size tokens of every KV head, in the
    layout of include/q4_attn.h. Slot p * page_size + i is row i of page p."""

    k_codes: object         # uint8 [pages, kv_heads, page_size * head_dim / 2]
    k_scales: object        # float16 [pages, kv_heads, page_size * head_dim / group]
    v_codes: object
    v_scales: object
    page_size: int
    head_dim: int
    group: int
    _struct: object = field(default=None, init=False, repr=False, compare=False)

    @property
    def pages(self) -> int:
        return self.k_codes.shape[0]

    @property
    def kv_heads(self) -> int:
        return self.k_codes.shape[1]

    @property
    def device(self):
        return self.k_codes.device

    def nbytes(self) -> int:
        return 2 * (self.k_codes.numel() + 2 * self.k_scales.numel())

    def __getstate__(self) -> dict:
        """Fields for a copy or a pickle: without the C structure, which holds this cache's addresses."""
        return {**self.__dict__, "_struct": None}

    def _check(self) -> None:
        """The buffers have the layout's types and sizes."""
        torch = torch_()
        if self.k_codes.dim() != 3:
            raise ValueError("k_codes must be [pages, kv_heads, page_size * head_dim / 2]")
        dev, shape = self.k_codes.get_device(), (self.pages, self.kv_heads)
        rows = self.page_size * self.head_dim
        codes, scales = rows // 2, rows // max(self.group, 1)
        for name, dtype, size in (("k_codes", torch.uint8, codes), ("v_codes", torch.uint8, codes),
                                  ("k_scales", torch.float16, scales), ("v_scales", torch.float16, scales)):
            array(getattr(self, name), name, dtype, (*shape, size), dev)

    def _c(self):
        """q4_paged_kv of this cache, by reference."""
        ptrs = (self.k_codes.data_ptr(), self.k_scales.data_ptr(), self.v_codes.data_ptr(), self.v_scales.data_ptr())
        if self._struct is None or self._struct[0] != ptrs:
            self._check()
            c = _lib.PagedKV(*ptrs, self.pages, self.page_size, self.kv_heads, self.head_dim, self.group)
            object.__setattr__(self, "_struct", (ptrs, c, ctypes.byref(c), self.kv_heads, self.k_codes.get_device()))
        return self._struct


def paged_kv_alloc(pages: int, page_size: int, kv_heads: int, head_dim: int, group: int = 128,
                   device="cuda") -> PagedKVCache4:
    """An empty cache. Its slots need no clearing: nothing reads one that no length covers."""
    import torch

    lib = _lib.load()
    codes = int(lib.q4_paged_codes_bytes(pages, page_size, kv_heads, head_dim))
    scales = int(lib.q4_paged_scales_count(pages, page_size, kv_heads, head_dim, group))
    if codes == 0 or scales == 0:
        raise Q4Error(5, lib.q4_last_error().decode())
    kc, vc = (torch.zeros((pages, kv_heads, codes // (pages * kv_heads)), dtype=torch.uint8, device=device)
              for _ in range(2))
    ks, vs = (torch.zeros((pages, kv_heads, scales // (pages * kv_heads)), dtype=torch.float16, device=device)
              for _ in range(2))
    return PagedKVCache4(kc, ks, vc, vs, page_size, head_dim, group)


def rope_table(positions: int, rot_dim: int, theta: float = 10000.0, device="cuda"):
    """q4_rope_table: float32 [positions, rot_dim / 2, 2], cosine and sine of position *
    theta^(-2 i / rot_dim). A model with scaled frequencies fills its own of this shape."""
    import torch

    if rot_dim <= 0 or rot_dim % 2 or positions < 0:
        raise ValueError("positions must be >= 0 and rot_dim a positive multiple of 16")
    table = torch.empty((positions, rot_dim // 2, 2), dtype=torch.float32, device=device)
    if not table.is_cuda:
        raise ValueError(f"device must be a GPU (got {table.device}); libq4 has no CPU path")
    call(_lib.load().q4_rope_table, table.get_device(), positions, rot_dim, theta, table.data_ptr())
    return table


def _rope_args(n, d, dev, positions, table, q_weight, k_weight):
    """(q_weight, k_weight, positions, table, table rows, rot_dim) as the C calls take them."""
    torch = torch_()
    pos = tab = rows = rot = 0
    if table is not None:
        if table.dim() != 3 or table.shape[2] != 2:
            raise ValueError("table must be [positions, rot_dim / 2, 2]")
        if positions is None:
            raise ValueError("a rotation needs positions")
        tab = array(table, "table", torch.float32, table.shape, dev)
        pos = array(positions, "positions", torch.int32, (n,), dev)
        rows, half, _ = table.shape
        rot = 2 * half
    return (0 if q_weight is None else array(q_weight, "q_weight", torch.float16, (d,), dev),
            0 if k_weight is None else array(k_weight, "k_weight", torch.float16, (d,), dev), pos, tab, rows, rot)


def _out_rows(out, name, shape, dev):
    """The output tensor (made where None) and its stride."""
    if out is None:
        torch = torch_()
        return torch.empty(shape, dtype=torch.float16, device=device(dev)), shape[1] * shape[2]
    *got, stride, at = _rows(out, name)
    if tuple(got) != shape or at != dev:
        raise ValueError(f"{name} must be {list(shape)} on cuda:{dev}")
    return out, stride


def qk_norm_rope(q, k, positions, table, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 q_out=None, k_out=None):
    """q4_qk_norm_rope: RMS norm of every q and k head and rotation by position, (q_out,
    k_out) float16. q [tokens, q_heads, head_dim] and k [tokens, kv_heads, head_dim] may
    be slices of one fused projection; q_out=q, k_out=k works in place. No weight, no
    norm; table=None, no rotation."""
    n, hq, d, qs, dev = _rows(q, "q")
    nk, hk, dk, ks, kdev = _rows(k, "k")
    if nk != n or dk != d:
        raise ValueError("q and k must agree in tokens and head_dim")
    on_device("k", kdev, dev)
    qw, kw, pos, tab, rows, rot = _rope_args(n, d, dev, positions, table, q_weight, k_weight)
    q_out, qos = _out_rows(q_out, "q_out", (n, hq, d), dev)
    k_out, kos = _out_rows(k_out, "k_out", (n, hk, d), dev)
    call(_lib.load().q4_qk_norm_rope, dev, q.data_ptr(), qs, k.data_ptr(), ks, n, hq, hk, d, qw, kw, eps, pos, tab, rows,
          rot, bool(interleaved), q_out.data_ptr(), qos, k_out.data_ptr(), kos)
    return q_out, k_out


def _append_args(k, v, cache: PagedKVCache4, slots):
    n, h, d, ks, dev = _rows(k, "k")
    nv, hv, dv, vs, vdev = _rows(v, "v")
    if (nv, hv, dv) != (n, h, d):
        raise ValueError("k and v must have the same shape")
    _, _, ref, heads, cdev = cache._c()
    if h != heads or d != cache.head_dim:
        raise ValueError(f"k and v must be [tokens, {heads}, {cache.head_dim}]")
    on_device("v", vdev, dev)
    on_device("the cache", cdev, dev)
    return n, d, ks, vs, dev, ref, array(slots, "slots", torch_().int32, (n,), dev)


def qk_norm_rope_append(q, k, v, positions, table, cache: PagedKVCache4, slots, q_weight=None, k_weight=None,
                        eps: float = 1e-6, interleaved: bool = False, q_out=None):
    """q4_qk_norm_rope_append: qk_norm_rope whose k, with v, is quantized into the cache's
    `slots` (int32 [tokens]; one outside the cache, -1 say, stores nothing). Returns q_out."""
    n, d, ks, vs, dev, ref, slot = _append_args(k, v, cache, slots)
    nq, hq, dq, qs, qdev = _rows(q, "q")
    if nq != n or dq != d:
        raise ValueError("q and k must agree in tokens and head_dim")
    on_device("q", qdev, dev)
    qw, kw, pos, tab, rows, rot = _rope_args(n, d, dev, positions, table, q_weight, k_weight)
    q_out, qos = _out_rows(q_out, "q_out", (n, hq, d), dev)
    call(_lib.load().q4_qk_norm_rope_append, dev, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, n, hq, qw, kw,
          eps, pos, tab, rows, rot, bool(interleaved), q_out.data_ptr(), qos, ref, slot)
    return q_out


def paged_kv_append(k, v, cache: PagedKVCache4, slots) -> None:
    """q4_paged_kv_append: k and v [tokens, kv_heads, head_dim], as they are, into `slots`."""
    n, _, ks, vs, dev, ref, slot = _append_args(k, v, cache, slots)
    call(_lib.load().q4_paged_kv_append, dev, k.data_ptr(), ks, v.data_ptr(), vs, n, ref, slot)


def paged_kv_dequant(cache: PagedKVCache4, slots):
    """q4_paged_kv_dequant: (k, v) float16 [tokens, kv_heads, head_dim] of `slots`, zeros
    for a slot outside the cache."""
    _, _, ref, heads, dev = cache._c()
    torch = torch_()
    if slots.dim() != 1:
        raise ValueError("slots must be [tokens]")
    n = slots.shape[0]
    slot = array(slots, "slots", torch.int32, (n,), dev)
    shape = (n, heads, cache.head_dim)
    k = torch.empty(shape, dtype=torch.float16, device=device(dev))
    v = torch.empty(shape, dtype=torch.float16, device=device(dev))
    call(_lib.load().q4_paged_kv_dequant, dev, ref, slot, n, k.data_ptr(), v.data_ptr())
    return k, v


def paged_attention_workspace_bytes(seqs: int, tokens: int, max_q: int, max_kv: int, q_heads: int, kv_heads: int,
                                    head_dim: int, group: int, window: int = 0) -> int:
    return int(_lib.load().q4_paged_attention_workspace_bytes(seqs, tokens, max_q, max_kv, q_heads, kv_heads, head_dim,
                                                              group, window))


def paged_attention(q, cache: PagedKVCache4, block_table, q_offsets, kv_lens, max_q: int, max_kv: int,
                    scale: float | None = None, window: int = 0, out=None, workspace=None):
    """q4_paged_attention: causal attention of each sequence's newest tokens over its pages.

    q: float16 [tokens, q_heads, head_dim], sequence n's rows q_offsets[n] ..
    q_offsets[n + 1] - 1 being the last of its kv_lens[n] tokens (k and v appended
    before); block_table: int32 [seqs, max_blocks], the page of each page_size tokens;
    max_q, max_kv: bounds of the rows and the length of any sequence (one form of the kernel
    serves the whole call: long chunks beside single tokens are faster in a call of their
    own). `out` must not overlap an input. scale defaults to
    1 / sqrt(head_dim); window > 0 hides keys more than window - 1 positions back. Returns
    float16 [tokens, q_heads, head_dim]; rows of no sequence keep what `out` held (an
    `out` made here holds anything there)."""
    torch = torch_()
    n, hq, d, qs, dev = _rows(q, "q")
    _, _, ref, heads, cdev = cache._c()
    if d != cache.head_dim:
        raise ValueError(f"q must have the cache's head_dim {cache.head_dim}")
    on_device("the cache", cdev, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [seqs, max_blocks]")
    seqs, blocks = shape = block_table.shape
    tab = array(block_table, "block_table", torch.int32, shape, dev)
    off = array(q_offsets, "q_offsets", torch.int32, (seqs + 1,), dev)
    lens = array(kv_lens, "kv_lens", torch.int32, (seqs,), dev)
    if out is None:
        out = torch.empty((n, hq, d), dtype=torch.float16, device=device(dev))
        to = out.data_ptr()
    else:
        to = array(out, "out", torch.float16, (n, hq, d), dev)
    lib = _lib.load()
    cur = enter(dev)  # the split, and with it the workspace, depends on the device
    try:
        need = lib.q4_paged_attention_workspace_bytes(seqs, n, max_q, max_kv, hq, heads, d, cache.group, window)
    finally:
        if cur != dev:
            torch.cuda.set_device(cur)
    ws, size = _workspace(q, need, workspace)
    call(lib.q4_paged_attention, dev, q.data_ptr(), qs, ref, tab, blocks, off, lens, seqs, n, max_q, max_kv, hq,
          d ** -0.5 if scale is None else scale, window, to, ws, size)
    return out


def paged_attention_shared_workspace_bytes(seqs: int, groups: int, tokens: int, max_q: int, max_kv: int, max_group_q: int,
                                           max_prefix: int, q_heads: int, kv_heads: int, head_dim: int,
                                           group: int) -> int:
    return int(_lib.load().q4_paged_attention_shared_workspace_bytes(seqs, groups, tokens, max_q, max_kv, max_group_q,
                                                                     max_prefix, q_heads, kv_heads, head_dim, group))


@lru_cache(maxsize=1024)  # of sizes alone; the split, and with it the workspace, depends on the device
def _shared_workspace(dev: int, *sizes) -> int:
    cur = enter(dev)
    try:
        return int(_lib.load().q4_paged_attention_shared_workspace_bytes(*sizes))
    finally:
        if cur != dev:
            torch_().cuda.set_device(cur)


def paged_attention_shared(q, cache: PagedKVCache4, prefix_table, prefix_lens, group_offsets, block_table, q_offsets,
                           kv_lens, max_q: int, max_kv: int, max_group_q: int, max_prefix: int,
                           scale: float | None = None, out=None, workspace=None):
    """q4_paged_attention_shared: paged_attention, without a window, of sequences that share prefixes.

    Sequences group_offsets[g] .. group_offsets[g + 1] - 1 (int32 [groups + 1], ascending) see
    the prefix_lens[g] tokens in the pages prefix_table[g] (int32 [groups, max_prefix_blocks])
    and then their own: block_table, kv_lens and max_kv count what lies behind the prefix.
    max_group_q, max_prefix: bounds of the rows of a group's sequences together and of the
    prefixes' lengths. The rest as in paged_attention."""
    torch = torch_()
    n, hq, d, qs, dev = _rows(q, "q")
    _, _, ref, heads, cdev = cache._c()
    if d != cache.head_dim:
        raise ValueError(f"q must have the cache's head_dim {cache.head_dim}")
    on_device("the cache", cdev, dev)
    if block_table.dim() != 2 or prefix_table.dim() != 2:
        raise ValueError("block_table must be [seqs, max_blocks] and prefix_table [groups, max_prefix_blocks]")
    i32 = torch.int32
    seqs, blocks = shape = block_table.shape
    tab = array(block_table, "block_table", i32, shape, dev)
    off = array(q_offsets, "q_offsets", i32, (seqs + 1,), dev)
    lens = array(kv_lens, "kv_lens", i32, (seqs,), dev)
    groups, prefix_blocks = shape = prefix_table.shape
    ptab = array(prefix_table, "prefix_table", i32, shape, dev)
    plens = array(prefix_lens, "prefix_lens", i32, (groups,), dev)
    goff = array(group_offsets, "group_offsets", i32, (groups + 1,), dev)
    if out is None:
        out = torch.empty((n, hq, d), dtype=torch.float16, device=device(dev))
        to = out.data_ptr()
    else:
        to = array(out, "out", torch.float16, (n, hq, d), dev)
    need = _shared_workspace(dev, seqs, groups, n, max_q, max_kv, max_group_q, max_prefix, hq, heads, d, cache.group)
    ws, size = _workspace(q, need, workspace)
    call(_lib.load().q4_paged_attention_shared, dev, q.data_ptr(), qs, ref, ptab, prefix_blocks, plens, goff, groups, tab, blocks,
         off, lens, seqs, n, max_q, max_kv, max_group_q, max_prefix, hq, d ** -0.5 if scale is None else scale, to, ws,
         size)
    return out
