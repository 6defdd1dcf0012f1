"""torch-facing wrappers of include/q4_attn.h (same names as the C calls): norm and
rotation of q and k, the paged INT4 KV cache and the attention over it.

As in ops.py, these functions check tensors, allocate outputs on the tensors' device
and pass raw pointers and torch's current HIP stream of that device to libq4; they
do no arithmetic of their own.
"""

from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

from . import _lib
from .ops import Q4Error, _check, _require_gpu, _stream, _workspace


def _on(t):
    """Context in which t's device is the current one (the library queries that device)."""
    import torch

    if t.device.index is None or t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _same_device(x, name, others) -> None:
    for other, t in others.items():
        if t is not None and t.device != x.device:
            raise ValueError(f"{other} ({t.device}) must be on {name}'s GPU ({x.device})")


def _rows(t, name: str):
    """(tokens, heads, head_dim, stride) of a float16 [tokens, heads, head_dim] GPU tensor
    whose heads are contiguous and whose tokens lie a fixed stride apart."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on a GPU (got {t.device}); libq4 has no CPU path")
    if t.dtype != torch.float16:
        raise TypeError(f"{name} must be torch.float16 (got {t.dtype})")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    n, h, d = t.shape
    if (d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return n, h, d, t.stride(0) if n > 1 else h * d


def _ints(t, name: str, shape) -> None:
    import torch

    _require_gpu(t, name, torch.int32)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}")


def _ptr(t):
    return None if t is None else t.data_ptr()


@dataclass
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

    def _c(self):
        return ctypes.byref(_lib.PagedKV(self.k_codes.data_ptr(), self.k_scales.data_ptr(), self.v_codes.data_ptr(),
                                         self.v_scales.data_ptr(), self.pages, self.page_size, self.kv_heads,
                                         self.head_dim, self.group))


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
    with _on(table):
        _check(_lib.load().q4_rope_table(positions, rot_dim, theta, table.data_ptr(), _stream(table)))
    return table


def _prep_rope(x, name, d, positions, table, q_weight, k_weight):
    import torch

    tokens = x.shape[0]
    if table is not None:
        _require_gpu(table, "table", torch.float32)
        if table.dim() != 3 or table.shape[2] != 2:
            raise ValueError("table must be [positions, rot_dim / 2, 2]")
        if positions is None:
            raise ValueError("a rotation needs positions")
        _ints(positions, "positions", (tokens,))
    for w, wname in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _require_gpu(w, wname, torch.float16)
            if tuple(w.shape) != (d,):
                raise ValueError(f"{wname} must be [{d}]")
    _same_device(x, name, {"positions": positions, "table": table, "q_weight": q_weight, "k_weight": k_weight})
    return (0, 0) if table is None else (table.shape[0], 2 * table.shape[1])


def _out_like(t, name, out):
    import torch

    if out is None:
        out = torch.empty(tuple(t.shape), dtype=torch.float16, device=t.device)
    if tuple(out.shape) != tuple(t.shape) or out.device != t.device:
        raise ValueError(f"{name} must be {list(t.shape)} on {t.device}")
    return out, _rows(out, name)[3]


def qk_norm_rope(q, k, positions, table, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 q_out=None, k_out=None):
    """q4_qk_norm_rope: RMS norm of every q and k head and rotation by position, (q_out,
    k_out) float16. q [tokens, q_heads, head_dim] and k [tokens, kv_heads, head_dim] may
    be slices of one fused projection; q_out=q, k_out=k works in place. No weight, no
    norm; table=None, no rotation."""
    n, hq, d, qs = _rows(q, "q")
    nk, hk, dk, ks = _rows(k, "k")
    if (nk, dk) != (n, d):
        raise ValueError("q and k must agree in tokens and head_dim")
    _same_device(q, "q", {"k": k})
    rows, rot = _prep_rope(q, "q", d, positions, table, q_weight, k_weight)
    q_out, qos = _out_like(q, "q_out", q_out)
    k_out, kos = _out_like(k, "k_out", k_out)
    with _on(q):
        _check(_lib.load().q4_qk_norm_rope(q.data_ptr(), qs, k.data_ptr(), ks, n, hq, hk, d, _ptr(q_weight),
                                           _ptr(k_weight), eps, _ptr(positions), _ptr(table), rows, rot,
                                           int(interleaved), q_out.data_ptr(), qos, k_out.data_ptr(), kos,
                                           _stream(q)))
    return q_out, k_out


def _prep_append(k, v, cache: PagedKVCache4, slots):
    n, h, d, ks = _rows(k, "k")
    if _rows(v, "v")[:3] != (n, h, d):
        raise ValueError("k and v must have the same shape")
    if (h, d) != (cache.kv_heads, cache.head_dim):
        raise ValueError(f"k and v must be [tokens, {cache.kv_heads}, {cache.head_dim}]")
    _ints(slots, "slots", (n,))
    _same_device(k, "k", {"v": v, "slots": slots, "the cache": cache})
    return n, ks, _rows(v, "v")[3]


def qk_norm_rope_append(q, k, v, positions, table, cache: PagedKVCache4, slots, q_weight=None, k_weight=None,
                        eps: float = 1e-6, interleaved: bool = False, q_out=None):
    """q4_qk_norm_rope_append: qk_norm_rope whose k, with v, is quantized into the cache's
    `slots` (int32 [tokens]; one outside the cache, -1 say, stores nothing). Returns q_out."""
    n, ks, vs = _prep_append(k, v, cache, slots)
    nq, hq, d, qs = _rows(q, "q")
    if (nq, d) != (n, cache.head_dim):
        raise ValueError("q and k must agree in tokens and head_dim")
    _same_device(q, "q", {"k": k})
    rows, rot = _prep_rope(q, "q", d, positions, table, q_weight, k_weight)
    q_out, qos = _out_like(q, "q_out", q_out)
    with _on(q):
        _check(_lib.load().q4_qk_norm_rope_append(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, n, hq,
                                                  _ptr(q_weight), _ptr(k_weight), eps, _ptr(positions), _ptr(table),
                                                  rows, rot, int(interleaved), q_out.data_ptr(), qos, cache._c(),
                                                  slots.data_ptr(), _stream(q)))
    return q_out


def paged_kv_append(k, v, cache: PagedKVCache4, slots) -> None:
    """q4_paged_kv_append: k and v [tokens, kv_heads, head_dim], as they are, into `slots`."""
    n, ks, vs = _prep_append(k, v, cache, slots)
    with _on(k):
        _check(_lib.load().q4_paged_kv_append(k.data_ptr(), ks, v.data_ptr(), vs, n, cache._c(), slots.data_ptr(),
                                              _stream(k)))


def paged_kv_dequant(cache: PagedKVCache4, slots):
    """q4_paged_kv_dequant: (k, v) float16 [tokens, kv_heads, head_dim] of `slots`, zeros
    for a slot outside the cache."""
    import torch

    if slots.dim() != 1:
        raise ValueError("slots must be [tokens]")
    _ints(slots, "slots", slots.shape)
    _same_device(slots, "slots", {"the cache": cache})
    n = slots.shape[0]
    k, v = (torch.empty((n, cache.kv_heads, cache.head_dim), dtype=torch.float16, device=cache.device)
            for _ in range(2))
    with _on(k):
        _check(_lib.load().q4_paged_kv_dequant(cache._c(), slots.data_ptr(), n, k.data_ptr(), v.data_ptr(),
                                               _stream(k)))
    return k, v


def paged_attention_workspace_bytes(seqs: int, tokens: int, max_q: int, max_kv: int, q_heads: int, kv_heads: int,
                                    head_dim: int, window: int = 0) -> int:
    return int(_lib.load().q4_paged_attention_workspace_bytes(seqs, tokens, max_q, max_kv, q_heads, kv_heads, head_dim,
                                                              window))


def paged_attention(q, cache: PagedKVCache4, block_table, q_offsets, kv_lens, max_q: int, max_kv: int,
                    scale: float | None = None, window: int = 0, out=None, workspace=None):
    """q4_paged_attention: causal attention of each sequence's newest tokens over its pages.

    q: float16 [tokens, q_heads, head_dim], sequence n's rows q_offsets[n] ..
    q_offsets[n + 1] - 1 being the last of its kv_lens[n] tokens (k and v appended
    before); block_table: int32 [seqs, max_blocks], the page of each page_size tokens;
    max_q, max_kv: bounds of the rows and the length of any sequence. scale defaults to
    1 / sqrt(head_dim); window > 0 hides keys more than window - 1 positions back. Returns
    float16 [tokens, q_heads, head_dim]; rows of no sequence keep what `out` held (an
    `out` made here holds anything there)."""
    import torch

    n, hq, d, qs = _rows(q, "q")
    if d != cache.head_dim:
        raise ValueError(f"q must have the cache's head_dim {cache.head_dim}")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [seqs, max_blocks]")
    seqs, blocks = block_table.shape
    _ints(block_table, "block_table", (seqs, blocks))
    _ints(q_offsets, "q_offsets", (seqs + 1,))
    _ints(kv_lens, "kv_lens", (seqs,))
    _same_device(q, "q", {"the cache": cache, "block_table": block_table, "q_offsets": q_offsets, "kv_lens": kv_lens})
    if out is None:
        out = torch.empty((n, hq, d), dtype=torch.float16, device=q.device)
    else:
        _require_gpu(out, "out", torch.float16)
        if tuple(out.shape) != (n, hq, d) or out.device != q.device:
            raise ValueError(f"out must be {[n, hq, d]} on {q.device}")
    lib = _lib.load()
    with _on(q):
        need = int(lib.q4_paged_attention_workspace_bytes(seqs, n, max_q, max_kv, hq, cache.kv_heads, d, window))
        ws_ptr, ws_bytes = _workspace(q, need, workspace)
        _check(lib.q4_paged_attention(q.data_ptr(), qs, cache._c(), block_table.data_ptr(), blocks,
                                      q_offsets.data_ptr(), kv_lens.data_ptr(), seqs, n, max_q, max_kv, hq,
                                      d ** -0.5 if scale is None else scale, window, out.data_ptr(), ws_ptr, ws_bytes,
                                      _stream(q)))
    return out
