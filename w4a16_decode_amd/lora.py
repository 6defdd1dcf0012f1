"""torch-facing wrapper of include/q4_lora.h: the W4A16 product with low-rank adapters."""

from __future__ import annotations

from dataclasses import dataclass

from . import _lib
from ._tensors import array, call, device, enter, on_device, torch_
from .ops import QuantizedWeight, _workspace


@dataclass
class LoraAdapters:
    """Adapters of one matrix: a float16 [adapters, rank, in_features], b float16
    [adapters, out_features, rank], scaling float32 [adapters], contiguous on one GPU."""

    a: object
    b: object
    scaling: object

    @property
    def count(self) -> int:
        return self.a.shape[0]

    @property
    def rank(self) -> int:
        return self.a.shape[1]


def workspace_bytes_lora(batch: int, out_features: int, in_features: int, group: int, rank: int) -> int:
    return int(_lib.load().q4_workspace_bytes_lora(batch, out_features, in_features, group, rank))


def gemm_lora(x, qw: QuantizedWeight, adapters: LoraAdapters, ids, out=None, workspace=None):
    """q4_gemm_lora: gemm plus scaling[i] * B_i (A_i x[b]) with i = ids[b] (int32 [B]; an id
    outside the adapters, -1 say, is a row without one). For QuantizedWeight; act-order and
    INT8 weights have no form with adapters."""
    torch = torch_()
    N, K, g = qw.out_features, qw.in_features, qw.group
    a, b, s = adapters.a, adapters.b, adapters.scaling
    if x.dim() != 2 or a.dim() != 3:
        raise ValueError(f"x must be [B, {K}] and adapters.a [adapters, rank, {K}]")
    B, dev = x.shape[0], x.get_device()
    n, rank, _ = a.shape
    src = array(x, "x", torch.float16, (B, K), dev)
    pa = array(a, "adapters.a", torch.float16, (n, rank, K), dev)
    pb = array(b, "adapters.b", torch.float16, (n, N, rank), dev)
    ps = array(s, "adapters.scaling", torch.float32, (n,), dev)
    pi = array(ids, "ids", torch.int32, (B,), dev)
    on_device("the weights", qw.packed.get_device(), dev)
    on_device("the scales", qw.scales.get_device(), dev)
    if out is None:
        out = torch.empty((B, N), dtype=torch.float16, device=device(dev))
    to = array(out, "out", torch.float16, (B, N), dev)
    lib = _lib.load()
    need = 0
    if B > 0:
        cur = enter(dev)  # the launch shape, and with it the workspace, depends on the device
        try:
            need = lib.q4_workspace_bytes_lora(B, N, K, g, rank)
        finally:
            if cur != dev:
                torch.cuda.set_device(cur)
    ws, size = _workspace(x, need, workspace)
    call(lib.q4_gemm_lora, dev, src, B, qw.packed.data_ptr(), qw.scales.data_ptr(),
         qw.zeros.data_ptr() if qw.asym else None, N, K, g, pa, pb, ps, n, rank, pi, to, ws, size)
    return out
