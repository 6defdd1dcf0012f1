"""Checks and launches shared by the wrappers whose calls take only microseconds.

A decode step's calls are so short on the GPU that the checks count: each tensor is asked
for as little as possible (get_device() instead of device, one stride() call), and
the stream is read as a raw handle.
"""

from __future__ import annotations

from .ops import _check

_t = None  # torch, once torch_() has imported it


def torch_():
    global _t
    if _t is None:
        import torch

        _t = torch
    return _t


def enter(dev: int):
    """Make dev the current device (the library queries that one); returns what to restore."""
    cur = torch_()._C._cuda_getDevice()
    if cur != dev:
        _t.cuda.set_device(dev)
    return cur


def call(fn, dev: int, *args) -> None:
    """Enqueue fn(*args, stream) on dev's current stream."""
    cur = enter(dev)
    try:
        st = fn(*args, _t._C._cuda_getCurrentRawStream(dev))
    finally:
        if cur != dev:
            _t.cuda.set_device(cur)
    if st:
        _check(st)


def complain(t, name: str, dtype) -> None:
    if not isinstance(t, torch_().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a GPU (got {t.device}); libq4 has no CPU path")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")


def array(t, name: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of the given type and shape on device dev."""
    if not isinstance(t, torch_().Tensor) or not t.is_cuda or t.dtype is not dtype:
        complain(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{name} (cuda:{t.get_device()}) must be on the same GPU as the other tensors (cuda:{dev})")
    return t.data_ptr()


def on_device(name: str, got: int, dev: int) -> None:
    if got != dev:
        raise ValueError(f"{name} (cuda:{got}) must be on the same GPU as the other tensors (cuda:{dev})")


_devices: list = []


def device(dev: int):
    """torch.device of an index, made once."""
    while len(_devices) <= dev:
        _devices.append(torch_().device("cuda", len(_devices)))
    return _devices[dev]
