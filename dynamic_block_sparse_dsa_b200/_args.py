"""Reading tensor arguments: address, type, device and layout checks.

The functions here define what a call accepts.  Where the native reader
(csrc/tensor_args.cpp) is built, it answers the ordinary case and hands
everything else to them.
"""
from __future__ import annotations

import sys

import torch

from . import build as _build

HEAD_DIM = 128


def _at(t: torch.Tensor, dtype, dev: int, name: str) -> int:
    """Address of a contiguous ``dtype`` tensor on device ``dev``."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    at = t.get_device()
    if at != dev:
        _wrong_device(at, dev, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _wrong_device(at: int, dev: int, name: str):
    if at < 0:
        raise ValueError("dynamic_block_sparse_dsa_b200 works on CUDA tensors only (no CPU path)")
    raise ValueError(f"{name} is on cuda:{at}, the call's other tensors on cuda:{dev}")


def _rows(t: torch.Tensor, dev: int, name: str):
    """(address, tokens, heads, elements from one token to the next) of bf16
    [tokens][heads][128] rows; only the tokens may be apart (slices of a packed
    projection)."""
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    at = t.get_device()
    if at != dev:
        _wrong_device(at, dev, name)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens][heads][{HEAD_DIM}], got {list(t.shape)}")
    n, heads, d = t.shape
    if d == HEAD_DIM and t.is_contiguous():
        return t.data_ptr(), n, heads, heads * HEAD_DIM
    s0, s1, s2 = t.stride()
    if d != HEAD_DIM or s2 != 1 or (s1 != HEAD_DIM and heads > 1):
        raise ValueError(f"{name} must be [tokens][heads][{HEAD_DIM}] with each token's heads contiguous, got "
                         f"{list(t.shape)} with strides {list(t.stride())}")
    # a single token has no next one; torch may give it any stride
    return t.data_ptr(), n, heads, s0 if n > 1 else heads * HEAD_DIM


py_at, py_rows = _at, _rows   # what the native reader falls back to

native = None   # the native reader's module


def connect(build: bool = False) -> None:
    """Put the native reader into use, if it is built from the sources that are here for this
    torch and Python; with ``build``, it is built first where it is not."""
    global native, _at, _rows
    if native is not None or (_build.args_stale() and not (build and _build.build_tensor_args())):
        return
    try:
        from . import _tensor_args
    except ImportError as e:
        sys.stderr.write(f"the native reader of tensor arguments does not load: {e}\n")
        return
    if _tensor_args.built_from != _build.args_key():   # one that this process had loaded before it was built anew
        return
    native = _tensor_args
    native.use(py_at, py_rows)
    _at, _rows = native.at, native.rows


connect()
