"""Python binding of the E4M3 block-scaled operators of include/fm_ops.h.

The pieces of a transformer layer whose linears run on E4M3 codes with one
fp32 scale per block of 128, on torch CUDA tensors:

    h, a, sa = ops.add_rmsnorm_e4m3(x, gain, residual=h)        # norm -> codes
    qkv = ops.gemm_e4m3(a, sa, *w_qkv, bias=b_qkv)              # linear
    q, k, v = ops.rope_axes(qkv, positions, pairs, n_q, n_kv, hd)
    u, su = ops.gated_e4m3(gate_up, "silu")                     # SwiGLU -> codes

with w_qkv = ops.quantize_weight_e4m3(w) made once.  `k` and `v` of a prefix
are what Expert.set_prefix takes ([batch, P, n_kv, hd] bf16).

Calls run on the tensors' device, on its current stream (or `stream`), are
asynchronous and can be captured in a CUDA graph.  Outputs are new tensors
unless given; a given one must not overlap an input or another output but where
its call says so.  The kernels are in libfm_expert.so, shapes and types are
checked in _ops.so (csrc/fm_ops_torch.cpp), and a missing library raises.  The
operators have no derivative: a tensor that requires grad is refused while
gradients are being recorded, one with a forward-mode tangent always.  Writing a
given output counts as an operation in place: a graph that saved it says so.
"""
from __future__ import annotations

import contextlib
import os
from typing import Sequence, Tuple

import numpy as np
import torch

from .binding import LIB_PATH, FmError, load

for _so in (LIB_PATH, os.path.join(os.path.dirname(LIB_PATH), "_ops.so")):
    if not os.path.exists(_so):
        raise FileNotFoundError(f"{_so} is missing: run `python -m vla_flow_matching_denoise_b200.build`")
from . import _ops  # noqa: E402

_ACT = {"none": 0, "silu": 1, "gelu_tanh": 2}


def _handle(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def add_rmsnorm_e4m3(x, gain=None, residual=None, *, eps: float = 1e-6, gain_offset: float = 0.0, h_out=None,
                     codes=None, scales=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(h, codes, scales): h = x + residual, then the RMS norm of h times
    (gain + gain_offset) as E4M3 codes with one scale per row and 128 columns.

    x: [rows, d] bf16 or fp32; residual: [rows, d] bf16 or fp32 (its type is
    h's) or None; gain: bf16 [d] or None.  h_out: where h goes (`residual`
    itself for an update in place); a new tensor with a residual, and x itself
    (nothing written) without one.  d: a multiple of 16 up to 16384."""
    return _ops.add_rmsnorm(x, gain, residual, eps, gain_offset, h_out, codes, scales, _handle(stream))


def gated_e4m3(x, act: str = "silu", *, codes=None, scales=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales) of act(x[:, :f]) * x[:, f:] ("silu", "gelu_tanh"; x is
    [rows, 2f]) or of x itself ("none"; x is [rows, f]), one scale per row and
    128 columns.  x: bf16 or fp32; f: a multiple of 16."""
    if act not in _ACT:
        raise ValueError(f"act {act!r}: expected one of {sorted(_ACT)}")
    return _ops.gated(x, _ACT[act], codes, scales, _handle(stream))


def quantize_weight_e4m3(w, *, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes [n, k], scales [ceil(n/128), ceil(k/128)]) of a bf16 weight
    [n, k], one scale per 128 x 128 block."""
    return _ops.quantize_weight(w, _handle(stream))


def gemm_e4m3(a, sa, w, sw, *, bias=None, out=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """out [m, n] = (a sa) (w sw)^T (+ bias): a [m, k] and w [n, k] E4M3 codes
    (float8_e4m3fn or uint8), sa [m, ceil(k/128)] and sw [ceil(n/128),
    ceil(k/128)] fp32, bias bf16 [n], out bf16 or fp32.  k: a multiple of 16."""
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise ValueError(f"out_dtype {out_dtype}: expected bfloat16 or float32")
    return _ops.gemm(a, sa, w, sw, bias, out, out_dtype is torch.float32, _handle(stream))


def rope_pairs(sections: Sequence[int], base: float = 10000.0, ladder: str = "shared",
               interleaved: bool = False) -> Tuple[np.ndarray, np.ndarray]:
    """The pair table of rope_axes: (axis uint8 [n], frequency float64 [n]) for
    sections[a] pairs on position axis a, n = sum(sections).

    ladder "shared": pair j has frequency base^(-j/n) whatever its axis (text
    tokens with equal positions on all axes then get plain RoPE); "per_axis":
    each section starts again, base^(-i/sections[a]) (image rows and columns).
    interleaved: the axes take pairs in turn until each has its share, instead
    of one block after the other (only with the shared ladder)."""
    sections = [int(s) for s in sections]
    if not sections or min(sections) < 0 or sum(sections) < 1:
        raise ValueError(f"sections {sections}: expected non-negative sizes with a positive sum")
    n = sum(sections)
    if ladder not in ("shared", "per_axis"):
        raise ValueError(f"ladder {ladder!r}: expected 'shared' or 'per_axis'")
    if interleaved and ladder != "shared":
        raise ValueError("interleaved axes need the shared ladder")
    if interleaved:
        left, axis = list(sections), []
        while len(axis) < n:
            for a in range(len(left)):
                if left[a]:
                    left[a] -= 1
                    axis.append(a)
    else:
        axis = [a for a, s in enumerate(sections) for _ in range(s)]
    if ladder == "per_axis":
        freq = [float(base) ** (-i / s) for s in sections for i in range(s)]
    else:
        freq = [float(base) ** (-j / n) for j in range(n)]
    return np.array(axis, dtype=np.uint8), np.array(freq, dtype=np.float64)


def rope_axes(x, positions, pairs, n_q: int, n_kv: int, head_dim: int, *, q_out=None, k_out=None, v_out=None,
              stream=None):
    """(q, k, v) of fused rows x [rows, (n_q + 2 n_kv) head_dim] (bf16 or fp32),
    q and k rotated: pair j is elements (j, j + n) of a head, its angle
    positions[axis[j]] * frequency[j], pairs = (axis, frequency) as rope_pairs
    makes them.  positions: int32 [n_axes, rows] (or [rows] for one axis).

    Outputs are [rows, heads, head_dim]: new tensors, the ones given (their own
    columns of x for an update in place), or None where False is given.  With
    v_out=False x may end after the key heads."""
    axis, freq = pairs
    return _ops.rope(x, positions, axis, freq, n_q, n_kv, head_dim, q_out, k_out, v_out, _handle(stream))


def sync(stream=None) -> None:
    """Waits for `stream` (a torch stream, a handle of the current device, or the
    current stream) and raises if a device-side wait of gemm_e4m3 gave up on the
    stream's device, whatever stream it ran on, since the calling thread's last
    sync there: what gemm_e4m3 gave since then is in doubt."""
    lib = load()
    if stream is None:
        stream = torch.cuda.current_stream()
    with contextlib.nullcontext() if isinstance(stream, int) else torch.cuda.device(stream.device):
        st = lib.fm_ops_sync(_handle(stream))
    if st:
        raise FmError("fm_ops_sync", st, lib.fm_last_error(None).decode())
