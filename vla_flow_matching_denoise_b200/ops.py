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
unless given.  This module only checks shapes and types and marshals; the
kernels are in libfm_expert.so, and a missing library raises.  The operators
have no backward: an input that requires grad is refused while gradients are
being recorded.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import numpy as np
import torch

from .binding import FmError, load

FP8 = torch.float8_e4m3fn
_TYPE = {torch.bfloat16: 0, torch.float32: 1}
_ACT = {"none": 0, "silu": 1, "gelu_tanh": 2}


def _fail(call: str, st: int):
    raise FmError(call, st, load().fm_last_error(None).decode())


def _run(call: str, dev: torch.device, stream, args) -> None:
    """The library's `call` on device `dev` and its current stream."""
    fn = getattr(load(), call)
    if dev.index == torch.cuda.current_device():
        s = torch.cuda.current_stream() if stream is None else stream
        st = fn(*args, s if isinstance(s, int) else s.cuda_stream)
    else:
        with torch.cuda.device(dev):
            s = torch.cuda.current_stream() if stream is None else stream
            st = fn(*args, s if isinstance(s, int) else s.cuda_stream)
    if st:
        _fail(call, st)


def _matrix(t, name: str, dtypes, dev: Optional[torch.device], rows: Optional[int] = None, cols: Optional[int] = None):
    """Row stride of `t`, a 2-D CUDA tensor with unit column stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}, expected one of {[str(d) for d in dtypes]}")
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{'rows' if rows is None else rows}, "
                         f"{'columns' if cols is None else cols}]")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows (column stride 1, got {t.stride(1)})")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad: this operator has no backward")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _vector(t, name: str, dtype, dev: torch.device, n: int) -> None:
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != dtype or t.dim() != 1 or t.shape[0] != n \
            or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} values on {dev}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad: this operator has no backward")


_CODES = (FP8, torch.uint8)
_REAL = (torch.bfloat16, torch.float32)
_F32 = (torch.float32,)


def _codes_out(codes, scales, rows: int, cols: int, dev):
    if codes is None:
        codes = torch.empty((rows, cols), dtype=FP8, device=dev)
        ldc = cols
    else:
        ldc = _matrix(codes, "codes", _CODES, dev, rows, cols)
    g = (cols + 127) // 128
    if scales is None:
        scales = torch.empty((rows, g), dtype=torch.float32, device=dev)
        lds = g
    else:
        lds = _matrix(scales, "scales", _F32, dev, rows, g)
    return codes, ldc, scales, lds


def add_rmsnorm_e4m3(x, gain=None, residual=None, *, eps: float = 1e-6, gain_offset: float = 0.0, h_out=None,
                     codes=None, scales=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(h, codes, scales): h = x + residual, then the RMS norm of h times
    (gain + gain_offset) as E4M3 codes with one scale per row and 128 columns.

    x: [rows, d] bf16 or fp32; residual: [rows, d] bf16 or fp32 (its type is
    h's) or None; gain: bf16 [d] or None.  h_out: where h goes (`residual`
    itself for an update in place); a new tensor with a residual, and x itself
    (nothing written) without one.  d: a multiple of 16 up to 16384."""
    ldx = _matrix(x, "x", _REAL, None)
    rows, d = x.shape
    dev = x.device
    ldr = ldh = 0
    h_type = x.dtype
    if residual is not None:
        ldr = _matrix(residual, "residual", _REAL, dev, rows, d)
        h_type = residual.dtype
        if h_out is None:
            h_out = torch.empty((rows, d), dtype=h_type, device=dev)
    elif h_out is not None:
        h_type = h_out.dtype
    if h_out is not None:
        ldh = _matrix(h_out, "h_out", (h_type,) if residual is not None else _REAL, dev, rows, d)
    if gain is not None:
        _vector(gain, "gain", torch.bfloat16, dev, d)
    codes, ldc, scales, lds = _codes_out(codes, scales, rows, d, dev)
    _run("fm_add_rmsnorm_e4m3", dev, stream,
         (x.data_ptr(), _TYPE[x.dtype], ldx, None if residual is None else residual.data_ptr(), _TYPE[h_type], ldr,
          None if gain is None else gain.data_ptr(), gain_offset, eps, rows, d,
          None if h_out is None else h_out.data_ptr(), ldh, codes.data_ptr(), ldc, scales.data_ptr(), lds))
    return (x if h_out is None else h_out), codes, scales


def gated_e4m3(x, act: str = "silu", *, codes=None, scales=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales) of act(x[:, :f]) * x[:, f:] ("silu", "gelu_tanh"; x is
    [rows, 2f]) or of x itself ("none"; x is [rows, f]), one scale per row and
    128 columns.  x: bf16 or fp32; f: a multiple of 16."""
    if act not in _ACT:
        raise ValueError(f"act {act!r}: expected one of {sorted(_ACT)}")
    ldx = _matrix(x, "x", _REAL, None)
    rows, f = x.shape
    if act != "none":
        if f % 2:
            raise ValueError(f"x has {f} columns: gate and up need an even number")
        f //= 2
    codes, ldc, scales, lds = _codes_out(codes, scales, rows, f, x.device)
    _run("fm_gated_e4m3", x.device, stream, (x.data_ptr(), _TYPE[x.dtype], ldx, _ACT[act], rows, f, codes.data_ptr(),
                                             ldc, scales.data_ptr(), lds))
    return codes, scales


def quantize_weight_e4m3(w, *, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes [n, k], scales [ceil(n/128), ceil(k/128)]) of a bf16 weight
    [n, k], one scale per 128 x 128 block."""
    ldw = _matrix(w, "w", (torch.bfloat16,), None)
    n, k = w.shape
    codes = torch.empty((n, k), dtype=FP8, device=w.device)
    scales = torch.empty(((n + 127) // 128, (k + 127) // 128), dtype=torch.float32, device=w.device)
    _run("fm_quantize_weight_e4m3_b128", w.device, stream, (w.data_ptr(), ldw, n, k, codes.data_ptr(), k,
                                                            scales.data_ptr(), scales.shape[1]))
    return codes, scales


def gemm_e4m3(a, sa, w, sw, *, bias=None, out=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """out [m, n] = (a sa) (w sw)^T (+ bias): a [m, k] and w [n, k] E4M3 codes,
    sa [m, ceil(k/128)] and sw [ceil(n/128), ceil(k/128)] fp32, bias bf16 [n],
    out bf16 or fp32.  k: a multiple of 16."""
    lda = _matrix(a, "a", _CODES, None)
    m, k = a.shape
    dev = a.device
    ldw = _matrix(w, "w", _CODES, dev, None, k)
    n, g = w.shape[0], (k + 127) // 128
    ldsa = _matrix(sa, "sa", _F32, dev, m, g)
    ldsw = _matrix(sw, "sw", _F32, dev, (n + 127) // 128, g)
    if bias is not None:
        _vector(bias, "bias", torch.bfloat16, dev, n)
    if out is None:
        if out_dtype not in _TYPE:
            raise ValueError(f"out_dtype {out_dtype}: expected bfloat16 or float32")
        out = torch.empty((m, n), dtype=out_dtype, device=dev)
        ldo = n
    else:
        ldo = _matrix(out, "out", _REAL, dev, m, n)
    _run("fm_gemm_e4m3_b128", dev, stream,
         (a.data_ptr(), lda, sa.data_ptr(), ldsa, w.data_ptr(), ldw, sw.data_ptr(), ldsw,
          None if bias is None else bias.data_ptr(), m, n, k, out.data_ptr(), _TYPE[out.dtype], ldo))
    return out


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


def _heads(t, name: str, x, rows: int, heads: int, hd: int):
    """(tensor, row stride) of a [rows, heads, hd] output; None makes one, False none."""
    if t is False or heads == 0:
        return (None, 0) if t is False else (torch.empty((rows, heads, hd), dtype=x.dtype, device=x.device), hd * heads)
    if t is None:
        return torch.empty((rows, heads, hd), dtype=x.dtype, device=x.device), heads * hd
    if not isinstance(t, torch.Tensor) or t.device != x.device or t.dtype != x.dtype \
            or tuple(t.shape) != (rows, heads, hd):
        raise ValueError(f"{name} must be a {x.dtype} tensor [{rows}, {heads}, {hd}] on {x.device}")
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != hd):
        raise ValueError(f"{name} must have contiguous heads in each row")
    return t, (t.stride(0) if rows > 1 else heads * hd)


def rope_axes(x, positions, pairs, n_q: int, n_kv: int, head_dim: int, *, q_out=None, k_out=None, v_out=None,
              stream=None):
    """(q, k, v) of fused rows x [rows, (n_q + 2 n_kv) head_dim] (bf16 or fp32),
    q and k rotated: pair j is elements (j, j + n) of a head, its angle
    positions[axis[j]] * frequency[j], pairs = (axis, frequency) as rope_pairs
    makes them.  positions: int32 [n_axes, rows] (or [rows] for one axis).

    Outputs are [rows, heads, head_dim]: new tensors, the ones given (their own
    columns of x for an update in place), or None where False is given.  With
    v_out=False x may end after the key heads."""
    ldx = _matrix(x, "x", _REAL, None)
    rows, dev = x.shape[0], x.device
    if n_q < 0 or n_kv < 0 or head_dim < 1:
        raise ValueError(f"n_q {n_q} / n_kv {n_kv} / head_dim {head_dim} out of range")
    want = (n_q + (1 if v_out is False else 2) * n_kv) * head_dim
    if x.shape[1] < want or (v_out is not False and x.shape[1] != want):
        raise ValueError(f"x has {x.shape[1]} columns, expected {want}")
    if positions.dim() == 1:
        positions = positions[None]
    ldp = _matrix(positions, "positions", (torch.int32,), dev, None, rows)
    axis, freq = pairs
    if axis.dtype != np.uint8 or freq.dtype != np.float64 or axis.ndim != 1 or axis.shape != freq.shape \
            or not axis.flags.c_contiguous or not freq.flags.c_contiguous:
        raise ValueError("pairs must be (uint8 [n], float64 [n]) contiguous arrays (see rope_pairs)")
    q, ldq = _heads(q_out, "q_out", x, rows, n_q, head_dim)
    k, ldk = _heads(k_out, "k_out", x, rows, n_kv, head_dim)
    v, ldv = _heads(v_out, "v_out", x, rows, n_kv, head_dim)
    _run("fm_rope_axes", dev, stream,
         (x.data_ptr(), _TYPE[x.dtype], ldx, rows, n_q, n_kv, head_dim, positions.data_ptr(), ldp, positions.shape[0],
          axis.ctypes.data, freq.ctypes.data, axis.shape[0], None if q is None else q.data_ptr(), ldq,
          None if k is None else k.data_ptr(), ldk, None if v is None else v.data_ptr(), ldv))
    return q, k, v


def sync(stream=None) -> None:
    """Waits for `stream` (default: the current one) and raises if a device-side
    wait of gemm_e4m3 gave up since the last call on this device."""
    s = torch.cuda.current_stream() if stream is None else stream
    st = load().fm_ops_sync(s if isinstance(s, int) else s.cuda_stream)
    if st:
        _fail("fm_ops_sync", st)
