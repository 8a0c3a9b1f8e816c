"""GPU parity of the E4M3 block-scaled operators (include/fm_ops.h) against
their definitions in 64 bits, through the Python binding.

Tolerances count roundings (u = 2^-24, half a step of fp32; a code is within
half an E4M3 step of the scaled value) and were set before the first run; each
is derived where it is used."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest

from oracle import fm_oracle as O
from vla_flow_matching_denoise_b200 import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from vla_flow_matching_denoise_b200 import ops  # noqa: E402
from vla_flow_matching_denoise_b200.binding import Expert, FmError, load  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _half_step(t):
    return torch.finfo(t).eps / 2


def _round_tol(dtype, ref):
    """One rounding to `dtype` of a value near `ref` (bf16's smallest normal is far below every test value)."""
    return _half_step(dtype) * ref.abs()


def _e4m3_half_step(v):
    _, e = torch.frexp(v.abs())
    return torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 4)


def _check_codes(codes, scales, y, tol):
    """codes, scales quantise y [rows, d] (64 bits) known to `tol` (absolute, per element)."""
    rows, d = y.shape
    g = (d + 127) // 128
    assert codes.shape == (rows, d) and scales.shape == (rows, g)
    pad = torch.zeros(rows, g * 128, dtype=torch.float64, device=y.device)
    padt = pad.clone()
    pad[:, :d], padt[:, :d] = y, tol
    amax = pad.view(rows, g, 128).abs().amax(2)
    s = torch.where(amax > 0, amax.clamp_min(2.0 ** -100) / 448, torch.ones_like(amax))
    # the scale: the largest element's own error, and the division
    assert torch.all((scales.double() - s).abs() <= padt.view(rows, g, 128).amax(2) / 448 + 2 * U * s)
    # the code: half a step of the scaled value (or of the code, across a power
    # of two), the value's error, and the roundings of 448 / a, of y r and of s
    sr = scales.double().repeat_interleave(128, 1)[:, :d]
    v = y / sr
    c = codes.view(FP8).double()
    bound = torch.maximum(_e4m3_half_step(v), _e4m3_half_step(c)) + tol / sr + 4 * U * v.abs()
    assert torch.all((c - v).abs() <= bound)


def _padded(t, extra, fill):
    """A copy of 2-D t inside a wider and longer buffer: (view, buffer)."""
    buf = torch.full((t.shape[0] + 2, t.shape[1] + extra), 0, dtype=t.dtype, device=t.device) if t.dtype in (FP8,) else \
        torch.full((t.shape[0] + 2, t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    if t.dtype == FP8:
        buf.view(torch.uint8).fill_(int(fill))
    view = buf[:t.shape[0], :t.shape[1]]
    view.copy_(t)
    return view, buf


# --------------------------------------------------------------------------- norm
NORM = [(1, 16), (1, 1024), (3, 128), (2, 2048), (50, 1024), (5, 144), (7, 1008), (306, 2048), (1, 4096), (9, 4112),
        (2, 8192), (1, 16384), (3, 16368), (513, 1024), (600, 2064), (1025, 496), (520, 16384), (4099, 144), (2000, 4112),
        (6001, 16), (1001, 8208)]


def _norm_ref(x, res, gain, offset, eps=1e-6):
    h = x.double() + (0 if res is None else res.double())
    rstd = (h.square().mean(1, keepdim=True) + eps).rsqrt()
    y = h * rstd * ((1.0 if gain is None else gain.double()) + offset)
    return h, y


def _norm_tol(y, d):
    # h one rounding; the squares: at most 32 sequential sums per lane, 5 shuffles
    # and 16 warps, 55 u on the sum, halved by the root; rsqrtf 2 ulp = 4 u, the
    # mean, + eps, the two products and gain + offset 5 u
    return (2 + 28 + 4 + 5) * U * y.abs()


@pytest.mark.parametrize("rows,d", NORM)
@pytest.mark.parametrize("xt,ht,resid,gain,offset", [(BF, BF, True, True, 0.0), (BF, F32, True, True, 1.0),
                                                     (F32, F32, False, False, 0.0), (F32, BF, True, True, 0.0),
                                                     (BF, BF, False, True, 1.0)])
def test_norm(rows, d, xt, ht, resid, gain, offset):
    g = _gen(rows * 31 + d)
    x = (torch.randn(rows, d, generator=g, device="cuda") * torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))).to(xt)
    r = torch.randn(rows, d, generator=g, device="cuda").to(ht) if resid else None
    w = (torch.randn(d, generator=g, device="cuda") * 0.3 + 1 - offset).to(BF) if gain else None
    h, codes, scales = ops.add_rmsnorm_e4m3(x, w, r, gain_offset=offset)
    h64, y64 = _norm_ref(x, r, w, offset)
    _check_codes(codes, scales, y64, _norm_tol(y64, d))
    if resid:
        assert h.dtype == ht
        assert torch.all((h.double() - h64).abs() <= _round_tol(ht, h64) * (1 + 2 ** -10) + U * h64.abs())
    else:
        assert h is x


def test_norm_in_place_strides_and_guards():
    g = _gen(3)
    rows, d = 37, 400
    x, _ = _padded(torch.randn(rows, d, generator=g, device="cuda").to(BF), 8, float("nan"))
    r0 = torch.randn(rows, d, generator=g, device="cuda")
    r, rbuf = _padded(r0, 4, 7.0)
    w = torch.randn(d, generator=g, device="cuda").to(BF)
    codes, cbuf = _padded(torch.zeros(rows, d, dtype=FP8, device="cuda"), 16, 0x55)
    scales, sbuf = _padded(torch.zeros(rows, 4, device="cuda"), 3, 7.0)
    h, c2, s2 = ops.add_rmsnorm_e4m3(x, w, r, h_out=r, codes=codes, scales=scales)
    assert h is r and c2 is codes and s2 is scales
    h64, y64 = _norm_ref(x, r0, w, 0.0)
    _check_codes(codes.contiguous(), scales.contiguous(), y64, _norm_tol(y64, d))
    assert torch.all((r.double() - h64).abs() <= 2 * U * h64.abs())
    assert torch.all(rbuf[rows:] == 7.0) and torch.all(rbuf[:, d:] == 7.0)
    cb = cbuf.view(torch.uint8)
    assert torch.all(cb[rows:] == 0x55) and torch.all(cb[:, d:] == 0x55)
    assert torch.all(sbuf[rows:] == 7.0) and torch.all(sbuf[:, 4:] == 7.0)
    # without a residual, into x itself and into another type
    x2 = torch.randn(5, 64, device="cuda").to(BF)
    keep = x2.clone()
    h, *_ = ops.add_rmsnorm_e4m3(x2, h_out=x2)
    assert h is x2 and torch.equal(x2, keep)
    h, *_ = ops.add_rmsnorm_e4m3(x2, h_out=torch.empty(5, 64, device="cuda"))
    assert torch.equal(h, keep.float())


def test_norm_special_rows():
    x = torch.randn(6, 256, generator=_gen(4), device="cuda")
    x[0] = 0                                   # zero row: codes 0, scale 1
    x[1, 5] = float("nan")                     # NaN anywhere: rstd is NaN, every code of the row
    x[2, 7] = float("inf")                     # rstd = 0: inf x 0 is NaN, the others 0
    x[3] *= 1e-30                              # far below eps: tiny values, still scaled
    x[4] *= 1e15
    _, codes, scales = ops.add_rmsnorm_e4m3(x)
    c = codes.view(torch.uint8)
    assert torch.all(c[0] == 0) and torch.all(scales[0] == 1)
    assert torch.all((c[1] & 0x7F) == 0x7F)
    assert (int(c[2, 7]) & 0x7F) == 0x7F and torch.all((c[2, torch.arange(256) != 7] & 0x7F) == 0)
    for i in (3, 4, 5):
        _, y = _norm_ref(x[i:i + 1], None, None, 0.0)
        _check_codes(codes[i:i + 1], scales[i:i + 1], y, _norm_tol(y, 256))


# --------------------------------------------------------------------------- gated
@pytest.mark.parametrize("rows,f", [(1, 16), (1, 4096), (3, 128), (50, 4096), (5, 144), (33, 1904), (2, 1920), (4, 2048),
                                    (7, 2064), (129, 11008), (1000, 48), (2, 65536),
                                    # several rows per thread, the last group with 1 .. 7 of its 16 pieces
                                    (2999, 4112), (40001, 144), (80001, 16), (5001, 1968), (9999, 304)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "none"])
@pytest.mark.parametrize("xt", [BF, F32])
def test_gated(rows, f, act, xt):
    g = _gen(rows + f)
    x = (torch.randn(rows, f if act == "none" else 2 * f, generator=g, device="cuda") * 3).to(xt)
    codes, scales = ops.gated_e4m3(x, act)
    x64 = x.double()
    if act == "none":
        y, tol = x64, torch.zeros_like(x64)
    else:
        gate, up = x64[:, :f], x64[:, f:]
        if act == "silu":
            t = gate
        else:
            t = 2 * 0.7978845608028654 * (gate + 0.044715 * gate ** 3)
        y = gate * torch.sigmoid(t) * up
        # exp: 2 ulp = 4 u and 2 u |t| for its scaled argument, t itself 5 u |t|;
        # 1 + e, the division and the product 4 u
        tol = (8 + 7 * t.abs()) * U * y.abs() + 1e-37
    _check_codes(codes, scales, y, tol)


def test_quantise_bit_exact():
    """act "none" is the group recipe itself: every step is one fp32 operation."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((24, 304)).astype(np.float32) * np.exp(rng.standard_normal((24, 1)) * 20).astype(np.float32)
    x[0, :128] = 0
    x[1] = 1e-42                                # subnormal
    x[2, 128:256] *= 0
    x[3, :] = np.float32(3e38)
    x[4, :16] = [448, 1.0625, -1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 2.0 ** -10 * 1.5, 240, 17, 19, 21, -21, 432, 464, 0, -0.0]
    x[4, 16:128] = 0.5                          # a = 464 there; ties of E4M3 where 448 / a is exact:
    x[5, :128] = np.arange(128, dtype=np.float32) / 8
    x[5, 0] = 448
    codes, scales = ops.gated_e4m3(torch.from_numpy(x).cuda(), "none")
    codes, scales = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
    for i in range(x.shape[0]):
        for g in range(3):
            v = x[i, 128 * g:min(304, 128 * g + 128)]
            a = np.abs(v).max()
            t = max(a, np.float32(2.0 ** -100))
            s = np.float32(t / np.float32(448)) if a > 0 else np.float32(1)
            r = np.float32(np.float32(448) / t) if a > 0 else np.float32(1)
            assert scales[i, g] == s
            assert np.array_equal(codes[i, 128 * g:128 * g + len(v)], O.e4m3_encode((v * r).astype(np.float32))), (i, g)
    y = torch.zeros(2, 256, device="cuda")
    y[0, 3], y[0, 4], y[1, 200], y[1, 201] = float("nan"), 2.0, float("inf"), 5.0
    codes, scales = ops.gated_e4m3(y, "none")
    c = codes.view(torch.uint8)
    assert (int(c[0, 3]) & 0x7F) == 0x7F and float(codes[0, 4].float()) == 448 and float(scales[0, 0]) == np.float32(2) / np.float32(448)
    assert float(scales[1, 1]) == float("inf") and (int(c[1, 200]) & 0x7F) == 0x7F and int(c[1, 201]) == 0
    assert float(scales[1, 0]) == 1.0


def test_gated_extremes_and_guards():
    f = 128
    gate = torch.tensor([-1e30, -200.0, -90.0, -30.0, 0.0, 30.0, 1e13, 3e38], device="cuda").repeat(f // 8)
    for act in ("silu", "gelu_tanh"):
        x = torch.cat([gate, torch.full((f,), 0.5, device="cuda")])[None]
        codes, scales = ops.gated_e4m3(x, act)
        y = torch.where(gate > 0, gate, torch.zeros_like(gate)).double() * 0.5      # exact beyond |gate| = 30 at this scale
        _check_codes(codes, scales, y[None], 4 * U * y.abs()[None] + 1e-10)
    x, _ = _padded(torch.randn(9, 288, generator=_gen(5), device="cuda").to(BF), 8, float("nan"))
    codes, cbuf = _padded(torch.zeros(9, 144, dtype=FP8, device="cuda"), 16, 0x55)
    scales, sbuf = _padded(torch.zeros(9, 2, device="cuda"), 1, 7.0)
    ops.gated_e4m3(x, "silu", codes=codes, scales=scales)
    a, b = ops.gated_e4m3(x.contiguous(), "silu")
    assert torch.equal(codes.view(torch.uint8), a.view(torch.uint8)) and torch.equal(scales, b)
    cb = cbuf.view(torch.uint8)
    assert torch.all(cb[9:] == 0x55) and torch.all(cb[:, 144:] == 0x55)
    assert torch.all(sbuf[9:] == 7.0) and torch.all(sbuf[:, 2:] == 7.0)


# --------------------------------------------------------------------------- weight quantiser
@pytest.mark.parametrize("n,k", [(128, 128), (1, 1), (200, 300), (129, 127), (256, 1024), (1003, 48)])
def test_weight_quantiser_bit_exact(n, k):
    rng = np.random.default_rng(n + k)
    bits = synth.f32_to_bf16_bits(rng.standard_normal((n, k + 3)).astype(np.float32) * 0.02)
    if n > 128:
        bits[128:, :128] = 0                    # a zero block (or its part): scale 1
    wide = torch.from_numpy(bits.view(np.int16)).cuda().view(BF)
    codes, scales = ops.quantize_weight_e4m3(wide[:, :k])
    w = synth.bf16_bits_to_f32(bits)[:, :k]
    codes, scales = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
    for i in range(0, n, 128):
        for j in range(0, k, 128):
            b = w[i:i + 128, j:j + 128]
            a = np.abs(b).max()
            s = np.float32(max(a, np.float32(2.0 ** -100)) / np.float32(448)) if a > 0 else np.float32(1)
            assert scales[i // 128, j // 128] == s
            assert np.array_equal(codes[i:i + 128, j:j + 128], O.e4m3_encode((b / s).astype(np.float32)))


# --------------------------------------------------------------------------- matrix product
def _operands(m, n, k, seed):
    g = _gen(seed)
    a, sa = ops.gated_e4m3(torch.randn(m, k, generator=g, device="cuda") *
                           torch.exp(torch.randn(m, 1, generator=g, device="cuda")), "none")
    w, sw = ops.quantize_weight_e4m3((torch.randn(n, k, generator=g, device="cuda") * 0.05).to(BF))
    sw = sw * (1 + torch.rand(sw.shape, generator=g, device="cuda"))
    bias = torch.randn(n, generator=g, device="cuda").to(BF)
    return a, sa, w, sw, bias


def _gemm_ref(a, sa, w, sw, bias=None):
    """The product in 64 bits and the sum of the magnitudes of its terms."""
    k, n = a.shape[1], w.shape[0]
    A = a.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    W = w.double() * sw.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    out, mag = A @ W.t(), A.abs() @ W.abs().t()
    if bias is not None:
        out, mag = out + bias.double(), mag + bias.double().abs()
    return out, mag


def _gemm_tol(out, mag, k, dtype):
    # products of codes are exact; 128 sums inside a group (counted as
    # truncations, 2 u each), then a product of scales, a scaling and one sum per
    # group, at most 8 more sums where the groups are split, and the bias
    g = (k + 127) // 128
    tol = (2 * 128 + 2 * g + 8 + 4) * U * mag
    return tol + (0 if dtype == F32 else _half_step(BF) * (out.abs() + tol))


SIZES = [(m, n, k) for m in (1, 2, 9, 16, 17, 33, 50, 64, 65, 127, 128, 129, 300) for n, k in ((130, 144), (1024, 1024))]
SIZES += [(1, 1, 16), (1, 5, 112), (3, 127, 128), (777, 1003, 2064), (130, 257, 16), (1, 2560, 1024), (1, 8192, 4096),
          (50, 8192, 1024), (50, 1024, 4096), (8, 2048, 16384), (31, 640, 8208), (257, 128, 16384), (600, 4100, 512),
          (2048, 8200, 272), (4100, 513, 640), (1, 1, 16384), (5000, 16, 32), (256, 1000, 2048), (100, 384, 384)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype,with_bias", [(BF, True), (F32, False)])
def test_gemm(m, n, k, dtype, with_bias):
    a, sa, w, sw, bias = _operands(m, n, k, m * 7 + n * 3 + k)
    bias = bias if with_bias else None
    out = ops.gemm_e4m3(a, sa, w, sw, bias=bias, out_dtype=dtype)
    ops.sync()
    ref, mag = _gemm_ref(a, sa, w, sw, bias)
    assert out.dtype == dtype and out.shape == (m, n)
    assert torch.all((out.double() - ref).abs() <= _gemm_tol(ref, mag, k, dtype))
    assert torch.equal(out, ops.gemm_e4m3(a, sa, w, sw, bias=bias, out_dtype=dtype))


@pytest.mark.parametrize("m,n,k", [(1, 130, 256), (40, 300, 1040), (64, 256, 512), (200, 390, 528), (300, 512, 2048)])
def test_gemm_exact(m, n, k):
    """Small integers and power-of-two scales: every sum is exact, so the order cannot matter."""
    g = _gen(9)
    a = torch.randint(-3, 4, (m, k), generator=g, device="cuda").float().to(FP8)
    w = torch.randint(-3, 4, (n, k), generator=g, device="cuda").float().to(FP8)
    gk = (k + 127) // 128
    sa = torch.exp2(torch.randint(-1, 2, (m, gk), generator=g, device="cuda").float())
    sw = torch.exp2(torch.randint(-1, 2, ((n + 127) // 128, gk), generator=g, device="cuda").float())
    out = ops.gemm_e4m3(a, sa, w, sw, out_dtype=F32)
    assert torch.equal(out.double(), _gemm_ref(a, sa, w, sw)[0])


@pytest.mark.parametrize("m,n,k", [(5, 70, 144), (40, 300, 272), (130, 300, 272), (260, 515, 400)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gemm_strides_and_guards(m, n, k, dtype):
    """Every operand strided inside a buffer of NaN: nothing outside is read or written."""
    a, sa, w, sw, bias = _operands(m, n, k, 11)
    ref, mag = _gemm_ref(a, sa, w, sw, bias)
    a2, _ = _padded(a, 48, 0x7F)
    w2, _ = _padded(w, 16, 0x7F)
    sa2, _ = _padded(sa, 1, float("nan"))
    sw2, _ = _padded(sw, 2, float("nan"))
    b2 = torch.full((n + 9,), float("nan"), device="cuda", dtype=BF)
    b2[1:n + 1] = bias
    obuf = torch.full((m + 2, n + 7), 7.0, device="cuda", dtype=dtype)
    out = obuf[1:m + 1, 3:n + 3]                # rows at odd element offsets
    got = ops.gemm_e4m3(a2, sa2, w2, sw2, bias=b2[1:n + 1], out=out)
    assert got is out and torch.all((out.double() - ref).abs() <= _gemm_tol(ref, mag, k, dtype))
    assert torch.all(obuf[0] == 7) and torch.all(obuf[m + 1:] == 7)
    assert torch.all(obuf[:, :3] == 7) and torch.all(obuf[:, n + 3:] == 7)


@pytest.mark.parametrize("m", [3, 50, 200])
def test_gemm_non_finite_values_stay_in_their_row_and_column(m):
    a, sa, w, sw, _ = _operands(m, 200, 400, 12)
    clean = ops.gemm_e4m3(a, sa, w, sw, out_dtype=F32)
    a.view(torch.uint8)[1, 390] = 0x7F
    w.view(torch.uint8)[150, 3] = 0xFF
    sa[2, 1] = float("inf")
    out = ops.gemm_e4m3(a, sa, w, sw, out_dtype=F32)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1], bad[2], bad[:, 150] = True, True, True
    assert torch.all(out[1].isnan()) and torch.all(out[:, 150].isnan()) and not torch.any(out[2].isfinite())
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("m,n,k", [(1, 300001, 128), (3, 200000, 32), (700, 4099, 144), (3000, 901, 1168), (259, 40000, 96)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gemm_wide_and_odd(m, n, k, dtype):
    """Many channels of few rows, odd rows of a large output, bias, a short last group."""
    a, sa, w, sw, bias = _operands(m, n, k, m + n)
    out = ops.gemm_e4m3(a, sa, w, sw, bias=bias, out_dtype=dtype)
    ops.sync()
    for j in range(0, n, 50048):                # a multiple of 128
        e = min(n, j + 50048)
        ref, mag = _gemm_ref(a, sa, w[j:e], sw[j // 128:(e + 127) // 128], bias[j:e])
        assert torch.all((out[:, j:e].double() - ref).abs() <= _gemm_tol(ref, mag, k, dtype))


def test_gemm_scales_of_every_size():
    m, n, k = 40, 260, 512
    a, sa, w, sw, _ = _operands(m, n, k, 13)
    sa = sa * torch.exp2(torch.arange(m, device="cuda").float() * 2 - 40)[:, None]
    sw = sw * 2.0 ** 30
    sa[5] = 0
    out = ops.gemm_e4m3(a, sa, w, sw, out_dtype=F32)
    ref, mag = _gemm_ref(a, sa, w, sw)
    assert torch.all((out.double() - ref).abs() <= _gemm_tol(ref, mag, k, F32))
    assert torch.all(out[5] == 0)


# --------------------------------------------------------------------------- RoPE
def _rope_ref(x, pos, pairs, nq, nkv, hd):
    axis, freq = pairs
    n, rows = len(axis), x.shape[0]
    ang = pos.double()[torch.from_numpy(axis).long().cuda()].t() * torch.from_numpy(freq).cuda()
    t = x.double().view(rows, -1, hd)
    r = t[:, :nq + nkv]
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    lo, hi = r[..., :n], r[..., n:2 * n]
    out = torch.cat([lo * c - hi * s, hi * c + lo * s, r[..., 2 * n:]], -1)
    # cos and sin: the fraction of a turn one rounding (0.5 u turns = pi u), the
    # 64-bit product of position and frequency, sincospif 2 ulp; then 3 roundings
    tol = torch.zeros_like(out)
    ang_err = 4 * U + 2.0 ** -51 * ang.abs()[:, None]
    tol[..., :n] = (lo.abs() + hi.abs()) * (ang_err + 8 * U)
    tol[..., n:2 * n] = tol[..., :n]
    return out, tol, t[:, nq + nkv:]


ROPE = [  # rows, nq, nkv, hd, sections, ladder, interleaved, far
    (1, 16, 2, 128, (16, 24, 24), "shared", False, 4096), (306, 16, 2, 128, (16, 24, 24), "shared", False, 4096),
    (50, 4, 1, 64, (32,), "shared", False, 2 ** 31 - 1), (7, 8, 8, 256, (48, 40, 40), "shared", True, 1000000),
    (33, 3, 1, 80, (20, 20), "per_axis", False, 300), (5, 2, 2, 72, (12, 12, 12), "shared", False, 300),
    (9, 0, 3, 64, (8, 8), "shared", False, 300), (11, 2, 0, 96, (7, 9, 11, 5), "shared", True, 5000),
    (4100, 2, 1, 64, (16,), "shared", False, 70000), (3, 1, 1, 2, (1,), "shared", False, 10),
    (700, 7, 1, 128, (32, 16), "per_axis", False, 300), (2, 64, 8, 128, (64,), "shared", False, 131072),
]


@pytest.mark.parametrize("rows,nq,nkv,hd,sections,ladder,inter,far", ROPE)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope(rows, nq, nkv, hd, sections, ladder, inter, far, dtype):
    g = _gen(rows + hd)
    x = torch.randn(rows, (nq + 2 * nkv) * hd, generator=g, device="cuda").to(dtype)
    pos = torch.randint(-far, far, (len(sections), rows), generator=g, device="cuda").to(torch.int32)
    pairs = ops.rope_pairs(sections, ladder=ladder, interleaved=inter)
    q, k, v = ops.rope_axes(x, pos, pairs, nq, nkv, hd)
    ref, tol, vref = _rope_ref(x, pos, pairs, nq, nkv, hd)
    out = torch.cat([q, k], 1)
    assert torch.all((out.double() - ref).abs() <= tol + _half_step(dtype) * (ref.abs() + tol))
    assert torch.equal(v, x.view(rows, -1, hd)[:, nq + nkv:])
    n = sum(sections)
    assert torch.equal(out[..., 2 * n:], x.view(rows, -1, hd)[:, :nq + nkv, 2 * n:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hd,sections,off", [(64, (16, 16), 0), (64, (8, 8), 0), (64, (16, 16), 1), (72, (12, 24), 0)])
def test_rope_in_place_strides_and_missing_outputs(dtype, hd, sections, off):
    rows, nq, nkv = 45, 4, 2
    g = _gen(8)
    wide = (nq + 2 * nkv) * hd
    x0 = torch.randn(rows, wide, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 50, (2, rows), generator=g, device="cuda").to(torch.int32)
    pairs = ops.rope_pairs(sections)
    q, k, v = ops.rope_axes(x0, pos, pairs, nq, nkv, hd)
    buf = torch.full((rows + 1, wide + 16), 7.0, device="cuda", dtype=dtype)
    x = buf[:rows, off:off + wide]
    x.copy_(x0)
    heads = x.unflatten(1, (-1, hd))
    pbuf = torch.full((2, rows + 5), -9, device="cuda", dtype=torch.int32)
    pbuf[:, :rows] = pos
    r = ops.rope_axes(x, pbuf[:, :rows], pairs, nq, nkv, hd, q_out=heads[:, :nq], k_out=heads[:, nq:nq + nkv], v_out=False)
    assert r[2] is None
    assert torch.equal(heads[:, :nq], q) and torch.equal(heads[:, nq:nq + nkv], k) and torch.equal(heads[:, nq + nkv:], v)
    assert torch.all(buf[rows:] == 7) and torch.all(buf[:, :off] == 7) and torch.all(buf[:, off + wide:] == 7)
    # only the key heads, from rows without value heads
    cut = x0[:, :(nq + nkv) * hd].contiguous()
    none, k2, none2 = ops.rope_axes(cut, pos, pairs, nq, nkv, hd, q_out=False, v_out=False)
    assert none is None and none2 is None and torch.equal(k2, k)
    # into a cache with its own row stride
    cache = torch.full((rows, 3, nkv, hd), 7.0, device="cuda", dtype=dtype)
    ops.rope_axes(x0, pos, pairs, nq, nkv, hd, q_out=False, k_out=cache[:, 1], v_out=cache[:, 2])
    assert torch.equal(cache[:, 1], k) and torch.equal(cache[:, 2], v) and torch.all(cache[:, 0] == 7)


def test_rope_equal_positions_are_plain_rope():
    """Text tokens have one position on every axis: the oracle's one-axis RoPE."""
    rows, nq, nkv, hd = 20, 4, 2, 64
    x = torch.randn(rows, (nq + 2 * nkv) * hd, generator=_gen(2), device="cuda")
    pos = torch.arange(100, 100 + rows, device="cuda", dtype=torch.int32)
    q, k, _ = ops.rope_axes(x, pos.repeat(3, 1), ops.rope_pairs((8, 12, 12)), nq, nkv, hd)
    xs = x.double().cpu().numpy().reshape(rows, -1, hd)
    ref = O.rope(xs[:, :nq + nkv], pos.cpu().numpy(), 10000.0)
    got = torch.cat([q, k], 1).double().cpu().numpy()
    assert np.max(np.abs(got - ref)) <= 16 * U * np.max(np.abs(xs)) * 2


# --------------------------------------------------------------------------- all of them
def test_offsets_beyond_32_bits():
    """Row strides so wide that the last rows start past 2^32 bytes and 2^31 elements."""
    ld, rows = 2 ** 27, 34
    big = torch.empty(rows * ld, dtype=torch.uint8, device="cuda")          # 4.6 GB
    g = _gen(1)
    a, sa, w, sw, _ = _operands(rows, 128, 256, 1)
    av = big.view(FP8).as_strided((rows, 256), (ld, 1))
    av.copy_(a)
    want = ops.gemm_e4m3(a, sa, w, sw)
    assert torch.equal(ops.gemm_e4m3(av, sa, w, sw), want)
    assert torch.equal(ops.gemm_e4m3(w, torch.ones(128, 2, device="cuda"), av, sw[:1]),
                       ops.gemm_e4m3(w, torch.ones(128, 2, device="cuda"), a, sw[:1]))
    ov = big.view(BF).as_strided((rows, 128), (ld // 2, 1), 1024)
    ops.gemm_e4m3(a, sa, w, sw, out=ov)
    assert torch.equal(ov, want)
    del av, ov
    x = torch.randn(rows, 288, generator=g, device="cuda").to(BF)
    xv = big.view(BF).as_strided((rows, 288), (ld // 2, 1))
    xv.copy_(x)
    cv = big.view(FP8).as_strided((rows, 144), (ld, 1), 4096)
    c1, s1 = ops.gated_e4m3(x, "silu")
    _, s2 = ops.gated_e4m3(xv, "silu", codes=cv)
    assert torch.equal(cv.contiguous().view(torch.uint8), c1.view(torch.uint8)) and torch.equal(s1, s2)
    _, c1, s1 = ops.add_rmsnorm_e4m3(x)
    cv = big.view(FP8).as_strided((rows, 288), (ld, 1), 4096)
    _, _, s2 = ops.add_rmsnorm_e4m3(xv, codes=cv)
    assert torch.equal(cv.contiguous().view(torch.uint8), c1.view(torch.uint8)) and torch.equal(s1, s2)
    pos = torch.arange(rows, device="cuda", dtype=torch.int32)
    pairs = ops.rope_pairs((16,))
    q, k, v = ops.rope_axes(x, pos, pairs, 5, 2, 32)
    heads = xv.unflatten(1, (9, 32))
    ops.rope_axes(xv, pos, pairs, 5, 2, 32, q_out=heads[:, :5], k_out=heads[:, 5:7], v_out=heads[:, 7:])
    assert torch.equal(heads, torch.cat([q, k, v], 1))


def test_refusals_on_the_device():
    x = torch.randn(4, 256, device="cuda").to(BF)
    host = torch.randn(4, 256).to(BF).pin_memory()
    c = torch.empty(4, 256, dtype=torch.uint8, device="cuda")
    s = torch.empty(4, 2, device="cuda")
    lib = load()
    st = torch.cuda.current_stream().cuda_stream
    assert lib.fm_gated_e4m3(host.data_ptr(), 0, 256, 0, 4, 256, c.data_ptr(), 256, s.data_ptr(), 2, st) == 1
    assert b"x is not device memory" in lib.fm_last_error(None)
    assert lib.fm_gated_e4m3(x.data_ptr(), 0, 256, 0, 4, 256, c.data_ptr(), 256, host.data_ptr(), 2, st) == 1
    for bad in (x.float().double(), x.half(), x[:, ::2], x[0]):
        with pytest.raises(ValueError):
            ops.gated_e4m3(bad, "none")
    with pytest.raises(FmError, match="multiple of 16"):
        ops.gated_e4m3(x[:, :40].contiguous(), "none")
    with pytest.raises(FmError, match="16-byte"):
        ops.add_rmsnorm_e4m3(x[:, 4:132])
    with pytest.raises(ValueError, match="residual"):
        ops.add_rmsnorm_e4m3(x, residual=x[:3])
    with pytest.raises(ValueError, match="gain"):
        ops.add_rmsnorm_e4m3(x, torch.ones(256, device="cuda"))
    with pytest.raises(ValueError, match="requires grad"):
        ops.gated_e4m3(x.detach().requires_grad_(), "none")
    a, sa = ops.gated_e4m3(x, "none")
    with pytest.raises(ValueError, match="sw"):
        ops.gemm_e4m3(a, sa, a, sa)
    with pytest.raises(ValueError, match="w has shape"):
        ops.gemm_e4m3(a, sa, a[:, :128], sa[:1, :1])
    with pytest.raises(ValueError, match="out"):
        ops.gemm_e4m3(a, sa, a, sa[:1], out=torch.empty(4, 5, device="cuda"))
    pairs = ops.rope_pairs((32,))
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="columns"):
        ops.rope_axes(x, pos, pairs, 3, 1, 64)
    with pytest.raises(ValueError, match="positions"):
        ops.rope_axes(x, pos[:3], pairs, 2, 1, 64)
    with pytest.raises(ValueError, match="positions"):
        ops.rope_axes(x, pos.long(), pairs, 2, 1, 64)
    with pytest.raises(ValueError, match="pairs"):
        ops.rope_axes(x, pos, (pairs[0].astype(np.int64), pairs[1]), 2, 1, 64)
    with pytest.raises(FmError, match="axis 1 of 1"):
        ops.rope_axes(x, pos, (pairs[0] + np.uint8(1), pairs[1]), 2, 1, 64)
    e = ops.gemm_e4m3(a[:0], sa[:0], a, sa[:1])
    assert e.shape == (0, 4)
    q, k, v = ops.rope_axes(x[:0], pos[:0], pairs, 2, 1, 64)
    assert q.shape == (0, 2, 64) and v.shape == (0, 1, 64)
    ops.sync()


def _layer(x, h, gain, wq, bq, wgu, pos, pairs):
    h2, a, sa = ops.add_rmsnorm_e4m3(x, gain, residual=h)
    q, k, v = ops.rope_axes(ops.gemm_e4m3(a, sa, *wq, bias=bq), pos, pairs, 4, 2, 64)
    u, su = ops.gated_e4m3(ops.gemm_e4m3(a, sa, *wgu), "silu")
    return h2, q, k, v, u.view(torch.uint8), su


def _layer_inputs(rows, seed):
    g = _gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=rnd(rows, 256).to(BF), h=rnd(rows, 256), gain=rnd(256).to(BF),
                wq=ops.quantize_weight_e4m3((rnd(512, 256) * 0.05).to(BF)), bq=rnd(512).to(BF),
                wgu=ops.quantize_weight_e4m3((rnd(2048, 256) * 0.05).to(BF)),
                pos=torch.randint(0, 99, (3, rows), generator=g, device="cuda").to(torch.int32),
                pairs=ops.rope_pairs((8, 12, 12)))


@pytest.mark.parametrize("rows", [1, 50, 300])
def test_graph_streams_and_determinism(rows):
    ins = [_layer_inputs(rows, s) for s in (1, 2)]
    want = [_layer(**i) for i in ins]
    torch.cuda.synchronize()
    # two streams at once, several times
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        got = []
        for st, i in zip(streams, ins):
            with torch.cuda.stream(st):
                got.append(_layer(**i))
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, o))
    # two graphs, replayed in turn and at once, on new inputs in the same memory
    graphs, outs = [], []
    for i in ins:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_layer(**i))
        graphs.append(gr)
    new = [_layer_inputs(rows, s) for s in (3, 4)]
    for i, n in zip(ins, new):
        i["x"].copy_(n["x"])
        i["pos"].copy_(n["pos"])
    want = [_layer(**i) for i in ins]
    torch.cuda.synchronize()
    for st, gr in zip(streams, graphs):
        with torch.cuda.stream(st):
            gr.replay()
            gr.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(a, b) for a, b in zip(w, o))
    ops.sync()


def test_backbone_prefix_into_the_expert():
    """The operators in the use they are for: a block-scaled backbone projects
    the prefix's hidden states (norm, q|k|v product with bias, RoPE over three
    axes), its K and V go into the expert's cache, and the chunk is denoised.

    The keys and values agree with a 64-bit run of the same layers (the codes'
    own error taken from the codes), and the chunk with the oracle's on them."""
    s = synth.WORKLOADS["tiny"]
    P, d, nq, nkv, hd = 40, 512, s.n_q_heads, s.n_kv_heads, s.head_dim
    g = _gen(6)
    raw = synth.make_weights(s)
    pairs = ops.rope_pairs((8, 12, 12))
    pos = torch.randint(0, 64, (3, P), generator=g, device="cuda").to(torch.int32)
    ks, vs = [], []
    for _ in range(s.n_layers):
        x = torch.randn(P, d, generator=g, device="cuda").to(BF)
        gain = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(BF)
        w = (torch.randn((nq + 2 * nkv) * hd, d, generator=g, device="cuda") * 0.05).to(BF)
        bias = (torch.randn(w.shape[0], generator=g, device="cuda") * 0.1).to(BF)
        wc, ws = ops.quantize_weight_e4m3(w)
        _, a, sa = ops.add_rmsnorm_e4m3(x, gain)
        qkv = ops.gemm_e4m3(a, sa, wc, ws, bias=bias)
        _, k, v = ops.rope_axes(qkv, pos, pairs, nq, nkv, hd, q_out=False)
        ref, mag = _gemm_ref(a, sa, wc, ws, bias)
        tol = _gemm_tol(ref, mag, d, BF)
        vref = ref[:, (nq + nkv) * hd:]
        assert torch.all((v.double().flatten(1) - vref).abs() <= tol[:, (nq + nkv) * hd:])
        kref, ktol, _ = _rope_ref(ref, pos, pairs, nq, nkv, hd)
        t = tol.view(P, -1, hd)[:, nq:nq + nkv]
        t = t + t.roll(hd // 2, -1)                       # a rotation mixes the pair's errors
        kref, ktol = kref[:, nq:], ktol[:, nq:] * (1 + 2 ** -6)
        assert torch.all((k.double() - kref).abs() <= t + ktol + _half_step(BF) * (kref.abs() + t))
        # against the layer before quantisation: E4M3 steps of both operands,
        # each at most 2^-4 of a value, in sums of 512 terms of random sign
        _, y = _norm_ref(x, None, gain, 0.0)
        full = y @ w.double().t() + bias.double()
        assert float((ref - full).norm() / (full - bias.double()).norm()) <= 2 * 2 ** -4
        ks.append(k[None].contiguous())
        vs.append(v[None].contiguous())
    e = Expert(s, raw, max_prefix=P)
    e.set_prefix(ks, vs, 1, P)
    x0 = synth.make_x0(s)
    out = e.denoise(x0, 10)
    e.close()
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    ref = O.denoise(x0, 10, raw, [bits(k) for k in ks], [bits(v) for v in vs], s)
    cos = float(np.dot(out.ravel(), ref.ravel()) / (np.linalg.norm(out) * np.linalg.norm(ref)))
    assert cos >= 0.999 and np.max(np.abs(out - ref)) <= 5e-2      # the library's own bars of this workload


def test_given_stream():
    """`stream` as a torch stream or a handle: work and new outputs belong to it."""
    ins = _layer_inputs(70, 5)
    _, a, sa = ops.add_rmsnorm_e4m3(ins["x"], ins["gain"], residual=ins["h"])
    want = ops.gemm_e4m3(a, sa, *ins["wq"])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (st, st.cuda_stream):
        _, a2, sa2 = ops.add_rmsnorm_e4m3(ins["x"], ins["gain"], residual=ins["h"], stream=s)
        got = ops.gemm_e4m3(a2, sa2, *ins["wq"], stream=s)
        ops.sync(s)
        assert torch.equal(got, want)


_FIRST = """
import torch
from vla_flow_matching_denoise_b200 import ops
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(640, 2048, generator=g, device="cuda").bfloat16()
w = (torch.randn(4096, 1024, generator=g, device="cuda") * 0.05).bfloat16()
pos = torch.zeros(3, 640, dtype=torch.int32, device="cuda")
pairs = ops.rope_pairs((8, 12, 12))
def run():
    wc, ws = ops.quantize_weight_e4m3(w)
    u, su = ops.gated_e4m3(x)
    h, c, s = ops.add_rmsnorm_e4m3(x)
    y = ops.gemm_e4m3(u, su, wc, ws)                 # many rows
    z = ops.gemm_e4m3(u[:5], su[:5], wc, ws)         # few rows
    q, k, v = ops.rope_axes(y[:, :1024], pos, pairs, 8, 4, 64)
    return y, z, q, k, v, c.view(torch.uint8)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
want = run()
ops.sync()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing needs a call before the one that is captured."""
    r = subprocess.run([sys.executable, "-c", _FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-500:] + r.stderr[-1500:]


def test_calls_from_several_threads():
    ins = [_layer_inputs(64 + 8 * i, 20 + i) for i in range(4)]
    want = [_layer(**i) for i in ins]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(20):
                got = _layer(**ins[i])
                st.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)
        # a refusal's text belongs to its thread
        try:
            ops.gated_e4m3(ins[i]["x"][:, :16 * i + 8].contiguous(), "none")
        except FmError as e:
            if f"f {16 * i + 8} out of range" not in str(e):
                bad.append(str(e))
        else:
            bad.append("not refused")

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
