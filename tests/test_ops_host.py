"""Host-side checks of the E4M3 block-scaled operators (no GPU needed): every
refusal that does not depend on a device happens before one is touched, and
the RoPE pair table."""
import numpy as np
import pytest

from vla_flow_matching_denoise_b200.binding import load

P = 0x10000          # a 16-byte aligned address; every call below is refused before it is used
AX = np.zeros(64, dtype=np.uint8)
FR = np.ones(64, dtype=np.float64)


def _norm(lib, **kw):
    a = dict(x=P, xt=0, ldx=256, res=P, ht=0, ldr=256, gain=P, off=0.0, eps=1e-6, rows=4, d=256, h=P, ldh=256,
             codes=P, ldc=256, scales=P, lds=2, stream=None)
    a.update(kw)
    return lib.fm_add_rmsnorm_e4m3(*a.values())


def _gated(lib, **kw):
    a = dict(x=P, xt=0, ldx=512, act=1, rows=4, f=256, codes=P, ldc=256, scales=P, lds=2, stream=None)
    a.update(kw)
    return lib.fm_gated_e4m3(*a.values())


def _quant(lib, **kw):
    a = dict(w=P, ldw=256, n=128, k=256, codes=P, ldc=256, scales=P, lds=2, stream=None)
    a.update(kw)
    return lib.fm_quantize_weight_e4m3_b128(*a.values())


def _gemm(lib, **kw):
    a = dict(a=P, lda=256, sa=P, ldsa=2, w=P, ldw=256, sw=P, ldsw=2, bias=None, m=130, n=200, k=256, out=P, ot=0,
             ldo=200, stream=None)
    a.update(kw)
    return lib.fm_gemm_e4m3_b128(*a.values())


def _rope(lib, **kw):
    a = dict(x=P, t=0, ldx=1280, rows=4, nq=8, nkv=1, hd=128, pos=P, ldp=4, axes=3, axis=AX.ctypes.data,
             freq=FR.ctypes.data, n=64, q=P, ldq=1024, k=P, ldk=128, v=P, ldv=128, stream=None)
    a.update(kw)
    return lib.fm_rope_axes(*a.values())


INVALID, CUDA, UNSUPPORTED = 1, 4, 6


@pytest.mark.parametrize("call,kw,status,text", [
    (_norm, dict(xt=2), UNSUPPORTED, "x_type"),
    (_norm, dict(ht=-1), UNSUPPORTED, "h_type"),
    (_norm, dict(d=8), INVALID, "d 8"),
    (_norm, dict(d=250, ldx=256), INVALID, "multiple of 16"),
    (_norm, dict(d=16400), INVALID, "16384"),
    (_norm, dict(rows=-1), INVALID, "rows -1"),
    (_norm, dict(eps=-1.0), INVALID, "eps"),
    (_norm, dict(eps=float("nan")), INVALID, "eps"),
    (_norm, dict(x=None), INVALID, "x is NULL"),
    (_norm, dict(codes=None), INVALID, "codes is NULL"),
    (_norm, dict(scales=None), INVALID, "scales is NULL"),
    (_norm, dict(ldx=248), INVALID, "x: row stride"),
    (_norm, dict(ldr=128), INVALID, "residual: row stride"),
    (_norm, dict(ldh=0), INVALID, "h_out: row stride"),
    (_norm, dict(ldc=255), INVALID, "codes: row stride"),
    (_norm, dict(lds=1), INVALID, "scales: row stride"),
    (_norm, dict(x=P + 2), INVALID, "x: rows must start on 16"),
    (_norm, dict(ldx=260), INVALID, "x: rows must start on 16"),
    (_norm, dict(ldc=264), INVALID, "codes: rows must start on 16"),
    (_norm, dict(gain=P + 2), INVALID, "gain"),
    (_norm, dict(scales=P + 2), INVALID, "scales: rows must start on 4"),
    (_gated, dict(act=3), UNSUPPORTED, "act"),
    (_gated, dict(xt=5), UNSUPPORTED, "x_type"),
    (_gated, dict(f=0), INVALID, "f 0"),
    (_gated, dict(f=24), INVALID, "multiple of 16"),
    (_gated, dict(f=(1 << 20) + 16), INVALID, "2^20"),
    (_gated, dict(rows=(1 << 31) - 1, f=1 << 20), INVALID, "one launch"),
    (_gated, dict(ldx=504), INVALID, "x: row stride"),
    (_gated, dict(x=P + 8), INVALID, "x: rows"),
    (_quant, dict(n=-1), INVALID, "negative"),
    (_quant, dict(w=None), INVALID, "w is NULL"),
    (_quant, dict(w=P + 1), INVALID, "w: rows"),
    (_quant, dict(n=129, lds=1), INVALID, "scales: row stride"),
    (_gemm, dict(ot=2), UNSUPPORTED, "out_type"),
    (_gemm, dict(k=0), INVALID, "k 0"),
    (_gemm, dict(k=250), INVALID, "multiple of 16"),
    (_gemm, dict(m=-1), INVALID, "m -1"),
    (_gemm, dict(a=None), INVALID, "a is NULL"),
    (_gemm, dict(sw=None), INVALID, "sw is NULL"),
    (_gemm, dict(out=None), INVALID, "out is NULL"),
    (_gemm, dict(lda=128), INVALID, "a: row stride"),
    (_gemm, dict(ldw=264), INVALID, "w: rows must start on 16"),
    (_gemm, dict(a=P + 8), INVALID, "a: rows must start on 16"),
    (_gemm, dict(ldsa=1), INVALID, "sa: row stride"),
    (_gemm, dict(ldsw=1), INVALID, "sw: row stride"),
    (_gemm, dict(bias=P + 1), INVALID, "bias"),
    (_gemm, dict(ldo=199), INVALID, "out: row stride"),
    (_gemm, dict(out=P + 2, ot=1), INVALID, "out: rows must start on 4"),
    (_gemm, dict(m=2147483647, n=2147483647, ldo=2147483647), INVALID, "one launch"),
    (_rope, dict(t=2), UNSUPPORTED, "type"),
    (_rope, dict(hd=127), INVALID, "head_dim"),
    (_rope, dict(hd=258), INVALID, "head_dim"),
    (_rope, dict(n=0), INVALID, "n_pairs"),
    (_rope, dict(hd=64), INVALID, "n_pairs 64"),
    (_rope, dict(axes=0), INVALID, "n_axes"),
    (_rope, dict(axes=9), INVALID, "n_axes"),
    (_rope, dict(axis=None), INVALID, "pair_axis"),
    (_rope, dict(nq=1025), INVALID, "heads"),
    (_rope, dict(rows=-4), INVALID, "rows -4"),
    (_rope, dict(ldx=1272), INVALID, "x: row stride"),
    (_rope, dict(ldp=3), INVALID, "positions: row stride"),
    (_rope, dict(ldq=1023), INVALID, "q_out: row stride"),
    (_rope, dict(x=P + 1), INVALID, "x: rows"),
    (_rope, dict(pos=None), INVALID, "positions is NULL"),
])
def test_refusals_before_the_device_is_touched(lib, call, kw, status, text):
    assert call(lib, **kw) == status, lib.fm_last_error(None)
    assert text in lib.fm_last_error(None).decode()


def test_bad_pair_tables(lib):
    axis = AX.copy()
    axis[5] = 3
    assert _rope(lib, axis=axis.ctypes.data) == INVALID
    assert b"axis 3 of 3" in lib.fm_last_error(None)
    freq = FR.copy()
    freq[63] = np.inf
    assert _rope(lib, freq=freq.ctypes.data) == INVALID
    assert b"finite" in lib.fm_last_error(None)


@pytest.mark.parametrize("call,kw", [
    (_norm, dict(rows=0, x=None, codes=None, scales=None)),
    (_gated, dict(rows=0, x=None)),
    (_quant, dict(n=0, w=None)),
    (_quant, dict(k=0)),
    (_gemm, dict(m=0, a=None, out=None)),
    (_gemm, dict(n=0, w=None, out=None)),
    (_rope, dict(rows=0, x=None)),
    (_rope, dict(q=None, k=None, v=None)),
    (_rope, dict(nq=0, nkv=0)),
])
def test_nothing_to_do_is_ok(lib, call, kw):
    assert call(lib, **kw) == 0, lib.fm_last_error(None)
    assert lib.fm_last_error(None) == b""


def test_a_call_without_a_device_reports_it(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a device")
    assert _gemm(lib) == CUDA
    assert lib.fm_last_error(None)


def test_rope_pairs():
    torch = pytest.importorskip("torch")  # noqa: F841  (ops imports it)
    from vla_flow_matching_denoise_b200 import ops
    axis, freq = ops.rope_pairs([2, 3, 1])
    assert axis.tolist() == [0, 0, 1, 1, 1, 2] and axis.dtype == np.uint8
    assert np.allclose(freq, [10000.0 ** (-j / 6) for j in range(6)], rtol=1e-15)
    axis, freq = ops.rope_pairs([2, 3, 1], base=100.0, interleaved=True)
    assert axis.tolist() == [0, 1, 2, 0, 1, 1]
    assert np.allclose(freq, [100.0 ** (-j / 6) for j in range(6)], rtol=1e-15)
    axis, freq = ops.rope_pairs([2, 0, 3], ladder="per_axis")
    assert axis.tolist() == [0, 0, 2, 2, 2]
    assert np.allclose(freq, [1, 1e4 ** -0.5, 1, 1e4 ** (-1 / 3), 1e4 ** (-2 / 3)], rtol=1e-15)
    for bad in (dict(sections=[]), dict(sections=[0]), dict(sections=[-1, 3]), dict(sections=[2], ladder="x"),
                dict(sections=[2], ladder="per_axis", interleaved=True)):
        with pytest.raises(ValueError):
            ops.rope_pairs(**bad)


def test_python_checks_refuse_cpu_tensors_and_bad_shapes():
    torch = pytest.importorskip("torch")
    from vla_flow_matching_denoise_b200 import ops
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.add_rmsnorm_e4m3(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.gated_e4m3(x)
    with pytest.raises(ValueError, match="act"):
        ops.gated_e4m3(x, "relu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.quantize_weight_e4m3(x)


@pytest.mark.parametrize("args", [(5, 0, 0), (-1, 0, 0), (1, -1, 0), (1, 0, -1)])
def test_the_stall_hook_refuses_what_is_out_of_range(lib, args):
    assert lib.fm_ops_test_stall(*args) == INVALID
    assert b"fm_ops_test_stall" in lib.fm_last_error(None)
    assert lib.fm_ops_test_stall(0, 0, 0) == 0


def test_sync_asks_the_device_of_the_stream(monkeypatch):
    torch = pytest.importorskip("torch")
    import contextlib
    from types import SimpleNamespace

    from vla_flow_matching_denoise_b200 import ops
    current, asked = [0], []

    @contextlib.contextmanager
    def device(d):
        was, current[0] = current[0], d.index
        yield
        current[0] = was

    fake = SimpleNamespace(fm_ops_sync=lambda st: asked.append((current[0], st)) or 0)
    monkeypatch.setattr(ops, "load", lambda: fake)
    monkeypatch.setattr(torch.cuda, "device", device)
    ops.sync(SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=77))
    ops.sync(78)
    assert asked == [(1, 77), (0, 78)] and current == [0]
