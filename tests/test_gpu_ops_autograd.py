"""The operators beside autograd: what they write into given tensors is seen by
graphs that saved them, and what they cannot differentiate is refused."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from vla_flow_matching_denoise_b200 import ops  # noqa: E402

BF = torch.bfloat16
FP8 = torch.float8_e4m3fn


def _calls():
    """name -> (call, given output or input that stays) of every tensor that a call writes."""
    x = torch.randn(8, 256, device="cuda").to(BF)
    res = torch.randn(8, 256, device="cuda")
    a, sa = ops.gated_e4m3(x, "none")
    w, sw = ops.quantize_weight_e4m3(torch.randn(128, 256, device="cuda").to(BF))
    pos = torch.arange(8, device="cuda", dtype=torch.int32)
    pairs = ops.rope_pairs((16,))
    f = lambda *s, dtype=torch.float32: torch.zeros(*s, device="cuda", dtype=dtype)  # noqa: E731
    h, c, s, c2, s2 = f(8, 256), f(8, 256, dtype=torch.uint8), f(8, 2), f(8, 128, dtype=torch.uint8), f(8, 1)
    out, q, k, v = f(8, 128), f(8, 4, 32, dtype=BF), f(8, 2, 32, dtype=BF), f(8, 2, 32, dtype=BF)
    return {
        "norm in place": (lambda: ops.add_rmsnorm_e4m3(x, residual=res, h_out=res), [res], [x]),
        "norm": (lambda: ops.add_rmsnorm_e4m3(x, residual=res, h_out=h, codes=c, scales=s), [h, c, s], [x, res]),
        "gated": (lambda: ops.gated_e4m3(x, codes=c2, scales=s2), [c2, s2], [x]),
        "gemm": (lambda: ops.gemm_e4m3(a, sa, w, sw, out=out), [out], [a, sa, w, sw]),
        "rope": (lambda: ops.rope_axes(x, pos, pairs, 4, 2, 32, q_out=q, k_out=k, v_out=v), [q, k, v], [x, pos]),
        "rope, some": (lambda: ops.rope_axes(x, pos, pairs, 4, 2, 32, q_out=False, k_out=k), [k], [x, pos, q]),
    }


@pytest.mark.parametrize("name", ["norm in place", "norm", "gated", "gemm", "rope", "rope, some"])
def test_given_outputs_count_as_written_in_place(name):
    call, written, kept = _calls()[name]
    before = [t._version for t in written], [t._version for t in kept]
    call()
    assert [t._version for t in written] == [v + 1 for v in before[0]]
    assert [t._version for t in kept] == before[1]


def test_a_graph_that_saved_the_residual_refuses_its_backward():
    x = torch.randn(4, 256, device="cuda").to(BF)
    h = torch.randn(4, 256, device="cuda")
    w = torch.randn(256, device="cuda", requires_grad=True)
    loss = (h * w).sum()
    ops.add_rmsnorm_e4m3(x, residual=h, h_out=h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    view = torch.randn(2, 4, 256, device="cuda")              # through a view of what was saved
    loss = (view * w).sum()
    ops.add_rmsnorm_e4m3(x, residual=view[1], h_out=view[1])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_and_leaves_without_recording():
    with torch.inference_mode():
        x = torch.randn(4, 256, device="cuda").to(BF)
        codes = torch.empty(4, 128, dtype=torch.uint8, device="cuda")
        ops.gated_e4m3(x, codes=codes)
    ops.gated_e4m3(x, codes=codes)
    gain = torch.nn.Parameter(torch.ones(256, device="cuda", dtype=BF))
    with pytest.raises(ValueError, match="gain requires grad"):
        ops.add_rmsnorm_e4m3(x, gain)
    with torch.no_grad():
        ops.add_rmsnorm_e4m3(x, gain)


def test_forward_mode_tangents_are_refused():
    import torch.autograd.forward_ad as fwd
    x = torch.randn(4, 256, device="cuda")
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="x carries a forward-mode tangent"):
            ops.add_rmsnorm_e4m3(dual)
        with torch.no_grad(), pytest.raises(ValueError, match="residual carries a forward-mode tangent"):
            ops.add_rmsnorm_e4m3(x, residual=dual)
        ops.add_rmsnorm_e4m3(fwd.unpack_dual(dual).primal)
