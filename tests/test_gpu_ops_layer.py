"""A whole layer closed over the operators (the attention between them in 64 bits):
every operator's result against its definition on the inputs that it had, eagerly,
for one token and for many, and the same bits from a captured graph."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.test_gpu_ops import (BF, F32, U, _check_codes, _gemm_ref, _gemm_tol, _half_step, _norm_ref, _norm_tol,  # noqa: E402
                                _rope_ref)
from vla_flow_matching_denoise_b200 import ops  # noqa: E402

D, NQ, NKV, HD, F = 512, 8, 2, 64, 1408


def _weights(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def w(n, k):
        return ops.quantize_weight_e4m3((torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).to(BF))
    gain = lambda: (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(BF)  # noqa: E731
    return dict(g1=gain(), g2=gain(), g3=gain(), wqkv=w((NQ + 2 * NKV) * HD, D), wo=w(D, NQ * HD), wgu=w(2 * F, D), wd=w(D, F),
                bqkv=torch.randn((NQ + 2 * NKV) * HD, generator=g, device="cuda").to(BF) * 0.1,
                pairs=ops.rope_pairs((8, 12, 12)))


def _attend(q, k, v):
    """Causal attention of bf16 heads in 64 bits, rounded to bf16."""
    q, k, v = (t.double().transpose(0, 1) for t in (q, k, v))
    k, v = (t.repeat_interleave(NQ // NKV, 0) for t in (k, v))
    s = q @ k.transpose(1, 2) * HD ** -0.5
    s = s.masked_fill(torch.ones_like(s[0], dtype=torch.bool).triu(1), float("-inf"))
    return (torch.softmax(s, -1) @ v).transpose(0, 1).reshape(q.shape[1], NQ * HD).to(BF)


def _layer(h, pos, w, act, attend=_attend):
    """h: the fp32 residual stream, updated in place.  Every intermediate tensor by name."""
    t = {}
    _, t["a1"], t["s1"] = ops.add_rmsnorm_e4m3(h, w["g1"])
    t["qkv"] = ops.gemm_e4m3(t["a1"], t["s1"], *w["wqkv"], bias=w["bqkv"])
    t["q"], t["k"], t["v"] = ops.rope_axes(t["qkv"], pos, w["pairs"], NQ, NKV, HD)
    t["att"] = attend(t["q"], t["k"], t["v"])
    t["a2"], t["s2"] = ops.gated_e4m3(t["att"], "none")
    t["o"] = ops.gemm_e4m3(t["a2"], t["s2"], *w["wo"])
    _, t["a3"], t["s3"] = ops.add_rmsnorm_e4m3(t["o"], w["g2"], residual=h, h_out=h)
    t["h1"] = h.clone()
    t["gu"] = ops.gemm_e4m3(t["a3"], t["s3"], *w["wgu"])
    t["a4"], t["s4"] = ops.gated_e4m3(t["gu"], act)
    t["d"] = ops.gemm_e4m3(t["a4"], t["s4"], *w["wd"], out_dtype=F32)
    _, t["a5"], t["s5"] = ops.add_rmsnorm_e4m3(t["d"], w["g3"], residual=h, h_out=h)
    t["h2"] = h.clone()
    return t


@pytest.mark.parametrize("rows", [1, 50, 306])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_layer(rows, act):
    w = _weights(rows)
    g = torch.Generator(device="cuda").manual_seed(rows + 1)
    h0 = torch.randn(rows, D, generator=g, device="cuda")
    pos = torch.randint(0, 64, (3, rows), generator=g, device="cuda").to(torch.int32)
    t = _layer(h0.clone(), pos, w, act)
    ops.sync()

    def norm(x, res, gain, a, s):
        hh, y = _norm_ref(x, res, gain, 0.0)
        _check_codes(t[a], t[s], y, _norm_tol(y, D))
        return hh

    def product(a, s, wt, out, bias=None):
        ref, mag = _gemm_ref(t[a], t[s], *wt, bias)
        assert torch.all((t[out].double() - ref).abs() <= _gemm_tol(ref, mag, t[a].shape[1], t[out].dtype))

    norm(h0, None, w["g1"], "a1", "s1")
    product("a1", "s1", w["wqkv"], "qkv", w["bqkv"])
    ref, tol, v = _rope_ref(t["qkv"], pos, w["pairs"], NQ, NKV, HD)
    got = torch.cat([t["q"], t["k"]], 1).double()
    assert torch.all((got - ref).abs() <= tol + _half_step(BF) * (ref.abs() + tol)) and torch.equal(t["v"], v.to(BF))
    _check_codes(t["a2"], t["s2"], t["att"].double(), torch.zeros_like(t["att"], dtype=torch.float64))
    product("a2", "s2", w["wo"], "o")
    h1 = norm(t["o"], h0, w["g2"], "a3", "s3")
    assert torch.all((t["h1"].double() - h1).abs() <= 2 * U * h1.abs())
    product("a3", "s3", w["wgu"], "gu")
    gate, up = t["gu"].double().chunk(2, 1)
    e = gate if act == "silu" else 2 * 0.7978845608028654 * (gate + 0.044715 * gate ** 3)
    y = gate * torch.sigmoid(e) * up
    _check_codes(t["a4"], t["s4"], y, (13 + 8 * e.abs()) * U * y.abs())
    product("a4", "s4", w["wd"], "d")
    h2 = norm(t["d"], t["h1"], w["g3"], "a5", "s5")
    assert torch.all((t["h2"].double() - h2).abs() <= 2 * U * h2.abs())

    # the same bits from a graph, on inputs that arrive after the capture (what lies
    # between the operators has to be capturable: a fixed mixture of the heads)
    def mix(q, k, v):
        return (q + k.repeat_interleave(NQ // NKV, 1) + v.repeat_interleave(NQ // NKV, 1)).flatten(1)
    x, p = torch.zeros_like(h0), torch.zeros_like(pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _layer(x, p, w, act, mix)
    want = _layer(h0.clone(), pos, w, act, mix)
    for _ in range(2):
        x.copy_(h0)
        p.copy_(pos)
        graph.replay()
        assert all(torch.equal(out[n].view(torch.uint8), want[n].view(torch.uint8)) for n in want)
    ops.sync()


def test_norm_outside_the_range_of_its_sum_of_squares():
    """What the header says of rows whose squares leave fp32."""
    x = torch.full((3, 128), 2.0, device="cuda")
    x[0] *= 1e19
    x[1] *= 1e-24
    _, codes, scales = ops.add_rmsnorm_e4m3(x, eps=0.0)
    assert torch.all(codes[0].float() == 0) and torch.all(codes[1].float().isnan())
    assert torch.all(codes[2].float() == 448)
