"""fm_gated_e4m3 over the whole range of its gate: each gate in rows of its own, so
that every group's scale is one activation's value, which the scale then pins to a
few roundings (the codes alone know it to 2^-4)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.test_gpu_ops import BF, F32, U, _check_codes  # noqa: E402
from vla_flow_matching_denoise_b200 import ops  # noqa: E402

SILU = [-150.0, -130.7, -110.3, -104.0, -100.0, -95.2, -90.0, -89.0, -88.7, -88.0, -87.4, -87.0, -86.6, -86.0, -80.1, -60.3,
        -40.7, -30.0, -20.2, -10.3, -3.1, -1.0, -0.3, -1e-5, -1e-30, 1e-30, 1e-5, 0.3, 1.0, 3.1, 10.3, 17.0, 50.7, 86.6, 87.4,
        88.0, 90.0, 104.0, 1e3, 1e13, 1e30, 3e38]
GELU = [-12.2, -11.9, -11.1, -10.4, -10.1, -10.03, -9.96, -9.9, -9.5, -9.0, -7.7, -5.3, -3.1, -1.0, -0.3, -1e-5, -1e-30,
        1e-30, 1e-5, 0.3, 1.0, 3.1, 5.3, 7.7, 9.96, 10.03, 11.1, 50.0, 1e3, 1e13, 1e30, 3e38]


def _act(gate, act):
    """(activation, exponent in nats) in 64 bits."""
    t = gate if act == "silu" else 2 * 0.7978845608028654 * (gate + 0.044715 * gate ** 3)
    return gate * torch.sigmoid(t), t


def _tol(y, t, act):
    # 2^x and 1/x are 2 and 1 ulp (4 u and 2 u) and the three operations around
    # them u each, + the product with up; SiLU's exponent is made to 48 bits and
    # its correction is one more u.  GELU's is made of three fp32 operations and
    # two constants of three and two roundings: 8 u of the exponent.  Where
    # 1 / (1 + 2^x) leaves fp32's normal range it is 2^-x by two halves: 2 x 4 u,
    # three products and the correction's two.
    return (13 + (0 if act == "silu" else 8 * t.abs())) * U * y.abs()


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("act,gates", [("silu", SILU), ("gelu_tanh", GELU)])
@pytest.mark.parametrize("rows", [1, 6000])     # a row per thread, and several
def test_every_gate_in_its_own_rows(act, gates, xt, rows):
    g = torch.Generator(device="cuda").manual_seed(len(gates))
    f = 256
    n = max(len(gates), rows)
    gate = torch.tensor(gates, device="cuda").repeat((n + len(gates) - 1) // len(gates))[:n]
    # neighbours of the listed gate, for its rounding errors
    gate = gate[:, None] * (1 - torch.rand(n, f, generator=g, device="cuda") * 2 ** -6)
    gate = gate.to(xt)
    a, _ = _act(gate.double(), act)
    # `up` brings each value near 1, as far as its type goes, and past 2^-90
    k = torch.clamp(-torch.floor(torch.log2(a.abs().amax(1, keepdim=True))), -120, 126)
    up = ((1 + torch.rand(n, f, generator=g, device="cuda")) * 0.99).double() * torch.exp2(k) * \
        torch.where(torch.rand(n, f, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    up = up.to(xt)
    x = torch.cat([gate, up], 1)
    assert torch.all(x.isfinite())
    codes, scales = ops.gated_e4m3(x, act)
    a, t = _act(gate.double(), act)
    y = a * up.double()
    assert torch.all(y.abs().amax(1) > 2.0 ** -90)
    _check_codes(codes, scales, y, _tol(y, torch.where(t < 0, t, torch.zeros_like(t)), act))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_far_gates_next_to_ordinary_ones(act):
    """A gate out of the ordinary range changes its own element only."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(64, 512, generator=g, device="cuda")
    far = x.clone()
    far[:, 3:256:7] = torch.tensor([-1e30, -3e38, -200.0, -1000.0], device="cuda").repeat(16)[:, None]
    want, ws = ops.gated_e4m3(torch.where(far == x, x, torch.zeros_like(x)), act)
    got, gs = ops.gated_e4m3(far, act)
    assert torch.equal(gs, ws)
    # -0 and 0 are the same value
    assert torch.equal(got.float(), want.float())
    far[:, 3:256:7] = float("nan")
    got, gs = ops.gated_e4m3(far, act)
    assert torch.equal(gs, ws)
    nan = got.float().isnan()
    assert torch.all(nan[:, 3:256:7]) and int(nan.sum()) == 64 * len(range(3, 256, 7))
    assert torch.equal(got.float()[~nan], want.float()[~nan])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("rows,f", [(7, 48), (70, 400), (5000, 272), (3000, 2064)])
def test_a_far_gate_whose_up_makes_it_count(act, rows, f):
    """One value of a far gate among ordinary ones, large enough to be seen, and rows of zeros between them."""
    g = torch.Generator(device="cuda").manual_seed(f)
    gate, up = (torch.randn(rows, f, generator=g, device="cuda") for _ in range(2))
    r = torch.arange(rows, device="cuda")
    far = torch.tensor([-95.0, -92.0, -88.0, -101.0] if act == "silu" else [-10.3, -10.2, -10.1, -10.5], device="cuda")
    gate[r, (r * 17) % f] = far[r % 4]
    up[r, (r * 17) % f] = 1e38
    gate[1::3], up[1::3] = 0, 0
    gate[2::3], up[2::3] = torch.randn_like(gate[2::3]), torch.randn_like(up[2::3])
    codes, scales = ops.gated_e4m3(torch.cat([gate, up], 1), act)
    a, t = _act(gate.double(), act)
    y = a * up.double()
    _check_codes(codes, scales, y, _tol(y, torch.where(t < 0, t, torch.zeros_like(t)), act))
    assert torch.all(scales[1::3] == 1) and torch.all(codes[1::3].float() == 0)
