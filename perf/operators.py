"""Cases of the E4M3 block-scaled operators (vla_flow_matching_denoise_b200.ops).

Four operators that together make the linears of a transformer layer whose
weights and activations are E4M3 codes with fp32 scales per block of 128: the
backbone that fills the action expert's prefix cache, or any decoder next to
it.

  norm   h = x + residual, y = h (mean(h^2) + eps)^-1/2 (gain + offset),
         y as E4M3 codes with one scale per row and 128 columns
  gated  u = act(gate) * up (or u = x), as E4M3 codes with the same scales
  gemm   out = (codes_a s_a) (codes_w s_w)^T + bias, s_a per row and 128
         inputs, s_w per 128 outputs and 128 inputs
  rope   rotate-half RoPE with a position axis per frequency over the q and k
         heads of a fused q|k|v row, split into q, k and v

`own` False computes them with elementary torch operations; `own` True makes
the library's calls.
"""
import numpy as np
import torch

own = False

FP8 = torch.float8_e4m3fn
TINY = 2.0 ** -100          # smallest group maximum a scale is made from


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of one request: latency only
        dict(name="norm_token", op="norm", m=1, d=1024, xt="bf16", ht="bf16", resid=True, offset=0.0),
        # 64 chunks of 50 action tokens, fp32 residual stream, bf16 branch
        dict(name="norm_chunks_f32", op="norm", m=3200, d=1024, xt="bf16", ht="f32", resid=True, offset=1.0),
        # 64 prefixes of 256 tokens at a backbone width of 2048
        dict(name="norm_prefixes", op="norm", m=16384, d=2048, xt="bf16", ht="bf16", resid=True, offset=0.0),
        # SwiGLU of one action chunk
        dict(name="gated_chunk", op="gated", m=50, f=4096, xt="bf16", act="silu"),
        # GELU-gated feed-forward of 64 prefixes
        dict(name="gated_prefixes", op="gated", m=16384, f=4096, xt="bf16", act="gelu_tanh"),
        # q|k|v projection of one token: a stream of the weights
        dict(name="gemm_token", op="gemm", m=1, n=2560, k=1024, ot="bf16", bias=True),
        # gate|up projection of one action chunk
        dict(name="gemm_chunk", op="gemm", m=50, n=8192, k=1024, ot="bf16", bias=False),
        # three requests of odd lengths packed together, a narrow ragged head
        dict(name="gemm_ragged", op="gemm", m=777, n=1003, k=2064, ot="bf16", bias=True),
        # down projection of 64 chunks into an fp32 residual stream
        dict(name="gemm_down_f32", op="gemm", m=3200, n=1024, k=4096, ot="f32", bias=False),
        # gate|up projection of 64 prefixes: the tensor cores
        dict(name="gemm_prefixes", op="gemm", m=16384, n=8192, k=2048, ot="bf16", bias=False),
        # one request's prefix and chunk: three camera views and text, axes (t, h, w)
        dict(name="rope_request", op="rope", m=306, nq=16, nkv=2, hd=128, xt="bf16", sections="16,24,24",
             ladder="shared", interleaved=False, far=4096),
        # 64 prefixes of video, interleaved axes, far time positions
        dict(name="rope_prefixes", op="rope", m=16384, nq=16, nkv=2, hd=128, xt="bf16", sections="24,20,20",
             ladder="shared", interleaved=True, far=1000000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "gated", "gemm", "gemm", "rope"])
    xt = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        d = 16 * _log(rng, 4, 512)
        m = _log(rng, 1, min(16384, 16384 * 2048 // (d * (2 if xt == "f32" else 1))))
        resid = rng.random() < 0.75
        ht = rng.choice(["bf16", "f32"]) if resid and xt == "bf16" and m * d < 2 ** 23 else xt
        return dict(op=op, m=m, d=d, xt=xt, ht=ht, resid=resid, offset=rng.choice([0.0, 1.0]))
    if op == "gated":
        f = 16 * _log(rng, 1, 1024)
        m = _log(rng, 1, min(16384, 16384 * 4096 // (f * (2 if xt == "f32" else 1))))
        return dict(op=op, m=m, f=f, xt=xt, act=rng.choice(["silu", "gelu_tanh", "none"]))
    if op == "gemm":
        n, k = _log(rng, 16, 8192), 16 * _log(rng, 1, 1024)
        m = _log(rng, 1, max(1, min(16384, 16384 * 8192 * 1024 // (n * k))))
        return dict(op=op, m=m, n=n, k=k, ot=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    hd = rng.choice([64, 72, 80, 96, 128, 256])
    rot = rng.choice([hd, hd, hd // 2])
    axes = rng.randint(1, 4)
    cuts = sorted(rng.sample(range(1, rot // 2), axes - 1))
    sections = [b - a for a, b in zip([0] + cuts, cuts + [rot // 2])]
    nkv = rng.choice([1, 2, 4, 8])
    nq = nkv * rng.choice([0, 1, 2, 7, 8])
    m = _log(rng, 1, min(16384, 16384 * 20 * 128 // ((nq + 2 * nkv) * hd * (2 if xt == "f32" else 1))))
    ladder = rng.choice(["shared", "per_axis"])
    return dict(op="rope", m=m, nq=nq, nkv=nkv, hd=hd, xt=xt, sections=",".join(map(str, sections)), ladder=ladder,
                interleaved=ladder == "shared" and rng.random() < 0.5, far=rng.choice([300, 4096, 1000000]))


# ----------------------------------------------------------------- inputs
def _type(t):
    return torch.bfloat16 if t == "bf16" else torch.float32


def _groups(k):
    return (k + 127) // 128


def _stream_rows(g, m, d, dtype):
    """Rows of a residual stream: normal values, rows of different size, a few wide channels."""
    x = torch.randn(m, d, generator=g, device="cuda")
    x *= torch.exp(torch.randn(m, 1, generator=g, device="cuda") * 0.5)
    x *= torch.where(torch.rand(d, generator=g, device="cuda") < 0.004, 20.0, 1.0)
    return x.to(dtype)


def _codes(x, rows):
    """E4M3 codes and scales of an fp32 matrix in blocks of `rows` x 128."""
    n, k = x.shape
    pad = torch.zeros(_groups(n) * 128 if rows == 128 else n, _groups(k) * 128, device=x.device)
    pad[:n, :k] = x
    b = pad.view(-1, rows, _groups(k), 128)
    amax = b.abs().amax((1, 3), keepdim=True)
    s = torch.where(amax > 0, amax.clamp_min(TINY) / 448.0, torch.ones_like(amax))
    q = (b / s).clamp(-448, 448).to(FP8).view(pad.shape)[:n, :k].contiguous()
    return q, s[:, 0, :, 0].contiguous()


def _axis_of_pair(sections, interleaved):
    """Axis of each rotated pair: consecutive sections, or the axes in turn until each has its share."""
    if not interleaved:
        return [a for a, s in enumerate(sections) for _ in range(s)]
    left, out = list(sections), []
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _frequencies(case):
    """(axis, base-10000 frequency) of each rotated pair; per_axis restarts the ladder in each section."""
    sections = [int(s) for s in case["sections"].split(",")]
    axis = _axis_of_pair(sections, case["interleaved"])
    if case["ladder"] == "per_axis":
        freq = [10000.0 ** (-i / s) for s in sections for i in range(s)]
    else:
        freq = [10000.0 ** (-j / len(axis)) for j in range(len(axis))]
    return axis, freq


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, m = case["op"], case["m"]
    s = {"case": case}
    if op == "norm":
        s["x"] = _stream_rows(g, m, case["d"], _type(case["xt"]))
        s["residual"] = _stream_rows(g, m, case["d"], _type(case["ht"])) if case["resid"] else None
        gain = torch.randn(case["d"], generator=g, device="cuda") * 0.2 + (1.0 - case["offset"])
        s["gain"] = gain.to(torch.bfloat16)
    elif op == "gated":
        wide = case["f"] * (1 if case["act"] == "none" else 2)
        s["x"] = (torch.randn(m, wide, generator=g, device="cuda") * 2.0).to(_type(case["xt"]))
    elif op == "gemm":
        n, k = case["n"], case["k"]
        s["a"], s["sa"] = _codes(_stream_rows(g, m, k, torch.float32), 1)
        s["w"], s["sw"] = _codes(torch.randn(n, k, generator=g, device="cuda") * 0.02, 128)
        s["bias"] = (torch.randn(n, generator=g, device="cuda") * 0.1).to(torch.bfloat16) if case["bias"] else None
    else:
        hd = case["hd"]
        wide = (case["nq"] + 2 * case["nkv"]) * hd
        s["x"] = torch.randn(m, wide, generator=g, device="cuda").to(_type(case["xt"]))
        sections = [int(v) for v in case["sections"].split(",")]
        near = torch.randint(0, 64, (len(sections), m), generator=g, device="cuda", dtype=torch.int32)
        near[0] = torch.randint(0, case["far"], (m,), generator=g, device="cuda", dtype=torch.int32)
        s["pos"] = near
        axis, freq = _frequencies(case)
        s["axis"] = torch.tensor(axis, device="cuda")
        s["freq"] = torch.tensor(freq, device="cuda", dtype=torch.float64)
        # the table of pairs, as a program keeps it from its configuration
        s["pairs"] = (np.array(axis, dtype=np.uint8), np.array(freq, dtype=np.float64))
    return s


# ----------------------------------------------------------------- one pass
def _quantize_plain(y):
    m, k = y.shape
    pad = torch.zeros(m, _groups(k) * 128, device=y.device)
    pad[:, :k] = y
    b = pad.view(m, -1, 128)
    amax = b.abs().amax(2)
    some = amax > 0
    a = amax.clamp_min(TINY)
    scale = torch.where(some, a / 448.0, torch.ones_like(a))
    r = torch.where(some, 448.0 / a, torch.ones_like(a))
    codes = (b * r[:, :, None]).clamp(-448, 448).to(FP8).view(m, -1)[:, :k].contiguous()
    return codes, scale


def _norm_plain(s):
    c = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)
    codes, scale = _quantize_plain(h * rstd * (s["gain"].float() + c["offset"]))
    out = {"codes": codes, "scales": scale}
    if s["residual"] is not None:
        out["h"] = h.to(s["residual"].dtype)
    return out


def _gated_plain(s):
    act, x = s["case"]["act"], s["x"].float()
    if act != "none":
        f = s["case"]["f"]
        gate, up = x[:, :f], x[:, f:]
        if act == "silu":
            x = gate / (1.0 + torch.exp(-gate)) * up
        else:
            z = 0.7978845608028654 * (gate + 0.044715 * gate * gate * gate)
            x = 0.5 * gate * (1.0 + torch.tanh(z)) * up
    codes, scale = _quantize_plain(x)
    return {"codes": codes, "scales": scale}


def _gemm_plain(s):
    n, k = s["w"].shape
    sa = s["sa"].repeat_interleave(128, 1)[:, :k]
    sw = s["sw"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    out = (s["a"].float() * sa) @ (s["w"].float() * sw).t()
    if s["bias"] is not None:
        out = out + s["bias"].float()
    return {"out": out.to(_type(s["case"]["ot"]))}


def _rope_plain(s):
    c = s["case"]
    m, hd, nq, nkv = c["m"], c["hd"], c["nq"], c["nkv"]
    half = s["freq"].numel()
    angle = s["pos"].double()[s["axis"]].t() * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x = s["x"].view(m, nq + 2 * nkv, hd)
    r = x[:, :nq + nkv].float()
    lo, hi = r[:, :, :half], r[:, :, half:2 * half]
    r = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin, r[:, :, 2 * half:]], 2).to(x.dtype)
    return {"q": r[:, :nq].contiguous(), "k": r[:, nq:].contiguous(), "v": x[:, nq + nkv:].contiguous()}


def _run_own(s):
    from vla_flow_matching_denoise_b200 import ops
    c = s["case"]
    if c["op"] == "norm":
        h, codes, scales = ops.add_rmsnorm_e4m3(s["x"], s["gain"], residual=s["residual"], eps=1e-6,
                                                gain_offset=c["offset"])
        out = {"codes": codes, "scales": scales}
        if s["residual"] is not None:
            out["h"] = h
        return out
    if c["op"] == "gated":
        codes, scales = ops.gated_e4m3(s["x"], c["act"])
        return {"codes": codes, "scales": scales}
    if c["op"] == "gemm":
        return {"out": ops.gemm_e4m3(s["a"], s["sa"], s["w"], s["sw"], bias=s["bias"], out_dtype=_type(c["ot"]))}
    q, k, v = ops.rope_axes(s["x"], s["pos"], s["pairs"], c["nq"], c["nkv"], c["hd"])
    return {"q": q, "k": k, "v": v}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "gated": _gated_plain, "gemm": _gemm_plain, "rope": _rope_plain}[
        state["case"]["op"]](state)


# ----------------------------------------------------------------- what a pass has to move and compute
def work(case):
    op, m = case["op"], case["m"]
    size = 4 if case.get("xt") == "f32" else 2
    if op == "norm":
        d, hs = case["d"], 4 if case["ht"] == "f32" else 2
        stream = 2 * hs if case["resid"] else 0
        return {"bytes": m * d * (size + stream + 1) + m * _groups(d) * 4 + 2 * d, "flops": 8 * m * d}
    if op == "gated":
        f, wide = case["f"], case["f"] * (1 if case["act"] == "none" else 2)
        return {"bytes": m * wide * size + m * f + m * _groups(f) * 4, "flops": 10 * m * f}
    if op == "gemm":
        n, k = case["n"], case["k"]
        out = 4 if case["ot"] == "f32" else 2
        return {"bytes": m * k + n * k + 4 * _groups(k) * (m + _groups(n)) + m * n * out + (2 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    wide = (case["nq"] + 2 * case["nkv"]) * case["hd"]
    axes = case["sections"].count(",") + 1
    return {"bytes": 2 * m * wide * size + 4 * axes * m, "flops": 3 * m * wide}


# ----------------------------------------------------------------- the definitions in 64 bits
def _e4m3_64(v):
    """Nearest E4M3 value (ties to even, saturating) of float64 values, as float64."""
    _, e = torch.frexp(v)                           # |v| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 3)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def _groups_64(y):
    values, scales = torch.empty_like(y), []
    for c in range(0, y.shape[1], 128):
        part = y[:, c:c + 128]
        top = part.abs().max(1).values
        s = torch.where(top == 0, torch.ones_like(top), torch.clamp(top, min=TINY) / 448.0)
        values[:, c:c + 128] = _e4m3_64(part / s[:, None])
        scales.append(s)
    return values, torch.stack(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["d"] + 1e-6) * (s["gain"].double() + case["offset"])
        codes, scales = _groups_64(y)
        out = {"codes": codes, "scales": scales}
        if s["residual"] is not None:
            out["h"] = h
        return out
    if op == "gated":
        x = s["x"].double()
        if case["act"] != "none":
            gate, up = x.chunk(2, 1)
            if case["act"] == "silu":
                x = gate * torch.sigmoid(gate) * up
            else:
                x = torch.nn.functional.gelu(gate, approximate="tanh") * up
        codes, scales = _groups_64(x)
        return {"codes": codes, "scales": scales}
    if op == "gemm":
        k, n = case["k"], case["n"]
        total = torch.zeros(case["m"], n, dtype=torch.float64, device="cuda")
        block = torch.arange(n, device="cuda") // 128
        for g in range(_groups(k)):
            a, w = (s[t][:, 128 * g:128 * g + 128].double() for t in ("a", "w"))
            total += (a @ w.t()) * s["sa"][:, g:g + 1].double() * s["sw"][block, g].double()
        return {"out": total if s["bias"] is None else total + s["bias"].double()}
    m, hd, nq, nkv = case["m"], case["hd"], case["nq"], case["nkv"]
    axis, freq = _frequencies(case)
    x = s["x"].double().view(m, nq + 2 * nkv, hd)
    turned = x[:, :nq + nkv].clone()
    half = len(axis)
    for j in range(half):
        z = torch.polar(torch.ones(m, dtype=torch.float64, device="cuda"), s["pos"][axis[j]].double() * freq[j])
        w = torch.complex(x[:, :nq + nkv, j], x[:, :nq + nkv, j + half]) * z[:, None]
        turned[:, :, j], turned[:, :, j + half] = w.real, w.imag
    return {"q": turned[:, :nq], "k": turned[:, nq:], "v": x[:, nq + nkv:]}
