"""The gated feed-forward block and its compressed forms: the cases they are measured on, in plain torch operations
and through the library's own entry points.

Operators (bf16 unless said otherwise, [out][in] weights without biases):
  glu       h = act(x W_gᵀ) ⊙ (x W_uᵀ)                       act: exact GeLU or SiLU
  glu_bwd   from dh: dx, dW_g, dW_u (and h where asked for), with g and u recomputed from x
  ckpt      x to 8-bit codes with a power of two for each 32 channels, and back
  step8     glu, the checkpoint of its input, and glu_bwd reading that checkpoint
  w4        y = x Ŵᵀ,  Ŵ = s (q − 8) with 4-bit q and one bf16 scale s for each `group` inputs
  w4_glu    h = act(x Ŵ_gᵀ) ⊙ (x Ŵ_uᵀ)
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one token through a small layer: the shortest call, all latency
        dict(name="glu one token, small layer", op="glu", n=1, d=256, h=768, act="gelu"),
        # a decode batch of 16 through a 4096-wide layer's MLP (width 3 D): the weights' bytes
        dict(name="glu decode 16", op="glu", n=16, d=4096, h=12288, act="gelu"),
        # the decode workload's batch of 256: bytes and products weigh about the same
        dict(name="glu decode 256", op="glu", n=256, d=4096, h=12288, act="gelu"),
        # prefill of 8 sequences of 2048 tokens, D = 2048
        dict(name="glu prefill", op="glu", n=16384, d=2048, h=6144, act="gelu"),
        # a packed ragged batch through odd widths
        dict(name="glu_bwd ragged", op="glu_bwd", n=1999, d=1032, h=2888, act="silu", want_h=True),
        # a training step of 4 sequences of 4096 tokens, D = 4096
        dict(name="glu_bwd large", op="glu_bwd", n=16384, d=4096, h=12288, act="gelu", want_h=False),
        # a float32 activation of a few hundred tokens, with a last group that is not whole
        dict(name="ckpt float32, ragged", op="ckpt", n=300, c=264, dtype="float32"),
        # the long-sequence workload's activation, 32768 tokens of 4096 channels
        dict(name="ckpt large", op="ckpt", n=32768, c=4096, dtype="bfloat16"),
        # a layer's whole pass in training with the input kept in 8 bits
        dict(name="step8", op="step8", n=4096, d=2048, h=6144, act="gelu"),
        # one token through a square projection
        dict(name="w4 one token", op="w4", m=1, k=4096, rows=4096, group=128),
        # a few sequences, an odd number of outputs, smaller groups
        dict(name="w4 five tokens, ragged", op="w4", m=5, k=5632, rows=4104, group=64),
        # eight sequences through the gated MLP of a 4096-wide layer
        dict(name="w4_glu eight tokens", op="w4_glu", m=8, k=4096, rows=12288, group=128, act="gelu"),
    ]


def _log(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def _wide(rng, low, high):
    return 8 * _log(rng, low // 8, high // 8)


def draw(rng):
    op = rng.choice(["glu", "glu", "glu_bwd", "glu_bwd", "ckpt", "step8", "w4", "w4_glu"])
    act = rng.choice(["gelu", "silu"])
    if op == "glu":
        return dict(op=op, n=_log(rng, 1, 32768), d=_wide(rng, 64, 4096), h=_wide(rng, 64, 12288), act=act)
    if op == "glu_bwd":
        return dict(op=op, n=_log(rng, 1, 16384), d=_wide(rng, 64, 4096), h=_wide(rng, 64, 12288), act=act,
                    want_h=rng.random() < 0.5)
    if op == "ckpt":
        return dict(op=op, n=_log(rng, 1, 32768), c=_wide(rng, 8, 4096), dtype=rng.choice(["bfloat16", "float32"]))
    if op == "step8":
        return dict(op=op, n=_log(rng, 1, 8192), d=_wide(rng, 64, 4096), h=_wide(rng, 64, 12288), act=act)
    group = rng.choice([32, 64, 128])
    case = dict(op=op, m=_log(rng, 1, 64), k=group * _log(rng, 1, 8192 // group), rows=_wide(rng, 64, 16384), group=group)
    return dict(case, act=act) if op == "w4_glu" else case


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * std


def _quantized(g, rows, k, group):
    """Codes [rows][k/2] (even inputs in the low four bits) and scales [rows][k/group] of a LeCun-normal matrix."""
    w = _normal(g, rows, k // group, group, std=1.0 / math.sqrt(k))
    scale = (w.abs().amax(2) / 7.0).to(torch.bfloat16)
    q = (torch.round(w / scale.float().unsqueeze(2)).clamp(-8, 7) + 8).to(torch.uint8).view(rows, k // 2, 2)
    return (q[:, :, 0] | (q[:, :, 1] << 4)).contiguous(), scale.contiguous()


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("glu", "glu_bwd", "step8"):
        n, d, h = case["n"], case["d"], case["h"]
        s["x"] = _normal(g, n, d).to(torch.bfloat16)
        s["w_gate"] = _normal(g, h, d, std=1.0 / math.sqrt(d)).to(torch.bfloat16)
        s["w_up"] = _normal(g, h, d, std=1.0 / math.sqrt(d)).to(torch.bfloat16)
        if op != "glu":
            s["dh"] = _normal(g, n, h, std=0.05).to(torch.bfloat16)
    elif op == "ckpt":
        # activations: unit scale, and one channel in fifty much larger, as residual streams have
        size = 1.0 + 30.0 * (torch.rand(case["c"], generator=g, device=DEV) < 0.02).float()
        s["x"] = (_normal(g, case["n"], case["c"]) * size).to(getattr(torch, case["dtype"]))
    else:
        s["x"] = _normal(g, case["m"], case["k"]).to(torch.bfloat16)
        s["w"] = _quantized(g, case["rows"], case["k"], case["group"])
        if op == "w4_glu":
            s["w2"] = _quantized(g, case["rows"], case["k"], case["group"])
    return s


# ---- the plain forms: 32 bits throughout, rounded once at the end ----------------------------------------------------


def _act(g, act):
    return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5))) if act == "gelu" else g * torch.sigmoid(g)


def _act_slope(g, act):
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    r = torch.sigmoid(g)
    return r * (1.0 + g * (1.0 - r))


def _plain_glu(x, w_gate, w_up, act):
    return _act(x @ w_gate.float().t(), act) * (x @ w_up.float().t())


def _plain_glu_bwd(x, w_gate, w_up, dh, act, want_h):
    wg, wu, dh = w_gate.float(), w_up.float(), dh.float()
    g, u = x @ wg.t(), x @ wu.t()
    a = _act(g, act)
    dg, du = dh * u * _act_slope(g, act), dh * a
    out = dict(dx=(dg @ wg + du @ wu), dw_gate=dg.t() @ x, dw_up=du.t() @ x)
    if want_h:
        out["h"] = a * u
    return {k: v.to(torch.bfloat16) for k, v in out.items()}


def _plain_ckpt(x):
    """x as the 8-bit checkpoint holds it, in 32 bits: for each 32 channels the smallest e ≥ −127 with
    |round(x / 2^e)| ≤ 127, and x̂ = round(x / 2^e) 2^e."""
    n, c = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -c % 32)).view(n, -1, 32)
    amax = x.abs().amax(2, keepdim=True)
    e = (amax.view(torch.int32) >> 23) - 127 - 6
    e = torch.where(amax * _power(-e) >= 127.5, e + 1, e).clamp(min=-127)
    return (torch.round(x * _power(-e)) * _power(e)).view(n, -1)[:, :c]


def _power(e):
    """2^e, from its bits (torch.ldexp multiplies by a power that is not exact on every device); −127 ≤ e ≤ 127, and
    for a group of zeros, whose exponent is lower still, a power that its zeros do not change."""
    return torch.where(e > -127, (e + 127).clamp(max=254) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _plain_weight(codes, scale, group):
    rows, half = codes.shape
    q = torch.stack([codes & 15, codes >> 4], 2).view(rows, -1, group).float() - 8.0
    return (q * scale.float().unsqueeze(2)).view(rows, 2 * half)


def run(state):
    op = state["op"]
    if own:
        return _run_own(state, op)
    x = state["x"]
    if op == "glu":
        return _plain_glu(x.float(), state["w_gate"], state["w_up"], state["act"]).to(torch.bfloat16)
    if op == "glu_bwd":
        return _plain_glu_bwd(x.float(), state["w_gate"], state["w_up"], state["dh"], state["act"], state["want_h"])
    if op == "ckpt":
        return _plain_ckpt(x).to(x.dtype)
    if op == "step8":
        h = _plain_glu(x.float(), state["w_gate"], state["w_up"], state["act"]).to(torch.bfloat16)
        return dict(_plain_glu_bwd(_plain_ckpt(x), state["w_gate"], state["w_up"], state["dh"], state["act"], False), h=h)
    w = _plain_weight(*state["w"], state["group"])
    if op == "w4":
        return (x.float() @ w.t()).to(torch.bfloat16)
    return _plain_glu(x.float(), w, _plain_weight(*state["w2"], state["group"]), state["act"]).to(torch.bfloat16)


def _run_own(state, op):
    from gated_linear_rnn_conv1d_b200 import rglru

    x = state["x"]
    if op == "glu":
        return rglru.glu_forward(state["w_gate"], state["w_up"], x, activation=state["act"])
    if op == "glu_bwd":
        r = rglru.glu_backward(state["w_gate"], state["w_up"], x, state["dh"], activation=state["act"],
                               want_h=state["want_h"])
        out = dict(dx=r["dx"], dw_gate=r["dW_gate"], dw_up=r["dW_up"])
        return dict(out, h=r["h"]) if state["want_h"] else out
    if op == "ckpt":
        return rglru.act8_unpack(rglru.act8_pack(x))
    if op == "step8":
        h = rglru.glu_forward(state["w_gate"], state["w_up"], x, activation=state["act"])
        kept = rglru.act8_pack(x)
        r = rglru.glu_backward(state["w_gate"], state["w_up"], kept, state["dh"], activation=state["act"])
        return dict(dx=r["dx"], dw_gate=r["dW_gate"], dw_up=r["dW_up"], h=h)
    w = rglru.W4Weight(*state["w"], state["group"])
    if op == "w4":
        return rglru.w4_linear(w, x)
    return rglru.w4_glu(w, rglru.W4Weight(*state["w2"], state["group"]), x, activation=state["act"])


# ---- what a pass cannot do without ------------------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op in ("glu", "glu_bwd", "step8"):
        n, d, h = case["n"], case["d"], case["h"]
        forward = dict(bytes=2 * (n * d + 2 * h * d + n * h), flops=4 * n * d * h)
        # x, both weights and dh in; dx, both weight gradients (and h) out; g, u, dx, dW_g and dW_u
        wide = n * h * (2 if case.get("want_h") else 1)
        backward = dict(bytes=2 * (2 * n * d + 4 * h * d + wide), flops=12 * n * d * h)
        if op != "step8":
            return forward if op == "glu" else backward
        # the forward writes the checkpoint, the backward reads it in the place of x
        kept = n * d + n * -(-d // 32)
        return dict(bytes=forward["bytes"] + backward["bytes"] + 2 * kept - 2 * n * d,
                    flops=forward["flops"] + backward["flops"])
    if op == "ckpt":
        n, c = case["n"], case["c"]
        size = 2 if case["dtype"] == "bfloat16" else 4
        return dict(bytes=2 * n * (size * c + c + -(-c // 32)), flops=4 * n * c)
    m, k, rows = case["m"], case["k"], case["rows"] * (2 if op == "w4_glu" else 1)
    return dict(bytes=rows * k // 2 + 2 * rows * (k // case["group"]) + 2 * m * (k + case["rows"]), flops=2 * m * k * rows)


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------


def _exact_act(g, act):
    """act(g) and its derivative: g Φ(g) by the complementary error function, or g σ(g)."""
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
    r = 1 / (1 + torch.exp(-g))
    return g * r, r + g * r * (1 - r)


def _exact_ckpt(x):
    n, c = x.shape
    out = torch.zeros(n, -(-c // 32) * 32, dtype=torch.float64, device=x.device)
    out[:, :c] = x.double()
    groups = out.view(n, -1, 32)
    top = groups.abs().amax(2, keepdim=True)
    mantissa, exponent = torch.frexp(top)  # top = mantissa 2^exponent, 0.5 ≤ mantissa < 1
    exponent = exponent.double()
    e = torch.where(mantissa * 128 >= 127.5, exponent - 6, exponent - 7).clamp(min=-127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    step = torch.tensor([2.0**k for k in range(-127, 128)], dtype=torch.float64, device=x.device)[(e + 127).long()]
    return (torch.round(groups / step) * step).view(n, -1)[:, :c]


def _exact_weight(codes, scale, group):
    rows, half = codes.shape
    q = torch.empty(rows, 2 * half, dtype=torch.float64, device=codes.device)
    q[:, 0::2] = codes.remainder(16).double()
    q[:, 1::2] = codes.div(16, rounding_mode="floor").double()
    return (q - 8) * scale.double().repeat_interleave(group, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, x = case["op"], s["x"]
    if op == "ckpt":
        return _exact_ckpt(x)
    if op in ("w4", "w4_glu"):
        a = x.double() @ _exact_weight(*s["w"], case["group"]).T
        if op == "w4":
            return a
        return _exact_act(a, case["act"])[0] * (x.double() @ _exact_weight(*s["w2"], case["group"]).T)
    wg, wu = s["w_gate"].double(), s["w_up"].double()
    h = None
    if op != "glu_bwd":
        h = _exact_act(x.double() @ wg.T, case["act"])[0] * (x.double() @ wu.T)
        if op == "glu":
            return h
    x = _exact_ckpt(x) if op == "step8" else x.double()
    g, u = x @ wg.T, x @ wu.T
    a, slope = _exact_act(g, case["act"])
    if op == "glu_bwd" and case["want_h"]:
        h = a * u
    du = s["dh"].double() * a
    dg = s["dh"].double() * u * slope
    del a, slope, g, u
    out = dict(dx=torch.addmm(du @ wu, dg, wg), dw_gate=dg.T @ x, dw_up=du.T @ x)
    return out if h is None else dict(out, h=h)
