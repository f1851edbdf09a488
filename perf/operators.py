"""The 8-bit activation operators: what is measured, and their plain forms.

Four operators of a decoder layer whose weights are integer codes and whose
activations are E4M3 bytes with one f32 scale per row:

  norm   h = x + r, y = h * w / sqrt(mean(h^2) + eps), quantised per row
  quant  a row quantised: scale = max(max|x| / 448, 2^-126), code = e4m3(x / scale)
  mm     y = act(scale[o] * xs[s] * sum_i deq(W[o,i]) * e4m3(c[s,i]) + bias[o]) + res[s,o]
  glu    y = act(gate) * up, gate and up as in mm (bias, no residual)

run() computes them with elementary torch operations, or (own = True) through
the package's public calls.
"""
import math
import weakref

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BITS = {"i8": 8, "i4": 4, "i2": 2}


def listed():
    return [
        # one decode step's norm of the residual stream: latency only
        {"name": "norm_token", "op": "norm", "S": 1, "D": 6144, "type": "bf16", "res": True},
        # the norm over a 1571-token prompt
        {"name": "norm_prompt", "op": "norm", "S": 1571, "D": 6144, "type": "bf16", "res": True},
        # an odd hidden size, half precision, no residual, a long batch: rows that no vector load divides
        {"name": "norm_odd", "op": "norm", "S": 6007, "D": 5003, "type": "f16", "res": False},
        # a few tokens' gated activations before the down projection
        {"name": "quant_tokens", "op": "quant", "S": 4, "D": 12288, "type": "bf16"},
        # f32 activations of a long prompt, the largest pass over memory
        {"name": "quant_long", "op": "quant", "S": 8192, "D": 12288, "type": "f32"},
        # the down projection of one token, added to the residual stream
        {"name": "mm_token", "op": "mm", "fmt": "i4", "O": 6144, "I": 12288, "S": 1, "type": "bf16", "act": "none", "bias": False, "res": True},
        # a small decode batch on int8 weights, bias and activation, f32 out
        {"name": "mm_batch_i8", "op": "mm", "fmt": "i8", "O": 8192, "I": 8192, "S": 8, "type": "f32", "act": "gelu_tanh", "bias": True, "res": False},
        # odd sizes in every direction, int2 codes, a batch between decode and prompt
        {"name": "mm_odd_i2", "op": "mm", "fmt": "i2", "O": 5001, "I": 4097, "S": 77, "type": "f16", "act": "relu", "bias": True, "res": True},
        # the down projection over a 1571-token prompt
        {"name": "mm_prompt", "op": "mm", "fmt": "i4", "O": 6144, "I": 12288, "S": 1571, "type": "bf16", "act": "none", "bias": False, "res": True},
        # one token's gate and up projections
        {"name": "glu_token", "op": "glu", "fmt": "i4", "O": 12288, "I": 6144, "S": 1, "type": "bf16", "act": "silu", "bias": False},
        # a serving batch of 48 tokens on an int8 expert
        {"name": "glu_batch_i8", "op": "glu", "fmt": "i8", "O": 2048, "I": 6144, "S": 48, "type": "f32", "act": "silu", "bias": True},
        # gate and up over a 1571-token prompt: the most arithmetic
        {"name": "glu_prompt", "op": "glu", "fmt": "i4", "O": 12288, "I": 6144, "S": 1571, "type": "bf16", "act": "silu", "bias": False},
    ]


def _log_int(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "mm", "mm", "glu", "glu"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op in ("norm", "quant"):
        D = _log_int(rng, 64, 16384)
        S = _log_int(rng, 1, min(16384, 8192 * 12288 // D))
        case = {"op": op, "S": S, "D": D, "type": kind}
        if op == "norm":
            case["res"] = rng.random() < 0.6
        return case
    O, I = _log_int(rng, 64, 12288), _log_int(rng, 64, 12288)
    S = min(_log_int(rng, 1, 2048), 1571 * 6144 * 12288 // (O * I))
    case = {"op": op, "fmt": rng.choice(["i8", "i4", "i2"]), "O": O, "I": I, "S": S, "type": kind,
            "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), "bias": rng.random() < 0.5}
    if op == "mm":
        case["res"] = rng.random() < 0.5
    return case


def _rows(S, D, g):
    """Activations: normal, rows of different sizes, a few columns ten times as large as the rest."""
    x = torch.randn(S, D, generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn(S, 1, generator=g, device="cuda"))
    wide = torch.rand(D, generator=g, device="cuda") < 0.002
    return torch.where(wide, 10.0 * x, x)


def _weights(case, g):
    """Codes in the host layout [O, ceil(I * bits / 8)] and row scales that keep the products' spread near 1."""
    bits = BITS[case["fmt"]]
    O, I = case["O"], case["I"]
    codes = torch.randint(0, 256, (O, (I * bits + 7) // 8), generator=g, device="cuda", dtype=torch.uint8)
    spread = 2.0 ** bits / math.sqrt(12.0)
    scales = (0.5 + torch.rand(O, generator=g, device="cuda")) / (spread * math.sqrt(I))
    return codes, scales


def _upload(case, codes, scales):
    """The resident tensor that a user's program keeps; freed with the state."""
    import quantized_weight_quant_gb300 as q
    t = q.tensor_upload(q.FORMATS[case["fmt"]], case["O"], case["I"], codes.cpu().numpy(), scales.cpu().numpy())
    weakref.finalize(t, q.tensor_free, t.handle)
    return t


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = TYPES[case["type"]]
    S, st = case["S"], {"case": case}
    if case["op"] in ("norm", "quant"):
        D = case["D"]
        st["x"] = _rows(S, D, g).to(kind)
        if case["op"] == "norm":
            st["w"] = 0.5 + torch.rand(D, generator=g, device="cuda")
            if case["res"]:
                st["r"] = torch.randn(S, D, generator=g, device="cuda").to(kind)
        if own:
            import quantized_weight_quant_gb300 as q
            st["y"] = q.Q8Rows(S, D)
            st["h"] = torch.empty_like(st["x"])
        return st
    O, I = case["O"], case["I"]
    x = _rows(S, I, g)
    st["xs"] = torch.clamp(x.abs().amax(1) / E4M3_MAX, min=2.0 ** -126)
    st["xc"] = (x / st["xs"][:, None]).to(torch.float8_e4m3fn)
    for k in range(2 if case["op"] == "glu" else 1):
        codes, scales = _weights(case, g)
        st["codes%d" % k], st["scales%d" % k] = codes, scales
        if case["bias"]:
            st["bias%d" % k] = torch.randn(O, generator=g, device="cuda")
        if own:
            st["t%d" % k] = _upload(case, codes, scales)
    if case.get("res"):
        st["res"] = torch.randn(S, O, generator=g, device="cuda").to(kind)
    if own:
        import quantized_weight_quant_gb300 as q
        st["xq"] = q.Q8Rows(S, I)
        st["xq"].codes[:, :I].copy_(st["xc"].view(torch.uint8))
        st["xq"].scales.copy_(st["xs"])
        st["y"] = torch.empty(S, O, dtype=kind, device="cuda")
    return st


def _act(name, v):
    if name == "relu":
        return torch.clamp(v, min=0.0)
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _dequantised(codes, fmt, I):
    """f32 [O, I] values of the codes: int8 as they are, int4 code - 8 (low nibble first), int2 code - 2 (low bits first)."""
    if fmt == "i8":
        return codes.view(torch.int8).float()
    bits = BITS[fmt]
    shifts = torch.arange(0, 8, bits, device=codes.device, dtype=torch.uint8)
    fields = (codes[:, :, None] >> shifts) & (2 ** bits - 1)
    return (fields.reshape(codes.shape[0], -1)[:, :I]).float() - 2.0 ** (bits - 1)


def _product(st, k):
    case = st["case"]
    w = _dequantised(st["codes%d" % k], case["fmt"], case["I"])
    v = (st["xc"].float() @ w.t()) * st["xs"][:, None] * st["scales%d" % k]
    return v + st["bias%d" % k] if case["bias"] else v


def _quantised(y):
    s = torch.clamp(y.abs().amax(1) / E4M3_MAX, min=2.0 ** -126)
    return (y / s[:, None]).to(torch.float8_e4m3fn), s


def run(state):
    case = state["case"]
    op, S = case["op"], case["S"]
    if own:
        import quantized_weight_quant_gb300 as q
        if op == "norm":
            q.rmsnorm_q8(state["x"], state["w"], state["y"], S, case["D"], EPS, r=state.get("r"), h=state["h"] if case["res"] else None)
        elif op == "quant":
            q.quantize_q8(state["x"], state["y"], S, case["D"])
        elif op == "mm":
            q.matmul_q8(state["t0"], state["xq"], state["y"], S, bias=state.get("bias0"), act=q.ACTS[case["act"]], res=state.get("res"))
        else:
            q.glu_q8(state["t0"], state["t1"], state["xq"], state["y"], S, act=q.ACTS[case["act"]], bias_g=state.get("bias0"), bias_u=state.get("bias1"))
        if op in ("mm", "glu"):
            return state["y"]
        out = {"codes": state["y"].values(), "scales": state["y"].scales}
        if case.get("res"):
            out["h"] = state["h"]
        return out
    kind = TYPES[case["type"]]
    if op == "norm":
        h = state["x"].float()
        if case["res"]:
            h = h + state["r"].float()
        codes, s = _quantised(h * state["w"] / torch.sqrt((h * h).mean(1, keepdim=True) + EPS))
        out = {"codes": codes, "scales": s}
        if case["res"]:
            out["h"] = h.to(kind)
        return out
    if op == "quant":
        codes, s = _quantised(state["x"].float())
        return {"codes": codes, "scales": s}
    if op == "mm":
        y = _act(case["act"], _product(state, 0))
        return (y + state["res"].float() if case["res"] else y).to(kind)
    return (_act(case["act"], _product(state, 0)) * _product(state, 1)).to(kind)


def work(case):
    S, size = case["S"], TYPES[case["type"]].itemsize
    if case["op"] in ("norm", "quant"):
        D = case["D"]
        read = S * D * size * (2 if case.get("res") else 1) + (4 * D if case["op"] == "norm" else 0)
        write = S * D + 4 * S + (S * D * size if case.get("res") else 0)
        return {"bytes": read + write, "flops": S * D * (6 if case["op"] == "norm" else 3)}
    O, I, n = case["O"], case["I"], 2 if case["op"] == "glu" else 1
    weights = n * (O * ((I * BITS[case["fmt"]] + 7) // 8) + 4 * O * (2 if case["bias"] else 1))
    rows = S * I + 4 * S + S * O * size * (2 if case.get("res") else 1)
    return {"bytes": weights + rows, "flops": 2 * n * S * O * I}


# ---- the definitions in 64 bits, apart from the plain forms above

def _e4m3_64(v):
    """The E4M3 value nearest to v (ties to even): steps of 2^(e - 3), e the exponent, at least -6."""
    e = torch.clamp(torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** -30))), min=-6.0)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=v.device), e - 3.0)
    return torch.clamp(torch.round(v / step) * step, -E4M3_MAX, E4M3_MAX)


def _quant_64(y):
    s = torch.maximum(y.abs().max(dim=1).values / E4M3_MAX, torch.tensor(2.0 ** -126, dtype=torch.float64, device=y.device))
    return {"codes": _e4m3_64(y / s.unsqueeze(1)), "scales": s}


def _weight_64(codes, fmt, I):
    c = codes.to(torch.int64)
    if fmt == "i8":
        return torch.where(c > 127, c - 256, c).double()
    if fmt == "i4":
        return torch.stack((c % 16, c // 16), dim=2).flatten(1)[:, :I].double() - 8.0
    return torch.stack((c % 4, c // 4 % 4, c // 16 % 4, c // 64), dim=2).flatten(1)[:, :I].double() - 2.0


def _act_64(name, v):
    if name == "relu":
        return torch.maximum(v, torch.zeros_like(v))
    if name == "silu":
        return v * torch.special.expit(v)
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        return v * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def exact(case, seed):
    if case["op"] in ("mm", "glu") and case["S"] * case["O"] * case["I"] > 4e11:
        return None
    st = prepare(case, seed)
    if case["op"] == "quant":
        return _quant_64(st["x"].double())
    if case["op"] == "norm":
        h = st["x"].double()
        if case["res"]:
            h = h + st["r"].double()
        out = _quant_64(h * st["w"].double() / torch.sqrt(h.square().sum(1, keepdim=True) / case["D"] + EPS))
        if case["res"]:
            out["h"] = h
        return out
    x = st["xc"].float().double() * st["xs"].double().unsqueeze(1)
    v = []
    for k in range(2 if case["op"] == "glu" else 1):
        w = _weight_64(st["codes%d" % k], case["fmt"], case["I"]) * st["scales%d" % k].double().unsqueeze(1)
        y = torch.matmul(x, w.transpose(0, 1))
        v.append(y + st["bias%d" % k].double() if case["bias"] else y)
    y = _act_64(case["act"], v[0])
    if case["op"] == "glu":
        return y * v[1]
    return y + st["res"].double() if case["res"] else y
