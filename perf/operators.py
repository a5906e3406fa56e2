"""The 8-bit integer operators: the cases they are measured on, their inputs,
their plain form and their definition in 64 bits.

An int8 matrix is a row-major array of codes with one fp32 scale for each row
(a token of the activations, an output channel of the weights).  Operators:

    quantize         x -> codes, scales -> x_hat = code * scale
    linear           y = x_hat w_hat^T
    gated            h = act(x_hat wg_hat^T) * (x_hat wu_hat^T)
    gated_backward   dh -> dx, d_gate, d_up (the codes and scales are constants)
    linear_backward  dy -> dx = dy w_hat
"""
import math

import torch

own = False

# act: silu(a) = a sigmoid(a), gelu_tanh(a) = a sigmoid(2 u), u = c (a + 0.044715 a^3), c = sqrt(2 / pi)
GELU_C = math.sqrt(2.0 / math.pi)


def listed():
    return [
        # one token's hidden state on its way into a projection: latency
        dict(name="quantize_token", op="quantize", rows=1, cols=4096, dtype="bf16"),
        # a prefill chunk's fp32 activations, one row and one column short of the round size
        dict(name="quantize_chunk", op="quantize", rows=2047, cols=14335, dtype="f32"),
        # one token through an attention projection: latency and the weights' bytes
        dict(name="linear_token", op="linear", m=1, n=4096, k=4096, out="f32"),
        # a decode batch through a large gate projection: the weights' bytes
        dict(name="linear_batch", op="linear", m=16, n=28672, k=8192, out="bf16"),
        # prefill through a down projection: the integer tensor cores
        dict(name="linear_prefill", op="linear", m=2048, n=4096, k=14336, out="f32"),
        # one token through gate and up: the weights' bytes
        dict(name="gated_token", op="gated", m=1, f=14336, k=4096, act="silu", out="bf16"),
        # prefill through gate and up
        dict(name="gated_prefill", op="gated", m=2048, f=14336, k=4096, act="silu", out="bf16"),
        # odd sizes in every direction, the other activation, fp32 out
        dict(name="gated_odd", op="gated", m=200, f=1371, k=2003, act="gelu_tanh", out="f32"),
        # a training or calibration step's chunk through the whole block and back
        dict(name="gated_backward_step", op="gated_backward", m=512, f=14336, k=4096, act="silu"),
        dict(name="gated_backward_odd", op="gated_backward", m=61, f=1371, k=1001, act="gelu_tanh"),
        # gradients through a down projection: a long chunk and a short one through a larger layer
        dict(name="linear_backward_chunk", op="linear_backward", m=2048, n=4096, k=14336),
        dict(name="linear_backward_short", op="linear_backward", m=16, n=8192, k=28672),
    ]


LIMIT_FLOPS = 2.0 * 2048 * 4096 * 14336   # the largest listed cases' products
LIMIT_BYTES = 28672 * 8192


def _log_size(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:   # half of the sizes are round ones
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "linear", "gated", "gated_backward", "linear_backward"])
    while True:
        if op == "quantize":
            case = dict(op=op, rows=_log_size(rng, 1, 4096), cols=_log_size(rng, 16, 28672),
                        dtype=rng.choice(["bf16", "f32"]))
            if case["rows"] * case["cols"] <= 2047 * 14335:
                return case
            continue
        m, k = _log_size(rng, 1, 4096), _log_size(rng, 64, 28672)
        n = _log_size(rng, 64, 28672)
        passes = {"linear": 1, "gated": 2, "gated_backward": 4, "linear_backward": 1}[op]
        if 2.0 * m * n * k * passes > LIMIT_FLOPS or n * k * min(passes, 2) > LIMIT_BYTES:
            continue
        if op == "linear":
            return dict(op=op, m=m, n=n, k=k, out=rng.choice(["f32", "bf16"]))
        if op == "gated":
            return dict(op=op, m=m, f=n, k=k, act=rng.choice(["silu", "gelu_tanh"]), out=rng.choice(["f32", "bf16"]))
        if op == "gated_backward":
            return dict(op=op, m=m, f=n, k=k, act=rng.choice(["silu", "gelu_tanh"]))
        return dict(op=op, m=m, n=n, k=k)


def _size(t):
    return {"f32": 4, "bf16": 2}[t]


def work(case):
    op = case["op"]
    if op == "quantize":   # read, codes and scales written, read back as x_hat
        rc = case["rows"] * case["cols"]
        return {"bytes": rc * (2 * _size(case["dtype"]) + 1) + 4 * case["rows"], "flops": 4 * rc}
    m, k = case["m"], case["k"]
    if op == "linear":
        n = case["n"]
        return {"bytes": m * k + n * k + 4 * (m + n) + m * n * _size(case["out"]), "flops": 2 * m * n * k}
    if op == "linear_backward":
        n = case["n"]
        return {"bytes": n * k + 4 * n + 2 * m * n + 2 * m * k, "flops": 2 * m * n * k}
    f = case["f"]
    if op == "gated":
        return {"bytes": m * k + 2 * f * k + 4 * (m + 2 * f) + m * f * _size(case["out"]), "flops": 4 * m * f * k}
    return {"bytes": m * k + 2 * f * k + 4 * (m + 2 * f) + 6 * m * f + 2 * m * k, "flops": 8 * m * f * k}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, rows, cols, std, outliers, factor):
    """N(0, std) with a few columns `factor` times larger, as activations and weights of a model have."""
    x = torch.randn(rows, cols, generator=gen, device="cuda") * std
    pick = torch.randint(0, cols, (outliers,), generator=gen, device="cuda").unique()
    x[:, pick] *= factor
    return x


def _int8(x):
    """An int8 matrix of x: codes in rows of a pitch that is a multiple of 16 bytes, one scale a row."""
    rows, cols = x.shape
    scales = x.abs().amax(dim=1).clamp_min(1e-30) / 127.0
    codes = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :cols]
    codes.copy_(torch.round(x / scales[:, None]).clamp_(-127, 127))
    return codes, scales


_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "quantize":
        return {"x": _normal(gen, case["rows"], case["cols"], 1.0, 3, 20.0).to(_TYPES[case["dtype"]])}
    m, k = case["m"], case["k"]
    inp = {}
    if op != "linear_backward":
        inp["x"] = _int8(_normal(gen, m, k, 1.0, 3, 20.0))
    if op in ("linear", "linear_backward"):
        inp["w"] = _int8(_normal(gen, case["n"], k, 0.02, 4, 10.0))
    else:
        inp["w_gate"] = _int8(_normal(gen, case["f"], k, 0.02, 4, 10.0))
        inp["w_up"] = _int8(_normal(gen, case["f"], k, 0.02, 4, 10.0))
    if op == "linear_backward":
        inp["dy"] = (torch.randn(m, case["n"], generator=gen, device="cuda") * 0.01).to(torch.bfloat16)
    if op == "gated_backward":
        inp["dh"] = (torch.randn(m, case["f"], generator=gen, device="cuda") * 0.01).to(torch.bfloat16)
    return inp


def prepare(case, seed):
    inp = _inputs(case, seed)
    state = {"case": dict(case), "inp": inp}
    if not own:
        return state
    # what a user's program keeps: the matrices' handles, the outputs and a zeroed workspace
    import block_wise_mixed_b200 as mpq
    op = case["op"]
    mats = {n: mpq.i8_matrix(*v) for n, v in inp.items() if isinstance(v, tuple)}

    def new(rows, cols, t):
        return torch.empty(rows, cols, dtype=_TYPES[t], device="cuda")

    if op == "quantize":
        state["q"] = mpq.i8_empty(case["rows"], case["cols"], "cuda")
        state["out"] = new(case["rows"], case["cols"], case["dtype"])
        return state
    m, k = case["m"], case["k"]
    if op == "linear":
        size = mpq.i8_linear_workspace_size(m, case["n"], k)
        state["out"] = new(m, case["n"], case["out"])
    elif op == "gated":
        size = mpq.i8_gated_workspace_size(m, case["f"], k)
        state["out"] = new(m, case["f"], case["out"])
    elif op == "gated_backward":
        size = mpq.i8_gated_backward_workspace_size(m, case["f"], k)
        state["out"] = (new(m, k, "bf16"), new(m, case["f"], "bf16"), new(m, case["f"], "bf16"))
    else:
        size = mpq.i8_linear_backward_workspace_size(m, case["n"], k)
        state["out"] = new(m, k, "bf16")
    state["mats"] = mats
    state["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _gate(act, a):
    """sigmoid's argument t(a) and its derivative (act(a) = a sigmoid(t))."""
    if act == "silu":
        return a, torch.ones_like(a)
    return 2.0 * GELU_C * (a + 0.044715 * a * a * a), 2.0 * GELU_C * (1.0 + 3.0 * 0.044715 * a * a)


def _plain(state):
    case, inp = state["case"], state["inp"]
    op = case["op"]
    if op == "quantize":
        x = inp["x"].double()   # 64 bits: quotients next to a rounding border
        amax = x.abs().amax(dim=1)
        s = torch.clamp(amax / 127.0, min=2.0 ** -126).float()
        s = torch.where(amax == 0, torch.ones_like(s), s)
        finite = torch.isfinite(amax)
        s = torch.where(finite, s, torch.full_like(s, math.nan))
        q = torch.round(x / s.double()[:, None]).clamp_(-127, 127)
        q = torch.where(finite[:, None], q, torch.zeros_like(q))
        return (q.float() * s[:, None]).to(_TYPES[case["dtype"]]), s

    def product(x, w):
        return (x[0].float() @ w[0].float().t()) * w[1] * x[1][:, None]

    if op == "linear":
        return product(inp["x"], inp["w"]).to(_TYPES[case["out"]])
    if op == "linear_backward":
        w = inp["w"][0].float() * inp["w"][1][:, None]
        return (inp["dy"].float() @ w).to(torch.bfloat16)
    a = product(inp["x"], inp["w_gate"])
    b = product(inp["x"], inp["w_up"])
    t, dt = _gate(case["act"], a)
    sig = torch.sigmoid(t)
    if op == "gated":
        return (a * sig * b).to(_TYPES[case["out"]])
    dh = inp["dh"].float()
    d_gate = dh * b * (sig + a * sig * torch.sigmoid(-t) * dt)
    d_up = dh * (a * sig)
    wg = inp["w_gate"][0].float() * inp["w_gate"][1][:, None]
    wu = inp["w_up"][0].float() * inp["w_up"][1][:, None]
    dx = d_gate @ wg + d_up @ wu
    return dx.to(torch.bfloat16), d_gate.to(torch.bfloat16), d_up.to(torch.bfloat16)


def run(state):
    if not own:
        return _plain(state)
    import block_wise_mixed_b200 as mpq
    case, inp = state["case"], state["inp"]
    op = case["op"]
    if op == "quantize":
        q = mpq.i8_quantize(inp["x"], out=state["q"])
        return mpq.i8_dequantize(q, out=state["out"]), q.scales
    mats, ws = state["mats"], state["ws"]
    if op == "linear":
        return mpq.i8_linear(mats["x"], mats["w"], out=state["out"], ws=ws)
    if op == "gated":
        return mpq.i8_gated(mats["x"], mats["w_gate"], mats["w_up"], act=case["act"], out=state["out"], ws=ws)
    if op == "linear_backward":
        return mpq.i8_linear_backward(mats["w"], inp["dy"], out=state["out"], ws=ws)
    dx, d_gate, d_up = state["out"]
    return mpq.i8_gated_backward(mats["x"], mats["w_gate"], mats["w_up"], inp["dh"], act=case["act"], dx=dx,
                                 d_gate=d_gate, d_up=d_up, ws=ws)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    inp = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        x = inp["x"].to(torch.float64)
        top = x.abs().max(dim=1).values
        s32 = (top / 127).to(torch.float32)            # the scale is stored in 32 bits
        s32[s32 < 2.0 ** -126] = 2.0 ** -126
        s32[top == 0] = 1.0
        s = s32.to(torch.float64)
        return torch.round(x / s.unsqueeze(1)) * s.unsqueeze(1), s
    hat = {n: v[0].double() * v[1].double().unsqueeze(1) for n, v in inp.items() if isinstance(v, tuple)}
    if op == "linear":
        return torch.einsum("mk,nk->mn", hat["x"], hat["w"])
    if op == "linear_backward":
        return torch.einsum("mn,nk->mk", inp["dy"].double(), hat["w"])
    a = torch.einsum("mk,fk->mf", hat["x"], hat["w_gate"])
    b = torch.einsum("mk,fk->mf", hat["x"], hat["w_up"])
    if case["act"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-a))
        g, dg = a * sig, sig * (1.0 + a * (1.0 - sig))
    else:
        th = torch.tanh(GELU_C * (a + 0.044715 * a ** 3))
        g = 0.5 * a * (1.0 + th)
        dg = 0.5 * (1.0 + th) + 0.5 * a * (1.0 - th * th) * GELU_C * (1.0 + 0.134145 * a * a)
    if op == "gated":
        return g * b
    dh = inp["dh"].double()
    d_gate, d_up = dh * b * dg, dh * g
    dx = torch.einsum("mf,fk->mk", d_gate, hat["w_gate"]) + torch.einsum("mf,fk->mk", d_up, hat["w_up"])
    return dx, d_gate, d_up
