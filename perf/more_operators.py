"""Measured cases of the feed-forward block's products: the gated projection (gate and up projections, activation and
product) with its gradients, the quantisation of activation rows to 8-bit integers, and the 8-bit integer matrix
product with a scale for each token and each channel.

Where ``own`` is false, ``run`` computes each operator in elementary torch operations in 32 bits, rounded once at the
end; where it is true, it makes the library calls of ``gemv_moe_expert_gb300.binding``.  ``exact`` computes the same
from the definitions in 64 bits.

Kinds of case
  gated        x [m, k], weights [n, k] twice -> h = act(x Wg^T) * (x Wu^T); with ``save`` also both projections
  gradient     d_h and the saved projections -> d_x, d_w_gate, d_w_up
  quantize     rows of x -> codes in -127..127 and a scale for each row
  gemm_i8      codes [m, k] and [n, k] with their scales -> y [m, n]
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step: both weight matrices are read for one row
        {"name": "gated 1 token", "kind": "gated", "m": 1, "n": 11008, "k": 4096, "dtype": "bf16", "act": "silu",
         "save": False, "pad": 0},
        # a few tokens through an odd layer whose rows start anywhere
        {"name": "gated ragged", "kind": "gated", "m": 7, "n": 1537, "k": 1001, "dtype": "f16", "act": "gelu",
         "save": False, "pad": 3},
        # a decode batch: more tokens than a dot product per token pays for, fewer than fill a tile
        {"name": "gated batch", "kind": "gated", "m": 48, "n": 11008, "k": 4096, "dtype": "f16", "act": "silu",
         "save": False, "pad": 0},
        # a prompt through a large layer
        {"name": "gated prompt", "kind": "gated", "m": 4096, "n": 11008, "k": 4096, "dtype": "bf16", "act": "silu",
         "save": False, "pad": 0},
        # the forward pass of a training step, projections kept for the gradient, rows padded
        {"name": "gated training", "kind": "gated", "m": 2048, "n": 5504, "k": 2048, "dtype": "bf16",
         "act": "gelu_tanh", "save": True, "pad": 8},
        # the backward pass of such a step
        {"name": "gradient training", "kind": "gradient", "m": 4096, "n": 5504, "k": 2048, "dtype": "bf16",
         "act": "silu", "pad": 0},
        # the backward pass of a small layer in f32
        {"name": "gradient f32", "kind": "gradient", "m": 512, "n": 1408, "k": 2048, "dtype": "f32", "act": "relu",
         "pad": 0},
        # a decode batch's activations to 8 bits: nothing but latency
        {"name": "quantize 4 tokens", "kind": "quantize", "m": 4, "k": 4096, "dtype": "f16", "pad": 0},
        # a prompt's activations to 8 bits
        {"name": "quantize prompt", "kind": "quantize", "m": 8192, "k": 11008, "dtype": "bf16", "pad": 0},
        # one decode token through a dense 8-bit layer
        {"name": "gemm_i8 1 token", "kind": "gemm_i8", "m": 1, "n": 11008, "k": 4096, "dtype": "f16", "pad": 0},
        # an odd batch through an odd layer, rows that start anywhere, results in f32
        {"name": "gemm_i8 ragged", "kind": "gemm_i8", "m": 147, "n": 1537, "k": 2050, "dtype": "f32", "pad": 3},
        # a prompt through a large 8-bit layer
        {"name": "gemm_i8 prompt", "kind": "gemm_i8", "m": 4096, "n": 11008, "k": 4096, "dtype": "bf16", "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = [max(work(c)[key] for c in listed()) for key in ("bytes", "flops")]
    while True:
        kind = rng.choice(["gated", "gated", "gradient", "quantize", "gemm_i8", "gemm_i8"])
        c = {"kind": kind, "m": _log(rng, 1, 8192), "k": _log(rng, 64, 11008),
             "dtype": rng.choice(["bf16", "f16", "bf16", "f16", "f32"]), "pad": rng.choice([0, 0, 8, 3])}
        if kind != "quantize":
            c["n"] = _log(rng, 64, 11008)
        if kind in ("gated", "gradient"):
            c["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
        if kind == "gated":
            c["save"] = rng.random() < 0.3
        # even sizes are what programs mostly have; one in three stays as drawn
        if rng.random() < 0.67:
            for key in ("n", "k"):
                if key in c:
                    c[key] = max(64, c[key] // 64 * 64)
        w = work(c)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return c


def work(case):
    c, size = case, SIZE[case["dtype"]]
    m, k = c["m"], c["k"]
    if c["kind"] == "quantize":
        return {"bytes": m * k * (size + 1) + 4 * m, "flops": 2 * m * k}
    n = c["n"]
    if c["kind"] == "gated":
        return {"bytes": (m * k + 2 * n * k + (3 if c["save"] else 1) * m * n) * size, "flops": 4 * m * n * k}
    if c["kind"] == "gradient":
        # x, both weights, both projections and d_h read; d_x and both weights' gradients written
        return {"bytes": (2 * m * k + 4 * n * k + 3 * m * n) * size, "flops": 8 * m * n * k}
    return {"bytes": (m + n) * k + m * n * size + 4 * (m + n), "flops": 2 * m * n * k}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rows(g, m, n, pad, dtype, scale=1.0):
    """[m, n] normal values in rows n + pad elements apart."""
    x = torch.randn(m, n + pad, generator=g, device="cuda", dtype=torch.float32)
    return (x * scale).to(dtype)[:, :n]


def _codes(g, m, k, pad):
    """[m, k] 8-bit codes of normal values, in rows k + pad bytes apart."""
    x = torch.randn(m, k + pad, generator=g, device="cuda", dtype=torch.float32)
    return (40 * x).round().clamp(-127, 127).to(torch.int8)[:, :k]


def prepare(case, seed):
    c, dt, pad = case, DTYPES[case["dtype"]], case["pad"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    m, k, kind = c["m"], c["k"], c["kind"]
    size = SIZE[c["dtype"]]
    new = lambda *shape, dtype=dt: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if kind == "quantize":
        x = _rows(g, m, k, pad, dt)
        # tokens differ in size, single channels stand out, and a padded batch has rows of zeros
        x *= torch.exp(0.5 * torch.randn(m, 1, generator=g, device="cuda")).to(dt)
        x[:, :: 509] *= 8
        if m > 16:
            x[9::64] = 0
        s["x"] = x
        s["q"], s["scale"] = new(m, k + pad, dtype=torch.int8)[:, :k], new(m, dtype=torch.float32)
        return s
    n = c["n"]
    if kind == "gemm_i8":
        s["a"], s["b"] = _codes(g, m, k, pad), _codes(g, n, k, pad)
        s["scale_a"] = 0.02 * torch.exp(0.5 * torch.randn(m, generator=g, device="cuda"))
        s["scale_b"] = 0.02 / k ** 0.5 * (0.5 + torch.rand(n, generator=g, device="cuda"))
        s["y"] = new(m, n + pad)[:, :n]
        # a program sizes the workspace once: both operands in 16 bits hold every size here
        s["scratch"] = new(2 * (m + n) * (k + 64) + 4096, dtype=torch.uint8)
        return s
    s["x"] = _rows(g, m, k, pad, dt)
    s["w_gate"], s["w_up"] = (_rows(g, n, k, pad, dt, k ** -0.5) for _ in range(2))
    if kind == "gated":
        s["h"] = new(m, n + pad)[:, :n]
        s["gate"], s["up"] = ((new(m, n + pad)[:, :n] for _ in range(2)) if c["save"] else (None, None))
        # room for operands whose rows are laid out again, where rows do not start on multiples of 16 bytes
        s["scratch"] = new((m + 2 * n) * (k + 64) * size + 4096, dtype=torch.uint8)
        return s
    s["gate"], s["up"], s["d_h"] = (_rows(g, m, n, pad, dt) for _ in range(3))
    s["d_x"] = new(m, k + pad)[:, :k]
    s["d_w_gate"], s["d_w_up"] = (new(n, k + pad)[:, :k] for _ in range(2))
    s["scratch"] = new((2 * m * (n + 64) + (m + 2 * n) * (k + 64)) * size + 4096, dtype=torch.uint8)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["kind"]](state)


_R2, _RPI = math.sqrt(0.5), math.sqrt(2 / math.pi)


def _act(name, g):
    """The activation and its derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        p = 0.5 * (1 + torch.erf(g * _R2))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(_RPI * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * _RPI * (1 + 3 * 0.044715 * g * g)
    return torch.clamp_min(g, 0), (g > 0).to(g.dtype)


def _plain_gated(s):
    dt = s["x"].dtype
    x = s["x"].float()
    gate, up = x @ s["w_gate"].float().T, x @ s["w_up"].float().T
    out = {"h": (_act(s["act"], gate)[0] * up).to(dt)}
    if s["save"]:
        out["gate"], out["up"] = gate.to(dt), up.to(dt)
    return out


def _plain_gradient(s):
    dt = s["x"].dtype
    x, up, d_h = s["x"].float(), s["up"].float(), s["d_h"].float()
    a, slope = _act(s["act"], s["gate"].float())
    d_gate, d_up = d_h * up * slope, d_h * a
    d_x = d_gate @ s["w_gate"].float() + d_up @ s["w_up"].float()
    return {"d_x": d_x.to(dt), "d_w_gate": (d_gate.T @ x).to(dt), "d_w_up": (d_up.T @ x).to(dt)}


def _plain_quantize(s):
    x = s["x"].float()
    scale = x.abs().amax(dim=1) / 127
    # the nearest code by the stored scale: in 64 bits, since values may lie next to the middle of two codes
    q = torch.round(x.double() / torch.where(scale > 0, scale, 1.0).double()[:, None])
    return {"q": q.to(torch.int8), "scale": scale}


def _plain_gemm_i8(s):
    # sums of such codes stay far below 2^24, so that 32 bits hold them exactly
    y = s["a"].float() @ s["b"].float().T
    return {"y": (y * s["scale_a"][:, None] * s["scale_b"]).to(s["y"].dtype)}


_plain = {"gated": _plain_gated, "gradient": _plain_gradient, "quantize": _plain_quantize, "gemm_i8": _plain_gemm_i8}


def _library():
    from gemv_moe_expert_gb300 import binding
    return binding, torch.cuda.current_stream().cuda_stream


def _gate(gb, name):
    return {"silu": gb.GATE_SILU, "gelu": gb.GATE_GELU, "gelu_tanh": gb.GATE_GELU_TANH, "relu": gb.GATE_RELU}[name]


def _own_gated(s):
    gb, stream = _library()
    ld, out = s["k"] + s["pad"], s["n"] + s["pad"]
    gb.check(gb.gbmm_gated(s["dtype"], _gate(gb, s["act"]), s["m"], s["n"], s["k"], s["x"], ld, s["w_gate"], s["w_up"],
                           ld, s["h"], out, s["gate"], s["up"], out, s["scratch"], s["scratch"].numel(), stream))
    return {name: s[name] for name in (("h", "gate", "up") if s["save"] else ("h",))}


def _own_gradient(s):
    gb, stream = _library()
    ld, wide = s["k"] + s["pad"], s["n"] + s["pad"]
    gb.check(gb.gbmm_gated_backward(s["dtype"], _gate(gb, s["act"]), s["m"], s["n"], s["k"], s["x"], ld, s["w_gate"],
                                    s["w_up"], ld, s["gate"], s["up"], wide, s["d_h"], wide, s["d_x"], ld,
                                    s["d_w_gate"], s["d_w_up"], ld, s["scratch"], s["scratch"].numel(), stream))
    return {name: s[name] for name in ("d_x", "d_w_gate", "d_w_up")}


def _own_quantize(s):
    gb, stream = _library()
    ld = s["k"] + s["pad"]
    gb.check(gb.gbmm_quantize_i8(s["dtype"], s["m"], s["k"], s["x"], ld, s["q"], ld, s["scale"], stream))
    return {"q": s["q"], "scale": s["scale"]}


def _own_gemm_i8(s):
    gb, stream = _library()
    ld = s["k"] + s["pad"]
    gb.check(gb.gbmm_gemm_i8(s["dtype"], s["m"], s["n"], s["k"], s["a"], ld, s["scale_a"], s["b"], ld, s["scale_b"],
                             s["y"], s["n"] + s["pad"], s["scratch"], s["scratch"].numel(), stream))
    return {"y": s["y"]}


_own = {"gated": _own_gated, "gradient": _own_gradient, "quantize": _own_quantize, "gemm_i8": _own_gemm_i8}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _exact_gated, "gradient": _exact_gradient, "quantize": _exact_quantize,
            "gemm_i8": _exact_gemm_i8}[s["kind"]](s)


def _exact_act(name, g):
    f = torch.nn.functional
    return {"silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"), "relu": f.relu}[name](g)


def _exact_gated(s):
    x = s["x"].double()
    gate = torch.einsum("ik,jk->ij", x, s["w_gate"].double())
    up = torch.einsum("ik,jk->ij", x, s["w_up"].double())
    out = {"h": _exact_act(s["act"], gate) * up}
    if s["save"]:
        out["gate"], out["up"] = gate, up
    return out


def _exact_gradient(s):
    """The derivative of <d_h, h> by the chain rule of torch, from the saved projections down to x and the weights."""
    gate, up = (s[name].double().requires_grad_() for name in ("gate", "up"))
    with torch.enable_grad():
        d_gate, d_up = torch.autograd.grad(_exact_act(s["act"], gate) * up, (gate, up), s["d_h"].double())
    x, w_gate, w_up = (s[name].double() for name in ("x", "w_gate", "w_up"))
    d_x = torch.einsum("ij,jk->ik", d_gate, w_gate)
    d_x += torch.einsum("ij,jk->ik", d_up, w_up)
    return {"d_x": d_x, "d_w_gate": torch.einsum("ij,ik->jk", d_gate, x), "d_w_up": torch.einsum("ij,ik->jk", d_up, x)}


def _exact_quantize(s):
    """The nearer of the two codes around x / scale, the even one in the middle."""
    x = s["x"].double()
    scale = (x.abs().max(dim=1).values.float() / 127).double()
    t = x / torch.where(scale > 0, scale, 1.0)[:, None]
    low = torch.floor(t)
    part = t - low
    up = (part > 0.5) | ((part == 0.5) & (low % 2 == 1))
    return {"q": (low + up).to(torch.int8), "scale": scale}


def _exact_gemm_i8(s):
    y = torch.einsum("ik,jk->ij", s["a"].double(), s["b"].double())
    return {"y": y * s["scale_a"].double()[:, None] * s["scale_b"].double()[None, :]}
