"""Measured cases of the mixture-of-experts layer around the expert products: the top-k softmax router, the tokens'
way into expert order and back (with gradients), and matrix-vector products with 4-bit weights and group scales.

Where ``own`` is false, ``run`` computes each operator in elementary torch operations in 32 bits, rounded once at the
end; where it is true, it makes the library calls of ``gemv_moe_expert_gb300.binding``.  ``exact`` computes the same
from the definitions in 64 bits.

Kinds of case
  route        logits [m, experts] -> ids, weights; with ``grad`` also d_weights -> d_logits
  dispatch     ids -> offsets, order, position; x [m, n] -> the rows in expert order
  combine      rows in expert order, weights -> y [m, n]
  gradient     d_y -> d_rows, d_weights (combine), d_dispatched rows -> d_x (dispatch)
  gemv_q4      y[m, n] = x W^T, W 4-bit [n, k] with a scale (and a zero point) for each group of columns
  experts_q4   the same, W of the expert that each routed row names
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
        # one token of a decode step through a small router: nothing but latency
        {"name": "route 1 token", "kind": "route", "m": 1, "experts": 64, "top_k": 8, "dtype": "f32", "selected": True,
         "bias": False, "pad": 0, "grad": False},
        # a prompt's router in bf16, ids balanced by a selection bias: 16-bit logits tie often
        {"name": "route prompt", "kind": "route", "m": 4096, "experts": 128, "top_k": 8, "dtype": "bf16",
         "selected": True, "bias": True, "pad": 0, "grad": False},
        # a training batch's router, forward and backward, softmax over every expert
        {"name": "route training", "kind": "route", "m": 65536, "experts": 128, "top_k": 8, "dtype": "f32",
         "selected": False, "bias": False, "pad": 0, "grad": True},
        # a few tokens of a decode batch put in expert order
        {"name": "dispatch 4 tokens", "kind": "dispatch", "m": 4, "experts": 64, "top_k": 8, "n": 2048, "dtype": "f16",
         "drop": 0.0, "pad": 0},
        # a prompt put in expert order, popular experts first
        {"name": "dispatch prompt", "kind": "dispatch", "m": 4096, "experts": 128, "top_k": 8, "n": 4096,
         "dtype": "bf16", "drop": 0.0, "pad": 0},
        # an odd batch back in token order: odd row length, padded rows, some rows without an expert
        {"name": "combine ragged", "kind": "combine", "m": 147, "experts": 11, "top_k": 3, "n": 1537, "dtype": "f16",
         "drop": 0.1, "pad": 7},
        # a prompt's expert outputs (f32, as the expert-ID matmul writes them) back in token order
        {"name": "combine prompt", "kind": "combine", "m": 4096, "experts": 128, "top_k": 8, "n": 4096, "dtype": "f32",
         "drop": 0.02, "pad": 0},
        # a training batch's gradients through combine and dispatch
        {"name": "gradient training", "kind": "gradient", "m": 8192, "experts": 64, "top_k": 8, "n": 2048,
         "dtype": "bf16", "drop": 0.02, "pad": 0},
        # one decode token through a dense 4-bit layer
        {"name": "gemv_q4 1 token", "kind": "gemv_q4", "m": 1, "n": 11008, "k": 4096, "group": 128, "dtype": "f16",
         "zeros": False, "tight": False},
        # three tokens, ragged sizes, zero points, a last group that is not full
        {"name": "gemv_q4 ragged", "kind": "gemv_q4", "m": 3, "n": 4097, "k": 2050, "group": 64, "dtype": "bf16",
         "zeros": True, "tight": False},
        # a decode step of four tokens through 4-bit experts, f32 activations as the expert-ID matmul takes them
        {"name": "experts_q4 4 tokens", "kind": "experts_q4", "m": 4, "experts": 64, "top_k": 8, "n": 1408, "k": 2048,
         "group": 128, "dtype": "f32", "zeros": False, "tight": False},
        # a decode batch through 4-bit experts, small groups with zero points
        {"name": "experts_q4 batch", "kind": "experts_q4", "m": 16, "experts": 128, "top_k": 8, "n": 1536, "k": 4096,
         "group": 32, "dtype": "bf16", "zeros": True, "tight": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = [max(work(c)[key] for c in listed()) for key in ("bytes", "flops")]
    while True:
        kind = rng.choice(["route", "dispatch", "combine", "gradient", "gemv_q4", "experts_q4"])
        dtype = rng.choice(["f32", "f16", "bf16"])
        if kind == "route":
            experts = _log(rng, 4, 512)
            c = {"kind": kind, "m": _log(rng, 1, 65536), "experts": experts, "top_k": min(experts, _log(rng, 1, 16)),
                 "dtype": dtype, "selected": rng.random() < 0.5, "bias": rng.random() < 0.5,
                 "pad": rng.choice([0, 0, 3, 8]), "grad": rng.random() < 0.5}
        elif kind in ("dispatch", "combine", "gradient"):
            experts = _log(rng, 4, 512)
            c = {"kind": kind, "m": _log(rng, 1, 32768), "experts": experts, "top_k": min(experts, _log(rng, 1, 16)),
                 "n": _log(rng, 64, 8192), "dtype": dtype, "drop": rng.choice([0.0, 0.02, 0.3]),
                 "pad": rng.choice([0, 0, 3, 8])}
        elif kind == "gemv_q4":
            c = {"kind": kind, "m": _log(rng, 1, 16), "n": _log(rng, 256, 16384), "k": _log(rng, 256, 12288),
                 "group": rng.choice([32, 64, 128]), "dtype": dtype, "zeros": rng.random() < 0.5,
                 "tight": rng.random() < 0.25}
        else:
            experts = _log(rng, 8, 128)
            c = {"kind": kind, "m": _log(rng, 1, 16), "experts": experts, "top_k": min(experts, _log(rng, 1, 8)),
                 "n": _log(rng, 128, 2048), "k": _log(rng, 256, 4096), "group": rng.choice([32, 64, 128]),
                 "dtype": dtype, "zeros": rng.random() < 0.5, "tight": rng.random() < 0.25}
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
    kind = c["kind"]
    if kind == "route":
        grid, slots = c["m"] * c["experts"], c["m"] * c["top_k"]
        nbytes = grid * size + slots * 8 + (4 * c["experts"] if c["bias"] else 0)
        if c["grad"]:
            nbytes += grid * size + slots * 4
        return {"bytes": nbytes, "flops": grid * (8 if c["grad"] else 4)}
    if kind == "dispatch":
        rows = c["m"] * c["top_k"]
        return {"bytes": rows * 12 + 4 * (c["experts"] + 1) + (c["m"] + rows) * c["n"] * size, "flops": 0}
    if kind == "combine":
        rows = c["m"] * c["top_k"]
        live = rows * (1 - c["drop"])
        return {"bytes": rows * 8 + (c["m"] + live) * c["n"] * size, "flops": 2 * live * c["n"]}
    if kind == "gradient":
        rows = c["m"] * c["top_k"]
        live = rows * (1 - c["drop"])
        # ys and the dispatched rows' gradient read, d_ys written; d_y read, d_x written; weights, position, d_weights
        return {"bytes": rows * 12 + (2 * c["m"] + 2 * live + rows) * c["n"] * size, "flops": 4 * live * c["n"]}
    groups = -(-c["k"] // c["group"])
    matrix = c["n"] * ((c["k"] + 1) // 2) + c["n"] * groups * (2 + (1 if c["zeros"] else 0))
    if kind == "gemv_q4":
        return {"bytes": matrix + c["m"] * (c["k"] + c["n"]) * size, "flops": 2 * c["m"] * c["n"] * c["k"]}
    rows = c["m"] * c["top_k"]
    distinct = c["experts"] * (1 - (1 - c["top_k"] / c["experts"]) ** c["m"])  # ids drawn evenly
    return {"bytes": distinct * matrix + (c["m"] * c["k"] + rows * c["n"]) * size + rows * 4,
            "flops": 2 * rows * c["n"] * c["k"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(g, m, n, pad, dtype):
    """[m, n] normal values in rows n + pad elements apart."""
    return _randn(g, m, n + pad).to(dtype)[:, :n]


def _pick(g, m, experts, top_k, skew):
    """top_k distinct experts for each token, expert e drawn with weight (e + 1)^-skew."""
    u = torch.rand(m, experts, generator=g, device="cuda").clamp_min_(1e-12)
    rank = torch.arange(1, experts + 1, device="cuda", dtype=torch.float32)
    return torch.topk(-skew * rank.log() - (-u.log()).log(), top_k, dim=1).indices.to(torch.int32)


def _order(ids, experts):
    """offsets, order and position of the routed rows, as a program has them from the forward pass."""
    key = ids.reshape(-1).clamp_max(experts)
    ranked, order = torch.sort(key, stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device="cuda")
    edges = torch.arange(experts + 1, device="cuda", dtype=ranked.dtype)
    return torch.searchsorted(ranked, edges).to(torch.int32), order.to(torch.int32), position.to(torch.int32)


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    m, kind = c["m"], c["kind"]
    new = lambda *shape, dtype=dt: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if kind == "route":
        s["logits"] = _rows(g, m, c["experts"], c["pad"], dt)
        s["select_bias"] = 0.1 * _randn(g, c["experts"]) if c["bias"] else None
        s["ids"], s["weights"] = new(m, c["top_k"], dtype=torch.int32), new(m, c["top_k"], dtype=torch.float32)
        if c["grad"]:
            s["d_weights"], s["d_logits"] = _randn(g, m, c["top_k"]), new(m, c["experts"])
        return s
    if kind in ("gemv_q4", "experts_q4"):
        n, k, groups = c["n"], c["k"], -(-c["k"] // c["group"])
        stack = (c["experts"], n) if kind == "experts_q4" else (n,)
        # packed rows start 16 bytes apart, or (tight) wherever the row before them ends
        nbytes = (k + 1) // 2
        pitch = nbytes if c["tight"] else -(-nbytes // 16) * 16
        s["q"] = torch.randint(0, 256, (*stack, pitch), generator=g, device="cuda", dtype=torch.uint8)[..., :nbytes]
        s["scales"] = (0.02 / 4 * (0.5 + torch.rand(*stack, groups, generator=g, device="cuda"))).to(torch.float16)
        s["zeros"] = (torch.randint(5, 12, (*stack, groups), generator=g, device="cuda", dtype=torch.uint8)
                      if c["zeros"] else None)
        s["x"] = _randn(g, m, k).to(dt)
        if kind == "gemv_q4":
            s["out"] = new(m, n)
        else:
            s["ids"], s["out"] = _pick(g, m, c["experts"], c["top_k"], 0.0), new(m, c["top_k"], n)
        return s
    n, experts, top_k, pad = c["n"], c["experts"], c["top_k"], c["pad"]
    rows = m * top_k
    ids = _pick(g, m, experts, top_k, 1.1)
    if c["drop"]:  # rows that a capacity limit or padding left without an expert
        ids = torch.where(torch.rand(m, top_k, generator=g, device="cuda") < c["drop"], experts, ids).to(torch.int32)
    s["ids"] = ids
    if kind == "dispatch":
        s["x"], s["xs"] = _rows(g, m, n, pad, dt), new(rows, n + pad)[:, :n]
        for name, count in (("offsets", experts + 1), ("order", rows), ("position", rows)):
            s[name] = new(count, dtype=torch.int32)
        # a program sizes the sort's workspace once, for its largest batch: 8 bytes a routed row hold every size here
        s["scratch"] = new(8 * rows + 65536, dtype=torch.uint8)
        return s
    s["offsets"], s["order"], s["position"] = _order(ids, experts)
    s["weights"] = torch.softmax(_randn(g, m, top_k), dim=1) * (ids < experts)
    s["ys"] = _rows(g, rows, n, pad, dt)
    if kind == "combine":
        s["y"] = new(m, n + pad)[:, :n]
        return s
    s["d_y"], s["d_xs"] = _rows(g, m, n, pad, dt), _rows(g, rows, n, pad, dt)
    s["d_ys"], s["d_x"] = new(rows, n + pad)[:, :n], new(m, n + pad)[:, :n]
    s["d_weights"] = new(m, top_k, dtype=torch.float32)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["kind"]](state)


def _plain_route(s):
    x, experts, top_k = s["logits"].float(), s["experts"], s["top_k"]
    score = x if s["select_bias"] is None else x + s["select_bias"]
    live = score > -math.inf
    score, index = torch.sort(torch.where(live, score, -math.inf), dim=1, descending=True, stable=True)
    index, chosen = index[:, :top_k], score[:, :top_k] > -math.inf
    p = torch.where(live, x, -math.inf)
    if s["selected"]:
        p = torch.where(chosen, p.gather(1, index), -math.inf)
    top = p.amax(dim=1, keepdim=True)
    p = torch.exp(p - torch.where(top > -math.inf, top, 0.0))
    p = p / p.sum(dim=1, keepdim=True).clamp_min(1e-30)
    weights = torch.where(chosen, p if s["selected"] else p.gather(1, index), 0.0)
    out = {"ids": torch.where(chosen, index, experts).to(torch.int32), "weights": weights}
    if s["grad"]:
        d = torch.where(chosen, s["d_weights"], 0.0)
        dot = (weights * d).sum(dim=1, keepdim=True)
        if s["selected"]:
            d_logits = torch.zeros_like(x).scatter(1, index, weights * (d - dot))
        else:
            d_logits = p * (torch.zeros_like(x).scatter(1, index, d) - dot)
        out["d_logits"] = d_logits.to(s["logits"].dtype)
    return out


def _plain_dispatch(s):
    offsets, order, position = _order(s["ids"], s["experts"])
    valid = torch.arange(order.numel(), device=order.device) < offsets[-1]
    xs = torch.where(valid[:, None], s["x"][order // s["top_k"]], 0.0)
    return {"offsets": offsets, "order": order, "position": position, "xs": xs}


def _plain_combine(s):
    rows = s["ys"][s["position"]].float().view(s["m"], s["top_k"], -1)
    valid = (s["position"] < s["offsets"][-1]).view(s["m"], s["top_k"], 1)
    y = torch.where(valid, s["weights"][:, :, None] * rows, 0.0).sum(dim=1)
    return {"y": y.to(s["ys"].dtype)}


def _plain_gradient(s):
    m, top_k, dt = s["m"], s["top_k"], s["ys"].dtype
    pos = s["position"]
    valid = (pos < s["offsets"][-1]).view(m, top_k, 1)
    d_y = s["d_y"].float()[:, None, :]
    d_weights = torch.where(valid[..., 0], (s["ys"][pos].float().view(m, top_k, -1) * d_y).sum(dim=2), 0.0)
    d_rows = torch.where(valid, s["weights"][:, :, None] * d_y, 0.0).to(dt)
    d_ys = torch.empty_like(s["d_xs"])
    d_ys[pos] = d_rows.view(m * top_k, -1)
    d_x = torch.where(valid, s["d_xs"][pos].float().view(m, top_k, -1), 0.0).sum(dim=1).to(dt)
    return {"d_ys": d_ys, "d_weights": d_weights, "d_x": d_x}


def _weights(q, scales, zeros, k, group):
    """[.., n, k] f32 from packed nibbles [.., n, (k + 1) / 2] and one scale (and zero point) for each group."""
    w = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2)[..., :k].float()
    at = torch.arange(k, device=q.device) // group
    w -= 8.0 if zeros is None else zeros[..., at].float()
    w *= scales[..., at].float()
    return w


def _plain_gemv_q4(s):
    w = _weights(s["q"], s["scales"], s["zeros"], s["k"], s["group"])
    return {"y": (s["x"].float() @ w.T).to(s["x"].dtype)}


def _plain_experts_q4(s):
    ids = s["ids"].reshape(-1)
    zeros = None if s["zeros"] is None else s["zeros"][ids]
    w = _weights(s["q"][ids], s["scales"][ids], zeros, s["k"], s["group"])
    x = s["x"].float().repeat_interleave(s["top_k"], dim=0)
    y = torch.bmm(w, x[:, :, None])
    return {"y": y.view(s["m"], s["top_k"], -1).to(s["x"].dtype)}


_plain = {"route": _plain_route, "dispatch": _plain_dispatch, "combine": _plain_combine, "gradient": _plain_gradient,
          "gemv_q4": _plain_gemv_q4, "experts_q4": _plain_experts_q4}


def _library():
    from gemv_moe_expert_gb300 import binding
    return binding, torch.cuda.current_stream().cuda_stream


def _own_route(s):
    gb, stream = _library()
    mode = gb.SOFTMAX_SELECTED if s["selected"] else gb.SOFTMAX_ALL
    gb.check(gb.gbmm_moe_route(s["dtype"], s["m"], s["experts"], s["top_k"], mode, s["logits"], s["logits"].stride(0),
                               s["select_bias"], s["ids"], s["weights"], stream))
    if not s["grad"]:
        return {"ids": s["ids"], "weights": s["weights"]}
    gb.check(gb.gbmm_moe_route_backward(s["dtype"], s["m"], s["experts"], s["top_k"], mode, s["logits"],
                                        s["logits"].stride(0), s["select_bias"], s["ids"], s["weights"],
                                        s["d_weights"], s["d_logits"], s["experts"], stream))
    return {"ids": s["ids"], "weights": s["weights"], "d_logits": s["d_logits"]}


def _own_dispatch(s):
    gb, stream = _library()
    gb.check(gb.gbmm_moe_sort(s["m"], s["top_k"], s["experts"], s["ids"], s["offsets"], s["order"], s["position"],
                              s["scratch"], s["scratch"].numel(), stream))
    gb.check(gb.gbmm_moe_dispatch(s["dtype"], s["m"], s["top_k"], s["experts"], s["n"], s["x"], s["n"] + s["pad"],
                                  s["position"], s["offsets"], s["xs"], s["n"] + s["pad"], stream))
    return {name: s[name] for name in ("offsets", "order", "position", "xs")}


def _own_combine(s):
    gb, stream = _library()
    gb.check(gb.gbmm_moe_combine(s["dtype"], s["m"], s["top_k"], s["experts"], s["n"], s["ys"], s["n"] + s["pad"],
                                 s["weights"], s["position"], s["offsets"], s["y"], s["n"] + s["pad"], stream))
    return {"y": s["y"]}


def _own_gradient(s):
    gb, stream = _library()
    ld = s["n"] + s["pad"]
    gb.check(gb.gbmm_moe_combine_backward(s["dtype"], s["m"], s["top_k"], s["experts"], s["n"], s["ys"], ld,
                                          s["weights"], s["position"], s["offsets"], s["d_y"], ld, s["d_ys"], ld,
                                          s["d_weights"], stream))
    gb.check(gb.gbmm_moe_dispatch_backward(s["dtype"], s["m"], s["top_k"], s["experts"], s["n"], s["d_xs"], ld,
                                           s["position"], s["offsets"], s["d_x"], ld, stream))
    return {"d_ys": s["d_ys"], "d_weights": s["d_weights"], "d_x": s["d_x"]}


def _own_gemv_q4(s):
    gb, stream = _library()
    gb.check(gb.gbmm_gemv_q4(s["dtype"], s["m"], s["n"], s["k"], s["group"], s["q"], s["q"].stride(-2), s["scales"],
                             "f16", s["zeros"], s["x"], s["k"], s["out"], s["n"], stream))
    return {"y": s["out"]}


def _own_experts_q4(s):
    gb, stream = _library()
    gb.check(gb.gbmm_matmul_id_q4(s["dtype"], s["m"], s["n"], s["k"], s["top_k"], s["experts"],
                                  gb.INPUT_SHARED_PER_TOKEN, s["group"], s["q"], s["q"].stride(-2), s["q"].stride(0),
                                  s["scales"], "f16", s["zeros"], s["x"], s["ids"], s["out"], stream))
    return {"y": s["out"]}


_own = {"route": _own_route, "dispatch": _own_dispatch, "combine": _own_combine, "gradient": _own_gradient,
        "gemv_q4": _own_gemv_q4, "experts_q4": _own_experts_q4}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "dispatch": _exact_dispatch, "combine": _exact_combine,
            "gradient": _exact_gradient, "gemv_q4": _exact_gemv_q4, "experts_q4": _exact_experts_q4}[s["kind"]](s)


def _exact_route(s):
    """One expert after the other: the largest score that is left, the first of equals."""
    import numpy as np
    x = s["logits"].double().cpu().numpy()
    score = s["logits"].float().cpu().numpy().copy()
    if s["select_bias"] is not None:
        score = score + s["select_bias"].cpu().numpy()
    score = score.astype(np.float64)
    at, ids = np.arange(s["m"]), np.full((s["m"], s["top_k"]), s["experts"])
    for slot in range(s["top_k"]):
        ids[:, slot] = score.argmax(axis=1)  # numpy's argmax gives the first of equals
        score[at, ids[:, slot]] = -np.inf
    picked = np.exp(x[at[:, None], ids])
    every = np.exp(x)
    weights = picked / (picked if s["selected"] else every).sum(axis=1, keepdims=True)
    out = {"ids": ids.astype(np.int32), "weights": weights}
    if s["grad"]:
        d = s["d_weights"].double().cpu().numpy()
        # Jacobian of the softmax: d w_i / d l_e = w_i ((i is e) - p_e)
        p = np.zeros_like(x)
        if s["selected"]:
            p[at[:, None], ids] = weights
        else:
            p = every / every.sum(axis=1, keepdims=True)
        d_logits = -p * np.einsum("ts,ts->t", weights, d)[:, None]
        for slot in range(s["top_k"]):
            d_logits[at, ids[:, slot]] += weights[:, slot] * d[:, slot]
        out["d_logits"] = d_logits
    return out


def _exact_dispatch(s):
    import numpy as np
    ids, rows = s["ids"].reshape(-1).cpu().numpy(), s["m"] * s["top_k"]
    lists = [np.flatnonzero(ids == e) for e in range(s["experts"] + 1)]
    order = np.concatenate(lists)
    position = np.empty(rows, np.int64)
    position[order] = np.arange(rows)
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in lists[:-1]])])
    xs = torch.zeros(rows, s["n"], dtype=torch.float64, device="cuda")
    live = torch.from_numpy(order[: offsets[-1]]).cuda()
    xs[: offsets[-1]] = s["x"].double()[live // s["top_k"]]
    return {"offsets": offsets, "order": order, "position": position, "xs": xs}


def _exact_combine(s):
    y = torch.zeros(s["m"], s["n"], dtype=torch.float64, device="cuda")
    live, position = int(s["offsets"][-1]), s["position"].view(s["m"], -1).long()
    for slot in range(s["top_k"]):
        keep = torch.nonzero(position[:, slot] < live)[:, 0]
        y[keep] += s["weights"][keep, slot, None].double() * s["ys"][position[keep, slot]].double()
    return {"y": y}


def _exact_gradient(s):
    rows, m, n = s["m"] * s["top_k"], s["m"], s["n"]
    live, position = int(s["offsets"][-1]), s["position"].view(m, -1).long()
    d_ys, d_x = (torch.zeros(r, n, dtype=torch.float64, device="cuda") for r in (rows, m))
    d_weights = torch.zeros(m, s["top_k"], dtype=torch.float64, device="cuda")
    for slot in range(s["top_k"]):
        keep = torch.nonzero(position[:, slot] < live)[:, 0]
        at, d_y = position[keep, slot], s["d_y"][keep].double()
        d_ys[at] = s["weights"][keep, slot, None].double() * d_y
        d_weights[keep, slot] = torch.einsum("rn,rn->r", d_y, s["ys"][at].double())
        d_x[keep] += s["d_xs"][at].double()
    return {"d_ys": d_ys, "d_weights": d_weights, "d_x": d_x}


def _exact_matrix(s, *at):
    """W[n, k] in 64 bits, column by column pair."""
    q, scales = s["q"][at].long(), s["scales"][at].double()
    zeros = torch.full_like(scales, 8.0) if s["zeros"] is None else s["zeros"][at].double()
    w = torch.empty(s["n"], 2 * q.shape[1], dtype=torch.float64, device="cuda")
    w[:, 0::2], w[:, 1::2] = (q % 16).double(), (q // 16).double()
    w = w[:, : s["k"]]
    for i in range(scales.shape[1]):
        part = w[:, i * s["group"]:(i + 1) * s["group"]]
        part -= zeros[:, i, None]
        part *= scales[:, i, None]
    return w


def _exact_gemv_q4(s):
    return {"y": s["x"].double() @ _exact_matrix(s).T}


def _exact_experts_q4(s):
    y = torch.zeros(s["m"], s["top_k"], s["n"], dtype=torch.float64, device="cuda")
    for e in torch.unique(s["ids"]).tolist():
        t, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        y[t, slot] = s["x"][t].double() @ _exact_matrix(s, e).T
    return {"y": y}
