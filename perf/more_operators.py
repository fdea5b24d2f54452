"""What a training or serving step runs around and inside the experts beside perf/operators.py, as cases that can be
timed and compared.

Four operators:

  ffn        the gated feed-forward block, act(x w_gate^T) * (x w_up^T) w_down^T, for the rows of every expert or one
             dense block; for training it also keeps its two projections, in bf16 or in 8 bits with block scales
  ffn_grad   its gradients, with respect to the rows and all three weights, from what the forward kept
  norm       the block's output normalised, gated, scaled and added to the residual stream, and the norm after that
  norm_grad  the gradients of the stream, the block's output, both norm weights and the gate

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once at the end) or,
with ``own``, through the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# --- cases --------------------------------------------------------------------

def _ffn(name, op, rows, h, i, experts, act, save, masked=0.0):
    return {"name": name, "op": op, "rows": rows, "h": h, "i": i, "experts": experts, "act": act, "save": save,
            "masked": masked}


def _norm(name, op, rows, h, fp32, post, gate):
    return {"name": name, "op": op, "rows": rows, "h": h, "fp32": fp32, "post": post, "gate": gate}


def listed():
    return [
        # one token through a shared expert
        _ffn("ffn_one_token", "ffn", 1, 7168, 2048, 1, "silu", "none"),
        # a decode step of 64 requests through it
        _ffn("ffn_decode", "ffn", 64, 7168, 2048, 1, "silu", "none"),
        # a short ragged batch over a few experts, odd widths, kept in 8 bits
        _ffn("ffn_ragged_fp8", "ffn", 333, 1000, 640, 12, "gelu", "fp8", 0.1),
        # a training step of a many-expert layer (4096 tokens, 6 choices), kept in 8 bits
        _ffn("ffn_train_fp8", "ffn", 24576, 4096, 1408, 64, "silu", "fp8"),
        # the way back of the short batch, with a width that no tile divides, kept in bf16
        _ffn("ffn_grad_ragged", "ffn_grad", 333, 1000, 712, 12, "gelu", "bf16", 0.1),
        # the way back of the many-expert layer from its 8-bit checkpoint
        _ffn("ffn_grad_train_fp8", "ffn_grad", 24576, 4096, 1408, 64, "silu", "fp8"),
        # a dense block of Mixtral's widths in training, kept in bf16
        _ffn("ffn_grad_dense", "ffn_grad", 4096, 4096, 14336, 1, "silu", "bf16"),
        # one token's norms around a block, a gate for each token
        _norm("norm_one_token", "norm", 1, 7168, False, True, "row"),
        # a decode step of 8 ranks x 128 tokens, no norm after the block
        _norm("norm_decode", "norm", 1024, 7168, False, False, "none"),
        # a training step's tokens, residual stream in 32 bits, a gate for each channel
        _norm("norm_train", "norm", 8192, 7168, True, True, "channel"),
        # the way back of a short batch, odd sizes
        _norm("norm_grad_ragged", "norm_grad", 333, 1000, True, True, "row"),
        # the way back of a training step's tokens
        _norm("norm_grad_train", "norm_grad", 8192, 7168, False, True, "channel"),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over its logarithm; the larger ones are odd multiples."""
    m = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) // step
    return max(lo, min(hi, (m | 1 if m > 64 // step else m) * step))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_grad", "ffn_grad", "norm", "norm_grad"])
    if op in ("ffn", "ffn_grad"):
        experts = rng.choice([1, 1, 3, 8, 16, 64])
        save = rng.choice(["bf16", "fp8"] if op == "ffn_grad" else ["none", "none", "bf16", "fp8"])
        h = _log_int(rng, 256, 7168, 8)
        i = _log_int(rng, 128, 4096, 128 if save == "fp8" else 8)
        if experts > 16:
            h, i = min(h, 4096), min(i, 1408)
        c = _ffn("", op, _log_int(rng, 1, 16384), h, i, experts, rng.choice(["silu", "gelu"]), save,
                 rng.choice([0.0, 0.0, 0.1, 0.5]) if experts > 1 else 0.0)
    else:
        c = _norm("", op, _log_int(rng, 1, 8192), _log_int(rng, 128, 8192 if op == "norm" else 7168, 8),
                  rng.random() < 0.5, rng.random() < 0.5, rng.choice(["none", "row", "channel"]))
    del c["name"]
    return c


# --- inputs -------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * int(seed) + 29)
    return g


def _normal(g, shape, scale=1.0, dtype=torch.bfloat16):
    """N(0, scale^2) values, made in pieces so that no large 32-bit copy is held."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        n = min(1 << 26, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV).mul_(scale)
    return out


def _quantised(x):
    """bf16 rows as e4m3 with a 32-bit scale for each 128 elements."""
    b = x.float().view(x.shape[0], -1, 128)
    amax = b.abs().amax(2)
    sc = torch.where(amax > 0, amax / 448.0, 1.0)
    return (b / sc[:, :, None]).to(torch.float8_e4m3fn).view(x.shape), sc.contiguous()


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": c, "err": torch.zeros(1, dtype=torch.int32, device=DEV)}
    n, h = c["rows"], c["h"]

    def rows(width, dtype=torch.bfloat16):
        return torch.zeros((n, width), dtype=dtype, device=DEV)

    if c["op"] in ("norm", "norm_grad"):
        stream = torch.float32 if c["fp32"] else torch.bfloat16
        s["x"] = _normal(g, (n, h), 2.0, stream)
        s["o"] = _normal(g, (n, h))
        s["w_pre"] = _normal(g, (h,), 0.2, torch.float32).add_(1.0)
        s["w_post"] = _normal(g, (h,), 0.2, torch.float32).add_(1.0) if c["post"] else None
        s["gate"] = None
        if c["gate"] == "row":  # a gate's sigmoid for each token
            s["gate"] = torch.rand(n, generator=g, device=DEV)
        elif c["gate"] == "channel":  # a learned scale for each channel
            s["gate"] = _normal(g, (h,), 0.3, torch.float32)
        s["alpha"] = 0.5
        if c["op"] == "norm":
            s["r"], s["n"] = rows(h, stream), rows(h)
            return s
        s["grad_r"], s["grad_n"] = _normal(g, (n, h), 1.0, stream), _normal(g, (n, h))
        s["grad_x"], s["grad_o"] = rows(h, stream), rows(h)
        s["grad_w_pre"] = torch.empty(h, device=DEV)
        s["grad_w_post"] = torch.empty(h, device=DEV) if c["post"] else None
        s["grad_gate"] = torch.empty_like(s["gate"]) if s["gate"] is not None else None
        return s

    e, i = c["experts"], c["i"]
    if e > 1:  # experts of uneven popularity; rows behind the last expert's belong to no one
        pop = torch.rand(e, generator=g, device=DEV).mul_(2.0).exp_()
        ids = torch.multinomial(pop, n, replacement=True, generator=g)
        ids = torch.where(torch.rand(n, generator=g, device=DEV) < c["masked"], e, ids)
        counts = ids.bincount(minlength=e + 1)[:e]
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
        s["cap"] = max(1, int(counts.max()))
    else:
        s["offsets"], s["cap"] = None, n
    s["x"] = _normal(g, (n, h))
    s["w_gate"] = _normal(g, (e, i, h), h ** -0.5)
    s["w_up"] = _normal(g, (e, i, h), h ** -0.5)
    s["w_down"] = _normal(g, (e, h, i), i ** -0.5)
    s["gate"] = s["gate_scales"] = s["up"] = s["up_scales"] = None
    s["hidden"] = rows(i)
    if c["op"] == "ffn":
        s["y"] = rows(h)
        if c["save"] == "bf16":
            s["gate"], s["up"] = rows(i), rows(i)
        elif c["save"] == "fp8":
            s["gate"], s["up"] = rows(i, torch.uint8), rows(i, torch.uint8)
            s["gate_scales"], s["up_scales"] = rows(i // 128, torch.float32), rows(i // 128, torch.float32)
        return s
    s["gate"], s["up"] = _normal(g, (n, i)), _normal(g, (n, i))
    if c["save"] == "fp8":
        s["gate"], s["gate_scales"] = _quantised(s["gate"])
        s["up"], s["up_scales"] = _quantised(s["up"])
    s["grad_y"] = _normal(g, (n, h))
    s["grad_hidden_gate"], s["grad_hidden_up"] = rows(i), rows(i)
    s["grad_x"] = rows(h)
    s["grad_w_gate"], s["grad_w_up"] = torch.empty_like(s["w_gate"]), torch.empty_like(s["w_up"])
    s["grad_w_down"] = torch.empty_like(s["w_down"])
    return s


# --- the plain forms ----------------------------------------------------------

def _by_expert(s):
    """The rows as [experts][cap], which of those places are filled, and each row's place (rows of no expert: none)."""
    c = s["case"]
    n, e, cap = c["rows"], c["experts"], s["cap"]
    row = torch.arange(n, device=DEV)
    if s["offsets"] is None:
        return row[None], torch.ones((1, n), dtype=torch.bool, device=DEV), row, row < n
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(cap, device=DEV)
    filled = at < off[1:, None]
    mine = (torch.searchsorted(off, row, right=True) - 1).clamp(max=e - 1)
    place = mine * cap + row - off[mine]
    live = row < off[-1]
    return at.clamp(max=n - 1), filled, place.masked_fill(~live, 0), live


def _spread(t, at, filled):
    return t[at].float().masked_fill_(~filled[:, :, None], 0.0)


def _together(t, place, live):
    return t.reshape(-1, t.shape[2])[place].masked_fill_(~live[:, None], 0.0)


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3.0 * 0.044715 * g * g)


def _codes(t):
    b = t.view(t.shape[0], -1, 128)
    amax = b.abs().amax(2)
    sc = torch.where(amax > 0, amax / 448.0, 1.0)
    return (b / sc[:, :, None]).to(torch.float8_e4m3fn).view(t.shape), sc


def _ffn_plain(s):
    c = s["case"]
    at, filled, place, live = _by_expert(s)
    x = _spread(s["x"], at, filled)
    g = torch.bmm(x, s["w_gate"].float().transpose(1, 2))
    u = torch.bmm(x, s["w_up"].float().transpose(1, 2))
    hidden = _act(g, c["act"])[0] * u
    y = _together(torch.bmm(hidden, s["w_down"].float().transpose(1, 2)), place, live).to(torch.bfloat16)
    if c["save"] == "none":
        return y
    g, u = _together(g, place, live), _together(u, place, live)
    if c["save"] == "bf16":
        return y, g.to(torch.bfloat16), u.to(torch.bfloat16)
    (gq, gs), (uq, us) = _codes(g), _codes(u)
    gs, us = gs.masked_fill(~live[:, None], 0.0), us.masked_fill(~live[:, None], 0.0)
    return y, gq, gs, uq, us


def _kept(s, name, dtype):
    """The projection that the forward kept, in `dtype`."""
    t = s[name].to(dtype)
    if s["case"]["save"] == "fp8":
        t = (t.view(t.shape[0], -1, 128) * s[name + "_scales"].to(dtype)[:, :, None]).view(t.shape)
    return t


def _ffn_grad_plain(s):
    c = s["case"]
    at, filled, place, live = _by_expert(s)
    x, dy = _spread(s["x"], at, filled), _spread(s["grad_y"], at, filled)
    g, u = _spread(_kept(s, "gate", torch.float32), at, filled), _spread(_kept(s, "up", torch.float32), at, filled)
    a, da = _act(g, c["act"])
    dh = torch.bmm(dy, s["w_down"].float())
    dg, du = dh * u * da, dh * a
    dx = torch.bmm(dg, s["w_gate"].float()) + torch.bmm(du, s["w_up"].float())
    return (_together(dx, place, live).to(torch.bfloat16), torch.bmm(dg.transpose(1, 2), x).to(torch.bfloat16),
            torch.bmm(du.transpose(1, 2), x).to(torch.bfloat16),
            torch.bmm(dy.transpose(1, 2), a * u).to(torch.bfloat16))


def _norm_plain(s):
    x, o = s["x"].float(), s["o"].float()
    if s["w_post"] is not None:
        o = o * torch.rsqrt((o * o).mean(1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        o = o * (s["gate"][:, None] if s["case"]["gate"] == "row" else s["gate"])
    r = x + s["alpha"] * o
    n = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["w_pre"]
    return r.to(s["x"].dtype), n.to(torch.bfloat16)


def _norm_grad_plain(s):
    """x is the stream that the forward wrote."""
    c = s["case"]
    r, o, dn, dr = s["x"].float(), s["o"].float(), s["grad_n"].float(), s["grad_r"].float()
    q = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    hat = r * q
    dhat = dn * s["w_pre"]
    dr = dr + q * (dhat - hat * (dhat * hat).mean(1, keepdim=True))
    out = {"x": dr.to(s["x"].dtype), "w_pre": (dn * hat).sum(0)}
    p = 1.0
    ohat = o
    if c["post"]:
        p = torch.rsqrt((o * o).mean(1, keepdim=True) + EPS)
        ohat = o * p
    branch = ohat * s["w_post"] if c["post"] else ohat
    db = s["alpha"] * dr
    if c["gate"] == "row":
        out["gate"] = (db * branch).sum(1)
        db = db * s["gate"][:, None]
    elif c["gate"] == "channel":
        out["gate"] = (db * branch).sum(0)
        db = db * s["gate"]
    if c["post"]:
        out["w_post"] = (db * ohat).sum(0)
        db = db * s["w_post"]
        db = p * (db - ohat * (db * ohat).mean(1, keepdim=True))
    out["o"] = db.to(torch.bfloat16)
    return out


# --- the library's calls ------------------------------------------------------

def _ffn_desc(s, m):
    c = s["case"]
    if "desc" not in s:
        act = m.MOE_ACT_SILU if c["act"] == "silu" else m.MOE_ACT_GELU_TANH
        save = {"none": m.MOE_SAVE_NONE, "bf16": m.MOE_SAVE_BF16, "fp8": m.MOE_SAVE_FP8}[c["save"]]
        s["desc"] = m.MoeFfnDesc(c["rows"], c["h"], c["i"], c["experts"], 1, act, save, 0)
    return s["desc"]


def _ffn_own(s, m):
    c = s["case"]
    m.moe_ffn(_ffn_desc(s, m), s["offsets"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["hidden"], s["y"],
              s["gate"], s["gate_scales"], s["up"], s["up_scales"], s["err"])
    if c["save"] == "none":
        return s["y"]
    if c["save"] == "bf16":
        return s["y"], s["gate"], s["up"]
    f8 = torch.float8_e4m3fn
    return s["y"], s["gate"].view(f8), s["gate_scales"], s["up"].view(f8), s["up_scales"]


def _ffn_grad_own(s, m):
    m.moe_ffn_grad(_ffn_desc(s, m), s["offsets"], s["x"], s["gate"], s["gate_scales"], s["up"], s["up_scales"],
                   s["w_gate"], s["w_up"], s["w_down"], s["grad_y"], s["hidden"], s["grad_hidden_gate"],
                   s["grad_hidden_up"], s["grad_x"], s["grad_w_gate"], s["grad_w_up"], s["grad_w_down"], s["err"])
    return s["grad_x"], s["grad_w_gate"], s["grad_w_up"], s["grad_w_down"]


def _norm_desc(s, m):
    c = s["case"]
    if "desc" not in s:
        gate = {"none": m.MOE_GATE_NONE, "row": m.MOE_GATE_ROW, "channel": m.MOE_GATE_CHANNEL}[c["gate"]]
        s["desc"] = m.MoeNormDesc(c["rows"], c["h"], int(c["fp32"]), gate, EPS, s["alpha"])
    return s["desc"]


def _norm_own(s, m):
    m.moe_norm(_norm_desc(s, m), s["x"], s["o"], s["w_post"], s["gate"], s["w_pre"], s["r"], s["n"], s["err"])
    return s["r"], s["n"]


def _norm_grad_own(s, m):
    d = _norm_desc(s, m)
    if "work" not in s:
        s["work"] = torch.empty(max(1, m.moe_norm_workspace(d)), dtype=torch.uint8, device=DEV)
    m.moe_norm_grad(d, s["x"], s["o"], s["w_post"], s["gate"], s["w_pre"], s["grad_r"], s["grad_n"], s["grad_x"],
                    s["grad_o"], s["grad_w_post"], s["grad_gate"], s["grad_w_pre"], s["work"], s["err"])
    out = {"x": s["grad_x"], "w_pre": s["grad_w_pre"], "o": s["grad_o"]}
    if s["gate"] is not None:
        out["gate"] = s["grad_gate"]
    if s["w_post"] is not None:
        out["w_post"] = s["grad_w_post"]
    return out


_PLAIN = {"ffn": _ffn_plain, "ffn_grad": _ffn_grad_plain, "norm": _norm_plain, "norm_grad": _norm_grad_plain}
_OWN = {"ffn": _ffn_own, "ffn_grad": _ffn_grad_own, "norm": _norm_own, "norm_grad": _norm_grad_own}


def run(state):
    op = state["case"]["op"]
    if own:
        import combine_moe_layout_gb300 as m
        return _OWN[op](state, m)
    return _PLAIN[op](state)


# --- what a pass cannot do without --------------------------------------------

def work(case):
    c = case
    n, h = c["rows"], c["h"]
    if c["op"] in ("norm", "norm_grad"):
        b = 4 if c["fp32"] else 2
        vec = h * (1 + c["post"] + (c["gate"] == "channel")) + n * (c["gate"] == "row")
        if c["op"] == "norm":  # x, o in; r, n out
            return {"bytes": n * h * (2.0 * b + 4) + 4.0 * vec, "flops": 10.0 * n * h}
        return {"bytes": n * h * (3.0 * b + 6) + 8.0 * vec, "flops": 24.0 * n * h}
    i, e = c["i"], c["experts"]
    n = n * (1.0 - c["masked"])
    used = e * (1.0 - (1.0 - 1.0 / e) ** n) if e > 1 else 1  # experts with a row
    kept = {"none": 0.0, "bf16": 4.0 * i, "fp8": 2.0 * i + i / 16.0}[c["save"]]
    if c["op"] == "ffn":
        return {"bytes": n * (4.0 * h + kept) + 6.0 * used * h * i, "flops": 6.0 * n * h * i}
    return {"bytes": n * (6.0 * h + kept) + 6.0 * (used + e) * h * i, "flops": 12.0 * n * h * i}


# --- in 64 bits, from the definitions -----------------------------------------

def _runs(s):
    if s["offsets"] is None:
        return [(0, 0, s["case"]["rows"])]
    off = s["offsets"].tolist()
    return [(e, a, b) for e, (a, b) in enumerate(zip(off, off[1:]))]


def _activated(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def _exact_ffn(s, c):
    n, h, i = c["rows"], c["h"], c["i"]
    f64 = dict(dtype=torch.float64, device=DEV)
    y, gate, up = torch.zeros((n, h), **f64), torch.zeros((n, i), **f64), torch.zeros((n, i), **f64)
    for e, a, b in _runs(s):
        if a < b:
            x = s["x"][a:b].double()
            gate[a:b], up[a:b] = x @ s["w_gate"][e].double().t(), x @ s["w_up"][e].double().t()
            y[a:b] = (_activated(gate[a:b], c["act"]) * up[a:b]) @ s["w_down"][e].double().t()
    if c["save"] == "none":
        return y
    if c["save"] == "bf16":
        return y, gate, up
    out = [y]
    for t in (gate, up):  # the codes before they are rounded
        top = t.view(n, -1, 128).abs().amax(2)
        sc = top / 448.0
        out += [(t.view(n, -1, 128) / sc.masked_fill(top == 0, 1.0)[:, :, None]).view(n, i), sc]
    return tuple(out)


def _exact_ffn_grad(s, c):
    n, h, i, e_all = c["rows"], c["h"], c["i"], c["experts"]
    f64 = dict(dtype=torch.float64, device=DEV)
    dx = torch.zeros((n, h), **f64)
    dwg, dwu, dwd = torch.zeros((e_all, i, h), **f64), torch.zeros((e_all, i, h), **f64), torch.zeros((e_all, h, i), **f64)
    for e, a, b in _runs(s):
        if a == b:
            continue
        part = {"case": c}
        for k in ("gate", "up", "gate_scales", "up_scales"):
            part[k] = s[k][a:b] if s[k] is not None else None
        with torch.enable_grad():
            g = _kept(part, "gate", torch.float64).requires_grad_(True)
            u = _kept(part, "up", torch.float64).requires_grad_(True)
            hidden = _activated(g, c["act"]) * u
            dy = s["grad_y"][a:b].double()
            dg, du = torch.autograd.grad(hidden, (g, u), dy @ s["w_down"][e].double())
        x = s["x"][a:b].double()
        dx[a:b] = dg @ s["w_gate"][e].double() + du @ s["w_up"][e].double()
        dwg[e], dwu[e], dwd[e] = dg.t() @ x, du.t() @ x, dy.t() @ hidden.detach()
    return dx, dwg, dwu, dwd


def _stream(x, o, w_post, gate, w_pre, c, alpha):
    if w_post is not None:
        o = o / (o.square().mean(1, keepdim=True) + EPS).sqrt() * w_post
    if gate is not None:
        o = o * (gate.unsqueeze(1) if c["gate"] == "row" else gate.unsqueeze(0))
    r = x + alpha * o
    return r, r / (r.square().mean(1, keepdim=True) + EPS).sqrt() * w_pre


def _exact_norm(s, c):
    def wide(k):
        return s[k].double() if s[k] is not None else None
    return _stream(wide("x"), wide("o"), wide("w_post"), wide("gate"), wide("w_pre"), c, s["alpha"])


def _exact_norm_grad(s, c):
    """The forward's x is what leaves the stream that was kept once the block's part is taken off again."""
    with torch.enable_grad():
        t = {k: s[k].double().requires_grad_(True) for k in ("o", "w_post", "gate", "w_pre") if s[k] is not None}
        r0, _ = _stream(torch.zeros_like(s["x"], dtype=torch.float64), t["o"], t.get("w_post"), t.get("gate"),
                        t["w_pre"], c, s["alpha"])
        x = (s["x"].double() - r0.detach()).requires_grad_(True)
        r, n = _stream(x, t["o"], t.get("w_post"), t.get("gate"), t["w_pre"], c, s["alpha"])
        total = (r * s["grad_r"].double()).sum() + (n * s["grad_n"].double()).sum()
        want = ["x", "w_pre", "o"] + [k for k in ("gate", "w_post") if k in t]
        got = torch.autograd.grad(total, [x if k == "x" else t[k] for k in want])
    return dict(zip(want, got))


def exact(case, seed):
    s = prepare(case, seed)
    return {"ffn": _exact_ffn, "ffn_grad": _exact_ffn_grad, "norm": _exact_norm,
            "norm_grad": _exact_norm_grad}[case["op"]](s, case)
