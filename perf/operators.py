"""The operators around an MoE layer's experts, as cases that can be timed and compared.

Four operators, each with its backward pass where a layer is trained:

  gate    router logits -> the k experts of a token and their weights (and the logits' gradient)
  sort    token rows -> rows in expert order, with offsets and the map back (and the rows' gradient)
  unsort  expert-ordered rows -> the router-weighted sum per token (and both gradients)
  lora    a projection shared by all requests, with each request's low-rank adapter beside it

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once at the end) or,
with ``own``, through the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"


# --- cases --------------------------------------------------------------------

def _gate(name, n, e, k, score, renorm, bf16, train, groups=1, keep=1, top=1):
    return {"name": name, "op": "gate", "n": n, "e": e, "k": k, "score": score, "renorm": renorm, "bf16": bf16,
            "train": train, "groups": groups, "keep": keep, "top": top}


def _sort(name, op, ranks, t, h, e, k, dtype, train, masked=0.0):
    return {"name": name, "op": op, "ranks": ranks, "t": t, "h": h, "e": e, "k": k, "dtype": dtype, "train": train,
            "masked": masked}


def _lora(name, t, n_in, n_out, rank, adapters, mix):
    return {"name": name, "op": "lora", "t": t, "in": n_in, "out": n_out, "rank": rank, "adapters": adapters,
            "mix": mix}


def listed():
    return [
        # one token being decoded: top-8 of 256, softmax probabilities as they are
        _gate("gate_one_token", 1, 256, 8, "softmax", False, False, False),
        # a prompt's tokens, group-limited sigmoid routing (4 of 8 groups by their best two), bf16 logits
        _gate("gate_prompt_groups", 4096, 256, 8, "sigmoid", True, True, False, 8, 4, 2),
        # a training step's tokens, softmax over the chosen: ids, weights and the logits' gradient
        _gate("gate_train", 32768, 256, 8, "softmax", True, False, True),
        # a decode step of 8 ranks x 128 tokens, e4m3 rows with block scales
        _sort("sort_decode_fp8", "sort", 8, 128, 7168, 256, 8, "fp8", False),
        # a short ragged batch in training, some choices dropped, odd sizes
        _sort("sort_train_ragged", "sort", 1, 333, 1000, 12, 3, "bf16", True, 0.2),
        # a training step of a many-expert layer, forward and backward
        _sort("sort_train", "sort", 1, 8192, 7168, 256, 8, "bf16", True),
        # the way back of the decode step
        _sort("unsort_decode", "unsort", 8, 128, 7168, 256, 8, "bf16", False),
        # few experts, two choices, a prompt's tokens in training: forward and both gradients
        _sort("unsort_train", "unsort", 1, 8192, 4096, 8, 2, "bf16", True),
        # one token of one request
        _lora("lora_one_token", 1, 4096, 4096, 16, 8, "tokens"),
        # a decode step of 64 requests over 32 adapters
        _lora("lora_decode", 64, 7168, 2048, 16, 32, "tokens"),
        # two prompts' pieces and some single tokens in one batch, odd sizes
        _lora("lora_mixed", 389, 2056, 4104, 24, 12, "requests"),
        # a full batch of prompts
        _lora("lora_prompts", 8192, 7168, 2048, 64, 16, "requests"),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over its logarithm; the larger ones are odd multiples."""
    m = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) // step
    return max(lo, min(hi, (m | 1 if m > 64 // step else m) * step))


def draw(rng):
    op = rng.choice(["gate", "sort", "unsort", "lora"])
    if op == "gate":
        e = rng.choice([8, 16, 60, 64, 128, 160, 256])
        k = rng.choice([x for x in (1, 2, 4, 6, 8) if x <= e // 2])
        score = rng.choice(["softmax", "sigmoid"])
        c = _gate("", _log_int(rng, 1, 32768), e, k, score, rng.random() < 0.5, rng.random() < 0.5,
                  rng.random() < 0.5)
        if e % 8 == 0 and e >= 64 and score == "sigmoid" and rng.random() < 0.5:
            c["n"] = min(c["n"], 4096)
            c["groups"], c["keep"], c["top"] = 8, 4, 2
    elif op in ("sort", "unsort"):
        dtype = rng.choice(["bf16", "bf16", "fp8"]) if op == "sort" else "bf16"
        train = dtype == "bf16" and rng.random() < 0.6
        step = 128 if dtype == "fp8" else 8
        ranks = rng.choice([1, 1, 4, 8])
        e = rng.choice([8, 24, 64, 256])
        t, k = _log_int(rng, 1, 8192 // ranks), rng.choice([x for x in (1, 2, 3, 4, 6, 8) if x <= e // 2])
        c = _sort("", op, ranks, t, _log_int(rng, 128, 7168, step), e, k, dtype, train,
                  rng.choice([0.0, 0.0, 0.1, 0.5]) if ranks * t * k >= 64 else 0.0)
    else:
        mix = rng.choice(["tokens", "requests"])
        t = _log_int(rng, 1, 256) if mix == "tokens" else _log_int(rng, 64, 8192)
        c = _lora("", t, _log_int(rng, 512, 7168, 8), _log_int(rng, 512, 2048 if t > 1024 else 7168, 8),
                  rng.choice([8, 16, 24, 32, 64]), _log_int(rng, 1, 32), mix)
    del c["name"]
    return c


# --- inputs -------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * int(seed) + 17)
    return g


def _normal(g, shape, scale=1.0, dtype=torch.bfloat16):
    """N(0, scale^2) values, made in pieces so that no large 32-bit copy is held."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        n = min(1 << 26, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV).mul_(scale)
    return out


def _choices(g, n, e, k, masked):
    """k distinct experts a token from random scores, best first; a share of the choices masked, and a token in
    sixteen with no expert at all where any are."""
    ids = torch.rand((n, e), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32)
    if masked > 0:
        ids = ids.masked_fill(torch.rand((n, k), generator=g, device=DEV) < masked, -1)
        ids = ids.masked_fill(torch.rand((n, 1), generator=g, device=DEV) < 1 / 16, -1)
    return ids.contiguous()


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": c, "err": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if c["op"] == "gate":
        n, e, k = c["n"], c["e"], c["k"]
        s["logits"] = _normal(g, (n, e), 1.0, torch.bfloat16 if c["bf16"] else torch.float32)
        s["idx"] = torch.empty((n, k), dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty((n, k), device=DEV)
        if c["train"]:
            s["grad_weights"] = _normal(g, (n, k), 1.0, torch.float32)
            s["grad_logits"] = torch.empty_like(s["logits"])
        return s
    if c["op"] == "lora":
        t, a, r = c["t"], c["adapters"], c["rank"]
        s["x"] = _normal(g, (t, c["in"]))
        s["w"] = _normal(g, (c["out"], c["in"]), c["in"] ** -0.5)
        s["lora_a"] = _normal(g, (a, r, c["in"]), c["in"] ** -0.5)
        s["lora_b"] = _normal(g, (a, c["out"], r), r ** -0.5)
        s["scales"] = torch.rand(a, generator=g, device=DEV).mul_(0.75).add_(0.25)
        if c["mix"] == "tokens":  # a decode step: every token is a request of its own
            ids = torch.randint(0, a, (t,), generator=g, device=DEV)
            plain_share = torch.rand(t, generator=g, device=DEV)
        else:  # prompts and their pieces: a run of tokens has one request
            start = torch.rand(t, generator=g, device=DEV) < max(1.0 / 512, 4.0 / t)
            req = start.int().cumsum(0)
            ids = torch.randint(0, a, (t + 1,), generator=g, device=DEV)[req]
            plain_share = torch.rand(t + 1, generator=g, device=DEV)[req]
        s["adapter"] = ids.masked_fill(plain_share < 0.1, -1).to(torch.int32) if t > 1 else ids.to(torch.int32)
        s["u"] = torch.empty((t, r), dtype=torch.bfloat16, device=DEV)
        s["y"] = torch.empty((t, c["out"]), dtype=torch.bfloat16, device=DEV)
        return s
    n, h, k = c["ranks"] * c["t"], c["h"], c["k"]
    s["idx"] = _choices(g, n, c["e"], k, c["masked"])
    s["offsets"] = torch.zeros(c["e"] * c["ranks"] + 1, dtype=torch.int32, device=DEV)
    s["tok_packed"] = torch.empty((n, k), dtype=torch.int32, device=DEV)
    if c["op"] == "sort":
        s["x"] = _normal(g, (n, h))
        s["scales"] = s["packed_scales"] = None
        if c["dtype"] == "fp8":  # e4m3 rows with one scale per 128 elements
            b = s["x"].float().view(n, h // 128, 128)
            sc = b.abs().amax(2) / 448.0
            s["scales"] = sc.contiguous()
            s["x"] = (b / sc[:, :, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(n, h)
            s["packed_scales"] = torch.zeros((n * k, h // 128), device=DEV)
        s["packed"] = torch.zeros((n * k, h), dtype=torch.uint8 if c["dtype"] == "fp8" else torch.bfloat16, device=DEV)
        if c["train"]:
            s["grad_packed"] = _normal(g, (n * k, h))
            s["grad_x"] = torch.empty((n, h), dtype=torch.bfloat16, device=DEV)
        return s
    s["tok_packed"] = _order(s["idx"], c["ranks"], c["e"])[0].contiguous()
    s["y"] = _normal(g, (n * k, h))
    s["weights"] = torch.rand((n, k), generator=g, device=DEV).add_(0.05)
    s["weights"] /= s["weights"].sum(1, keepdim=True)
    s["out"] = torch.empty((n, h), dtype=torch.bfloat16, device=DEV)
    if c["train"]:
        s["grad_out"] = _normal(g, (n, h))
        s["grad_y"] = torch.zeros((n * k, h), dtype=torch.bfloat16, device=DEV)
        s["grad_weights"] = torch.empty((n, k), device=DEV)
    return s


# --- the plain forms ----------------------------------------------------------

def _order(idx, ranks, e):
    """The row of every choice in expert order (-1: masked), the choice of every row, which rows are filled, and
    the offsets of the (expert, rank) regions."""
    n, k = idx.shape
    flat = idx.reshape(-1).long()
    src = torch.arange(n * k, device=idx.device) // (n // ranks * k)
    key = torch.where(flat >= 0, flat * ranks + src, e * ranks)
    key, choice = torch.sort(key, stable=True)
    filled = key < e * ranks
    row = torch.arange(n * k, device=idx.device)
    tok = torch.empty_like(row)
    tok[choice] = torch.where(filled, row, -1)
    off = torch.searchsorted(key, torch.arange(e * ranks + 1, device=idx.device))
    return tok.view(n, k).int(), choice, filled, off.int()


def _gate_plain(s):
    c = s["case"]
    x = s["logits"].float()
    n, e, k = c["n"], c["e"], c["k"]
    if c["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    key = x
    if c["groups"] > 1:
        best = torch.sort(p.view(n, c["groups"], -1), dim=2, descending=True).values[:, :, :c["top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        drop = torch.ones((n, c["groups"]), dtype=torch.bool, device=x.device).scatter_(1, kept, False)
        key = x.masked_fill(drop.repeat_interleave(e // c["groups"], 1), -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = p.gather(1, idx)
    total = chosen.sum(1, keepdim=True)
    w = chosen / total if c["renorm"] else chosen
    if not c["train"]:
        return idx.int(), w
    g = s["grad_weights"]
    gs = (g - (g * w).sum(1, keepdim=True)) / total if c["renorm"] else g  # with respect to the chosen scores
    if c["score"] == "softmax":
        d = torch.zeros_like(x).scatter_(1, idx, gs * chosen) - p * (gs * chosen).sum(1, keepdim=True)
    else:
        d = torch.zeros_like(x).scatter_(1, idx, gs * chosen * (1.0 - chosen))
    return idx.int(), w, d.to(s["logits"].dtype)


def _sort_plain(s):
    c = s["case"]
    k = c["k"]
    tok, choice, filled, off = _order(s["idx"], c["ranks"], c["e"])
    x = s["x"].view(torch.uint8) if c["dtype"] == "fp8" else s["x"]
    packed = x[choice // k].masked_fill_(~filled[:, None], 0)
    if c["dtype"] == "fp8":
        sc = s["scales"][choice // k].masked_fill_(~filled[:, None], 0)
        return off, tok, packed.view(torch.float8_e4m3fn), sc
    if not c["train"]:
        return off, tok, packed
    g = s["grad_packed"][tok.clamp(min=0).long()].float() * (tok >= 0)[:, :, None]
    return off, tok, packed, g.sum(1).to(torch.bfloat16)


def _unsort_plain(s):
    c = s["case"]
    tok, w = s["tok_packed"], s["weights"]
    at, live = tok.clamp(min=0).long(), tok >= 0
    wl = w * live
    out = (s["y"][at].float() * wl[:, :, None]).sum(1).to(torch.bfloat16)
    if not c["train"]:
        return out
    g = s["grad_out"].float()
    rows = s["y"].shape[0]
    to = torch.where(live, tok.long(), rows).view(-1)
    gy = torch.zeros((rows + 1, c["h"]), dtype=torch.bfloat16, device=g.device)
    gy[to] = (g[:, None, :] * wl[:, :, None]).to(torch.bfloat16).view(-1, c["h"])
    gw = (s["y"][at].float() * g[:, None, :]).sum(2) * live
    return out, gy[:rows], gw


def _lora_plain(s):
    c = s["case"]
    t, a, r = c["t"], c["adapters"], c["rank"]
    x = s["x"].float()
    ids = s["adapter"].long()
    mine = ids[:, None] == torch.arange(a, device=x.device)
    u = (x @ s["lora_a"].view(a * r, c["in"]).float().t()).view(t, a, r)
    u = (u * (mine * s["scales"])[:, :, None]).view(t, a * r)
    b = s["lora_b"].float().permute(0, 2, 1).reshape(a * r, c["out"])
    return (x @ s["w"].float().t() + u @ b).to(torch.bfloat16)


# --- the library's calls ------------------------------------------------------

def _gate_own(s, m):
    c = s["case"]
    if "desc" not in s:
        s["desc"] = m.MoeDesc(1, c["n"], 8, c["e"], c["k"], c["n"], m.MOE_BF16, 0)
        s["opts"] = m.MoeGateOpts(m.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else m.MOE_SCORE_SIGMOID,
                                  int(c["renorm"]), c["groups"], c["keep"], c["top"], int(c["bf16"]), 1.0)
    m.moe_gate(s["desc"], s["opts"], s["logits"], None, s["idx"], s["weights"], s["err"])
    if not c["train"]:
        return s["idx"], s["weights"]
    m.moe_gate_grad(s["desc"], s["opts"], s["logits"], s["idx"], s["grad_weights"], s["grad_logits"], s["err"])
    return s["idx"], s["weights"], s["grad_logits"]


def _rows_desc(s, m):
    c = s["case"]
    if "desc" not in s:
        s["desc"] = m.MoeDesc(c["ranks"], c["t"], c["h"], c["e"], c["k"], c["t"],
                              m.MOE_FP8_E4M3 if c["dtype"] == "fp8" else m.MOE_BF16, 0)
    return s["desc"]


def _sort_own(s, m):
    c, d = s["case"], _rows_desc(s, m)
    m.moe_sort(d, s["idx"], s["x"], s["scales"], s["offsets"], s["packed"], s["packed_scales"], s["tok_packed"],
               s["err"])
    if c["dtype"] == "fp8":
        return s["offsets"], s["tok_packed"], s["packed"].view(torch.float8_e4m3fn), s["packed_scales"]
    if not c["train"]:
        return s["offsets"], s["tok_packed"], s["packed"]
    m.moe_sort_grad(d, s["grad_packed"], s["tok_packed"], s["grad_x"], s["err"])
    return s["offsets"], s["tok_packed"], s["packed"], s["grad_x"]


def _unsort_own(s, m):
    c, d = s["case"], _rows_desc(s, m)
    m.moe_unsort(d, s["y"], s["tok_packed"], s["weights"], s["out"], s["err"])
    if not c["train"]:
        return s["out"]
    m.moe_unsort_grad(d, s["y"], s["tok_packed"], s["weights"], s["grad_out"], s["grad_y"], s["grad_weights"],
                      s["err"])
    return s["out"], s["grad_y"], s["grad_weights"]


def _lora_own(s, m):
    c = s["case"]
    if "desc" not in s:
        s["desc"] = m.MoeLoraDesc(c["t"], c["in"], c["out"], c["rank"], c["adapters"], 0)
    m.moe_lora_linear(s["desc"], s["x"], s["w"], s["lora_a"], s["lora_b"], s["scales"], s["adapter"], s["u"], s["y"],
                      s["err"])
    return s["y"]


_PLAIN = {"gate": _gate_plain, "sort": _sort_plain, "unsort": _unsort_plain, "lora": _lora_plain}
_OWN = {"gate": _gate_own, "sort": _sort_own, "unsort": _unsort_own, "lora": _lora_own}


def run(state):
    op = state["case"]["op"]
    if own:
        import combine_moe_layout_gb300 as m
        return _OWN[op](state, m)
    return _PLAIN[op](state)


# --- what a pass cannot do without --------------------------------------------

def work(case):
    c = case
    if c["op"] == "gate":
        n, e, k, b = c["n"], c["e"], c["k"], 2 if c["bf16"] else 4
        by, fl = n * (e * b + 8 * k), 4.0 * n * e
        if c["train"]:  # the logits, ids and weights' gradients in, the logits' gradient out
            by, fl = by + n * (2 * e * b + 8 * k), fl + 4.0 * n * e
        return {"bytes": by, "flops": fl}
    if c["op"] == "lora":
        t, i, o, r, a = c["t"], c["in"], c["out"], c["rank"], c["adapters"]
        draws = t if c["mix"] == "tokens" else max(4, t // 512)
        used = a * (1.0 - (1.0 - 1.0 / a) ** draws)  # adapters that some token names
        return {"bytes": 2.0 * (t * i + o * i + t * o + used * r * (i + o)) + 4.0 * t,
                "flops": 2.0 * t * (i * o + r * (i + o))}
    n, h, k = c["ranks"] * c["t"], c["h"], c["k"]
    live = k * (1.0 - c["masked"]) * (15 / 16 if c["masked"] else 1.0)  # choices a token that name an expert
    if c["op"] == "sort":
        row = h + h // 128 * 4 if c["dtype"] == "fp8" else 2 * h
        by, fl = n * (row * (1 + live) + 8 * k) + 4 * c["e"] * c["ranks"], 0.0
        if c["train"]:
            by, fl = by + n * (2 * h * (1 + live) + 4 * k), 1.0 * n * live * h
        return {"bytes": by, "flops": fl}
    by, fl = n * (2 * h * (1 + live) + 8 * k), 2.0 * n * live * h
    if c["train"]:
        by, fl = by + n * (2 * h * (1 + 2 * live) + 12 * k), fl + 3.0 * n * live * h
    return {"bytes": by, "flops": fl}


# --- in 64 bits, from the definitions -----------------------------------------

def _exact_gate(s, c):
    z = s["logits"].double()
    n, e, k = c["n"], c["e"], c["k"]
    lse = torch.logsumexp(z, 1, keepdim=True)
    score = (z - lse).exp() if c["score"] == "softmax" else torch.sigmoid(z)
    allowed = torch.ones((n, e), dtype=torch.bool, device=z.device)
    if c["groups"] > 1:
        size = e // c["groups"]
        best = score.view(n, c["groups"], size).topk(c["top"], 2).values.sum(2)
        ranked = best.sort(1, descending=True).values
        near = (ranked[:, c["keep"] - 1] - ranked[:, c["keep"]]).abs()
        if bool(((near < 3e-7) & (near > 0)).any()):  # 32 bits cannot tell these groups apart
            return None
        place = (best[:, None, :] > best[:, :, None]).sum(2)
        tied = best[:, None, :] == best[:, :, None]
        lower = torch.ones((c["groups"], c["groups"]), device=z.device, dtype=torch.bool).tril(-1)
        place = place + (tied & lower).sum(2)
        allowed = (place < c["keep"]).repeat_interleave(size, 1)
    rest = z.masked_fill(~allowed, -math.inf)
    ids = []
    for _ in range(k):  # the largest that is left, the lowest index among equals
        top = rest.amax(1, keepdim=True)
        i = torch.where(rest == top, torch.arange(e, device=z.device), e).amin(1, keepdim=True)
        ids.append(i)
        rest = rest.scatter(1, i, -math.inf)
    ids = torch.cat(ids, 1)
    with torch.enable_grad():
        zz = z.clone().requires_grad_(True)
        sc = torch.softmax(zz, 1) if c["score"] == "softmax" else torch.sigmoid(zz)
        w = sc.gather(1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        if not c["train"]:
            return ids.int(), w.detach()
        (d,) = torch.autograd.grad((w * s["grad_weights"].double()).sum(), zz)
    return ids.int(), w.detach(), d


def _exact_rows(s, c):
    """The rows of the choices by counting: a choice comes after every choice of a lower expert and after the
    earlier choices of its own."""
    n, k, e, ranks = c["ranks"] * c["t"], c["k"], c["e"], c["ranks"]
    flat = s["idx"].view(-1).long()
    tok = torch.full((n * k,), -1, dtype=torch.int64, device=flat.device)
    off = torch.zeros(e * ranks + 1, dtype=torch.int64, device=flat.device)
    before = 0
    for x in range(e):
        at = (flat == x).nonzero().view(-1)
        tok[at] = before + torch.arange(at.numel(), device=at.device)
        per = (at // (c["t"] * k) if n else at).bincount(minlength=ranks)
        off[x * ranks + 1:(x + 1) * ranks + 1] = before + per.cumsum(0)
        before += at.numel()
    return tok.view(n, k), off


def _exact_sort(s, c):
    tok, off = _exact_rows(s, c)
    n, k, h = c["ranks"] * c["t"], c["k"], c["h"]
    packed = torch.zeros((n * k, h), dtype=torch.float64, device=DEV)
    sc = torch.zeros((n * k, h // 128), dtype=torch.float64, device=DEV) if c["dtype"] == "fp8" else None
    dx = torch.zeros((n, h), dtype=torch.float64, device=DEV)
    for j in range(k):
        t = (tok[:, j] >= 0).nonzero().view(-1)
        p = tok[t, j]
        packed[p] = s["x"].double()[t]
        if sc is not None:
            sc[p] = s["scales"][t].double()
        if c["train"]:
            dx[t] += s["grad_packed"][p].double()
    got = (off.int(), tok.int(), packed) + ((sc,) if sc is not None else ())
    return got + (dx,) if c["train"] else got


def _exact_unsort(s, c):
    tok, _ = _exact_rows(s, c)
    n, k, h = c["ranks"] * c["t"], c["k"], c["h"]
    out = torch.zeros((n, h), dtype=torch.float64, device=DEV)
    gy = torch.zeros((n * k, h), dtype=torch.float64, device=DEV) if c["train"] else None
    gw = torch.zeros((n, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        t = (tok[:, j] >= 0).nonzero().view(-1)
        p = tok[t, j]
        w = s["weights"][t, j].double()[:, None]
        y = s["y"][p].double()
        out[t] += w * y
        if c["train"]:
            g = s["grad_out"][t].double()
            gy[p] = w * g
            gw[t, j] = (y * g).sum(1)
    return (out, gy, gw) if c["train"] else out


def _exact_lora(s, c):
    x = s["x"].double()
    y = x @ s["w"].double().t()
    for a in range(c["adapters"]):
        t = (s["adapter"] == a).nonzero().view(-1)
        if t.numel():
            y[t] += s["scales"][a].double() * ((x[t] @ s["lora_a"][a].double().t()) @ s["lora_b"][a].double().t())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": _exact_gate, "sort": _exact_sort, "unsort": _exact_unsort, "lora": _exact_lora}[case["op"]](s, case)
