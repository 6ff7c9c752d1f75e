"""Timing cases of the 8-bit integer products and of the products grouped by
expert, with a plain form of each.

  linear       channel_linear: product in 8-bit integers with one fp32 scale for
               each token and one for each output channel of the weight
  experts      forward with an "int8" bank: the same product over the experts
  grouped      grouped_matmul: bf16 rows sorted by expert times their expert's
               weight, groups of any size
  input_grad   grouped_input_grad: its gradient with respect to the rows
  weight_grad  grouped_weight_grad: its gradient with respect to the weights

With `own` false, run() computes them in elementary torch operations in
float32 (the codes of a quantiser from products in float64, where a value next
to the border between two codes is not moved); with `own` true it calls the
library.
"""
import functools
import math

import torch

own = False

H, F, E, K = 2688, 1856, 128, 6  # the layer: width, expert width, experts, top-k
SHARED = 3712                    # width of the shared expert
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    full = {"H": H, "F": F, "E": E, "k": K}
    up, down = {"E": E, "N": F, "K": H}, {"E": E, "N": H, "K": F}
    return [
        # one dense projection (shared expert's up part): one token, an odd
        # verify batch, a prompt chunk
        {"name": "linear M=1", "op": "linear", "M": 1, "N": SHARED, "K": H, "y": "bf16"},
        {"name": "linear M=77", "op": "linear", "M": 77, "N": SHARED, "K": H, "y": "bf16"},
        {"name": "linear M=4096", "op": "linear", "M": 4096, "N": SHARED, "K": H, "y": "bf16"},
        # the routed experts: a speculative batch, 64 requests, a prompt chunk
        {"name": "experts T=5", "op": "experts", "T": 5, **full},
        {"name": "experts T=64", "op": "experts", "T": 64, **full},
        {"name": "experts T=4096", "op": "experts", "T": 4096, **full},
        # one projection of the routed experts: the up part of four decoding
        # requests, the down part of a training batch of 4096 tokens
        {"name": "grouped R=24", "op": "grouped", "R": 24, "pad": 0, "y": "bf16", **up},
        {"name": "grouped R=24576", "op": "grouped", "R": 24576, "pad": 0, "y": "bf16", **down},
        # training on 250 tokens in a buffer of 256, and on 4096 tokens
        {"name": "input_grad R=1500", "op": "input_grad", "R": 1500, "pad": 36, "y": "bf16", **up},
        {"name": "input_grad R=24576", "op": "input_grad", "R": 24576, "pad": 0, "y": "bf16", **up},
        # the weights' gradient: of a short batch in the weights' type, of 4096
        # tokens in float32 for an optimizer that keeps such gradients
        {"name": "weight_grad R=1500", "op": "weight_grad", "R": 1500, "pad": 36, "y": "bf16", **down},
        {"name": "weight_grad R=24576", "op": "weight_grad", "R": 24576, "pad": 0, "y": "f32", **down},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "experts", "grouped", "input_grad", "weight_grad"])
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 64, SHARED), "K": 16 * _log(rng, 4, H // 16),
                "y": rng.choice(["bf16", "f32"])}
    if op == "experts":
        return {"op": op, "T": _log(rng, 1, 4096), "H": 64 * _log(rng, 2, H // 64), "F": 64 * _log(rng, 1, F // 64),
                "E": 16 * rng.randint(1, E // 16), "k": rng.randint(1, K)}
    return {"op": op, "R": _log(rng, 1, 24576), "pad": rng.choice([0, 0, rng.randint(1, 300)]), "E": rng.randint(1, E),
            "N": 8 * _log(rng, 8, F // 8), "K": 8 * _log(rng, 8, H // 8), "y": rng.choice(["bf16", "f32"])}


# ---------------------------------------------------------------- plain pieces
def _codes(v):
    """(integer values in float32, scales [.., 1] in float32): one scale for each
    row of v (float32), amax / 127; a code is the integer nearest to value *
    float32(127 / amax), ties to even."""
    amax = v.abs().amax(-1, keepdim=True)
    live = amax >= 2.0 ** -100
    inv = torch.where(live, torch.full_like(amax, 127.0) / torch.where(live, amax, 1.0), 0.0)
    s = torch.where(live, amax / torch.full_like(amax, 127.0), 0.0)
    return torch.round(v.double() * inv.double()).float(), s


# ---------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _use_bias(g, e):
    """Bias of the router: experts are used unevenly (rank^-1/2)."""
    rank = torch.randperm(e, generator=g, device=g.device) + 1
    return -0.5 * torch.log(rank.float())


def _weights(g, e, n, k):
    """bf16 [e, n, k], ~N(0, 1 / fan-in)."""
    return torch.empty((e, n, k), dtype=torch.bfloat16, device="cuda").normal_(0, 1 / math.sqrt(k), generator=g)


def _inputs(c, seed):
    """What the inputs of a case are made of: tensors in the operator's types."""
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    if c["op"] == "linear":
        x = _randn(g, c["M"], c["K"])
        x[::10] *= 4.0  # outlier tokens
        return {"x": x.bfloat16(), "w": (_randn(g, c["N"], c["K"]) / math.sqrt(c["K"])).bfloat16()}
    if c["op"] == "experts":
        d = {"x": _randn(g, c["T"], c["H"]).bfloat16()}
        top, ids = (_randn(g, c["T"], c["E"]) + _use_bias(g, c["E"])).topk(c["k"], dim=1)
        d["ids"], d["gates"] = ids.int(), torch.softmax(top, 1)
        d["up"], d["down"] = _weights(g, c["E"], c["F"], c["H"]), _weights(g, c["E"], c["H"], c["F"])
        return d
    # rows by expert, as a router's picks fall; `pad` rows of no expert behind them
    share = torch.softmax(_use_bias(g, c["E"]), 0)
    picks = torch.multinomial(share, c["R"], replacement=True, generator=g)
    off = torch.zeros(c["E"] + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(picks, minlength=c["E"]).cumsum(0)
    d = {"offsets": off}
    rows = c["R"] + c["pad"]
    if c["op"] != "input_grad":
        d["x"] = _randn(g, rows, c["K"]).bfloat16()
    if c["op"] != "grouped":
        d["dy"] = (1e-2 * _randn(g, rows, c["N"])).bfloat16()
    if c["op"] != "weight_grad":
        d["w"] = _weights(g, c["E"], c["N"], c["K"])
    return d


def prepare(case, seed):
    """The inputs, and the weights as a serving program keeps them: packed by the
    library where `own` is true, as codes and scales otherwise.  Of the grouped
    products the row bounds on the host for the plain form's loop, and the buffer
    of the output (its rows of no expert stay as they are)."""
    c, d = case, _inputs(case, seed)
    d["case"] = c
    if c["op"] == "linear":
        if own:
            import sparse_moe_routed_amd as moe
            d["w"] = moe.channel_pack(d["w"])
            if c["M"] > moe.CHANNEL_FEW_ROWS:
                d["ws"] = moe.channel_linear_workspace(c["M"], c["K"])
        else:
            q, s = _codes(d["w"].float())
            d["w"] = (q.to(torch.int8), s)
        return d
    if c["op"] == "experts":
        if own:
            import sparse_moe_routed_amd as moe
            d["dims"] = moe.LayerDims(c["H"], c["F"], c["E"], c["k"])
            d["bank"] = moe.quantize_experts(d.pop("up"), d.pop("down"), "int8", d["dims"])
            d["ws"] = moe.workspace(d["dims"], "int8", c["T"])
        else:
            for p in ("up", "down"):
                got = [_codes(w.float()) for w in d[p].split(16)]
                d[p] = torch.cat([q.to(torch.int8) for q, _ in got])
                d[p + "_s"] = torch.cat([s for _, s in got])
        return d
    if not own:
        d["bounds"] = d["offsets"].tolist()
    rows, out = c["R"] + c["pad"], TYPES[c["y"]]
    shape = {"grouped": (rows, c["N"]), "input_grad": (rows, c["K"]), "weight_grad": (c["E"], c["N"], c["K"])}[c["op"]]
    d["out"] = torch.zeros(shape, dtype=out, device="cuda")
    return d


# ---------------------------------------------------------------- one pass
def run(state):
    return {"linear": _run_linear, "experts": _run_experts, "grouped": _run_grouped, "input_grad": _run_input_grad,
            "weight_grad": _run_weight_grad}[state["case"]["op"]](state)


def _run_linear(d):
    out = TYPES[d["case"]["y"]]
    if own:
        import sparse_moe_routed_amd as moe
        return moe.channel_linear(d["x"], d["w"], y_dtype=out, ws=d.get("ws"))
    q, s = d["w"]
    xq, xs = _codes(d["x"].float())
    return ((xq @ q.float().T) * xs * s.T).to(out)


def _run_experts(d):
    c = d["case"]
    if own:
        import sparse_moe_routed_amd as moe
        return moe.forward(d["x"], d["ids"], d["gates"], d["bank"], d["dims"], y_dtype=torch.bfloat16, ws=d["ws"])
    e, f, h, t, k = c["E"], c["F"], c["H"], c["T"], c["k"]
    xq, xs = _codes(d["x"].float())
    if t * k <= e:  # few rows: the weights of each row's expert
        r = d["ids"].reshape(-1).long()
        hid = torch.bmm(d["up"][r].float(), xq.repeat_interleave(k, 0).unsqueeze(2)).squeeze(2)
        hid = hid * xs.repeat_interleave(k, 0) * d["up_s"][r].squeeze(2)
        aq, a_s = _codes(hid.clamp_(min=0).square_().bfloat16().float())
        o = torch.bmm(d["down"][r].float(), aq.unsqueeze(2)).squeeze(2)
        o = (o * a_s * d["down_s"][r].squeeze(2)).view(t, k, h)
    else:  # every expert on every token; a token's slots are picked at the end
        up = (d["up"].float() * d["up_s"]).view(e * f, h)
        hid = (up @ (xq * xs).T).view(e, f, t).transpose(1, 2).contiguous()
        del up
        hid = hid.clamp_(min=0).square_().bfloat16()
        o = torch.empty((e, t, h), device="cuda")
        for i in range(e):
            aq, a_s = _codes(hid[i].float())
            torch.matmul(aq * a_s, d["down"][i].float().T * d["down_s"][i].T, out=o[i])
        o = o[d["ids"].long(), torch.arange(t, device="cuda").unsqueeze(1)]  # [T, k, H]
    return (o * d["gates"].unsqueeze(2)).sum(1).bfloat16()


def _groups(d):
    b = d["bounds"]
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1)]


def _run_grouped(d):
    if own:
        import sparse_moe_routed_amd as moe
        return moe.grouped_matmul(d["x"], d["w"], d["offsets"], y=d["out"])
    for e, a, b in _groups(d):
        if b > a:
            d["out"][a:b] = d["x"][a:b].float() @ d["w"][e].float().T
    return d["out"]


def _run_input_grad(d):
    if own:
        import sparse_moe_routed_amd as moe
        return moe.grouped_input_grad(d["dy"], d["w"], d["offsets"], dx=d["out"])
    for e, a, b in _groups(d):
        if b > a:
            d["out"][a:b] = d["dy"][a:b].float() @ d["w"][e].float()
    return d["out"]


def _run_weight_grad(d):
    if own:
        import sparse_moe_routed_amd as moe
        return moe.grouped_weight_grad(d["dy"], d["x"], d["offsets"], dw=d["out"])
    for e, a, b in _groups(d):
        d["out"][e] = d["dy"][a:b].float().T @ d["x"][a:b].float()
    return d["out"]


# ---------------------------------------------------------------- work
@functools.lru_cache(maxsize=None)
def _experts_used(e, tokens, k):
    """Distinct experts that the inputs' uneven use gives `tokens` tokens of k picks
    (the mean of eight samples; k = 0: picks one by one)."""
    g = torch.Generator()
    g.manual_seed(e * 1000003 + tokens * 11 + k)
    if k and tokens * k >= 40 * e:
        return e
    total = 0
    for _ in range(8):
        bias = _use_bias(g, e)
        if k:
            picks = (torch.randn((tokens, e), generator=g) + bias).topk(k, dim=1)[1]
        else:
            picks = torch.multinomial(torch.softmax(bias, 0), tokens, replacement=True, generator=g)
        total += torch.unique(picks).numel()
    return total / 8


def work(case):
    c = case
    if c["op"] == "linear":
        m, n, k = c["M"], c["N"], c["K"]
        return {"bytes": 2 * m * k + n * k + 4 * n + (2 if c["y"] == "bf16" else 4) * m * n, "flops": 2 * m * n * k}
    if c["op"] == "experts":
        t, h, f, e, k = c["T"], c["H"], c["F"], c["E"], c["k"]
        size = _experts_used(e, t, k) * (2 * f * h + 4 * (f + h)) + 2 * t * h + 2 * t * h + 8 * t * k
        return {"bytes": size, "flops": 4 * t * k * f * h}
    r, e, n, k = c["R"], c["E"], c["N"], c["K"]
    out = 2 if c["y"] == "bf16" else 4
    rows = 4 * (e + 1)
    if c["op"] == "grouped":
        rows += 2 * r * k + out * r * n
    elif c["op"] == "input_grad":
        rows += 2 * r * n + out * r * k
    else:
        rows += 2 * r * (n + k)
    weights = out * e * n * k if c["op"] == "weight_grad" else 2 * _experts_used(e, r, 0) * n * k
    return {"bytes": rows + weights, "flops": 2 * r * n * k}


# ---------------------------------------------------------------- in 64 bits
def _exact_rows(v):
    """Rows of v (float32) in 64 bits after 8-bit codes with a scale for each row;
    127 / amax and amax / 127 are float32 quotients, the format's definition."""
    top = v.abs().max(dim=-1, keepdim=True).values
    c127 = torch.tensor(127.0, device=v.device)
    keep = top >= 2.0 ** -100
    inv = torch.where(keep, c127 / top.clamp(min=2.0 ** -100), torch.zeros_like(top)).double()
    scale = torch.where(keep, top / c127, torch.zeros_like(top)).double()
    p = v.double() * inv
    n = torch.floor(p)
    part = p - n  # exact: the product has 32 significant bits
    n = n + ((part > 0.5) | ((part == 0.5) & (torch.remainder(n, 2.0) == 1.0))).double()
    return n * scale


def _bf16_once(v):
    """bf16 of float64 v rounded once: float32 with the lost part kept odd first."""
    f = v.float()
    off = f.double() != v
    low = torch.where(f.double().abs() > v.abs(), torch.nextafter(f, torch.zeros_like(f)), f)
    bits = low.view(torch.int32)
    return torch.where(off, bits | 1, bits).view(torch.float32).bfloat16().float()


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    if c["op"] == "linear":
        return _exact_rows(d["x"].float()) @ _exact_rows(d["w"].float()).t()
    if c["op"] == "experts":
        t, k = c["T"], c["k"]
        x = _exact_rows(d["x"].float())
        flat = d["ids"].reshape(-1).long()
        y = torch.zeros((t * k, c["H"]), dtype=torch.float64, device="cuda")
        for e in torch.unique(flat).tolist():
            r = (flat == e).nonzero().squeeze(1)
            h = x[r // k] @ _exact_rows(d["up"][e].float()).t()
            a = _bf16_once(h.clamp(min=0).square())
            y[r] = _exact_rows(a) @ _exact_rows(d["down"][e].float()).t()
        return (y.view(t, k, -1) * d["gates"].double().unsqueeze(2)).sum(1)
    rows, off = c["R"] + c["pad"], d["offsets"].tolist()
    shape = {"grouped": (rows, c["N"]), "input_grad": (rows, c["K"]), "weight_grad": (c["E"], c["N"], c["K"])}[c["op"]]
    out = torch.zeros(shape, dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        s = slice(off[e], off[e + 1])
        if s.start == s.stop:
            continue
        if c["op"] == "grouped":
            out[s] = d["x"][s].double() @ d["w"][e].double().t()
        elif c["op"] == "input_grad":
            out[s] = d["dy"][s].double() @ d["w"][e].double()
        else:
            out[e] = d["dy"][s].double().t() @ d["x"][s].double()
    return out
