"""Measured cases of the experts' feed-forward block on the expert-major slabs: the gated
up-projection with its activation (and a checkpoint of what the activation saw, in bf16 or in
8 bits), the down-projection, the gradient of the down-projection through the activation, the
gradient of the up-projection with respect to the rows, and the gradients of the weights.

An expert's rows lie one behind the other in its rank's slab, experts in ascending order; rows
past the slab's end are dropped. Each operator has a plain form (elementary torch operations in
fp32, experts of like numbers of rows batched, one rounding at the end) and, where `own` is
true, the call of this package. `exact` restates the definitions in 64 bits.

The 8-bit checkpoint holds E4M3 codes and one bf16 scale per 128 channels. Rows of a slab that
no expert owns are part of the outputs too and keep the zeros they were made with.
"""
import math

import torch

own = False

BLOCK = 128      # channels that share one scale of the 8-bit checkpoint
E4M3_MAX = 448.0
GELU_A, GELU_B = 1.5957691216057308, 0.044715  # gelu(v) = v * sigmoid(GELU_A * (v + GELU_B * v^3)), the tanh form


# --------------------------------------------------------------------------- cases

def _case(name, op, T, H, F, E, k, R, skew, empty, room, **more):
    # H: the model's width; F: an expert's; skew: exponent of the experts' popularity; empty: share of
    # top-k slots that hold -1; room: rows of a rank's slab over its mean load
    return {"name": name, "op": op, "T": T, "H": H, "F": F, "E": E, "k": k, "R": R, "skew": skew, "empty": empty,
            "room": room, **more}


def listed():
    return [
        # one decoded token through eight experts' up-projections: the weights' stream
        _case("gate_up_token", "gate_up", 1, 7168, 2048, 256, 8, 32, 0.0, 0.0, 32.0, act="silu", save="none"),
        # a decode batch: a few rows for every expert
        _case("gate_up_decode", "gate_up", 128, 7168, 2048, 256, 8, 32, 0.0, 0.0, 2.0, act="silu", save="none"),
        # a training batch with the 8-bit checkpoint
        _case("gate_up_batch", "gate_up", 4096, 7168, 2048, 256, 8, 32, 0.0, 0.0, 1.25, act="silu", save="8bit"),
        # a training batch of uneven popularity, many rows an expert, the checkpoint in bf16
        _case("gate_up_skewed", "gate_up", 16384, 4096, 2048, 128, 8, 64, 1.2, 0.0, 2.0, act="gelu", save="bf16"),
        # the way back for one decoded token
        _case("down_token", "down", 1, 7168, 2048, 256, 8, 32, 0.0, 0.0, 32.0),
        # the way back of a training or prompt batch
        _case("down_batch", "down", 4096, 7168, 2048, 256, 8, 32, 0.0, 0.0, 1.25),
        # gradient through the activation of a small batch: latency
        _case("down_bwd_small", "down_bwd", 127, 1024, 512, 16, 4, 4, 0.0, 0.0, 1.5, act="gelu", save="bf16"),
        # gradient through the activation of a training batch, from the 8-bit checkpoint
        _case("down_bwd_batch", "down_bwd", 4096, 7168, 2048, 256, 8, 32, 0.0, 0.0, 1.25, act="silu", save="8bit"),
        # gradient of the rows: ragged widths, empty slots, slabs too small for the hottest ranks
        _case("gate_up_bwd_ragged", "gate_up_bwd", 777, 1032, 1000, 64, 6, 16, 1.2, 0.15, 1.5),
        # gradient of the rows, many rows an expert
        _case("gate_up_bwd_skewed", "gate_up_bwd", 16384, 4096, 2048, 128, 8, 64, 1.2, 0.0, 2.0),
        # gradient of the weights: a small ragged batch, experts without rows among the others
        _case("wgrad_small", "wgrad", 130, 1000, 328, 32, 4, 4, 0.8, 0.2, 1.5, of="down"),
        # gradient of the up-projection's weights, many rows an expert
        _case("wgrad_skewed", "wgrad", 16384, 4096, 2048, 128, 8, 64, 1.2, 0.0, 2.0, of="gate_up"),
    ]


_MOST_BYTES, _MOST_FLOPS = 15e9, 2.2e12  # of one pass of a drawn case, below the largest listed ones'


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["gate_up", "gate_up", "down", "down_bwd", "gate_up_bwd", "wgrad"])
        H, F = 8 * _log_int(rng, 8, 1024), 8 * _log_int(rng, 4, 512)
        E = rng.choice([1, 8, 16, 32, 64, 96, 128, 160, 256])
        k = rng.randint(1, min(E, 10))
        R = rng.choice([r for r in (1, 4, 8, 16, 32) if E % r == 0])
        T = _log_int(rng, 1, 16384)
        more = {}
        if op in ("gate_up", "down_bwd"):
            more = {"act": rng.choice(["silu", "gelu"]), "save": rng.choice(["bf16", "8bit"])}
            if op == "gate_up" and rng.random() < 0.5:
                more["save"] = "none"
            if more["save"] == "8bit":
                F = BLOCK * _log_int(rng, 1, 32)
        elif op == "wgrad":
            more = {"of": rng.choice(["gate_up", "down"])}
        case = _case("", op, T, H, F, E, k, R, rng.choice([0.0, 0.0, 0.8, 1.2]), rng.choice([0.0, 0.0, 0.1]),
                     1.0 if R == 1 else rng.choice([1.25, 1.5, 2.0]), **more)
        w = work(case)
        if w["bytes"] <= _MOST_BYTES and w["flops"] <= _MOST_FLOPS and 2 * 3 * E * F * H <= 24e9:
            del case["name"]
            return case


def _expected(case):
    """Rows that the slabs hold and experts that have any, on average."""
    T, E, k, R = case["T"], case["E"], case["k"], case["R"]
    p = [(i + 1.0) ** -case["skew"] for i in range(E)]
    hit = [min(1.0, k * v / sum(p)) for v in p]
    for _ in range(20):  # no expert twice in a token: what the hottest cannot take, the others do
        scale = k / sum(hit)
        hit = [min(1.0, h * scale) for h in hit]
    hit = [h * (1.0 - case["empty"]) for h in hit]
    rows = T * sum(hit) if R == 1 else min(T * sum(hit), case["room"] * T * k)
    return rows, sum(1.0 - (1.0 - h) ** T for h in hit)


def work(case):
    H, F, E = case["H"], case["F"], case["E"]
    rows, experts = _expected(case)
    op = case["op"]
    saved = {"none": 0, "bf16": 4 * F, "8bit": 2 * F + 4 * (F // BLOCK)}.get(case.get("save"), 0)
    if op == "gate_up":
        n, flops = 4 * experts * F * H + rows * (2 * H + 2 * F + saved), 4 * rows * H * F
    elif op == "down":
        n, flops = 2 * experts * F * H + rows * (2 * F + 2 * H), 2 * rows * H * F
    elif op == "down_bwd":
        n, flops = 2 * experts * F * H + rows * (2 * H + saved + 4 * F + 2 * F), 2 * rows * H * F
    elif op == "gate_up_bwd":
        n, flops = 4 * experts * F * H + rows * (4 * F + 2 * H), 4 * rows * H * F
    else:
        width = 2 * F if case["of"] == "gate_up" else F
        n, flops = 2 * E * width * H + rows * 2 * (width + H), 2 * rows * width * H
    return {"bytes": int(n + 4 * (E + 1)), "flops": int(flops)}


# --------------------------------------------------------------------------- inputs

def _normal(gen, shape, scale=1.0):
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    return t.mul_(scale) if scale != 1.0 else t


def _offsets(case, gen):
    """First row of every expert, all ranks' rows counted through: distinct experts per token
    (Gumbel top-k over the experts' popularity)."""
    T, E, k = case["T"], case["E"], case["k"]
    perm = torch.randperm(E, generator=gen, device="cuda")
    logp = -case["skew"] * torch.log(perm.float() + 1.0)
    gumbel = -torch.log(-torch.log(torch.rand((T, E), generator=gen, device="cuda").clamp(1e-20, 1 - 1e-7)))
    idx = torch.topk(logp + gumbel, k, dim=1).indices
    idx = torch.where(torch.rand((T, k), generator=gen, device="cuda") < case["empty"], E, idx)
    counts = torch.bincount(idx.reshape(-1), minlength=E + 1)[:E]
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


_AT_ONCE = 1 << 29  # elements of the weights that a group of experts of the plain form may have


def _groups(offsets, E, R, rows, weights):
    """The plain form's plan: experts of like numbers of rows, so that a group is one batched product. Of
    each group: its experts, the slab rows of each one (padded by its first row), which of them are
    there, their places among all of the group's, and the slab rows that these stand for."""
    o, per = offsets.tolist(), E // R
    spans = []
    for e in range(E):
        first = o[e] - o[e // per * per]
        n = min(first + o[e + 1] - o[e], rows) - first
        if n > 0:
            spans.append((n, e, e // per * rows + first))
    spans.sort(key=lambda v: (-v[0], v[1]))
    groups = []
    while spans:
        most = spans[0][0]
        n = sum(2 * v[0] > most for v in spans)
        n = max(1, min(n, _AT_ONCE // weights))
        size, expert, first = torch.tensor(spans[:n], device=offsets.device).unbind(1)
        spans = spans[n:]
        i = torch.arange(most, device=offsets.device)
        there = i < size[:, None]
        row = first[:, None] + torch.where(there, i, 0)
        at = there.view(-1).nonzero()[:, 0]
        groups.append({"experts": expert, "rows": row, "there": there, "at": at, "to": row.view(-1)[at]})
    return groups


def _checkpoint(pre, save):
    """What the up-projection kept of its sums: bf16, or codes and scales."""
    if save == "bf16":
        return {"pre": pre, "pre_q": None, "pre_scales": None}
    blocks = pre.float().view(*pre.shape[:-1], -1, BLOCK)
    scales = (blocks.abs().amax(-1) / E4M3_MAX).to(torch.bfloat16)
    divisor = torch.where(scales > 0, scales.float(), 1.0)[..., None]
    q = (blocks / divisor).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(pre.shape)
    return {"pre": None, "pre_q": q, "pre_scales": scales}


def _zeros(shape, dtype):
    return torch.zeros(shape, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device="cuda").view(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, T, H, F, E, k, R = (case[n] for n in ("op", "T", "H", "F", "E", "k", "R"))
    rows = math.ceil(case["room"] * T * k / R)
    bf16 = torch.bfloat16
    s = {"op": op, "H": H, "F": F, "E": E, "R": R, "rows": rows, "act": case.get("act"),
         "offsets": _offsets(case, gen), "status": _zeros((1,), torch.int32)}
    # what a plain program keeps from sizing its slabs
    s["groups"] = _groups(s["offsets"], E, R, rows, (1 if case.get("of", op).startswith("down") else 2) * F * H)
    if op == "gate_up":
        s["x"] = _normal(gen, (R, rows, H))
        s["w_gate_up"] = _normal(gen, (E, 2 * F, H), H ** -0.5)
        s["h"] = _zeros((R, rows, F), bf16)
        s["pre"] = _zeros((R, rows, 2 * F), bf16) if case["save"] == "bf16" else None
        s["pre_q"] = _zeros((R, rows, 2 * F), torch.float8_e4m3fn) if case["save"] == "8bit" else None
        s["pre_scales"] = _zeros((R, rows, 2 * F // BLOCK), bf16) if case["save"] == "8bit" else None
    elif op == "down":
        s["h"] = _normal(gen, (R, rows, F), 0.5)
        s["w_down"] = _normal(gen, (E, H, F), F ** -0.5)
        s["y"] = _zeros((R, rows, H), bf16)
    elif op == "down_bwd":
        s["dy"] = _normal(gen, (R, rows, H), 0.02)
        s["w_down"] = _normal(gen, (E, H, F), F ** -0.5)
        s.update(_checkpoint(_normal(gen, (R, rows, 2 * F), 1.0), case["save"]))
        s["dpre"] = _zeros((R, rows, 2 * F), bf16)
        s["h"] = _zeros((R, rows, F), bf16)
    elif op == "gate_up_bwd":
        s["dpre"] = _normal(gen, (R, rows, 2 * F), 0.02)
        s["w_gate_up"] = _normal(gen, (E, 2 * F, H), H ** -0.5)
        s["dx"] = _zeros((R, rows, H), bf16)
    else:
        n, m = (2 * F, H) if case["of"] == "gate_up" else (H, F)
        s["dout"] = _normal(gen, (R, rows, n), 0.02)
        s["in"] = _normal(gen, (R, rows, m))
        s["dw"] = _zeros((E, n, m), bf16)
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _gate(act, v):
    """sigmoid(p(v)) and the derivative of p, for the activation v * sigmoid(p(v))"""
    if act == "silu":
        return 1.0 / (1.0 + torch.exp(-v)), 1.0
    return 1.0 / (1.0 + torch.exp(-GELU_A * (v + GELU_B * v * v * v))), GELU_A * (1.0 + 3.0 * GELU_B * v * v)


def _rows(t, g):
    """The rows of a group's experts in fp32: [experts][most rows][width]."""
    return t.view(-1, t.shape[-1])[g["rows"]].float()


def _put(t, g, v):
    """Rows of a group back into their slabs, rounded."""
    t.view(-1, t.shape[-1])[g["to"]] = v.to(t.dtype)


def _plain_gate_up(s):
    F = s["F"]
    out = {n: torch.zeros_like(s[n]) for n in ("h", "pre", "pre_q", "pre_scales") if s[n] is not None}
    for g in s["groups"]:
        pre = torch.bmm(_rows(s["x"], g), s["w_gate_up"][g["experts"]].float().transpose(1, 2))
        pre = pre.view(-1, 2 * F)[g["at"]]
        gate, up = pre[:, :F], pre[:, F:]
        sig, _ = _gate(s["act"], gate)
        _put(out["h"], g, gate * sig * up)
        if s["pre"] is not None:
            _put(out["pre"], g, pre)
        if s["pre_q"] is not None:
            kept = _checkpoint(pre, "8bit")
            _put(out["pre_q"].view(torch.uint8), g, kept["pre_q"].view(torch.uint8))
            _put(out["pre_scales"], g, kept["pre_scales"])
    return out


def _plain_down(s):
    y = torch.zeros_like(s["y"])
    for g in s["groups"]:
        v = torch.bmm(_rows(s["h"], g), s["w_down"][g["experts"]].float().transpose(1, 2))
        _put(y, g, v.view(-1, s["H"])[g["at"]])
    return {"y": y}


def _plain_down_bwd(s):
    F = s["F"]
    dpre, h = torch.zeros_like(s["dpre"]), torch.zeros_like(s["h"])
    for g in s["groups"]:
        dh = torch.bmm(_rows(s["dy"], g), s["w_down"][g["experts"]].float()).view(-1, F)[g["at"]]
        if s["pre"] is not None:
            pre = s["pre"].view(-1, 2 * F)[g["to"]].float()
        else:
            q = s["pre_q"].view(-1, 2 * F // BLOCK, BLOCK).view(torch.uint8)[g["to"]].view(torch.float8_e4m3fn)
            pre = (q.float() * s["pre_scales"].view(-1, 2 * F // BLOCK)[g["to"]].float()[..., None]).view(-1, 2 * F)
        gate, up = pre[:, :F], pre[:, F:]
        sig, slope = _gate(s["act"], gate)
        dgate, dup = dh * up * (sig + gate * sig * (1.0 - sig) * slope), dh * (gate * sig)
        _put(dpre, g, torch.cat([dgate, dup], dim=1))
        _put(h, g, gate * sig * up)
    return {"dpre": dpre, "h": h}


def _plain_gate_up_bwd(s):
    dx = torch.zeros_like(s["dx"])
    for g in s["groups"]:
        v = torch.bmm(_rows(s["dpre"], g), s["w_gate_up"][g["experts"]].float())
        _put(dx, g, v.view(-1, s["H"])[g["at"]])
    return {"dx": dx}


def _plain_wgrad(s):
    dw = torch.zeros_like(s["dw"])
    for g in s["groups"]:
        dout = _rows(s["dout"], g) * g["there"][:, :, None]
        dw[g["experts"]] = torch.bmm(dout.transpose(1, 2), _rows(s["in"], g)).to(dw.dtype)
    return {"dw": dw}


_plain = {"gate_up": _plain_gate_up, "down": _plain_down, "down_bwd": _plain_down_bwd,
          "gate_up_bwd": _plain_gate_up_bwd, "wgrad": _plain_wgrad}


def _act(ep, s):
    return {"silu": ep.ACT_SILU, "gelu": ep.ACT_GELU}[s["act"]]


def _own_gate_up(s):
    import combine_ep_get_05_gb300 as ep

    ep.ep_expert_gate_up(s["x"], s["w_gate_up"], s["offsets"], _act(ep, s), s["h"], s["pre"], s["pre_q"],
                         s["pre_scales"], s["status"])
    return {n: s[n] for n in ("h", "pre", "pre_q", "pre_scales") if s[n] is not None}


def _own_down(s):
    import combine_ep_get_05_gb300 as ep

    ep.ep_expert_down(s["h"], s["w_down"], s["offsets"], s["y"], s["status"])
    return {"y": s["y"]}


def _own_down_bwd(s):
    import combine_ep_get_05_gb300 as ep

    ep.ep_expert_down_bwd(s["dy"], s["w_down"], s["pre"], s["pre_q"], s["pre_scales"], s["offsets"], _act(ep, s),
                          s["dpre"], s["h"], s["status"])
    return {"dpre": s["dpre"], "h": s["h"]}


def _own_gate_up_bwd(s):
    import combine_ep_get_05_gb300 as ep

    ep.ep_expert_gate_up_bwd(s["dpre"], s["w_gate_up"], s["offsets"], s["dx"], s["status"])
    return {"dx": s["dx"]}


def _own_wgrad(s):
    import combine_ep_get_05_gb300 as ep

    ep.ep_expert_wgrad(s["dout"], s["in"], s["offsets"], s["dw"], s["status"])
    return {"dw": s["dw"]}


_own = {"gate_up": _own_gate_up, "down": _own_down, "down_bwd": _own_down_bwd, "gate_up_bwd": _own_gate_up_bwd,
        "wgrad": _own_wgrad}


# --------------------------------------------------------------------------- 64 bits

def _exact_act(act, v):
    """The activation and its derivative."""
    if act == "silu":
        sig = torch.sigmoid(v)
        return v * sig, sig * (1.0 + v * (1.0 - sig))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * v * v)


def exact(case, seed):
    if work(case)["flops"] > 1.2e13:  # 64-bit products run at about a TFLOP/s
        return None
    s = prepare(case, seed)
    op, F, E, R = case["op"], case["F"], case["E"], case["R"]
    o, per = s["offsets"].cpu().long(), E // R
    base = o[:-1].view(R, per)[:, :1]
    first = (o[:-1].view(R, per) - base).clamp(max=s["rows"]).view(-1).tolist()
    after = (o[1:].view(R, per) - base).clamp(max=s["rows"]).view(-1).tolist()

    def made(name):
        return torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")

    def of(name, e):
        return s[name][e // per].narrow(0, first[e], after[e] - first[e])

    def put(t, e, v):
        t[e // per].narrow(0, first[e], after[e] - first[e]).copy_(v)

    outputs = {"gate_up": ("h", "pre", "pre_q", "pre_scales"), "down": ("y",), "down_bwd": ("dpre", "h"),
               "gate_up_bwd": ("dx",), "wgrad": ("dw",)}[op]
    out = {n: made(n) for n in outputs if s[n] is not None}
    for e in range(E):
        if after[e] == first[e]:
            continue
        if op == "gate_up":
            gate, up = torch.einsum("th,cfh->ctf", of("x", e).double(),
                                    s["w_gate_up"][e].double().view(2, F, -1)).unbind(0)
            put(out["h"], e, _exact_act(case["act"], gate)[0] * up)
            pre = torch.cat([gate, up], dim=1)
            if case["save"] == "bf16":
                put(out["pre"], e, pre)
            elif case["save"] == "8bit":  # before the roundings, the codes' at the scale that is kept
                scales = torch.stack([c.abs().max(1).values for c in pre.split(BLOCK, dim=1)], dim=1) / 448.0
                kept = scales.to(torch.bfloat16).double().repeat_interleave(BLOCK, dim=1)
                put(out["pre_q"], e, (pre / kept).clamp(-448.0, 448.0))
                put(out["pre_scales"], e, scales)
        elif op == "down":
            put(out["y"], e, torch.einsum("tf,hf->th", of("h", e).double(), s["w_down"][e].double()))
        elif op == "down_bwd":
            dh = torch.einsum("th,hf->tf", of("dy", e).double(), s["w_down"][e].double())
            if case["save"] == "bf16":
                pre = of("pre", e).double()
            else:
                pre = of("pre_q", e).double().view(-1, 2 * F // BLOCK, BLOCK)
                pre = (pre * of("pre_scales", e).double()[:, :, None]).view(-1, 2 * F)
            gate, up = pre.split(F, dim=1)
            a, da = _exact_act(case["act"], gate)
            put(out["dpre"], e, torch.cat([dh * up * da, dh * a], dim=1))
            put(out["h"], e, a * up)
        elif op == "gate_up_bwd":
            put(out["dx"], e, torch.einsum("tf,fh->th", of("dpre", e).double(), s["w_gate_up"][e].double()))
        else:
            out["dw"][e] = torch.einsum("tn,tm->nm", of("dout", e).double(), of("in", e).double())
    return out
