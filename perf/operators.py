"""Measured cases of the operators around the expert-major path: the residual's
addition with the root-mean-square norm (bf16 and E4M3 outputs) and its gradient,
E4M3 rows sorted by expert, the gradient of the sort, and the gradient of the
weighted return from expert order.

Each operator has a plain form (elementary torch operations in fp32, one rounding
at the end) and, where `own` is true, the call of this package. `exact` restates the
definitions in 64 bits.

Outputs held in E4M3 are float8_e4m3fn tensors next to their fp32 scales; rows of a
slab that no token is sent to are part of the outputs too and keep the zeros they
were made with.
"""
import math

import torch

own = False

BLOCK = 128      # channels that share one E4M3 scale
E4M3_MAX = 448.0
EPS = 1e-6


# --------------------------------------------------------------------------- cases

def _norm(name, T, H, carry, residual, outputs, weight):
    return {"name": name, "op": "norm", "T": T, "H": H, "carry": carry, "residual": residual, "outputs": outputs,
            "weight": weight}


def _norm_bwd(name, T, H, carry, residual, weight):
    return {"name": name, "op": "norm_bwd", "T": T, "H": H, "carry": carry, "residual": residual, "weight": weight}


def _route(name, op, T, H, E, k, R, skew, empty, room, **more):
    # skew: exponent of the experts' popularity; empty: share of top-k slots that hold -1;
    # room: rows of a rank's slab over its mean load (rows past the slab's end are dropped)
    return {"name": name, "op": op, "T": T, "H": H, "E": E, "k": k, "R": R, "skew": skew, "empty": empty,
            "room": room, **more}


def listed():
    return [
        # one decoded token in front of an expert layer: the launch's latency
        _norm("norm_token", 1, 7168, "bf16", True, "yq", "bf16"),
        # a decode batch; the residual stream kept in fp32
        _norm("norm_decode", 128, 7168, "f32", True, "yq", "f32"),
        # a prompt or training batch: bf16 rows for the router, E4M3 rows for the dispatch
        _norm("norm_batch", 4096, 7168, "bf16", True, "yq", "bf16"),
        # the norm without a residual and without E4M3, a ragged width
        _norm("norm_ragged", 8191, 4104, "f32", False, "y", "f32"),
        # gradient for a small batch, fp32 stream
        _norm_bwd("norm_bwd_small", 127, 1024, "f32", True, "f32"),
        # gradient for a training batch
        _norm_bwd("norm_bwd_batch", 4096, 7168, "bf16", True, "bf16"),
        # E4M3 rows of a decode batch into expert order, layout included
        _route("sort_q_decode", "sort_q_ll", 128, 7168, 256, 8, 32, 0.0, 0.0, 2.0),
        # E4M3 rows of a training or prompt batch, layout at hand
        _route("sort_q_batch", "sort_q", 4096, 7168, 256, 8, 32, 0.0, 0.0, 1.25),
        # gradient of the sort: a small ragged batch with empty slots, with the router's gradient of x
        _route("sort_bwd_small", "sort_bwd", 130, 1000, 16, 4, 4, 0.0, 0.2, 1.5, add=True),
        # gradient of the sort on one rank, popularity as uneven as the skewed workload's
        _route("sort_bwd_skewed", "sort_bwd", 16384, 4096, 128, 8, 1, 1.2, 0.0, 1.0, add=True),
        # gradient of the weighted return: ragged, empty slots, slabs too small for the hottest ranks
        _route("return_bwd_ragged", "return_bwd", 777, 1032, 64, 6, 16, 1.2, 0.15, 1.5),
        # gradient of the weighted return of a training batch
        _route("return_bwd_batch", "return_bwd", 4096, 7168, 256, 8, 32, 0.0, 0.0, 1.25),
    ]


_COSTLIEST = 0.95e9  # bytes of one pass of a drawn case, below the largest listed one's


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm_bwd", "sort_q", "sort_q_ll", "sort_bwd", "return_bwd"])
        H = 8 * _log_int(rng, 8, 1024)
        if op in ("sort_q", "sort_q_ll"):
            H = BLOCK * _log_int(rng, 1, 64)
        if op == "norm":
            outputs = rng.choice(["y", "q", "yq"])
            if outputs != "y":
                H = BLOCK * _log_int(rng, 1, 64)
            case = _norm("", _log_int(rng, 1, 16384), H, rng.choice(["bf16", "f32"]), rng.random() < 0.8, outputs,
                         rng.choice(["bf16", "f32"]))
        elif op == "norm_bwd":
            case = _norm_bwd("", _log_int(rng, 1, 16384), H, rng.choice(["bf16", "f32"]), rng.random() < 0.8,
                             rng.choice(["bf16", "f32"]))
        else:
            k = rng.randint(1, 10)
            E = rng.choice([16, 32, 64, 96, 128, 160, 256, 512])
            R = rng.choice([r for r in (1, 4, 8, 16, 32) if E % r == 0])
            T = _log_int(rng, 1, 800 if op == "sort_q_ll" else 16384)
            case = _route("", op, T, H, E, k, R, rng.choice([0.0, 0.0, 0.8, 1.2]), rng.choice([0.0, 0.0, 0.1]),
                          1.0 if R == 1 else rng.choice([1.25, 1.5, 2.0]))
            if op == "sort_bwd":
                case["add"] = rng.random() < 0.5
        if H != 3072 and work(case)["bytes"] <= _COSTLIEST:
            del case["name"]
            return case


def work(case):
    T, H = case["T"], case["H"]
    carry = 4 if case.get("carry") == "f32" else 2
    w = 4 if case.get("weight") == "f32" else 2
    if case["op"] == "norm":
        n = 2 * T * H + w * H                                        # x, weight
        n += 2 * carry * T * H if case["residual"] else 0            # the stream in and out
        n += 2 * T * H if "y" in case["outputs"] else 0
        n += T * H + 4 * T * (H // BLOCK) if "q" in case["outputs"] else 0
        return {"bytes": n, "flops": 8 * T * H}
    if case["op"] == "norm_bwd":
        n = (2 + carry) * T * H + w * H                              # dy, z, weight
        n += carry * T * H if case["residual"] else 0                # the stream's gradient in
        n += carry * T * H + 4 * H + (2 * T * H if carry == 4 else 0)  # dz, dweight, dx
        return {"bytes": n, "flops": 14 * T * H}
    E, k = case["E"], case["k"]
    rows = T * k * (1.0 - case["empty"])
    routing = T * k * (8 + 4) + 4 * (E + 1)                          # ids, slots, offsets
    if case["op"] in ("sort_q", "sort_q_ll"):
        row = H + 4 * (H // BLOCK)
        return {"bytes": int(T * row + rows * (row + 8) + 4 * T * k + routing), "flops": 0}
    if case["op"] == "sort_bwd":
        return {"bytes": int(2 * rows * H + 4 * rows + 2 * T * H * (2 if case["add"] else 1) + 4 * T * k + routing),
                "flops": int(rows * H)}
    return {"bytes": int(4 * rows * H + 2 * T * H + 8 * T * k + routing), "flops": int(3 * rows * H)}


# --------------------------------------------------------------------------- inputs

def _normal(gen, shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _activations(gen, T, H, scale, dtype):
    """Rows as a residual stream has them: channels of different magnitude, tokens too."""
    channel = torch.exp(0.5 * torch.randn(H, generator=gen, device="cuda"))
    token = torch.exp(0.3 * torch.randn((T, 1), generator=gen, device="cuda"))
    return (torch.randn((T, H), generator=gen, device="cuda") * channel * token * scale).to(dtype)


def _routing(case, gen):
    """Distinct experts per token (Gumbel top-k over the experts' popularity), weights that
    sum to 1 over the token's slots, and the expert layout of the batch."""
    T, E, k = case["T"], case["E"], case["k"]
    perm = torch.randperm(E, generator=gen, device="cuda")
    logp = -case["skew"] * torch.log(perm.float() + 1.0)
    gumbel = -torch.log(-torch.log(torch.rand((T, E), generator=gen, device="cuda").clamp(1e-20, 1 - 1e-7)))
    idx = torch.topk(logp + gumbel, k, dim=1).indices
    idx = torch.where(torch.rand((T, k), generator=gen, device="cuda") < case["empty"], -1, idx)
    w = torch.softmax(_normal(gen, (T, k)), dim=1)
    w = torch.where(idx >= 0, w, 0.0).contiguous()

    flat = idx.reshape(-1)
    key = torch.where(flat >= 0, flat, E)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    slot = torch.where(flat >= 0, place - offsets[flat.clamp(min=0)], -1).reshape(T, k)
    return idx.contiguous(), w, offsets.to(torch.int32), slot.to(torch.int32).contiguous()


def _quantised(gen, T, H):
    """E4M3 rows as the norm hands them over: every block's largest code is +-448."""
    q = (torch.randn((T, H), generator=gen, device="cuda") * 120.0).clamp(-E4M3_MAX, E4M3_MAX)
    scales = torch.exp(0.5 * torch.randn((T, H // BLOCK), generator=gen, device="cuda")) / E4M3_MAX * 4.0
    return q.to(torch.float8_e4m3fn), scales


def _zeros(shape, dtype):
    return torch.zeros(shape, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device="cuda").view(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, H, op = case["T"], case["H"], case["op"]
    s = {"op": op, "T": T, "H": H}
    carry = torch.float32 if case.get("carry") == "f32" else torch.bfloat16
    if op in ("norm", "norm_bwd"):
        wdt = torch.float32 if case["weight"] == "f32" else torch.bfloat16
        s["weight"] = (1.0 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(wdt)
        s["carry"] = carry
    if op == "norm":
        s["x"] = _activations(gen, T, H, 0.7, torch.bfloat16)
        s["residual"] = _activations(gen, T, H, 2.0, carry) if case["residual"] else None
        s["residual_out"] = _zeros((T, H), carry) if case["residual"] else None
        s["y"] = _zeros((T, H), torch.bfloat16) if "y" in case["outputs"] else None
        s["y_q"] = _zeros((T, H), torch.float8_e4m3fn) if "q" in case["outputs"] else None
        s["y_scales"] = _zeros((T, H // BLOCK), torch.float32) if "q" in case["outputs"] else None
        return s
    if op == "norm_bwd":
        s["dy"] = _normal(gen, (T, H), 0.02, torch.bfloat16)
        s["z"] = _activations(gen, T, H, 2.0, carry)
        s["dz_in"] = _normal(gen, (T, H), 0.03, carry) if case["residual"] else None
        s["dz"] = _zeros((T, H), carry)
        s["dx"] = _zeros((T, H), torch.bfloat16) if carry == torch.float32 else None
        s["dweight"] = _zeros((H,), torch.float32)
        s["workspace"] = None  # made by the first pass that needs one and kept
        return s
    idx, w, offsets, slot = _routing(case, gen)
    E, k, R = case["E"], case["k"], case["R"]
    rows = math.ceil(case["room"] * T * k / R)
    s.update(topk_idx=idx, topk_w=w, E=E, k=k, R=R, rows=rows, status=_zeros((1,), torch.int32))
    if op == "sort_q_ll":
        s.update(offsets=_zeros((E + 1,), torch.int32), slot=_zeros((T, k), torch.int32))
    else:
        s.update(offsets=offsets, slot=slot)
    if op in ("sort_q", "sort_q_ll"):
        s["x_q"], s["x_scales"] = _quantised(gen, T, H)
        s["perm_q"] = _zeros((R, rows, H), torch.float8_e4m3fn)
        s["perm_scales"] = _zeros((R, rows, H // BLOCK), torch.float32)
        s["perm_src"] = _zeros((R, rows), torch.int32)
        s["perm_w"] = _zeros((R, rows), torch.float32)
    elif op == "sort_bwd":
        s["dperm_x"] = _normal(gen, (R, rows, H), 0.02, torch.bfloat16)
        s["dperm_w"] = _normal(gen, (R, rows), 0.5)
        s["dx_in"] = _normal(gen, (T, H), 0.01, torch.bfloat16) if case["add"] else None
        s["dx"] = _zeros((T, H), torch.bfloat16)
        s["dtopk_w"] = _zeros((T, k), torch.float32)
    else:
        s["dout"] = _normal(gen, (T, H), 0.02, torch.bfloat16)
        s["y"] = _normal(gen, (R, rows, H), 1.0, torch.bfloat16)
        s["dy"] = _zeros((R, rows, H), torch.bfloat16)
        s["dtopk_w"] = _zeros((T, k), torch.float32)
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _plain_norm(s):
    z = s["x"].float()
    if s["residual"] is not None:
        z = z + s["residual"].float()
    v = z * torch.rsqrt((z * z).mean(1, keepdim=True) + EPS) * s["weight"].float()
    out = {}
    if s["residual"] is not None:
        out["residual_out"] = z.to(s["carry"])
    if s["y"] is not None:
        out["y"] = v.to(torch.bfloat16)
    if s["y_q"] is not None:
        blocks = v.view(s["T"], s["H"] // BLOCK, BLOCK)
        scales = blocks.abs().amax(2) / E4M3_MAX
        q = blocks / torch.where(scales > 0, scales, 1.0)[:, :, None]
        out["y_q"], out["y_scales"] = q.to(torch.float8_e4m3fn).view(s["T"], s["H"]), scales
    return out


def _plain_norm_bwd(s):
    z, dy = s["z"].float(), s["dy"].float()
    r = torch.rsqrt((z * z).mean(1, keepdim=True) + EPS)
    g = dy * s["weight"].float()
    dz = r * g - z * (r * r * r * (g * z).mean(1, keepdim=True))
    if s["dz_in"] is not None:
        dz = dz + s["dz_in"].float()
    out = {"dz": dz.to(s["carry"]), "dweight": (dy * z * r).sum(0)}
    if s["dx"] is not None:
        out["dx"] = dz.to(torch.bfloat16)
    return out


def _rows_of(s, offsets, slot):
    """Row of every (token, slot) in the slabs seen as one array; the row after the last
    stands for entries that were not sent."""
    per_rank = s["E"] // s["R"]
    e = s["topk_idx"].clamp(min=0)
    rank = e // per_rank
    p = offsets.long()[e] - offsets.long()[rank * per_rank] + slot
    sent = (slot >= 0) & (p < s["rows"])
    return torch.where(sent, rank * s["rows"] + p, s["R"] * s["rows"]), sent


def _plain_layout(s):
    flat = s["topk_idx"].reshape(-1)
    hit = (flat[:, None] == torch.arange(s["E"], device=flat.device)).to(torch.int32)
    upto = hit.cumsum(0, dtype=torch.int32)
    offsets = torch.cat([upto.new_zeros(1), upto[-1].cumsum(0, dtype=torch.int32)])
    slot = torch.where(flat >= 0, upto.gather(1, flat.clamp(min=0)[:, None])[:, 0] - 1, -1)
    return offsets, slot.view(s["T"], s["k"])


def _scattered(s, rows, values, like):
    """values[t][j] (or values[t]) into its row of zeroed slabs shaped as `like`."""
    flat = torch.zeros((s["R"] * s["rows"] + 1,) + tuple(like.shape[2:]), dtype=values.dtype, device=values.device)
    flat[rows] = values
    return flat[:-1].view(like.shape)


def _plain_sort_q(s):
    offsets, slot = (s["offsets"], s["slot"]) if s["op"] == "sort_q" else _plain_layout(s)
    rows, _ = _rows_of(s, offsets, slot)
    token = torch.arange(s["T"], dtype=torch.int32, device=rows.device)
    out = {"perm_q": _scattered(s, rows, s["x_q"].view(torch.uint8)[:, None], s["perm_q"]).view(torch.float8_e4m3fn),
           "perm_scales": _scattered(s, rows, s["x_scales"][:, None], s["perm_scales"]),
           "perm_src": _scattered(s, rows, token[:, None], s["perm_src"]),
           "perm_w": _scattered(s, rows, s["topk_w"], s["perm_w"])}
    if s["op"] == "sort_q_ll":
        out.update(offsets=offsets, slot=slot)
    return out


def _plain_sort_bwd(s):
    rows, sent = _rows_of(s, s["offsets"], s["slot"])
    rows = torch.where(sent, rows, 0)
    d = s["dperm_x"].view(-1, s["H"])[rows].float() * sent[:, :, None]
    dx = d.sum(1)
    if s["dx_in"] is not None:
        dx = dx + s["dx_in"].float()
    return {"dx": dx.to(torch.bfloat16), "dtopk_w": torch.where(sent, s["dperm_w"].view(-1)[rows], 0.0)}


def _plain_return_bwd(s):
    rows, sent = _rows_of(s, s["offsets"], s["slot"])
    dout = s["dout"].float()
    dy = _scattered(s, rows, (dout[:, None] * s["topk_w"][:, :, None]).to(torch.bfloat16), s["dy"])
    y = s["y"].view(-1, s["H"])[torch.where(sent, rows, 0)].float()
    return {"dy": dy, "dtopk_w": torch.where(sent, (y * dout[:, None]).sum(2), 0.0)}


_plain = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "sort_q": _plain_sort_q, "sort_q_ll": _plain_sort_q,
          "sort_bwd": _plain_sort_bwd, "return_bwd": _plain_return_bwd}


def _own_norm(s):
    import combine_ep_get_05_gb300 as ep

    ep.ep_rmsnorm(s["x"], s["residual"], s["weight"], EPS, s["residual_out"], s["y"], s["y_q"], s["y_scales"])
    return {n: s[n] for n in ("residual_out", "y", "y_q", "y_scales") if s[n] is not None}


def _own_norm_bwd(s):
    import combine_ep_get_05_gb300 as ep

    if s["workspace"] is None:
        size = ep.ep_rmsnorm_bwd_workspace_size(s["T"], s["H"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    ep.ep_rmsnorm_bwd(s["dy"], s["z"], s["weight"], s["dz_in"], EPS, s["dz"], s["dx"], s["dweight"], s["workspace"])
    return {n: s[n] for n in ("dz", "dx", "dweight") if s[n] is not None}


def _own_sort_q(s):
    import combine_ep_get_05_gb300 as ep

    ep.ep_dispatch_permuted_fp8(s["x_q"], s["x_scales"], s["topk_idx"], s["topk_w"], s["offsets"], s["slot"], s["E"],
                                s["R"], s["rows"], s["perm_q"], s["perm_scales"], s["perm_src"], s["perm_w"],
                                s["status"])
    return {n: s[n] for n in ("perm_q", "perm_scales", "perm_src", "perm_w")}


def _own_sort_q_ll(s):
    import combine_ep_get_05_gb300 as ep

    ep.ep_dispatch_permuted_fp8_ll(s["x_q"], s["x_scales"], s["topk_idx"], s["topk_w"], s["E"], s["R"], s["rows"],
                                   s["offsets"], s["slot"], s["perm_q"], s["perm_scales"], s["perm_src"], s["perm_w"],
                                   s["status"])
    return {n: s[n] for n in ("perm_q", "perm_scales", "perm_src", "perm_w", "offsets", "slot")}


def _own_sort_bwd(s):
    import combine_ep_get_05_gb300 as ep

    ep.ep_dispatch_permuted_bwd(s["dperm_x"], s["dperm_w"], s["dx_in"], s["topk_idx"], s["offsets"], s["slot"], s["E"],
                                s["dx"], s["dtopk_w"], s["status"])
    return {"dx": s["dx"], "dtopk_w": s["dtopk_w"]}


def _own_return_bwd(s):
    import combine_ep_get_05_gb300 as ep

    ep.ep_combine_permuted_bwd(s["dout"], s["y"], s["topk_idx"], s["topk_w"], s["offsets"], s["slot"], s["E"], s["dy"],
                               s["dtopk_w"], s["status"])
    return {"dy": s["dy"], "dtopk_w": s["dtopk_w"]}


_own = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "sort_q": _own_sort_q, "sort_q_ll": _own_sort_q_ll,
        "sort_bwd": _own_sort_bwd, "return_bwd": _own_return_bwd}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        z = s["x"].double() + (s["residual"].double() if s["residual"] is not None else 0.0)
        sigma = torch.sqrt(torch.linalg.vector_norm(z, dim=1) ** 2 / case["H"] + EPS)
        v = torch.einsum("th,t,h->th", z, 1.0 / sigma, s["weight"].double())
        out = {}
        if case["residual"]:
            out["residual_out"] = z
        if "y" in case["outputs"]:
            out["y"] = v
        if "q" in case["outputs"]:  # before the rounding to 8 bits, as the others are before theirs
            scales = torch.stack([c.abs().max(1).values for c in v.split(BLOCK, dim=1)], dim=1) / 448.0
            out["y_q"] = torch.cat([c / scales[:, i:i + 1] for i, c in enumerate(v.split(BLOCK, dim=1))], dim=1)
            out["y_scales"] = scales
        return out
    if op == "norm_bwd":
        z, dy = s["z"].double(), s["dy"].double()
        sigma = torch.sqrt(torch.linalg.vector_norm(z, dim=1) ** 2 / case["H"] + EPS)
        n = z / sigma[:, None]
        g = dy * s["weight"].double()
        dz = (g - n * (torch.einsum("th,th->t", g, n) / case["H"])[:, None]) / sigma[:, None]
        if case["residual"]:
            dz = dz + s["dz_in"].double()
        out = {"dz": dz, "dweight": torch.einsum("th,th->h", dy, n)}
        if case["carry"] == "f32":
            out["dx"] = dz
        return out
    T, E, k, R, room = case["T"], case["E"], case["k"], case["R"], s["rows"]
    idx, w = s["topk_idx"].cpu(), s["topk_w"].double()
    count = [0] * E       # rows of each expert so far, then the first row of each in its rank
    order = []            # (token, slot, expert, place among the expert's rows)
    for t, row in enumerate(idx.tolist()):
        for j, e in enumerate(row):
            if e >= 0:
                order.append((t, j, e, count[e]))
                count[e] += 1
    first = [sum(count[e - e % (E // R):e]) for e in range(E)]
    kept = [(t, j, e // (E // R), first[e] + c) for t, j, e, c in order if first[e] + c < room]
    kept = torch.tensor(kept, dtype=torch.int64, device=w.device).reshape(-1, 4)
    t, j, r, p = kept.unbind(1)
    if op in ("sort_q", "sort_q_ll"):
        q = torch.zeros(s["perm_q"].shape, dtype=torch.float64, device=w.device)
        q[r, p] = s["x_q"].double()[t]
        scales = torch.zeros(s["perm_scales"].shape, dtype=torch.float64, device=w.device)
        scales[r, p] = s["x_scales"].double()[t]
        pw = torch.zeros(s["perm_w"].shape, dtype=torch.float64, device=w.device)
        pw[r, p] = w[t, j]
        out = {"perm_q": q, "perm_scales": scales, "perm_src": None, "perm_w": pw}
        if op == "sort_q_ll":
            out.update(offsets=None, slot=None)
        return out
    dw = torch.zeros((T, k), dtype=torch.float64, device=w.device)
    if op == "sort_bwd":
        dx = s["dx_in"].double() if case["add"] else torch.zeros(s["dx"].shape, dtype=torch.float64, device=w.device)
        for slot in range(k):
            of = j == slot
            dx[t[of]] += s["dperm_x"][r[of], p[of]].double()
        dw[t, j] = s["dperm_w"].double()[r, p]
        return {"dx": dx, "dtopk_w": dw}
    dy = torch.zeros(s["dy"].shape, dtype=torch.float64, device=w.device)
    for slot in range(k):
        of = j == slot
        d = s["dout"].double()[t[of]]
        dy[r[of], p[of]] = d * w[t[of], slot, None]
        dw[t[of], slot] = torch.einsum("nh,nh->n", d, s["y"][r[of], p[of]].double())
    return {"dy": dy, "dtopk_w": dw}
