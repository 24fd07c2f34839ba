"""A mixture-of-experts layer on the expert-major path, trained and served.

    python examples/moe_layer.py

Training: residual addition + RMS norm -> router -> rows into expert order -> experts ->
weighted return, with every gradient of the norm, the sort and the return from this
library (as torch.autograd functions); the router and the experts are plain matmuls. The
gradients are compared with the same layer written in fp32 torch operations.

Serving: a decode batch through the same layer with the norm's E4M3 rows, sorted by expert
in one launch, compared with the bf16 path.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import combine_ep_get_05_gb300 as ep  # noqa: E402

EPS = 1e-6


class Norm(torch.autograd.Function):
    """(x, residual, weight) -> (y, x + residual)"""

    @staticmethod
    def forward(ctx, x, residual, weight):
        n = ep.rmsnorm(x, weight, EPS, residual)
        ctx.save_for_backward(n.residual, weight)
        return n.y, n.residual

    @staticmethod
    def backward(ctx, dy, dz):
        z, weight = ctx.saved_tensors
        dres, dx, dw = ep.rmsnorm_bwd(dy.contiguous(), z, weight, EPS, dz.contiguous())
        return dx, dres, dw.to(weight.dtype)


class Sort(torch.autograd.Function):
    """Rows into expert order."""

    @staticmethod
    def forward(ctx, x, topk_idx, layout, num_ranks, max_rows):
        ctx.topk_idx, ctx.layout = topk_idx, layout
        return ep.dispatch_permuted(x, topk_idx, None, layout, num_ranks, max_rows).perm_x

    @staticmethod
    def backward(ctx, dperm):
        dx, _ = ep.dispatch_permuted_bwd(dperm.contiguous(), ctx.topk_idx, ctx.layout)
        return dx, None, None, None, None


class Return(torch.autograd.Function):
    """Rows back to token order, times their weights."""

    @staticmethod
    def forward(ctx, y, topk_w, topk_idx, layout):
        ctx.save_for_backward(y, topk_w)
        ctx.topk_idx, ctx.layout = topk_idx, layout
        return ep.combine_permuted(y, topk_idx, topk_w, layout)

    @staticmethod
    def backward(ctx, dout):
        y, topk_w = ctx.saved_tensors
        dy, dw = ep.combine_permuted_bwd(dout.contiguous(), y, ctx.topk_idx, topk_w, ctx.layout)
        return dy, dw, None, None


def route(logits, k):
    """Top-k experts and weights that sum to 1; ids in ascending order of score, ties by id."""
    w, idx = torch.topk(torch.softmax(logits.float(), dim=1), k, dim=1)
    return idx.contiguous(), (w / w.sum(1, keepdim=True)).contiguous()


def experts(rows, offsets, w):
    """y = rows @ w[e] for every expert's rows of one rank's slab (rows past the last stay zero)."""
    parts = [rows[offsets[e]:offsets[e + 1]] @ w[e] for e in range(w.shape[0])]
    tail = rows[offsets[w.shape[0]]:]
    return torch.cat(parts + [torch.zeros_like(tail)])


def layer(x, residual, p, k, num_ranks):
    """One layer: returns (out, the residual stream after it, the experts picked)."""
    y, z = Norm.apply(x, residual, p["norm"])
    topk_idx, topk_w = route(y @ p["router"], k)
    E = p["router"].shape[1]
    lay = ep.get_expert_layout(topk_idx, E)
    off = lay.offsets.tolist()
    per = E // num_ranks
    max_rows = max(1, max(off[(r + 1) * per] - off[r * per] for r in range(num_ranks)))
    px = Sort.apply(y, topk_idx, lay, num_ranks, max_rows)
    local = [[o - off[r * per] for o in off[r * per:(r + 1) * per + 1]] for r in range(num_ranks)]
    py = torch.stack([experts(px[r], local[r], p["experts"][r * per:(r + 1) * per]) for r in range(num_ranks)])
    return Return.apply(py, topk_w, topk_idx, lay), z, topk_idx


def layer_fp32(x, residual, p, topk_idx):
    """The same layer in fp32 torch operations, every expert on every token; the experts to
    take are given, since rounding may turn a near tie of the router round."""
    z = x + residual
    y = z * torch.rsqrt((z * z).mean(1, keepdim=True) + EPS) * p["norm"]
    topk_w = torch.softmax(y @ p["router"], dim=1).gather(1, topk_idx)
    topk_w = topk_w / topk_w.sum(1, keepdim=True)
    all_y = torch.einsum("th,ehg->teg", y, p["experts"])
    picked = all_y.gather(1, topk_idx[:, :, None].expand(-1, -1, all_y.shape[2]))
    return (picked * topk_w[:, :, None]).sum(1), z


def make(T, H, E, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    p = {"norm": 1.0 + 0.1 * randn(H), "router": randn(H, E) * H ** -0.5, "experts": randn(E, H, H) * H ** -0.5}
    p = {n: t.to(torch.bfloat16) for n, t in p.items()}
    return randn(T, H).to(torch.bfloat16), randn(T, H).to(torch.bfloat16), p


def relative(a, b):
    return float(((a.float() - b.float()).norm() / b.float().norm()).detach())


def train(T=256, H=512, E=16, k=4, num_ranks=4, seed=0):
    """One step; returns the relative difference of every gradient from the fp32 layer's."""
    x, residual, p = make(T, H, E, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    gout, gz = (torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    leaves = [t.requires_grad_() for t in (x, residual, p["norm"], p["router"], p["experts"])]
    out, z, topk_idx = layer(x, residual, p, k, num_ranks)
    grads = torch.autograd.grad((out * gout).sum() + (z * gz).sum(), leaves)

    f = [t.detach().float().requires_grad_() for t in leaves]
    ref = {"norm": f[2], "router": f[3], "experts": f[4]}
    out32, z32 = layer_fp32(f[0], f[1], ref, topk_idx)
    grads32 = torch.autograd.grad((out32 * gout.float()).sum() + (z32 * gz.float()).sum(), f)
    names = ("x", "residual", "norm", "router", "experts")
    return {"out": relative(out, out32), **{n: relative(a, b) for n, a, b in zip(names, grads, grads32)}}


@torch.no_grad()
def decode(T=32, H=512, E=16, k=4, num_ranks=4, seed=0):
    """A decode batch with E4M3 rows; returns its relative difference from the bf16 path."""
    x, residual, p = make(T, H, E, seed)
    n = ep.rmsnorm(x, p["norm"], EPS, residual, fp8=True)
    topk_idx, topk_w = route(n.y @ p["router"], k)
    max_rows = T * k  # whatever the routing, without asking the GPU
    slabs = ep.alloc_permuted(num_ranks, max_rows, H, fp8=True)
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    slot = torch.empty((T, k), dtype=torch.int32, device="cuda")
    ep.ep_dispatch_permuted_fp8_ll(n.y_q, n.y_scales, topk_idx, topk_w, E, num_ranks, max_rows, off, slot,
                                   slabs.perm_x, slabs.perm_scales, slabs.perm_src, slabs.perm_w, slabs.status)
    rows = (slabs.perm_x.float() * slabs.perm_scales.repeat_interleave(128, dim=2)).to(torch.bfloat16)
    o, per = off.tolist(), E // num_ranks
    py = torch.stack([experts(rows[r], [v - o[r * per] for v in o[r * per:(r + 1) * per + 1]],
                              p["experts"][r * per:(r + 1) * per]) for r in range(num_ranks)])
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    ep.ep_combine_permuted_ll(py, topk_idx, topk_w, off, slot, E, out, slabs.status)
    assert ep.read_flags(slabs.status) == 0
    ref, _, _ = layer(x, residual, p, k, num_ranks)
    return relative(out, ref)


if __name__ == "__main__":
    ep.build_library()
    print("relative difference from the fp32 layer:", {n: f"{v:.2e}" for n, v in train().items()})
    print("decode batch with E4M3 rows against bf16 rows:", f"{decode():.2e}")
