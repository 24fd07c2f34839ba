"""Convenience layer over the C ABI: allocate the caller-owned buffers with torch
and chain the entry points. It adds no computation: every step still runs in
the library's kernels (see _lib.py).

A helper with `stream` allocates, zero-fills and frees on that stream, where its kernels run,
and what it returns may also be used and freed on the stream that was current (once that has
been made to wait for `stream`, as for any work there). Inputs are the caller's: they have to
be ready on `stream` and to live until its work is done."""
from __future__ import annotations

from dataclasses import dataclass, fields
from typing import Optional

import torch

from . import _lib as L


class _On:
    """with _On(stream) as on: `stream` is the current one (None: the current one stays).
    on.made(m): m, a tensor or a dataclass of tensors that was allocated there and goes to the
    caller; its memory is taken back only after the caller's stream is done with it too."""

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        if self.stream is not None:
            s = self.stream
            if not isinstance(s, torch.cuda.Stream):
                s = torch.cuda.ExternalStream(s.cuda_stream)
            self.callers = torch.cuda.current_stream()
            self.inside = torch.cuda.stream(s)
            self.inside.__enter__()
        return self

    def __exit__(self, *exception):
        if self.stream is not None:
            self.inside.__exit__(*exception)

    def made(self, m):
        if self.stream is not None:
            for t in [m] if isinstance(m, torch.Tensor) else [getattr(m, f.name) for f in fields(m)]:
                if isinstance(t, torch.Tensor):
                    t.record_stream(self.callers)
        return m


@dataclass
class Layout:
    tokens_per_expert: torch.Tensor  # int32 [E]
    tokens_per_rank: torch.Tensor    # int32 [R]
    tokens_per_node: Optional[torch.Tensor]  # int32 [N] or None
    is_token_in_rank: torch.Tensor   # uint8 [T][R]
    is_token_in_node: Optional[torch.Tensor]  # uint8 [T][N] or None
    slot: torch.Tensor               # int32 [T][R]
    workspace: torch.Tensor          # uint8, zero-filled once, reusable
    status: torch.Tensor             # int32 [1]
    num_experts: int
    num_ranks: int
    ranks_per_node: int


@dataclass
class Dispatched:
    recv_x: torch.Tensor              # bf16 or uint8 (e4m3) [R][max_tokens][H]
    recv_scales: Optional[torch.Tensor]   # fp32 [R][max_tokens][H/128] (e4m3 only)
    recv_src_idx: Optional[torch.Tensor]  # int32 [R][max_tokens]
    recv_topk_idx: Optional[torch.Tensor]  # int32 [R][max_tokens][k]
    recv_topk_w: Optional[torch.Tensor]    # fp32 [R][max_tokens][k]
    status: torch.Tensor
    max_tokens: int


def alloc_layout(T: int, num_experts: int, num_ranks: int, ranks_per_node: int = 0, device="cuda") -> Layout:
    dev = torch.device(device)
    N = num_ranks // ranks_per_node if ranks_per_node > 0 else 0
    ws_bytes = L.ep_layout_workspace_size(T, num_experts, num_ranks, ranks_per_node)
    i32 = dict(dtype=torch.int32, device=dev)
    return Layout(
        tokens_per_expert=torch.empty(num_experts, **i32),
        tokens_per_rank=torch.empty(num_ranks, **i32),
        tokens_per_node=torch.empty(N, **i32) if N else None,
        is_token_in_rank=torch.empty((T, num_ranks), dtype=torch.uint8, device=dev),
        is_token_in_node=torch.empty((T, N), dtype=torch.uint8, device=dev) if N else None,
        slot=torch.empty((T, num_ranks), **i32),
        workspace=torch.zeros(max(ws_bytes, 256), dtype=torch.uint8, device=dev),
        status=torch.zeros(1, **i32),
        num_experts=num_experts, num_ranks=num_ranks, ranks_per_node=ranks_per_node,
    )


def alloc_dispatch(num_ranks: int, max_tokens: int, H: int, k: int, fp8: bool = False, metadata: bool = True,
                   device="cuda") -> Dispatched:
    dev = torch.device(device)
    shape = (num_ranks, max_tokens, H)
    return Dispatched(
        recv_x=torch.empty(shape, dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev),
        recv_scales=torch.empty((num_ranks, max_tokens, H // 128), dtype=torch.float32, device=dev) if fp8 else None,
        recv_src_idx=torch.empty((num_ranks, max_tokens), dtype=torch.int32, device=dev) if metadata else None,
        recv_topk_idx=torch.empty((num_ranks, max_tokens, k), dtype=torch.int32, device=dev) if metadata else None,
        recv_topk_w=torch.empty((num_ranks, max_tokens, k), dtype=torch.float32, device=dev) if metadata else None,
        status=torch.zeros(1, dtype=torch.int32, device=dev),
        max_tokens=max_tokens,
    )


def get_layout(topk_idx: torch.Tensor, num_experts: int, num_ranks: int, ranks_per_node: int = 0,
               out: Optional[Layout] = None, stream=None) -> Layout:
    T = topk_idx.shape[0]
    with _On(stream) as on:
        lay = out if out is not None else on.made(
            alloc_layout(T, num_experts, num_ranks, ranks_per_node, topk_idx.device))
        L.ep_get_layout(topk_idx, num_experts, num_ranks, ranks_per_node, lay.tokens_per_expert, lay.tokens_per_rank,
                        lay.tokens_per_node, lay.is_token_in_rank, lay.is_token_in_node, lay.slot, lay.workspace,
                        lay.status, stream)
    return lay


def dispatch(x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor, layout: Layout, max_tokens: int,
             fp8: bool = False, out: Optional[Dispatched] = None, stream=None) -> Dispatched:
    T, H = x.shape
    k = topk_idx.shape[1]
    with _On(stream) as on:
        d = out if out is not None else on.made(
            alloc_dispatch(layout.num_ranks, max_tokens, H, k, fp8, device=x.device))
        L.ep_dispatch(x, L.DTYPE_E4M3 if fp8 else L.DTYPE_BF16, topk_idx, topk_w, layout.slot, layout.num_experts,
                      layout.num_ranks, max_tokens, d.recv_x, d.recv_scales, d.recv_src_idx, d.recv_topk_idx,
                      d.recv_topk_w, d.status, stream)
    return d


def combine(y: torch.Tensor, layout: Layout, max_tokens: int, out: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    T = layout.slot.shape[0]
    H = y.shape[2]
    with _On(stream) as on:
        o = out if out is not None else on.made(torch.empty((T, H), dtype=torch.bfloat16, device=y.device))
        L.ep_combine(y, layout.slot, max_tokens, o, status, stream)
    return o


def read_flags(status: torch.Tensor) -> int:
    """Synchronise and return the asynchronous EP_FLAG_* bits of a status word."""
    return int(status.item())


def combine_fp8(y, y_scales, layout: Layout, max_tokens: int, out=None, status=None) -> torch.Tensor:
    """Combine of FP8 expert outputs (E4M3 codes [R][max_tokens][H] + scales) into bf16 [T][H]."""
    R, _, H = y.shape
    T = layout.slot.shape[0]
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    L.ep_combine_fp8(y, y_scales, layout.slot, max_tokens, out, status)
    return out


def combine_weights(recv_topk_w, layout: Layout, max_tokens: int, out=None, status=None) -> torch.Tensor:
    """The combined top-k weights [T][k]: the received weight rows summed back to token order."""
    T = layout.slot.shape[0]
    if out is None:
        out = torch.empty((T, recv_topk_w.shape[2]), dtype=torch.float32, device=recv_topk_w.device)
    L.ep_combine_weights(recv_topk_w, layout.slot, max_tokens, out, status)
    return out



# --------------------------------------------------------------------------- expert-major path

@dataclass
class ExpertLayout:
    offsets: torch.Tensor    # int32 [E+1]: first row of every expert, all ranks' rows counted through
    slot: torch.Tensor       # int32 [T][k]: place among the expert's rows, -1 where not counted
    workspace: torch.Tensor  # uint8, zero-filled once, reusable
    status: torch.Tensor     # int32 [1]
    num_experts: int


@dataclass
class Permuted:
    perm_x: torch.Tensor                  # bf16 rows or E4M3 codes [R][max_rows][H]
    perm_scales: Optional[torch.Tensor]   # fp32 [R][max_rows][H/128] (E4M3 only)
    perm_src: torch.Tensor                # int32 [R][max_rows]
    perm_w: Optional[torch.Tensor]        # fp32 [R][max_rows]
    status: torch.Tensor


@dataclass
class Normed:
    residual: torch.Tensor                # x + residual (the one of them that there is, itself)
    y: Optional[torch.Tensor]             # bf16 [T][H]
    y_q: Optional[torch.Tensor]           # float8_e4m3fn [T][H]
    y_scales: Optional[torch.Tensor]      # fp32 [T][H/128]


def rmsnorm(x: Optional[torch.Tensor], weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
            bf16: bool = True, fp8: bool = False, stream=None) -> Normed:
    """x + residual (either may be None, not both) and its RMS norm, as bf16 rows, as E4M3 rows with 1x128
    scales, or both."""
    given = x if x is not None else residual
    if given is None:
        raise ValueError("x or residual is required")
    T, H = given.shape
    dev = given.device
    with _On(stream) as on:
        n = on.made(Normed(
            residual=torch.empty_like(residual) if x is not None and residual is not None else None,
            y=torch.empty((T, H), dtype=torch.bfloat16, device=dev) if bf16 else None,
            y_q=torch.empty((T, H), dtype=torch.float8_e4m3fn, device=dev) if fp8 else None,
            y_scales=torch.empty((T, H // 128), dtype=torch.float32, device=dev) if fp8 else None))
        L.ep_rmsnorm(x, residual, weight, eps, n.residual, n.y, n.y_q, n.y_scales, stream)
    if n.residual is None:
        n.residual = given
    return n


def rmsnorm_bwd(dy: torch.Tensor, z: torch.Tensor, weight: torch.Tensor, eps: float,
                dz: Optional[torch.Tensor] = None, stream=None):
    """Gradient of rmsnorm at z = Normed.residual, with the gradient dz that arrives along the
    stream: (gradient of residual in the stream's type, gradient of x in bf16, fp32 dweight)."""
    T, H = z.shape
    with _On(stream) as on:
        out = on.made(torch.empty_like(z))
        dx = out
        if z.dtype != torch.bfloat16:
            dx = on.made(torch.empty((T, H), dtype=torch.bfloat16, device=z.device))
        dw = on.made(torch.empty(H, dtype=torch.float32, device=z.device))
        ws = torch.empty(L.ep_rmsnorm_bwd_workspace_size(T, H), dtype=torch.uint8, device=z.device)
        L.ep_rmsnorm_bwd(dy, z, weight, dz, eps, out, dx if dx is not out else None, dw, ws, stream)
    return out, dx, dw


def get_expert_layout(topk_idx: torch.Tensor, num_experts: int, stream=None) -> ExpertLayout:
    T, k = topk_idx.shape
    dev = topk_idx.device
    i32 = dict(dtype=torch.int32, device=dev)
    with _On(stream) as on:
        ws = torch.zeros(L.ep_expert_layout_workspace_size(T, num_experts), dtype=torch.uint8, device=dev)
        lay = on.made(ExpertLayout(torch.empty(num_experts + 1, **i32), torch.empty((T, k), **i32), ws,
                                   torch.zeros(1, **i32), num_experts))
        L.ep_get_expert_layout(topk_idx, num_experts, lay.offsets, lay.slot, ws, lay.status, stream)
    return lay


def alloc_permuted(num_ranks: int, max_rows: int, H: int, fp8: bool = False, weights: bool = True,
                   device="cuda") -> Permuted:
    """Zero-filled slabs: rows that no token is sent to stay zero."""
    dev = torch.device(device)
    x = torch.zeros((num_ranks, max_rows, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
    return Permuted(
        perm_x=x.view(torch.float8_e4m3fn) if fp8 else x,
        perm_scales=torch.zeros((num_ranks, max_rows, H // 128), dtype=torch.float32, device=dev) if fp8 else None,
        perm_src=torch.full((num_ranks, max_rows), -1, dtype=torch.int32, device=dev),
        perm_w=torch.zeros((num_ranks, max_rows), dtype=torch.float32, device=dev) if weights else None,
        status=torch.zeros(1, dtype=torch.int32, device=dev),
    )


def dispatch_permuted(x: torch.Tensor, topk_idx: torch.Tensor, topk_w: Optional[torch.Tensor], layout: ExpertLayout,
                      num_ranks: int, max_rows: int, scales: Optional[torch.Tensor] = None,
                      out: Optional[Permuted] = None, stream=None) -> Permuted:
    """Rows into expert order: bf16 rows, or E4M3 codes with their scales."""
    with _On(stream) as on:
        p = out if out is not None else on.made(
            alloc_permuted(num_ranks, max_rows, x.shape[1], scales is not None, topk_w is not None, x.device))
        if scales is None:
            L.ep_dispatch_permuted(x, topk_idx, topk_w, layout.offsets, layout.slot, layout.num_experts, num_ranks,
                                   max_rows, p.perm_x, p.perm_src, p.perm_w, p.status, stream)
        else:
            L.ep_dispatch_permuted_fp8(x, scales, topk_idx, topk_w, layout.offsets, layout.slot, layout.num_experts,
                                       num_ranks, max_rows, p.perm_x, p.perm_scales, p.perm_src, p.perm_w, p.status,
                                       stream)
    return p


def dispatch_permuted_bwd(dperm_x: torch.Tensor, topk_idx: torch.Tensor, layout: ExpertLayout,
                          dperm_w: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                          status: Optional[torch.Tensor] = None, stream=None):
    """Gradient of dispatch_permuted, added to `dx` (another gradient of x) where given: (dx, dtopk_w or None)."""
    T, k = topk_idx.shape
    dev = dperm_x.device
    with _On(stream) as on:
        out = on.made(torch.empty((T, dperm_x.shape[2]), dtype=torch.bfloat16, device=dev))
        dw = on.made(torch.empty((T, k), dtype=torch.float32, device=dev)) if dperm_w is not None else None
        L.ep_dispatch_permuted_bwd(dperm_x, dperm_w, dx, topk_idx, layout.offsets, layout.slot, layout.num_experts,
                                   out, dw, status, stream)
    return out, dw


def combine_permuted(y: torch.Tensor, topk_idx: torch.Tensor, topk_w: Optional[torch.Tensor], layout: ExpertLayout,
                     status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows back to token order, weighted where topk_w is given."""
    with _On(stream) as on:
        out = on.made(torch.empty((topk_idx.shape[0], y.shape[2]), dtype=torch.bfloat16, device=y.device))
        L.ep_combine_permuted(y, topk_idx, topk_w, layout.offsets, layout.slot, layout.num_experts, out, status,
                              stream)
    return out


def combine_permuted_bwd(dout: torch.Tensor, y: torch.Tensor, topk_idx: torch.Tensor, topk_w: Optional[torch.Tensor],
                         layout: ExpertLayout, status: Optional[torch.Tensor] = None, stream=None):
    """Gradient of combine_permuted: (dy with zeros in rows that hold no entry, dtopk_w or None where unweighted)."""
    with _On(stream) as on:
        dy = on.made(torch.zeros_like(y))
        dw = on.made(torch.empty_like(topk_w)) if topk_w is not None else None
        L.ep_combine_permuted_bwd(dout, y, topk_idx, topk_w, layout.offsets, layout.slot, layout.num_experts, dy, dw,
                                  status, stream)
    return dy, dw
