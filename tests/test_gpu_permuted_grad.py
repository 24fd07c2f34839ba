"""The E4M3 sort and the gradients of the expert-major path against plain restatements.

The sort copies, so it is compared bit for bit. The gradient of the sort is an fp32 sum in
a stated order and dy a single product: both bit for bit too. dtopk_w is a dot product in
fp32 over H channels: at most 64 fused terms per thread and 13 additions across the block,
within 80 u of the sum of the terms' magnitudes (u = 2^-24).
"""
import numpy as np
import pytest
import torch

import combine_ep_get_05_gb300 as ep
import oracle
import workloads
from gpu_helpers import GUARD, SENT_BF16, SENT_F32, SENT_I32, check_guards, guarded, host_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


class Batch:
    """A routed batch on the GPU with its expert layout (from the oracle) and slab rows."""

    def __init__(self, T, H, E, k, R, max_rows=None, empty=0.0, bad=False, seed=0):
        rng = np.random.Generator(np.random.PCG64(seed))
        idx = workloads.routing_uniform(rng, T, E, k)
        if empty:
            idx[rng.random((T, k)) < empty] = -1
        if bad and T > 1:
            idx[0, 0] = E + 3            # out of range: not counted
            if k > 1:
                idx[1, 1] = idx[1, 0]    # a repeat: counted once
            idx[T // 2, :] = -1          # a token that goes nowhere
        self.T, self.H, self.E, self.k, self.R = T, H, E, k, R
        self.idx, self.w = idx, workloads._weights(rng, np.where(idx < E, idx, -1))
        self.EL = oracle.expert_layout(idx, E) if T else {"expert_offsets": np.zeros(E + 1, np.int32),
                                                         "expert_slot": np.zeros((0, k), np.int32)}
        off, slot = self.EL["expert_offsets"], self.EL["expert_slot"]
        per = E // R
        loads = off[per::per] - off[:-1:per]
        self.M = int(max(1, loads.max())) if max_rows is None else max_rows
        e = np.clip(idx, 0, E - 1)
        p = off[e] - off[(e // per) * per] + slot
        self.sent = (slot >= 0) & (p < self.M)
        self.dropped = bool(((slot >= 0) & (p >= self.M)).any())
        self.rows = np.where(self.sent, (e // per) * self.M + p, -1).astype(np.int64)
        cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.t_idx, self.t_w, self.t_off, self.t_slot = cu(idx), cu(self.w), cu(off), cu(slot)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def flags(self):
        return ep.FLAG_CAPACITY if self.dropped else 0


def rand_bf16(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


CASES = [dict(T=1, H=128, E=4, k=2, R=2), dict(T=128, H=1024, E=16, k=4, R=4, bad=True),
         dict(T=77, H=640, E=24, k=5, R=8, empty=0.3), dict(T=300, H=7168, E=64, k=8, R=16),
         dict(T=200, H=384, E=32, k=6, R=4, max_rows=100, bad=True), dict(T=65, H=256, E=64, k=32, R=1),
         dict(T=33, H=256, E=8, k=1, R=8, max_rows=0), dict(T=50, H=128, E=4, k=3, R=1, empty=1.0),
         dict(T=1024, H=128, E=16, k=8, R=4, bad=True), dict(T=256, H=128, E=1024, k=32, R=8, bad=True),
         dict(T=910, H=256, E=40, k=9, R=8, empty=0.2), dict(T=481, H=1152, E=32, k=17, R=2, bad=True),
         dict(T=1024, H=16384, E=8, k=1, R=8), dict(T=3, H=16512, E=8, k=2, R=2)]


# --------------------------------------------------------------------------- E4M3 sort

def fp8_inputs(b, seed=3):
    rng = np.random.Generator(np.random.PCG64(seed))
    q = rng.integers(0, 256, (b.T, b.H), dtype=np.uint8)  # every code, NaNs among them: copied as they are
    s = rng.standard_normal((b.T, b.H // 128)).astype(np.float32)
    return q, s


def fp8_expected(b, q, s):
    R, M = b.R, b.M
    out = {"q": np.full((R * M, b.H), 0x7E, np.uint8), "s": np.full((R * M, b.H // 128), SENT_F32, np.float32),
           "src": np.full(R * M, SENT_I32, np.int32), "w": np.full(R * M, SENT_F32, np.float32)}
    t, j = np.nonzero(b.sent)
    rows = b.rows[t, j]
    out["q"][rows], out["s"][rows], out["src"][rows], out["w"][rows] = q[t], s[t], t, b.w[t, j]
    return out


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
@pytest.mark.parametrize("ll", [False, True])
@pytest.mark.parametrize("meta", [True, False])
def test_fp8_sort_bit_exact(case, ll, meta):
    b = Batch(**case)
    q, s = fp8_inputs(b)
    want = fp8_expected(b, q, s)
    R, M, nb = b.R, b.M, b.H // 128
    pq, pqb = guarded((R, M, b.H), torch.uint8, 0x7E)
    ps, psb = guarded((R, M, nb), torch.float32, SENT_F32)
    src, srcb = guarded((R, M), torch.int32, SENT_I32)
    pw, pwb = guarded((R, M), torch.float32, SENT_F32)
    pq.fill_(0x7E), ps.fill_(SENT_F32), src.fill_(SENT_I32), pw.fill_(SENT_F32)
    tq, ts = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    m = (src, pw) if meta else (None, None)
    if ll:
        off, slot = torch.full_like(b.t_off, -7), torch.full_like(b.t_slot, -7)
        ep.ep_dispatch_permuted_fp8_ll(tq, ts, b.t_idx, b.t_w, b.E, R, M, off, slot, pq, ps, *m, b.status)
        assert torch.equal(off, b.t_off) and torch.equal(slot, b.t_slot)
        bad = bool((b.idx >= b.E).any()) or any(len(set(r[r >= 0])) < (r >= 0).sum() for r in b.idx)
        assert ep.read_flags(b.status) == b.flags() | (ep.FLAG_BAD_EXPERT if bad else 0)
    else:
        ep.ep_dispatch_permuted_fp8(tq, ts, b.t_idx, b.t_w, b.t_off, b.t_slot, b.E, R, M, pq, ps, *m, b.status)
        assert ep.read_flags(b.status) == b.flags()
    assert np.array_equal(host_bits(pq).reshape(R * M, b.H), want["q"])
    assert np.array_equal(host_bits(ps).reshape(R * M, nb), want["s"])
    if meta:
        assert np.array_equal(host_bits(src).reshape(-1), want["src"])
        assert np.array_equal(host_bits(pw).reshape(-1), want["w"])
    for back, n, fill in ((pqb, R * M * b.H, 0x7E), (psb, R * M * nb, SENT_F32), (srcb, R * M, SENT_I32),
                          (pwb, R * M, SENT_F32)):
        check_guards(back, n, fill)


def test_fp8_sort_after_the_norm_is_the_bf16_sort_quantised():
    """Norm -> E4M3 rows -> sort: every slab row is its token's E4M3 row, and the codes may be
    handed over as float8_e4m3fn."""
    b = Batch(T=96, H=1024, E=16, k=4, R=4)
    x = rand_bf16((b.T, b.H), 1)
    weight = torch.ones(b.H, device="cuda")
    y_q = torch.empty((b.T, b.H), dtype=torch.float8_e4m3fn, device="cuda")
    y_s = torch.empty((b.T, b.H // 128), device="cuda")
    ep.ep_rmsnorm(x, None, weight, 1e-6, None, None, y_q, y_s)
    pq = torch.zeros((b.R, b.M, b.H), dtype=torch.float8_e4m3fn, device="cuda")
    ps = torch.zeros((b.R, b.M, b.H // 128), device="cuda")
    ep.ep_dispatch_permuted_fp8(y_q, y_s, b.t_idx, None, b.t_off, b.t_slot, b.E, b.R, b.M, pq, ps)
    t, j = np.nonzero(b.sent)
    rows = torch.from_numpy(b.rows[t, j]).cuda()
    tt = torch.from_numpy(t).cuda()
    assert torch.equal(pq.view(torch.uint8).view(-1, b.H)[rows], y_q.view(torch.uint8)[tt])
    assert torch.equal(ps.view(-1, b.H // 128)[rows], y_s[tt])


@pytest.mark.parametrize("ll", [False, True])
def test_fp8_sort_offsets_past_32_bits(ll):
    """Slab rows whose first byte lies past 2^32."""
    T, H, E, k, R, M = 700, 16384, 2, 2, 2, 135_000
    b = Batch(T=T, H=H, E=E, k=k, R=R, max_rows=M)
    q, s = fp8_inputs(b)
    tq, ts = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    pq = torch.zeros((R, M, H), dtype=torch.uint8, device="cuda")
    ps = torch.zeros((R, M, H // 128), device="cuda")
    src = torch.full((R, M), -1, dtype=torch.int32, device="cuda")
    if ll:
        ep.ep_dispatch_permuted_fp8_ll(tq, ts, b.t_idx, b.t_w, E, R, M, b.t_off, b.t_slot, pq, ps, src)
    else:  # the second rank's rows at the end of its slab, by way of the offsets
        off = torch.tensor([0, T, T], dtype=torch.int32, device="cuda")
        slot = b.t_slot + torch.where(b.t_idx == 1, M - T, 0).to(torch.int32)
        ep.ep_dispatch_permuted_fp8(tq, ts, b.t_idx, b.t_w, off, slot, E, R, M, pq, ps, src)
    first = 0 if ll else M - T
    assert torch.equal(pq[1, first:first + T], tq) and torch.equal(ps[1, first:first + T], ts)
    assert torch.equal(pq[0, :T], tq)
    assert int((src >= 0).sum()) == 2 * T


# --------------------------------------------------------------------------- gradient of the sort

def sort_bwd_expected(b, dperm_x, dperm_w, dx_in):
    acc = dx_in.float() if dx_in is not None else torch.zeros((b.T, b.H), device="cuda")
    dw = torch.zeros((b.T, b.k), device="cuda")
    flat, fw = dperm_x.view(-1, b.H), dperm_w.view(-1)
    for j in range(b.k):
        t = torch.from_numpy(np.nonzero(b.sent[:, j])[0]).cuda()
        rows = torch.from_numpy(b.rows[b.sent[:, j], j]).cuda()
        acc[t] = acc[t] + flat[rows].float()
        dw[t, j] = fw[rows]
    return acc.to(torch.bfloat16), dw


GRAD_CASES = CASES + [dict(T=130, H=1000, E=16, k=4, R=4, empty=0.2), dict(T=1, H=8, E=1, k=1, R=1),
                      dict(T=9, H=16392, E=8, k=3, R=2), dict(T=40, H=8200, E=16, k=9, R=2),
                      dict(T=700, H=392, E=16, k=4, R=4, bad=True), dict(T=5000, H=1024, E=32, k=5, R=4, empty=0.1),
                      dict(T=10000, H=64, E=16, k=8, R=2, max_rows=36000), dict(T=2600, H=264, E=16, k=3, R=4),
                      dict(T=2500, H=2048, E=8, k=1, R=8, bad=True), dict(T=400, H=4104, E=8, k=2, R=1),
                      dict(T=3000, H=2056, E=16, k=1, R=4), dict(T=500, H=7168, E=16, k=10, R=2, empty=0.3)]


@pytest.mark.parametrize("case", GRAD_CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
@pytest.mark.parametrize("add", [False, True])
def test_sort_gradient_bit_exact(case, add):
    b = Batch(**case)
    # rows that hold no entry are NaN: reading one would show
    dperm_x = torch.full((b.R, b.M, b.H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dperm_w = torch.full((b.R, b.M), float("nan"), device="cuda")
    used = torch.from_numpy(b.rows[b.sent]).cuda()
    dperm_x.view(-1, b.H)[used] = rand_bf16((used.numel(), b.H), 2)
    dperm_w.view(-1)[used] = torch.randn(used.numel(), device="cuda")
    dx_in = rand_bf16((b.T, b.H), 3) if add else None
    want, want_w = sort_bwd_expected(b, dperm_x, dperm_w, dx_in)
    dx, dxb = guarded((b.T, b.H), torch.bfloat16, SENT_BF16)
    dw, dwb = guarded((b.T, b.k), torch.float32, SENT_F32)
    ep.ep_dispatch_permuted_bwd(dperm_x, dperm_w, dx_in, b.t_idx, b.t_off, b.t_slot, b.E, dx, dw, b.status)
    assert ep.read_flags(b.status) == b.flags()
    assert np.array_equal(host_bits(dx), host_bits(want)) and torch.equal(dw, want_w)
    check_guards(dxb, b.T * b.H, SENT_BF16)
    check_guards(dwb, b.T * b.k, SENT_F32)
    if add:  # in place, without the weights
        ep.ep_dispatch_permuted_bwd(dperm_x, None, dx_in, b.t_idx, b.t_off, b.t_slot, b.E, dx_in)
        assert np.array_equal(host_bits(dx_in), host_bits(want))


def test_sort_gradient_is_the_unweighted_return():
    b = Batch(T=200, H=1024, E=32, k=6, R=8, empty=0.1)
    d = rand_bf16((b.R, b.M, b.H), 4)
    dx, out = (torch.empty((b.T, b.H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ep.ep_dispatch_permuted_bwd(d, None, None, b.t_idx, b.t_off, b.t_slot, b.E, dx)
    ep.ep_combine_permuted(d, b.t_idx, None, b.t_off, b.t_slot, b.E, out)
    assert torch.equal(dx, out)


# --------------------------------------------------------------------------- gradient of the return

def return_bwd_expected(b, dout, y):
    dy = torch.full((b.R * b.M, b.H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros((b.T, b.k), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(dw)
    for j in range(b.k):
        t = torch.from_numpy(np.nonzero(b.sent[:, j])[0]).cuda()
        rows = torch.from_numpy(b.rows[b.sent[:, j], j]).cuda()
        dy[rows] = (dout[t].float() * b.t_w[t, j, None]).to(torch.bfloat16)
        prod = dout[t].double() * y.view(-1, b.H)[rows].double()
        dw[t, j], mag[t, j] = prod.sum(1), prod.abs().sum(1)
    return dy.view(b.R, b.M, b.H), dw, mag


@pytest.mark.parametrize("case", GRAD_CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_return_gradient_against_formula(case):
    b = Batch(**case)
    dout, y = rand_bf16((b.T, b.H), 5), rand_bf16((b.R, b.M, b.H), 6)
    want, want_w, mag = return_bwd_expected(b, dout, y)
    nan = int(np.array(0x7FC0, np.uint16))
    dy, dyb = guarded((b.R, b.M, b.H), torch.bfloat16, SENT_BF16)
    dy.view(torch.int16).fill_(nan)
    dw, dwb = guarded((b.T, b.k), torch.float32, SENT_F32)
    ep.ep_combine_permuted_bwd(dout, y, b.t_idx, b.t_w, b.t_off, b.t_slot, b.E, dy, dw, b.status)
    assert ep.read_flags(b.status) == b.flags()
    assert torch.equal(torch.isnan(dy), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(dy), torch.nan_to_num(want))
    assert torch.all((dw.double() - want_w).abs() <= 80 * U * mag)
    assert torch.all(dw[~torch.from_numpy(b.sent).cuda()] == 0)
    check_guards(dyb, b.R * b.M * b.H, SENT_BF16)
    check_guards(dwb, b.T * b.k, SENT_F32)
    again = torch.empty_like(dw)
    only = torch.empty_like(dy)
    only.view(torch.int16).fill_(nan)
    ep.ep_combine_permuted_bwd(dout, y, b.t_idx, b.t_w, b.t_off, b.t_slot, b.E, y, again)  # dy over y
    ep.ep_combine_permuted_bwd(dout, None, b.t_idx, b.t_w, b.t_off, b.t_slot, b.E, only)   # dy alone
    assert torch.equal(again, dw)
    used = torch.from_numpy(b.rows[b.sent]).cuda()
    for d in (y, only):
        assert torch.equal(d.view(-1, b.H)[used], dy.view(-1, b.H)[used])


def test_return_gradient_unweighted_copies_the_rows():
    b = Batch(T=60, H=520, E=8, k=3, R=2, empty=0.2)
    dout = rand_bf16((b.T, b.H), 7)
    dy = torch.zeros((b.R, b.M, b.H), dtype=torch.bfloat16, device="cuda")
    ep.ep_combine_permuted_bwd(dout, None, b.t_idx, None, b.t_off, b.t_slot, b.E, dy)
    perm = torch.zeros_like(dy)
    ep.ep_dispatch_permuted(dout, b.t_idx, None, b.t_off, b.t_slot, b.E, b.R, b.M, perm)
    assert torch.equal(dy, perm)


def test_gradients_of_the_layer_against_differences():
    """loss = <g, combine(w, y(x))> with y = 2 x (a linear expert): differences of the definition
    in 64 bits along random directions of x and of the weights. The path is linear in each, so
    the difference is exact up to rounding; the gradients carry bf16 rounding (2^-8 each, twice)."""
    b = Batch(T=48, H=256, E=8, k=3, R=4, empty=0.1)
    x, g = rand_bf16((b.T, b.H), 8), rand_bf16((b.T, b.H), 9)
    px = torch.zeros((b.R, b.M, b.H), dtype=torch.bfloat16, device="cuda")
    ep.ep_dispatch_permuted(x, b.t_idx, b.t_w, b.t_off, b.t_slot, b.E, b.R, b.M, px)
    y = 2 * px
    dy = torch.zeros_like(y)
    dw = torch.empty((b.T, b.k), device="cuda")
    ep.ep_combine_permuted_bwd(g, y, b.t_idx, b.t_w, b.t_off, b.t_slot, b.E, dy, dw)
    dx = torch.empty_like(x)
    ep.ep_dispatch_permuted_bwd(2 * dy, None, None, b.t_idx, b.t_off, b.t_slot, b.E, dx)
    sent = torch.from_numpy(b.sent).cuda().double()

    def loss(xx, ww):
        return float((g.double() * (2 * xx) * (ww * sent).sum(1, keepdim=True)).sum())

    gen = torch.Generator(device="cuda").manual_seed(10)
    for _ in range(3):
        dirx = torch.randn((b.T, b.H), generator=gen, device="cuda", dtype=torch.float64)
        dirw = torch.randn((b.T, b.k), generator=gen, device="cuda", dtype=torch.float64)
        w64, x64 = b.t_w.double(), x.double()
        fx = (loss(x64 + dirx, w64) - loss(x64 - dirx, w64)) / 2
        fw = (loss(x64, w64 + dirw) - loss(x64, w64 - dirw)) / 2
        magx = float((dx.double().abs() * dirx.abs()).sum())
        magw = float((dw.double().abs() * dirw.abs()).sum())
        assert abs(float((dx.double() * dirx).sum()) - fx) <= 2 * 2.0 ** -8 * magx
        assert abs(float((dw.double() * dirw).sum()) - fw) <= 1e-5 * magw


def test_gradients_with_rows_past_32_bits():
    T, H, E, k, R, M = 64, 16384, 2, 2, 2, 135_000
    b = Batch(T=T, H=H, E=E, k=k, R=R, max_rows=M)
    off = torch.tensor([0, T, T], dtype=torch.int32, device="cuda")
    slot = b.t_slot + torch.where(b.t_idx == 1, M - T, 0).to(torch.int32)
    dout = rand_bf16((T, H), 11)
    dy = torch.zeros((R, M, H), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((R, M, H), dtype=torch.bfloat16, device="cuda")
    y[1, M - T:] = 1.0
    dw = torch.empty((T, k), device="cuda")
    ep.ep_combine_permuted_bwd(dout, y, b.t_idx, b.t_w, off, slot, E, dy, dw)
    w1 = (b.t_w * (b.t_idx == 1)).sum(1)
    assert torch.equal(dy[1, M - T:], (dout.float() * w1[:, None]).to(torch.bfloat16))
    ref = dout.double().sum(1)
    assert torch.all(((dw * (b.t_idx == 1)).sum(1).double() - ref).abs() <= 80 * U * dout.double().abs().sum(1))
    dx = torch.empty_like(dout)
    ep.ep_dispatch_permuted_bwd(dy, None, None, b.t_idx, off, slot, E, dx)
    first = torch.where(b.t_idx[:, 0] == 0, 0, 1)
    rows = torch.stack([dy[0, :T], dy[1, M - T:]])
    a = rows[first, torch.arange(T, device="cuda")].float() + rows[1 - first, torch.arange(T, device="cuda")].float()
    assert torch.equal(dx, a.to(torch.bfloat16))


def test_empty_batches_write_nothing():
    b = Batch(T=0, H=256, E=8, k=2, R=2)
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    slab = torch.full((2, 1, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((0, 2), device="cuda")
    ep.ep_combine_permuted_bwd(x, slab, b.t_idx, b.t_w, b.t_off, b.t_slot, 8, slab, dw)
    ep.ep_dispatch_permuted_bwd(slab, None, None, b.t_idx, b.t_off, b.t_slot, 8, x)
    q = torch.empty((0, 256), dtype=torch.uint8, device="cuda")
    s = torch.empty((0, 2), device="cuda")
    pq = torch.full((2, 1, 256), 9, dtype=torch.uint8, device="cuda")
    ps = torch.full((2, 1, 2), 9.0, device="cuda")
    off = torch.full((9,), -1, dtype=torch.int32, device="cuda")
    ep.ep_dispatch_permuted_fp8(q, s, b.t_idx, b.t_w, b.t_off, b.t_slot, 8, 2, 1, pq, ps)
    ep.ep_dispatch_permuted_fp8_ll(q, s, b.t_idx, b.t_w, 8, 2, 1, off, b.t_slot, pq, ps)
    assert torch.all(slab == 5) and torch.all(pq == 9) and torch.all(ps == 9) and torch.all(off == 0)
    assert GUARD > 0
