"""The experts' feed-forward block as it is used: rows of the dispatch, streams, graphs, repeated and
concurrent calls, offsets past 2^31, many experts, values that are not finite, offsets that are wrong."""
import math

import pytest
import torch

import combine_ep_get_05_gb300 as ep
from expert_cases import (ACTS, SENTINEL, Rows, act_of, check_down, check_down_bwd, check_gate_up, check_gate_up_bwd,
                          check_wgrad, decode, normal, out, slab)
from gpu_helpers import GUARD

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


def zero_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Block:
    """All five operators on one set of rows."""

    def __init__(self, rows, H, F, seed=1, act="silu", eight=False, make=out):
        self.rows, self.H, self.F, self.act, self.eight = rows, H, F, act, eight
        self.x, self.dy = slab(rows, seed, H, 2.0), slab(rows, seed + 1, H, 0.1)
        self.w1 = normal(seed + 2, rows.E, 2 * F, H, scale=H ** -0.5)
        self.w2 = normal(seed + 3, rows.E, H, F, scale=F ** -0.5)
        self.h, self.y, self.dpre, self.h2, self.dx = (make(rows, n) for n in (F, H, 2 * F, F, H))
        self.pre = None if eight else make(rows, 2 * F)
        self.q = make(rows, 2 * F, torch.float8_e4m3fn) if eight else None
        self.s = make(rows, 2 * F // 128) if eight else None
        self.dw1 = torch.full((rows.E, 2 * F, H), SENTINEL, dtype=torch.bfloat16, device="cuda")
        self.dw2 = torch.full((rows.E, H, F), SENTINEL, dtype=torch.bfloat16, device="cuda")
        self.status = zero_status()

    def run(self, stream=None):
        off, a = self.rows.offsets, ACTS[self.act]
        ep.ep_expert_gate_up(self.x, self.w1, off, a, self.h, self.pre, self.q, self.s, self.status, stream)
        ep.ep_expert_down(self.h, self.w2, off, self.y, self.status, stream)
        ep.ep_expert_down_bwd(self.dy, self.w2, self.pre, self.q, self.s, off, a, self.dpre, self.h2, self.status,
                              stream)
        ep.ep_expert_gate_up_bwd(self.dpre, self.w1, off, self.dx, self.status, stream)
        ep.ep_expert_wgrad(self.dpre, self.x, off, self.dw1, self.status, stream)
        ep.ep_expert_wgrad(self.dy, self.h2, off, self.dw2, self.status, stream)

    def outputs(self):
        return [t for t in (self.h, self.y, self.dpre, self.h2, self.dx, self.dw1, self.dw2, self.pre, self.q, self.s)
                if t is not None]

    def clear(self):
        for t in self.outputs():
            t.view(torch.uint8).fill_(0x55)

    def check(self):
        r = self.rows
        check_gate_up(self.x, self.w1, r, self.act, self.h, self.pre, self.q, self.s)
        check_down(self.h, self.w2, r, self.y)
        check_down_bwd(self.dy, self.w2, decode(self.q, self.s) if self.eight else self.pre, r, self.act, self.dpre,
                       self.h2)
        check_gate_up_bwd(self.dpre, self.w1, r, self.dx)
        check_wgrad(self.dpre, self.x, r, self.dw1)
        check_wgrad(self.dy, self.h2, r, self.dw2)
        assert ep.read_flags(self.status) == (ep.FLAG_CAPACITY if r.dropped else 0)


def bits(tensors):
    return [t.view(torch.uint8).clone() for t in tensors]


@pytest.mark.parametrize("eight", [False, True])
def test_chained_calls_repeat_bit_for_bit(eight):
    """Each call reads what the one before wrote, thirty times over in a row."""
    b = Block(Rows([70, 0, 129, 300, 5, 33], 2, 512), 264, 384, act="gelu", eight=eight)
    b.run()
    b.check()
    want = bits(b.outputs())
    for _ in range(30):
        b.run()
    assert all(torch.equal(a, t) for a, t in zip(bits(b.outputs()), want))
    owned = b.rows.owned()
    b.clear()
    b.run()
    for t, w in zip(b.outputs(), want):
        if t.shape[:2] == owned.shape:
            assert torch.equal(t.view(torch.uint8).view(*owned.shape, -1)[owned], w.view(*owned.shape, -1)[owned])
        else:
            assert torch.equal(t.view(torch.uint8), w)


def guarded(rows, width, dtype=torch.bfloat16):
    n = rows.R * rows.max_rows * width
    g = torch.full((n + 2 * GUARD,), SENTINEL, dtype=torch.float32, device="cuda").to(dtype)
    GUARDS.append((g, n))
    return g[GUARD:GUARD + n].view(rows.R, rows.max_rows, width)


GUARDS = []


@pytest.mark.parametrize("counts,R,M,H,F", [([3, 40, 0, 21], 2, 43, 72, 128), ([257, 100], 1, 357, 264, 256)])
def test_nothing_is_written_outside_the_outputs(counts, R, M, H, F):
    GUARDS.clear()
    for eight in (False, True):
        b = Block(Rows(counts, R, M), H, F, eight=eight, make=guarded)
        b.run()
        b.check()
    E = len(counts)
    for n, m in ((2 * F, H), (H, F)):
        g = torch.full((E * n * m + 2 * GUARD,), SENTINEL, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_wgrad(slab(b.rows, 5, n), slab(b.rows, 6, m), b.rows.offsets, g[GUARD:-GUARD].view(E, n, m))
        GUARDS.append((g, E * n * m))
    for g, n in GUARDS:
        v = g.float()
        sentinel = v[0].item()
        assert bool((v[:GUARD] == sentinel).all()) and bool((v[GUARD + n:] == sentinel).all())


def test_streams_and_concurrent_calls():
    """Two blocks at a time on two streams, one of them given, one current; neither is the inputs' stream."""
    blocks = [Block(Rows([200, 17, 0, 90], 2, 256), 520, 256, seed=10 * i + 1) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(10):
        blocks[0].run(streams[0])
        with torch.cuda.stream(streams[1]):
            blocks[1].run()
    torch.cuda.synchronize()
    for b in blocks:
        b.check()


def test_captured_and_replayed_with_other_rows():
    """A graph reads the offsets, rows and weights of its replay, not of its capture."""
    first, second = Rows([10, 0, 64, 33], 2, 150), Rows([0, 149, 2, 5], 2, 150)
    b, c = Block(first, 136, 256, eight=True), Block(second, 136, 256, seed=50, eight=True)
    b.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    g.replay()
    b.check()
    b.rows.offsets.copy_(second.offsets)
    for n in ("x", "dy", "w1", "w2"):
        getattr(b, n).copy_(getattr(c, n))
    for t in (b.h, b.y, b.dpre, b.h2, b.dx, b.s):
        t.fill_(SENTINEL)
    b.q.copy_(torch.full(b.q.shape, SENTINEL, device="cuda").to(b.q.dtype))
    g.replay()
    b.rows.spans, b.rows.dropped = second.spans, second.dropped
    b.check()
    c.run()
    assert all(torch.equal(p, q) for p, q in zip(bits(b.outputs()), bits(c.outputs())))


def test_rows_past_2_31_elements():
    rows = Rows([0, 0, 3, 37], 2, 290000)
    H = 8192  # the second slab begins at element 2.4e9
    x = torch.zeros((2, 290000, H), dtype=torch.bfloat16, device="cuda")
    x[1, :40] = normal(1, 40, H)
    w = normal(2, 4, 2 * 64, H, scale=H ** -0.5)
    h = out(rows, 64)
    ep.ep_expert_gate_up(x, w, rows.offsets, 0, h)
    check_gate_up(x, w, rows, "silu", h)
    dw = torch.empty((4, 64, H), dtype=torch.bfloat16, device="cuda")
    dout = normal(3, 2, 290000, 64)
    ep.ep_expert_wgrad(dout, x, rows.offsets, dw)
    check_wgrad(dout, x, rows, dw)
    w2 = normal(4, 4, H, 64, scale=0.1)
    ep.ep_expert_down(h, w2, rows.offsets, x)
    for e in (2, 3):
        r, a, b = rows.spans[e]
        want = h[r, a:b].double() @ w2[e].double().T
        assert bool(((x[r, a:b].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-3).all())
    assert not x[1, 40:100].any() and not x[0, -100:].any()


def test_weights_past_2_31_elements():
    rows = Rows([0] * 35 + [20], 1, 20)
    H, F = 8192, 4096  # the last expert's weights begin at element 2.3e9
    w = torch.zeros((36, 2 * F, H), dtype=torch.bfloat16, device="cuda")
    w[35] = normal(2, 2 * F, H, scale=H ** -0.5)
    x, h, dx = slab(rows, 1, H), out(rows, F), out(rows, H)
    ep.ep_expert_gate_up(x, w, rows.offsets, 0, h)
    check_gate_up(x, w, rows, "silu", h)
    dpre = slab(rows, 3, 2 * F, 0.1)
    ep.ep_expert_gate_up_bwd(dpre, w, rows.offsets, dx)
    check_gate_up_bwd(dpre, w, rows, dx)
    ep.ep_expert_wgrad(dpre, x, rows.offsets, w)
    check_wgrad(dpre, x, rows, w)


@pytest.mark.parametrize("E,R", [(385, 1), (1024, 16), (3000, 8), (8192, 256)])
def test_many_experts(E, R):
    g = torch.Generator().manual_seed(E)
    counts = torch.randint(0, 3, (E,), generator=g).tolist()
    counts[E - 1] = 70
    per = E // R
    rows = Rows(counts, R, max(sum(counts[r * per:(r + 1) * per]) for r in range(R)))
    b = Block(rows, 16, 128, eight=True)
    b.run()
    b.check()


def test_values_that_are_not_finite_stay_in_their_row_and_expert():
    rows = Rows([40, 40], 1, 80)
    x, w = slab(rows, 1, 128), normal(2, 2, 256, 128, scale=0.1)
    good = out(rows, 128)
    ep.ep_expert_gate_up(x, w, rows.offsets, 0, good)
    x[0, 7, 3], x[0, 50, 5] = math.nan, math.inf
    h = out(rows, 128)
    ep.ep_expert_gate_up(x, w, rows.offsets, 0, h)
    other = torch.ones(80, dtype=torch.bool, device="cuda")
    other[[7, 50]] = False
    assert torch.equal(h[0, other], good[0, other])
    assert bool(h[0, 7].isnan().all()) and not bool(torch.isfinite(h[0, 50]).any())
    dw = torch.empty((2, 128, 128), dtype=torch.bfloat16, device="cuda")
    dout = slab(rows, 3, 128)
    x[0, 50, 5] = 1.0
    ep.ep_expert_wgrad(dout, x, rows.offsets, dw)
    assert bool(dw[0, :, 3].isnan().all()) and bool(torch.isfinite(dw[0, :, 4:]).all()) and bool(torch.isfinite(dw[1]).all())


def test_checkpoint_of_zeros_infinities_and_nan():
    """One channel of x selects what the sums are: the weights' first column times x's first channel."""
    rows = Rows([8], 1, 8)
    H, F = 8, 128
    w = torch.zeros((1, 2 * F, H), dtype=torch.bfloat16, device="cuda")
    w[0, :, 0] = torch.linspace(-3, 3, 2 * F, device="cuda").to(torch.bfloat16)
    w[0, 5, 1], w[0, F + 9, 1] = 1.0, 1.0  # one gate and one up channel of their own
    x = torch.zeros((1, 8, H), dtype=torch.bfloat16, device="cuda")
    x[0, :, 0] = torch.tensor([0, 1, 2.0 ** -110, 1, 1, -2, 2.0 ** 100, 1e-20], device="cuda").to(torch.bfloat16)
    x[0, 3, 1], x[0, 4, 1] = math.inf, math.nan
    h, q, s = out(rows, F), out(rows, 2 * F, torch.float8_e4m3fn), out(rows, 2)
    ep.ep_expert_gate_up(x, w, rows.offsets, 0, h, None, q, s)
    q, s = q[0].float(), s[0].float()
    assert not s[0].any() and not q[0].any()
    assert not s[2].any() and not q[2].any()        # below 2^-100
    assert bool(s[3].isinf().all())
    for c in (5, F + 9):
        assert bool(q[3, c].isnan())
    keep = torch.ones(2 * F, dtype=torch.bool, device="cuda")
    keep[[5, F + 9]] = False
    assert bool(q[4].isnan().all())  # NaN times a zero weight is NaN: the whole row
    assert not q[3, keep & (w[0, :, 0] != 0)].isinf().any()
    for r in (1, 5, 6, 7):
        c = x[0, r, 0].double() * w[0, :, 0].double()
        wide = s[r].double().repeat_interleave(128)
        assert bool(((q[r].double() * wide - c).abs() <= 2.0 ** -4 * c.abs() + 2.0 ** -10 * wide + 2.0 ** -20 * c.abs()).all()), r


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90, 64], [0, -5, 10, 10, 10], [-40, -30, 5, 6, 7],
                                     [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0, 5], [0, 1 << 30, 5, 1 << 30, 9]])
def test_offsets_that_are_wrong_stay_inside_the_slabs(offsets):
    """Rows are taken from inside the slab whatever the offsets say, and nothing else is written."""
    rows = Rows([16] * 4, 2, 64)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    GUARDS.clear()
    x, w, dy = normal(1, 2, 64, 64), normal(2, 4, 256, 64), normal(3, 2, 64, 128)
    h, status = guarded(rows, 128), zero_status()
    ep.ep_expert_gate_up(x, w, off, 0, h, status=status)
    dw = torch.full((4, 128, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_wgrad(dy, x, off, dw, status)
    assert bool(torch.isfinite(dw).all())
    assert ep.read_flags(status) & ~ep.FLAG_CAPACITY == 0
    for g, n in GUARDS:
        assert bool((g[:GUARD].float() == SENTINEL).all()) and bool((g[GUARD + n:].float() == SENTINEL).all())


def reference(x, topk_idx, topk_w, w1, w2, act):
    """The layer in 64 bits, token by token."""
    F = w2.shape[2]
    c = torch.einsum("th,efh->tef", x, w1)
    y = torch.einsum("tef,ehf->teh", act_of(act, c[..., :F])[0] * c[..., F:], w2)
    picked = y.gather(1, topk_idx[:, :, None].expand(-1, -1, y.shape[2]))
    return (picked * topk_w[:, :, None]).sum(1)


@pytest.mark.parametrize("save", ["bf16", "8bit"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_layer_and_its_gradients(act, save):
    """Dispatch, block, weighted return and every gradient, by the helpers, against 64 bits, the gradients
    also against differences of the 64-bit layer. Between two operators rows are rounded to bf16, 2^-8 of
    a value at most and half of that on average: seven roundings on the longest way (h, y, dy, dpre, h,
    dx, the gradient) give at most 7 * 2^-8 = 2.7 % in the 2-norm. The 8-bit checkpoint is off by up to
    2^-4 an element, 2.6 % on average, in gate and in up: at most 2 * 2^-4 more."""
    T, H, F, E, k, R = 150, 128, 256, 8, 3, 4
    bound = 7 * 2.0 ** -8 + (2 * 2.0 ** -4 if save == "8bit" else 0)
    x, dout = normal(1, T, H), normal(2, T, H)
    w1, w2 = normal(3, E, 2 * F, H, scale=H ** -0.5), normal(4, E, H, F, scale=F ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(5)
    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.contiguous()
    tw = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1).contiguous()
    a = ACTS[act]

    lay = ep.get_expert_layout(idx, E)
    M = T * k
    px = ep.dispatch_permuted(x, idx, tw, lay, R, M).perm_x
    up = ep.expert_gate_up(px, w1, lay, a, save)
    y = ep.expert_down(up.h, w2, lay)
    o = ep.combine_permuted(y, idx, tw, lay)
    dy, dtw = ep.combine_permuted_bwd(dout, y, idx, tw, lay)
    dpre, h = ep.expert_down_bwd(dy, w2, up, lay, a)
    dw2 = ep.expert_wgrad(dy, h, lay)
    dw1 = ep.expert_wgrad(dpre, px, lay)
    dx, _ = ep.dispatch_permuted_bwd(ep.expert_gate_up_bwd(dpre, w1, lay), idx, lay)

    leaves = [t.double().requires_grad_() for t in (x, tw, w1, w2)]
    ref = reference(leaves[0], idx, leaves[1], leaves[2], leaves[3], act)
    grads = torch.autograd.grad((ref * dout.double()).sum(), leaves)
    far = lambda p, q: float((p.double() - q).norm() / q.norm())  # noqa: E731
    assert far(o, ref.detach()) < 7 * 2.0 ** -8
    for name, got, want in zip(("x", "topk_w", "w1", "w2"), (dx, dtw, dw1, dw2), grads):
        assert far(got, want) < bound, name
    # differences: the change of the output along a direction is the gradient's product with it
    for i, got in enumerate((dx, dtw, dw1, dw2)):
        d = torch.randn(leaves[i].shape, generator=g, device="cuda", dtype=torch.float64)
        d = d * leaves[i].detach().std() + grads[i] * (leaves[i].detach().norm() / grads[i].norm())
        eps = 1e-5
        moved = [[t.detach() + (s * eps * d if j == i else 0) for j, t in enumerate(leaves)] for s in (1, -1)]
        diff = sum(s * (reference(m[0], idx, m[1], m[2], m[3], act) * dout.double()).sum()
                   for s, m in zip((1, -1), moved)) / (2 * eps)
        assert abs(float((got.double() * d).sum() - diff)) < bound * float(got.double().norm() * d.norm()), i
        assert abs(float((grads[i] * d).sum() - diff)) < 1e-6 * float(grads[i].norm() * d.norm()), i


def test_random_shapes():
    g = torch.Generator().manual_seed(11)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    for i in range(24):
        R = pick(1, 4)
        E = R * pick(1, 6)
        most = [3, 40, 300][i % 3]
        counts = [pick(0, most) if pick(0, 3) else 0 for _ in range(E)]
        per = E // R
        load = max(sum(counts[r * per:(r + 1) * per]) for r in range(R))
        eight = i % 2 == 0
        rows = Rows(counts, R, max(1, load + pick(-2, 5)))
        b = Block(rows, 8 * pick(1, 90), 128 * pick(1, 5) if eight else 8 * pick(1, 80), seed=100 + 10 * i,
                  act=["silu", "gelu"][pick(0, 1)], eight=eight)
        b.run()
        b.check()


def test_arguments_of_cuda_tensors():
    rows = Rows([4, 4], 2, 8)
    b = Block(rows, 64, 128, eight=True)
    off = rows.offsets
    calls = {
        ep.ep_expert_gate_up: dict(x=b.x, w_gate_up=b.w1, expert_offsets=off, act=0, h=b.h, pre=b.dpre, pre_q=b.q,
                                   pre_scales=b.s, status=b.status),
        ep.ep_expert_down: dict(h=b.h, w_down=b.w2, expert_offsets=off, y=b.y, status=b.status),
        ep.ep_expert_down_bwd: dict(dy=b.dy, w_down=b.w2, pre=None, pre_q=b.q, pre_scales=b.s, expert_offsets=off,
                                    act=0, dpre=b.dpre, h=b.h2, status=b.status),
        ep.ep_expert_gate_up_bwd: dict(dpre=b.dpre, w_gate_up=b.w1, expert_offsets=off, dx=b.dx, status=b.status),
        ep.ep_expert_wgrad: dict(dout=b.dpre, rows=b.x, expert_offsets=off, dw=b.dw1, status=b.status),
    }
    optional = {"pre", "status"}
    for f, base in calls.items():
        f(**base)
        for n, v in base.items():
            if not isinstance(v, torch.Tensor):
                continue
            changes = [v.to(torch.float64), v.cpu(), v[None]]
            if n != "status":
                changes.append(torch.cat([v.view(torch.uint8), v.view(torch.uint8)]).view(v.dtype))
            if v.dim() > 1:
                changes.append(v.view(torch.uint8 if v.element_size() == 1 else torch.int16).transpose(0, 1).contiguous()
                               .transpose(0, 1).view(v.dtype))
            if n not in optional and not (n == "h" and f is ep.ep_expert_down_bwd):
                changes.append(None)
            for bad in changes:
                with pytest.raises((ValueError, ep.EpError)):
                    f(**{**base, n: bad})
                    pytest.fail(f"{f.__name__} took a wrong {n}")
    with pytest.raises(ep.EpError, match="EP_ERR_INVALID"):
        ep.ep_expert_gate_up(b.x, b.w1, off, 2, b.h)
    with pytest.raises(ValueError, match="either pre or pre_q"):
        ep.ep_expert_down_bwd(b.dy, b.w2, b.dpre, b.q, b.s, off, 0, b.dpre)
    torch.cuda.synchronize()


def test_helpers_on_another_stream():
    """Helpers allocate and run on the stream that they are given."""
    rows = Rows([60, 10], 1, 80)
    lay = ep.ExpertLayout(rows.offsets, None, None, None, 2)
    x, w1, w2 = slab(rows, 1, 128), normal(2, 2, 512, 128, scale=0.1), normal(3, 2, 128, 256, scale=0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    up = ep.expert_gate_up(x, w1, lay, save="bf16", stream=s)
    y = ep.expert_down(up.h, w2, lay, stream=s)
    dpre, h = ep.expert_down_bwd(y, w2, up, lay, stream=s)
    dx = ep.expert_gate_up_bwd(dpre, w1, lay, stream=s)
    dw = ep.expert_wgrad(dpre, x, lay, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    owned = rows.owned()
    assert not up.h[~owned].any() and not y[~owned].any() and not dpre[~owned].any() and not dx[~owned].any()
    up.pre[~owned] = SENTINEL
    for t in (up.h, y, dpre, dx, h):
        t[~owned] = SENTINEL
    check_gate_up(x, w1, rows, "silu", up.h, up.pre)
    check_down(up.h, w2, rows, y)
    check_down_bwd(y, w2, up.pre, rows, "silu", dpre, h)
    check_gate_up_bwd(dpre, w1, rows, dx)
    check_wgrad(dpre, x, rows, dw)


@pytest.mark.parametrize("I,J", [(16, 64), (40, 72), (104, 520), (232, 200), (264, 1000)])
def test_weights_gradient_of_many_small_tiles(I, J):
    """Tiles that follow one another at once, with every number of chunks a group of warps can have, experts
    without rows among them: none of the sums that are on their way out is overwritten."""
    g = torch.Generator().manual_seed(I)
    counts = torch.randint(-2, 4, (2400,), generator=g).clamp(min=0).tolist()
    rows = Rows(counts, 8, max(sum(counts[r * 300:(r + 1) * 300]) for r in range(8)))
    dout, x = normal(1, 8, rows.max_rows, I), normal(2, 8, rows.max_rows, J)
    dw = torch.full((2400, I, J), SENTINEL, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        ep.ep_expert_wgrad(dout, x, rows.offsets, dw)
    want = torch.zeros((2400, I, J), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    flat = [(e, r * rows.max_rows + p) for e, (r, a, b) in enumerate(rows.spans) for p in range(a, b)]
    e, p = torch.tensor(flat, device="cuda").unbind(1)
    d, v = dout.view(-1, I)[p].double(), x.view(-1, J)[p].double()
    want.index_add_(0, e, d[:, :, None] * v[:, None, :])
    size.index_add_(0, e, (d[:, :, None] * v[:, None, :]).abs())
    assert bool(((dw.double() - want).abs() <= 2.0 ** -8 * want.abs() + 3 * 2.0 ** -23 * size).all())
