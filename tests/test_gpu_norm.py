"""ep_rmsnorm and ep_rmsnorm_bwd against their definitions in 64 bits.

Tolerances, with u = 2^-24 (half an ulp of fp32, relative). A row's sum is at most 32
fused terms per thread and 10 additions across the block, so the sum of squares is within
42 u of itself and rstd within 21 u plus 4 u for the mean, eps and the reciprocal root; two
products and the addition of the residual add 3 u: v is within 32 u < 2^-18. A bf16 output
is the rounding of some value within that bound: it lies between the roundings of the
bound's two ends. E4M3 adds half a step of its grid, scales 2 u. In the gradient the sum of g z is within
42 u of the sum of magnitudes; with the factors and the final additions every element is
within 128 u of the sum of the magnitudes of its terms. A channel of dweight is a sum of at
most T terms in any order: within (T + 16) u of the sum of the terms' magnitudes (16: each
term's own roundings and rstd's).
"""
import numpy as np
import pytest
import torch

import combine_ep_get_05_gb300 as ep
from gpu_helpers import check_guards, guarded, host_bits, SENT_BF16, SENT_F32

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


def rand(shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def weights(H, dtype, seed=5):
    return (1.0 + 0.3 * rand((H,), seed, dtype=torch.float32)).to(dtype)


def definition(x, residual, weight, eps=EPS):
    z = 0.0
    if x is not None:
        z = z + x.double()
    if residual is not None:
        z = z + residual.double()
    v = z / torch.sqrt((z * z).mean(1, keepdim=True) + eps) * weight.double()
    return z, v


def rounds_from(got, ref, bound):
    """Every bf16 of `got` is the rounding of some value within `bound` of `ref` (rounding is
    monotone, so it lies between the roundings of the two ends)."""
    lo, hi = (ref - bound).to(torch.bfloat16), (ref + bound).to(torch.bfloat16)
    return bool(torch.all((got >= lo) & (got <= hi)))


def e4m3_step(a):
    """Spacing of the E4M3 grid around |a| (subnormal spacing 2^-9)."""
    e = torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 3)


def check_quantised(q, scales, v):
    """Codes and scales of rows whose blocks are finite, against v in 64 bits."""
    T, H = v.shape
    blocks = v.view(T, H // 128, 128)
    ref = blocks.abs().amax(2) / 448.0
    assert torch.all((scales.double() - ref).abs() <= ref * 2.0 ** -18 + 2.0 ** -149)
    a = blocks / torch.where(ref > 0, ref, 1.0)[:, :, None]
    got = q.view(torch.float8_e4m3fn).double().view(T, H // 128, 128)
    slack = a.abs() * 2.0 ** -17
    assert torch.all((got - a).abs() <= 0.5 * e4m3_step(a.abs() + slack) + slack)


SIZES = [(1, 8), (3, 136), (1, 7168), (2, 128), (33, 1000), (257, 1024), (130, 4104), (5, 16384), (64, 2176), (7, 8192)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("carry", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32])
def test_norm_against_definition(T, H, carry, wdt):
    x = rand((T, H), 1)
    residual = rand((T, H), 2, 3.0, carry)
    weight = weights(H, wdt)
    fp8 = H % 128 == 0
    sent = SENT_BF16 if carry == torch.bfloat16 else SENT_F32
    rout, rback = guarded((T, H), carry, sent)
    y, yback = guarded((T, H), torch.bfloat16, SENT_BF16)
    q, qback = guarded((T, H), torch.uint8, 0x7E) if fp8 else (None, None)
    sc, sback = guarded((T, H // 128), torch.float32, SENT_F32) if fp8 else (None, None)
    ep.ep_rmsnorm(x, residual, weight, EPS, rout, y, q, sc)
    torch.cuda.synchronize()
    z, v = definition(x, residual, weight)
    assert torch.equal(rout, (x.float() + residual.float()).to(carry))
    assert rounds_from(y, v, v.abs() * 2.0 ** -18)
    check_guards(rback, T * H, sent)
    check_guards(yback, T * H, SENT_BF16)
    if fp8:
        check_quantised(q, sc, v)
        check_guards(qback, T * H, 0x7E)
        check_guards(sback, T * H // 128, SENT_F32)


@pytest.mark.parametrize("T,H", [(20000, 8), (12000, 264), (12001, 512), (5000, 1032), (1500, 4104), (1200, 7168),
                                 (400, 16384), (153, 128)])
@pytest.mark.parametrize("carry", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inputs", ["x", "residual", "both"])
def test_norm_of_many_rows(T, H, carry, inputs):
    """More rows than fit the GPU at once: every form of the kernel takes several rows a CTA."""
    x = rand((T, H), 61) if inputs != "residual" else None
    residual = rand((T, H), 62, 3.0, carry) if inputs != "x" else None
    weight = weights(H, torch.float32 if T % 2 else torch.bfloat16)
    fp8 = H % 128 == 0
    sent = SENT_BF16 if carry == torch.bfloat16 else SENT_F32
    rout, rback = guarded((T, H), carry, sent)
    y, yback = guarded((T, H), torch.bfloat16, SENT_BF16)
    q, qback = guarded((T, H), torch.uint8, 0x7E) if fp8 else (None, None)
    sc, sback = guarded((T, H // 128), torch.float32, SENT_F32) if fp8 else (None, None)
    ep.ep_rmsnorm(x, residual, weight, EPS, rout, y, q, sc)
    torch.cuda.synchronize()
    z, v = definition(x, residual, weight)
    assert torch.equal(rout, (x.float() + residual.float() if inputs == "both" else
                              x.float() if inputs == "x" else residual.float()).to(carry))
    assert rounds_from(y, v, v.abs() * 2.0 ** -18)
    check_guards(rback, T * H, sent)
    check_guards(yback, T * H, SENT_BF16)
    if fp8:
        check_quantised(q, sc, v)
        check_guards(qback, T * H, 0x7E)
        check_guards(sback, T * H // 128, SENT_F32)


@pytest.mark.parametrize("H", [128, 1024, 7168])
@pytest.mark.parametrize("case", ["x only", "residual only", "fp8 only", "y only", "residual_out of x"])
def test_norm_subsets_of_inputs_and_outputs(H, case):
    T = 19
    x = rand((T, H), 3) if case != "residual only" else None
    residual = rand((T, H), 4, 2.0, torch.float32) if case in ("residual only", "fp8 only") else None
    weight = weights(H, torch.float32)
    z, v = definition(x, residual, weight)
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda") if case != "fp8 only" else None
    q = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda") if case != "y only" else None
    sc = torch.empty((T, H // 128), device="cuda") if q is not None else None
    rout = torch.empty((T, H), device="cuda") if case == "residual_out of x" else None
    ep.ep_rmsnorm(x, residual, weight, EPS, rout, y, q, sc)
    torch.cuda.synchronize()
    if y is not None:
        assert rounds_from(y, v, v.abs() * 2.0 ** -18)
    if q is not None:
        check_quantised(q, sc, v)
    if rout is not None:
        assert torch.equal(rout, x.float())


@pytest.mark.parametrize("carry", [torch.bfloat16, torch.float32])
def test_norm_in_place(carry):
    T, H = 37, 1024
    x, residual, weight = rand((T, H), 6), rand((T, H), 7, 2.0, carry), weights(H, torch.bfloat16)
    rout, y = torch.empty_like(residual), torch.empty_like(x)
    ep.ep_rmsnorm(x, residual, weight, EPS, rout, y)
    x2, r2 = x.clone(), residual.clone()
    ep.ep_rmsnorm(x2, r2, weight, EPS, r2, x2)
    assert torch.equal(r2, rout) and torch.equal(x2, y)


@pytest.mark.parametrize("H", [128, 7168])
def test_norm_of_zero_rows_zero_blocks_and_zero_weights(H):
    T = 4
    x = rand((T, H), 8)
    x[1] = 0.0
    x[2] = -0.0
    weight = weights(H, torch.float32)
    if H > 128:
        weight[128:256] = 0.0
    y = torch.empty_like(x)
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sc = torch.empty((T, H // 128), device="cuda")
    ep.ep_rmsnorm(x, None, weight, EPS, None, y, q, sc)
    minus = (weight < 0).to(torch.uint8) * 0x80  # +0 times a negative weight is -0
    assert torch.all(y[1] == 0) and torch.equal(q[1], minus) and torch.all(sc[1] == 0)
    assert torch.all(y[2] == 0) and torch.equal(q[2], minus ^ 0x80) and torch.all(sc[2] == 0)
    if H > 128:
        assert torch.all(sc[:, 1] == 0) and torch.all((q[:, 128:256] & 0x7F) == 0)
    _, v = definition(x, None, weight)
    check_quantised(q, sc, v)


def test_norm_eps_zero_and_tiny_rows():
    """Rows far below and above 1: the norm brings them to the same size; with eps = 0 a
    zero row is 0 * inf = NaN, as the formula says."""
    H = 1024
    x = rand((4, H), 9)
    x[0] *= 2.0 ** -40
    x[1] *= 2.0 ** 40
    x[3] = 0.0
    weight = weights(H, torch.bfloat16)
    y = torch.empty_like(x)
    q = torch.empty((4, H), dtype=torch.uint8, device="cuda")
    sc = torch.empty((4, H // 128), device="cuda")
    ep.ep_rmsnorm(x, None, weight, 0.0, None, y, q, sc)
    _, v = definition(x[:3], None, weight, 0.0)
    assert rounds_from(y[:3], v, v.abs() * 2.0 ** -18)
    check_quantised(q[:3], sc[:3], v)
    assert torch.all(torch.isnan(y[3]))


def test_norm_of_nan_and_infinity():
    """A NaN makes its row NaN; an infinity its own element NaN and the rest of its row 0;
    other rows are untouched. NaNs have the NaN code in E4M3."""
    H = 1024
    x = rand((4, H), 10)
    clean = x.clone()
    x[1, 5] = float("nan")
    x[2, 300] = float("inf")
    weight = weights(H, torch.bfloat16)
    outs = []
    for xx in (clean, x):
        y = torch.empty_like(x)
        q = torch.empty((4, H), dtype=torch.uint8, device="cuda")
        sc = torch.empty((4, H // 128), device="cuda")
        ep.ep_rmsnorm(xx, None, weight, EPS, None, y, q, sc)
        outs.append((y, q, sc))
    (y0, q0, s0), (y1, q1, s1) = outs
    for r in (0, 3):
        assert torch.equal(y0[r], y1[r]) and torch.equal(q0[r], q1[r]) and torch.equal(s0[r], s1[r])
    assert torch.all(torch.isnan(y1[1])) and torch.all((q1[1] & 0x7F) == 0x7F)
    assert torch.isnan(y1[2, 300]) and int(q1[2, 300]) & 0x7F == 0x7F
    rest = torch.ones(H, dtype=torch.bool, device="cuda")
    rest[300] = False
    assert torch.all(y1[2][rest] == 0) and torch.all((q1[2][rest] & 0x7F) == 0) and torch.all(s1[2] == 0)


def test_norm_quantises_as_the_fp8_dispatch_does():
    """One row format: with weights of 1 and rows whose rstd is a power of two, v is a bf16
    value, and the codes and scales are those the FP8 dispatch makes of it."""
    T, H = 16, 1024
    x = torch.where(rand((T, H), 11).float() > 0, 2.0, -2.0).to(torch.bfloat16)
    weight = torch.ones(H, device="cuda")
    weight[::3] = 0.375
    y = torch.empty_like(x)
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sc = torch.empty((T, H // 128), device="cuda")
    ep.ep_rmsnorm(x, None, weight, 0.0, None, y, q, sc)
    topk = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    tw = torch.ones((T, 1), device="cuda")
    lay = ep.get_layout(topk, 1, 1)
    d = ep.dispatch(y, topk, tw, lay, T, fp8=True)
    assert torch.equal(d.recv_x[0], q) and torch.equal(d.recv_scales[0], sc)


@pytest.mark.parametrize("carry", [torch.bfloat16, torch.float32])
def test_norm_quantises_blocks_whose_scale_is_subnormal(carry):
    """Blocks around 2^-130, whose scale has no finite reciprocal, next to ordinary ones: the
    division itself, as the FP8 dispatch makes it of the same bf16 values."""
    T, H = 9, 1024
    x = torch.where(rand((T, H), 14).float() > 0, 2.0, -2.0)
    weight = torch.ones(H, device="cuda")
    weight[::3] = 0.375
    weight[::5] = 0.5
    weight[128:384] *= 2.0 ** -130
    weight[640:768] *= 2.0 ** -118
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sc = torch.empty((T, H // 128), device="cuda")
    ep.ep_rmsnorm(None, x.to(carry), weight, 0.0, None, y, q, sc)
    topk = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    lay = ep.get_layout(topk, 1, 1)
    d = ep.dispatch(y, topk, torch.ones((T, 1), device="cuda"), lay, T, fp8=True)
    assert torch.all(sc[:, 1:3] < 2.0 ** -126) and torch.all(sc[:, 1:3] > 0)
    assert torch.equal(d.recv_scales[0], sc) and torch.equal(d.recv_x[0], q)


def test_norm_rounds_codes_once_where_scales_are_small():
    """Values at and beside the midpoints of codes, with scales from 2^-126 to 2^-80: a quotient whose
    correction underflows is off by an fp32 ulp, which shows here. The codes are those of the IEEE division."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mids = (codes[:-1] + codes[1:]) / 2
    r = np.random.default_rng(31)
    blocks = 127
    H = 128 * (blocks + 1)
    w = np.full(H, 448.0, dtype=np.float32)  # the first block shows that the root mean square is exactly 1
    for b in range(blocks):
        keep = r.integers(4, 24)  # leading bits of the scale
        m = 1.0 + np.floor(r.random() * 2.0 ** keep) / 2.0 ** keep
        amax = np.float32(448.0 * m * 2.0 ** (-126 + b % 47))
        scale = amax / np.float32(448.0)
        v = (r.choice(mids, 127) * np.float64(scale)).astype(np.float32)
        beside = np.nextafter(v, np.float32(1)), np.nextafter(v, np.float32(0))
        v = np.where(np.arange(127) % 4 < 2, v, np.where(np.arange(127) % 4 == 2, beside[0], beside[1]))
        w[128 * (b + 1):128 * (b + 2)] = np.append(v, amax)
    x = torch.where(rand((3, H), 32).float() > 0, 1.0, -1.0).bfloat16()
    for carry in (torch.bfloat16, torch.float32):
        q = torch.empty((3, H), dtype=torch.uint8, device="cuda")
        sc = torch.empty((3, H // 128), device="cuda")
        ep.ep_rmsnorm(None, x.to(carry), torch.from_numpy(w).cuda(), 0.0, None, None, q, sc)
        sc = sc.cpu()
        assert torch.all(sc[:, 0] == 1.0)
        want = w.reshape(-1, 128) / sc[0].numpy()[:, None]
        want = torch.from_numpy(want.reshape(H)).to(torch.float8_e4m3fn).view(torch.uint8)
        sign = (x < 0).to(torch.uint8).cpu() << 7
        assert torch.equal(q.cpu(), want[None] | sign)
        assert torch.equal(sc[0], sc[1]) and torch.equal(sc[0], sc[2])


def test_norm_offsets_past_32_bits():
    T, H = 140_000, 16384
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[-3:] = rand((3, H), 12)
    weight = weights(H, torch.bfloat16)
    y = torch.empty_like(x)
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sc = torch.empty((T, H // 128), device="cuda")
    ep.ep_rmsnorm(x, None, weight, EPS, None, y, q, sc)
    _, v = definition(x[-3:], None, weight)
    assert rounds_from(y[-3:], v, v.abs() * 2.0 ** -18)
    check_quantised(q[-3:], sc[-3:], v)
    assert torch.all(y[:1000] == 0) and torch.all((q[-1000:-3] & 0x7F) == 0)
    del y, q
    dz = torch.empty_like(x)
    dw = torch.empty(H, device="cuda")
    ws = torch.empty(ep.ep_rmsnorm_bwd_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    dy = torch.zeros_like(x)
    dy[-3:] = rand((3, H), 13)
    ep.ep_rmsnorm_bwd(dy, x, weight, None, EPS, dz, None, dw, ws)
    d, bound, wref, wmag = gradient(dy[-3:], x[-3:], weight, None)
    assert rounds_from(dz[-3:], d, bound)
    assert torch.all((dw.double() - wref).abs() <= (3 + 16) * U * wmag)


# --------------------------------------------------------------------------- gradient

def gradient(dy, z, weight, dz_in, eps=EPS):
    """d, its fp32 error bound, dweight and the sum of the magnitudes of dweight's terms."""
    z, dy, w = z.double(), dy.double(), weight.double()
    rstd = 1.0 / torch.sqrt((z * z).mean(1, keepdim=True) + eps)
    g = dy * w
    mean = (g * z).mean(1, keepdim=True)
    d = rstd * (g - z * rstd ** 2 * mean)
    mag = rstd * (g.abs() + z.abs() * rstd ** 2 * (g * z).abs().mean(1, keepdim=True))
    if dz_in is not None:
        d = d + dz_in.double()
        mag = mag + dz_in.double().abs()
    terms = dy * z * rstd
    return d, 128 * U * mag + 2.0 ** -140, terms.sum(0), terms.abs().sum(0)


def run_bwd(dy, z, weight, dz_in, dx=True, dweight=True):
    T, H = z.shape
    sent = SENT_BF16 if z.dtype == torch.bfloat16 else SENT_F32
    dz, dzback = guarded((T, H), z.dtype, sent)
    dxt = torch.empty((T, H), dtype=torch.bfloat16, device="cuda") if dx else None
    dw, dwback = guarded((H,), torch.float32, SENT_F32) if dweight else (None, None)
    size = ep.ep_rmsnorm_bwd_workspace_size(T, H)
    ws, wsback = guarded((size,), torch.uint8, 0x55) if dweight else (None, None)
    ep.ep_rmsnorm_bwd(dy, z, weight, dz_in, EPS, dz, dxt, dw, ws)
    torch.cuda.synchronize()
    check_guards(dzback, T * H, sent)
    if dweight:
        check_guards(dwback, H, SENT_F32)
        check_guards(wsback, size, 0x55)
    return dz, dxt, dw


@pytest.mark.parametrize("T,H", SIZES + [(1500, 264), (700, 7168), (20000, 264), (3000, 1032), (9000, 8), (400, 16384)])
@pytest.mark.parametrize("carry", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32])
def test_norm_gradient_against_formula(T, H, carry, wdt):
    dy, z, weight = rand((T, H), 21), rand((T, H), 22, 2.0, carry), weights(H, wdt)
    dz_in = rand((T, H), 23, 0.5, carry) if T % 2 else None
    d, bound, wref, wmag = gradient(dy, z, weight, dz_in)
    dz, dx, dw = run_bwd(dy, z, weight, dz_in)
    if carry == torch.bfloat16:
        assert rounds_from(dz, d, bound)
    else:
        assert torch.all((dz.double() - d).abs() <= bound + d.abs() * U)
    assert rounds_from(dx, d, bound)
    assert torch.all((dw.double() - wref).abs() <= (T + 16) * U * wmag)


@pytest.mark.parametrize("T,H", [(3, 136), (40, 1024), (9, 7168)])
def test_norm_gradient_against_differences(T, H):
    """Central differences of the definition in 64 bits along random directions of z and of
    the weight: step 1e-4 relative, truncation below 1e-6 of the gradient's size."""
    dy, z, weight = rand((T, H), 31), rand((T, H), 32, 2.0, torch.float32), weights(H, torch.float32)
    dz, _, dw = run_bwd(dy, z, weight, None)

    def loss(zz, ww):
        v = zz / torch.sqrt((zz * zz).mean(1, keepdim=True) + EPS) * ww
        return float((v * dy.double()).sum())

    g = torch.Generator(device="cuda").manual_seed(33)
    for _ in range(3):
        dir_z = torch.randn((T, H), generator=g, device="cuda", dtype=torch.float64)
        dir_w = torch.randn((H,), generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        fz = (loss(z.double() + h * dir_z, weight.double()) - loss(z.double() - h * dir_z, weight.double())) / (2 * h)
        fw = (loss(z.double(), weight.double() + h * dir_w) - loss(z.double(), weight.double() - h * dir_w)) / (2 * h)
        size_z = float(dz.double().norm() * dir_z.norm() / np.sqrt(T * H))
        size_w = float(dw.double().norm() * dir_w.norm() / np.sqrt(H))
        assert abs(float((dz.double() * dir_z).sum()) - fz) <= 2e-5 * size_z * np.sqrt(T * H)
        assert abs(float((dw.double() * dir_w).sum()) - fw) <= 2e-5 * size_w * np.sqrt(H)


def test_norm_gradient_in_place_without_dweight_and_repeatable():
    T, H = 301, 2176
    dy, z, weight = rand((T, H), 41), rand((T, H), 42, 2.0), weights(H, torch.bfloat16)
    dz_in = rand((T, H), 43)
    dz, _, dw = run_bwd(dy, z, weight, dz_in, dx=False)
    again, _, dw2 = run_bwd(dy, z, weight, dz_in, dx=False)
    assert torch.equal(dz, again) and torch.equal(dw, dw2)
    alone, _, _ = run_bwd(dy, z, weight, dz_in, dx=False, dweight=False)
    assert torch.equal(dz, alone)
    buf = dz_in.clone()
    ep.ep_rmsnorm_bwd(dy, z, weight, buf, EPS, buf)
    assert torch.equal(buf, dz)


def test_norm_gradient_of_an_empty_batch():
    H = 256
    empty = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((H,), 3.0, device="cuda")
    ws = torch.empty(0, dtype=torch.uint8, device="cuda")
    ep.ep_rmsnorm(empty, None, weights(H, torch.bfloat16), EPS, None, empty)
    ep.ep_rmsnorm_bwd(empty, empty, weights(H, torch.bfloat16), None, EPS, empty, None, dw, ws)
    assert torch.all(dw == 0)


def test_norm_on_another_stream_and_in_a_graph():
    T, H = 64, 1024
    x, residual, weight = rand((T, H), 51), rand((T, H), 52), weights(H, torch.bfloat16)
    ref_r, ref_y = torch.empty_like(x), torch.empty_like(x)
    ep.ep_rmsnorm(x, residual, weight, EPS, ref_r, ref_y)
    dz_ref, _, dw_ref = run_bwd(ref_y, ref_r, weight, None, dx=False)
    rout, y, dz, dw = (torch.zeros_like(t) for t in (x, x, x, dw_ref))
    ws = torch.empty(ep.ep_rmsnorm_bwd_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ep.ep_rmsnorm(x, residual, weight, EPS, rout, y)
        ep.ep_rmsnorm_bwd(y, rout, weight, None, EPS, dz, None, dw, ws)
    for _ in range(3):
        for t in (rout, y, dz, dw):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(rout, ref_r) and torch.equal(y, ref_y) and torch.equal(dz, dz_ref) and torch.equal(dw, dw_ref)
    with torch.cuda.stream(side):
        y.zero_()
        ep.ep_rmsnorm(x, residual, weight, EPS, rout, y)
    side.synchronize()
    assert torch.equal(y, ref_y)
    assert host_bits(y).shape == (T, H)
