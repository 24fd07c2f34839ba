"""The buffer helpers on a stream of their own while the caller's stream is busy, and allocates and
fills memory of the same sizes: results as on one stream, then and after the caller's stream is done."""
import pytest
import torch

import combine_ep_get_05_gb300 as ep

pytestmark = pytest.mark.gpu

T, H, E, k, R = 512, 1024, 16, 4, 4
M = 1024
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


def inputs():
    g = torch.Generator(device="cuda").manual_seed(71)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    idx = torch.argsort(torch.rand((T, E), generator=g, device="cuda"), dim=1)[:, :k].contiguous()
    w = torch.rand((T, k), generator=g, device="cuda")
    return dict(x=bf(T, H), residual=torch.randn((T, H), generator=g, device="cuda"), weight=bf(H), idx=idx, w=w,
                dy=bf(T, H), slab=bf(R, M, H), slab_w=torch.rand((R, M), generator=g, device="cuda"),
                ranks=bf(R, T, H))


def everything(i, stream):
    n = ep.rmsnorm(i["x"], i["weight"], EPS, i["residual"], fp8=True, stream=stream)
    dz, dx, dweight = ep.rmsnorm_bwd(i["dy"], n.residual, i["weight"], EPS, stream=stream)
    lay = ep.get_expert_layout(i["idx"], E, stream=stream)
    p = ep.dispatch_permuted(n.y, i["idx"], i["w"], lay, R, M, stream=stream)
    p8 = ep.dispatch_permuted(n.y_q, i["idx"], i["w"], lay, R, M, scales=n.y_scales, stream=stream)
    back = ep.combine_permuted(i["slab"], i["idx"], i["w"], lay, stream=stream)
    dslab, dw = ep.combine_permuted_bwd(i["dy"], i["slab"], i["idx"], i["w"], lay, stream=stream)
    dsort, dsw = ep.dispatch_permuted_bwd(i["slab"], i["idx"], lay, i["slab_w"], i["dy"], stream=stream)
    ranks = ep.get_layout(i["idx"], E, R, stream=stream)
    d = ep.dispatch(i["x"], i["idx"], i["w"], ranks, T, stream=stream)
    out = ep.combine(i["ranks"], ranks, T, stream=stream)
    return [n.residual, n.y, n.y_q, n.y_scales, dz, dx, dweight, lay.offsets, lay.slot, lay.status, p.perm_x, p.perm_src,
            p.perm_w, p.status, p8.perm_x, p8.perm_scales, p8.perm_src, p8.perm_w, back, dslab, dw, dsort, dsw,
            ranks.slot, ranks.tokens_per_rank, ranks.status, d.status, out]


def same(got, want):
    return [i for i, (g, w) in enumerate(zip(got, want))
            if not torch.equal(g.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8))]


def test_helpers_on_another_stream_while_the_callers_is_busy():
    i = inputs()
    want = everything(i, None)
    sizes = [(t.shape, t.dtype) for t in want]
    torch.cuda.synchronize()
    for t in sizes:  # memory of these sizes in the caller's pool, full of ones
        torch.empty(t[0], dtype=torch.uint8, device="cuda").fill_(255)
    big = torch.ones((8192, 8192), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for _ in range(10):
            big = big @ big * 2.0 ** -13  # the caller's stream has some tens of milliseconds to do
        got = everything(i, side)
        filled = [torch.empty(s, dtype=t, device="cuda").view(torch.uint8).fill_(255) for s, t in sizes]
        side.synchronize()
        with torch.cuda.stream(side):
            assert not same(got, want)
        torch.cuda.synchronize()
        assert not same(got, want)
        del got, filled


def test_what_a_helper_returns_may_be_freed_by_the_callers_stream():
    """The caller's stream reads a result late; the result is dropped and the side stream allocates
    that much again before the read is done."""
    i = inputs()
    want = ep.rmsnorm(i["x"], i["weight"], EPS, i["residual"]).y.clone()
    big = torch.ones((8192, 8192), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        n = ep.rmsnorm(i["x"], i["weight"], EPS, i["residual"], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(10):
            big = big @ big * 2.0 ** -13
        copy = n.y.clone()
        del n
        again = [ep.rmsnorm(i["dy"], i["weight"], EPS, i["residual"], stream=side) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
        del again


def test_a_stream_may_be_anything_with_a_handle():
    """What the entry points ask of a stream, its cuda_stream, is enough for the helpers too."""
    i = inputs()
    want = everything(i, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    got = everything(i, Handle())
    torch.cuda.synchronize()
    assert not same(got, want)
    external = everything(i, torch.cuda.ExternalStream(side.cuda_stream))
    torch.cuda.synchronize()
    assert not same(external, want)
