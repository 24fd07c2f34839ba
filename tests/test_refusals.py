"""What the norm, the E4M3 sort and the gradients refuse: at the C entry before anything is
launched (EP_ERR_INVALID), and in the binding before the library is called (ValueError).
CPU only; the pointers are never dereferenced."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
OK, INVALID = 0, 1
F = P(4096)      # a 16-byte aligned address
ODD = P(4096 + 4)


@pytest.fixture(scope="module", autouse=True)
def L():
    from combine_ep_get_05_gb300 import _lib, build

    build.build()
    return _lib.lib()


def call(fn, defaults, **change):
    args = dict(defaults)
    assert set(change) <= set(args), change
    args.update(change)
    return fn(*args.values())


NORM = dict(x=F, residual=F, weight=F, stream_dtype=0, weight_dtype=0, eps=1e-6, T=4, H=256, residual_out=F, y=F, y_q=F,
            y_scales=F, stream=None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(H=0), dict(H=-8), dict(H=260), dict(H=16392), dict(H=136), dict(stream_dtype=1),
    dict(stream_dtype=3), dict(weight_dtype=1), dict(weight_dtype=-1), dict(eps=-1.0), dict(eps=float("nan")),
    dict(x=None, residual=None), dict(weight=None), dict(y_q=None), dict(y_scales=None),
    dict(residual_out=None, y=None, y_q=None, y_scales=None), dict(x=ODD), dict(residual=ODD), dict(weight=ODD),
    dict(residual_out=ODD), dict(y=ODD), dict(y_q=ODD), dict(y_scales=ODD)], ids=str)
def test_norm_refuses(L, change):
    assert call(L.ep_rmsnorm, NORM, **change) == INVALID


def test_norm_of_no_rows_is_ok(L):
    assert call(L.ep_rmsnorm, NORM, T=0, x=None, residual=None, weight=None) == OK


BWD = dict(dy=F, z=F, weight=F, dz_in=F, stream_dtype=0, weight_dtype=0, eps=1e-6, T=4, H=256, dz=F, dx=F, dweight=F,
           workspace=F, workspace_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(H=0), dict(H=12), dict(H=16392), dict(stream_dtype=1), dict(weight_dtype=5), dict(eps=-1e-3),
    dict(dy=None), dict(z=None), dict(weight=None), dict(dz=None), dict(workspace=None), dict(workspace_bytes=4095),
    dict(dy=ODD), dict(z=ODD), dict(weight=ODD), dict(dz_in=ODD), dict(dz=ODD), dict(dx=ODD), dict(dweight=ODD),
    dict(workspace=ODD)], ids=str)
def test_norm_gradient_refuses(L, change):
    assert call(L.ep_rmsnorm_bwd, BWD, **change) == INVALID


def test_norm_gradient_workspace_is_host_arithmetic(L):
    size = L.ep_rmsnorm_bwd_workspace_size
    assert size(0, 256) == 0 and size(-1, 256) == 0 and size(4, 0) == 0 and size(4, 16392) == 0
    assert size(4, 256) == 4 * 256 * 4
    assert size(1 << 20, 16384) == size(1 << 21, 16384) < 1 << 26  # bounded for any batch
    assert call(L.ep_rmsnorm_bwd, BWD, T=0, dweight=None, workspace=None, dy=None) == OK


SORT = dict(x_q=F, x_scales=F, topk_idx=F, topk_w=F, expert_offsets=F, expert_slot=F, T=4, H=256, k=2, E=8, R=4,
            max_rows=4, perm_q=F, perm_scales=F, perm_src=F, perm_w=F, status=None, stream=None)
ROUTING = [dict(T=-1), dict(k=0), dict(k=33), dict(R=0), dict(R=257, E=257), dict(E=9), dict(E=2), dict(E=8196),
           dict(max_rows=-1), dict(R=4, max_rows=1 << 30), dict(topk_idx=None), dict(expert_offsets=None),
           dict(expert_slot=None), dict(topk_idx=ODD), dict(expert_offsets=ODD), dict(expert_slot=ODD)]


@pytest.mark.parametrize("change", ROUTING + [
    dict(H=0), dict(H=192), dict(H=65664), dict(x_q=None), dict(x_scales=None), dict(perm_q=None),
    dict(perm_scales=None), dict(topk_w=None), dict(x_q=ODD), dict(x_scales=ODD), dict(perm_q=ODD),
    dict(perm_scales=ODD), dict(perm_src=ODD), dict(perm_w=ODD), dict(topk_w=ODD)], ids=str)
def test_fp8_sort_refuses(L, change):
    assert call(L.ep_dispatch_permuted_fp8, SORT, **change) == INVALID
    order = ("x_q", "x_scales", "topk_idx", "topk_w", "T", "H", "k", "E", "R", "max_rows", "expert_offsets",
             "expert_slot", "perm_q", "perm_scales", "perm_src", "perm_w", "status", "stream")
    assert call(L.ep_dispatch_permuted_fp8_ll, {n: SORT[n] for n in order}, **change) == INVALID


def test_fp8_sort_limits_of_the_one_launch_form(L):
    order = ("x_q", "x_scales", "topk_idx", "topk_w", "T", "H", "k", "E", "R", "max_rows", "expert_offsets",
             "expert_slot", "perm_q", "perm_scales", "perm_src", "perm_w", "status", "stream")
    base = {n: SORT[n] for n in order}
    assert call(L.ep_dispatch_permuted_fp8_ll, base, T=1025, k=1) == INVALID
    assert call(L.ep_dispatch_permuted_fp8_ll, base, T=1024, k=9) == INVALID
    assert call(L.ep_dispatch_permuted_fp8_ll, base, E=1028) == INVALID
    assert call(L.ep_dispatch_permuted_fp8, SORT, T=0, x_q=None, x_scales=None, topk_idx=None) == OK


SORT_BWD = dict(dperm_x=F, dperm_w=F, dx_in=F, topk_idx=F, expert_offsets=F, expert_slot=F, T=4, H=256, k=2, E=8, R=4,
                max_rows=4, dx=F, dtopk_w=F, status=None, stream=None)


@pytest.mark.parametrize("change", ROUTING + [
    dict(H=0), dict(H=100), dict(dperm_x=None), dict(dperm_w=None), dict(dx=None), dict(dperm_x=ODD),
    dict(dperm_w=ODD), dict(dx_in=ODD), dict(dx=ODD), dict(dtopk_w=ODD)], ids=str)
def test_sort_gradient_refuses(L, change):
    assert call(L.ep_dispatch_permuted_bwd, SORT_BWD, **change) == INVALID


RETURN_BWD = dict(dout=F, y=F, topk_idx=F, topk_w=F, expert_offsets=F, expert_slot=F, T=4, H=256, k=2, E=8, R=4,
                  max_rows=4, dy=F, dtopk_w=F, status=None, stream=None)


@pytest.mark.parametrize("change", ROUTING + [
    dict(H=0), dict(H=100), dict(dout=None), dict(y=None), dict(dy=None), dict(topk_w=None), dict(dout=ODD),
    dict(y=ODD), dict(topk_w=ODD), dict(dy=ODD), dict(dtopk_w=ODD)], ids=str)
def test_return_gradient_refuses(L, change):
    assert call(L.ep_combine_permuted_bwd, RETURN_BWD, **change) == INVALID


def test_binding_refuses_host_tensors_wrong_types_and_shapes():
    import combine_ep_get_05_gb300 as ep

    T, H, k, E, R, M = 4, 256, 2, 8, 4, 4
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    f32, i32 = (lambda *s: torch.zeros(s)), (lambda *s: torch.zeros(s, dtype=torch.int32))
    q, sc = torch.zeros((T, H), dtype=torch.uint8), f32(T, H // 128)
    idx, off, slot = torch.zeros((T, k), dtype=torch.int64), i32(E + 1), i32(T, k)
    with pytest.raises(ValueError, match="x or residual"):
        ep.ep_rmsnorm(None, None, bf(H), 1e-6, None, bf(T, H))
    with pytest.raises(ValueError, match="residual stream"):
        ep.ep_rmsnorm(bf(T, H), bf(T, H), bf(H), 1e-6, f32(T, H))
    with pytest.raises(ValueError, match="residual stream"):
        ep.ep_rmsnorm(bf(T, H), torch.zeros((T, H), dtype=torch.float16), bf(H), 1e-6, None, bf(T, H))
    with pytest.raises(ValueError, match="residual stream"):
        ep.ep_rmsnorm_bwd(bf(T, H), torch.zeros((T, H), dtype=torch.float16), bf(H), None, 1e-6, bf(T, H))
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ep.ep_rmsnorm(bf(T, H), None, bf(H), 1e-6, None, bf(T, H))
    with pytest.raises(ValueError, match="dy must be a CUDA tensor"):
        ep.ep_rmsnorm_bwd(bf(T, H), bf(T, H), bf(H), None, 1e-6, bf(T, H))
    with pytest.raises(ValueError, match="x_q must be a CUDA tensor"):
        ep.ep_dispatch_permuted_fp8(q, sc, idx, None, off, slot, E, R, M, q, sc)
    with pytest.raises(ValueError, match="x_q must be a CUDA tensor"):
        ep.ep_dispatch_permuted_fp8_ll(q, sc, idx, None, E, R, M, off, slot, q, sc)
    with pytest.raises(ValueError, match="dperm_x must be a CUDA tensor"):
        ep.ep_dispatch_permuted_bwd(bf(R, M, H), None, None, idx, off, slot, E, bf(T, H))
    with pytest.raises(ValueError, match="dout must be a CUDA tensor"):
        ep.ep_combine_permuted_bwd(bf(T, H), bf(R, M, H), idx, f32(T, k), off, slot, E, bf(R, M, H), f32(T, k))
