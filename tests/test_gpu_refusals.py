"""What the norm, the E4M3 sort and the gradients refuse of CUDA tensors: types, shapes,
strides, missing arguments and integers out of range raise before anything is launched, and
the outputs keep what they held."""
import pytest
import torch

import combine_ep_get_05_gb300 as ep

pytestmark = pytest.mark.gpu

T, H, k, E, R, M = 4, 256, 2, 8, 4, 5


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def f32(*shape):
    return z(*shape, dtype=torch.float32)


def i32(*shape):
    return z(*shape, dtype=torch.int32)


def arguments():
    idx = z(T, k, dtype=torch.int64)
    q = z(T, H, dtype=torch.uint8)
    routing = dict(topk_idx=idx, expert_offsets=i32(E + 1), expert_slot=i32(T, k))
    sort = dict(x_q=q, x_scales=f32(T, 2), topk_w=f32(T, k), num_experts=E, num_ranks=R, max_rows=M,
                perm_q=z(R, M, H, dtype=torch.float8_e4m3fn), perm_scales=f32(R, M, 2), perm_src=i32(R, M),
                perm_w=f32(R, M), status=i32(1), **routing)
    return {
        ep.ep_rmsnorm: dict(x=z(T, H), residual=f32(T, H), weight=f32(H), eps=1e-6, residual_out=f32(T, H), y=z(T, H),
                            y_q=q, y_scales=f32(T, 2)),
        ep.ep_rmsnorm_bwd: dict(dy=z(T, H), z=f32(T, H), weight=z(H), dz_in=f32(T, H), eps=1e-6, dz=f32(T, H),
                                dx=z(T, H), dweight=f32(H), workspace=z(1 << 16, dtype=torch.uint8)),
        ep.ep_dispatch_permuted_fp8: sort,
        ep.ep_dispatch_permuted_fp8_ll: dict(sort),
        ep.ep_dispatch_permuted_bwd: dict(dperm_x=z(R, M, H), dperm_w=f32(R, M), dx_in=z(T, H), num_experts=E, dx=z(T, H),
                                          dtopk_w=f32(T, k), status=i32(1), **routing),
        ep.ep_combine_permuted_bwd: dict(dout=z(T, H), y=z(R, M, H), topk_w=f32(T, k), num_experts=E, dy=z(R, M, H),
                                         dtopk_w=f32(T, k), status=i32(1), **routing),
    }


OPTIONAL = {"residual", "residual_out", "y", "x", "dz_in", "dx", "dweight", "topk_w", "perm_src", "perm_w", "status",
            "dx_in", "dtopk_w"}


@pytest.mark.parametrize("name", [f.__name__ for f in arguments()] if torch.cuda.is_available() else [])
def test_every_tensor_argument_is_checked(name):
    f = getattr(ep, name)
    base = arguments()[f]
    f(**base)
    torch.cuda.synchronize()
    tensors = [n for n, v in base.items() if isinstance(v, torch.Tensor)]
    for n in tensors:
        v = base[n]
        wrong = torch.float16 if v.dtype != torch.float16 else torch.int32
        changes = [("type", v.to(wrong)), ("host", v.cpu()), ("rank", v[None]), ("list", [1.0])]
        if n not in ("workspace", "status"):
            changes.append(("shape", torch.cat([v, v])))
        if v.dim() > 1 and v.numel() > v.shape[-1]:
            changes.append(("strides", v.view(torch.uint8 if v.element_size() == 1 else v.dtype)
                            .transpose(0, 1).contiguous().transpose(0, 1).view(v.dtype)))
        if n not in OPTIONAL:
            changes.append(("missing", None))
        for what, bad in changes:
            with pytest.raises((ValueError, ep.EpError)):
                f(**{**base, n: bad})
                pytest.fail(f"{name} took {n} with a wrong {what}")


def test_refusals_name_the_argument():
    base = arguments()
    with pytest.raises(ValueError, match=r"y must have shape \(4, 256\), got \(4, 128\)"):
        ep.ep_rmsnorm(**{**base[ep.ep_rmsnorm], "y": z(T, 128)})
    with pytest.raises(ValueError, match="dy must be torch.bfloat16, got torch.float32"):
        ep.ep_rmsnorm_bwd(**{**base[ep.ep_rmsnorm_bwd], "dy": f32(T, H)})
    with pytest.raises(ValueError, match="topk_idx must be contiguous"):
        ep.ep_dispatch_permuted_bwd(**{**base[ep.ep_dispatch_permuted_bwd],
                                       "topk_idx": z(k, T, dtype=torch.int64).transpose(0, 1)})
    with pytest.raises(ValueError, match="max_rows is too large"):
        ep.ep_dispatch_permuted_fp8(**{**base[ep.ep_dispatch_permuted_fp8], "max_rows": 1 << 31})
    with pytest.raises(TypeError):
        ep.ep_rmsnorm(**{**base[ep.ep_rmsnorm], "eps": "small"})
    with pytest.raises(AttributeError):
        ep.ep_rmsnorm(**{**base[ep.ep_rmsnorm], "stream": 7})
    with pytest.raises(ep.EpError, match="EP_ERR_INVALID"):
        ep.ep_rmsnorm(**{**base[ep.ep_rmsnorm], "eps": -1.0})
    with pytest.raises(ep.EpError, match="EP_ERR_INVALID"):
        ep.ep_rmsnorm_bwd(**{**base[ep.ep_rmsnorm_bwd], "workspace": z(16, dtype=torch.uint8)})


def test_a_refused_call_writes_nothing():
    y = torch.full((T, H), 3.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(z(T, H), None, z(128), 1e-6, None, y)
    torch.cuda.synchronize()
    assert torch.all(y == 3)
