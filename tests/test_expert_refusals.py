"""What the experts' feed-forward block refuses: at the C entry before anything is launched
(EP_ERR_INVALID), and in the binding before the library is called (ValueError). CPU only; the
pointers are never dereferenced."""
import ctypes

import pytest
import torch

import combine_ep_get_05_gb300 as ep

P = ctypes.c_void_p
OK, INVALID = 0, 1
F = P(4096)      # a 16-byte aligned address
ODD = P(4096 + 4)


@pytest.fixture(scope="module", autouse=True)
def L():
    ep.build_library()
    return ep.lib()


def call(fn, defaults, **change):
    assert set(change) <= set(defaults), change
    return fn(*{**defaults, **change}.values())


SIZES = dict(H=256, F=128, E=8, R=4, max_rows=16)
GATE_UP = dict(x=F, w=F, offsets=F, act=0, **SIZES, h=F, pre=F, pre_q=F, pre_scales=F, status=None, stream=None)
DOWN = dict(h=F, w=F, offsets=F, **SIZES, y=F, status=None, stream=None)
DOWN_BWD = dict(dy=F, w=F, pre=None, pre_q=F, pre_scales=F, offsets=F, act=0, **SIZES, dpre=F, h=F, status=None,
                stream=None)
GATE_UP_BWD = dict(dpre=F, w=F, offsets=F, **SIZES, dx=F, status=None, stream=None)
WGRAD = dict(dout=F, rows=F, offsets=F, I=256, J=128, E=8, R=4, max_rows=16, dw=F, status=None, stream=None)
CALLS = {"gate_up": GATE_UP, "down": DOWN, "down_bwd": DOWN_BWD, "gate_up_bwd": GATE_UP_BWD, "wgrad": WGRAD}

EXPERTS = [dict(E=0), dict(E=9), dict(E=8196), dict(R=0), dict(R=257, E=257), dict(max_rows=-1),
           dict(R=4, max_rows=1 << 30), dict(offsets=None), dict(offsets=ODD)]
WIDTHS = [dict(H=0), dict(H=-8), dict(H=260), dict(H=65544), dict(F=0), dict(F=132), dict(F=65544)]


@pytest.mark.parametrize("name", list(CALLS))
def test_every_entry_refuses(L, name):
    fn, base = getattr(L, "ep_expert_" + name), CALLS[name]
    changes = list(EXPERTS)
    changes += WIDTHS if "H" in base else [dict(I=0), dict(I=12), dict(I=131080), dict(J=0), dict(J=-8), dict(J=131080)]
    if "act" in base:
        changes += [dict(act=2), dict(act=-1), dict(F=136)]
    optional = {"gate_up": {"pre"}, "down_bwd": {"pre", "h"}}.get(name, set())
    for n, v in base.items():
        if v is F:
            changes.append({n: ODD})
            if n not in optional:
                changes.append({n: None})
    for change in changes:
        assert call(fn, base, **change) == INVALID, change
    if name != "wgrad":
        assert call(fn, base, max_rows=0, offsets=None) == OK  # no rows: nothing is read or launched


def test_one_checkpoint_is_read(L):
    assert call(L.ep_expert_down_bwd, DOWN_BWD, pre=F) == INVALID
    assert call(L.ep_expert_down_bwd, DOWN_BWD, pre_q=None, pre_scales=None) == INVALID


def bf(*s):
    return torch.empty(s, dtype=torch.bfloat16)


E, R, M, H, W = 8, 4, 16, 256, 128
OFF = torch.empty(E + 1, dtype=torch.int32)


def test_binding_refuses_host_tensors_and_wrong_ranks():
    for f, args in ((ep.ep_expert_gate_up, (bf(R, M, H), bf(E, 2 * W, H), OFF, 0, bf(R, M, W))),
                    (ep.ep_expert_down, (bf(R, M, W), bf(E, H, W), OFF, bf(R, M, H))),
                    (ep.ep_expert_down_bwd, (bf(R, M, H), bf(E, H, W), bf(R, M, 2 * W), None, None, OFF, 0,
                                             bf(R, M, 2 * W))),
                    (ep.ep_expert_gate_up_bwd, (bf(R, M, 2 * W), bf(E, 2 * W, H), OFF, bf(R, M, H))),
                    (ep.ep_expert_wgrad, (bf(R, M, H), bf(R, M, W), OFF, bf(E, H, W)))):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            f(*args)
        with pytest.raises(ValueError, match="must have 3 dimensions, got 2"):
            f(args[0][0], *args[1:])
        with pytest.raises(ValueError, match="is required"):
            f(None, *args[1:])


def test_binding_names_what_it_refuses():
    with pytest.raises(ValueError, match="w_gate_up must have an even number of rows an expert, got 255"):
        ep.ep_expert_gate_up(bf(R, M, H), bf(E, 255, H), OFF, 0, bf(R, M, 127))
    with pytest.raises(ValueError, match="w_gate_up must have an even number of rows an expert, got 255"):
        ep.ep_expert_gate_up_bwd(bf(R, M, 255), bf(E, 255, H), OFF, bf(R, M, H))
    wide = torch.empty((1, 1, 1 << 31), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="^x is too large"):
        ep.ep_expert_gate_up(wide, bf(E, 2 * W, H), OFF, 0, bf(R, M, W))


def test_helpers_refuse_before_they_allocate():
    lay = ep.ExpertLayout(OFF, None, None, None, E)
    with pytest.raises(ValueError, match="save must be"):
        ep.expert_gate_up(bf(R, M, H), bf(E, 2 * W, H), lay, save="fp8")
    with pytest.raises(ValueError, match="kept no checkpoint"):
        ep.expert_down_bwd(bf(R, M, H), bf(E, H, W), ep.GateUp(bf(R, M, W), None, None, None), lay)
