"""Refusals of the transformer operators' entry points: every check runs on
the host before anything is launched, so these need no GPU (the addresses
are never followed)."""
import ctypes

import pytest

from video_vae_causal_implicit_b200 import build as cbuild
from video_vae_causal_implicit_b200 import cc3d


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cc3d.lib()


def P(a):
    return None if a is None else ctypes.c_void_p(a)


def norm(lib, **kw):
    a = dict(x=0x100000, residual=None, gamma=0x1000, beta=None, rows=4, c=64, eps=1e-6, silu=0,
             h=None, y=0x200000, q=None, scales=None, scale=0.0)
    a.update(kw)
    return lib.cc3d_add_rms_norm(P(a["x"]), P(a["residual"]), P(a["gamma"]), P(a["beta"]),
                                 a["rows"], a["c"], a["eps"], a["silu"], P(a["h"]), P(a["y"]),
                                 P(a["q"]), P(a["scales"]), a["scale"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), cc3d.ERR_INVALID_ARG), (dict(gamma=None), cc3d.ERR_INVALID_ARG),
    (dict(rows=-1), cc3d.ERR_INVALID_ARG), (dict(c=0), cc3d.ERR_INVALID_ARG),
    (dict(eps=-1.0), cc3d.ERR_INVALID_ARG), (dict(eps=float("nan")), cc3d.ERR_INVALID_ARG),
    (dict(y=None), cc3d.ERR_INVALID_ARG),                                  # no output
    (dict(q=0x300000), cc3d.ERR_INVALID_ARG),                              # no scale
    (dict(q=0x300000, scales=0x400000, scale=0.5), cc3d.ERR_INVALID_ARG),  # two
    (dict(q=0x300000, scale=1e-38), cc3d.ERR_INVALID_ARG),
    (dict(q=0x300000, scale=float("inf")), cc3d.ERR_INVALID_ARG),
    (dict(scales=0x400000), cc3d.ERR_INVALID_ARG),                         # scales, no codes
    (dict(c=60), cc3d.ERR_UNSUPPORTED), (dict(c=16392), cc3d.ERR_UNSUPPORTED),
    (dict(x=0x100008), cc3d.ERR_ALIGNMENT), (dict(y=0x200002), cc3d.ERR_ALIGNMENT),
    (dict(q=0x300004, scale=0.5), cc3d.ERR_ALIGNMENT),
    (dict(gamma=0x1004), cc3d.ERR_ALIGNMENT),
    (dict(scales=0x400002, q=0x300000), cc3d.ERR_ALIGNMENT),
    (dict(y=0x100010), cc3d.ERR_ALIAS), (dict(h=0x200010), cc3d.ERR_ALIAS),
    (dict(residual=0x180000, h=0x180010), cc3d.ERR_ALIAS),
    (dict(q=0x100000, scale=0.5), cc3d.ERR_ALIAS),                         # codes over x
    (dict(q=0x300000, scales=0x300008), cc3d.ERR_ALIAS),
    (dict(y=0x1000), cc3d.ERR_ALIAS),                                      # over gamma
])
def test_add_rms_norm_refusals(lib, kw, status):
    before = cc3d.cc3d_launch_count()
    assert norm(lib, **kw) == status
    assert cc3d.cc3d_launch_count() == before


def linear(lib, **kw):
    a = dict(x=0x1000000, ldx=64, w=0x2000000, ldw=64, bias=None, res=None, ldr=0, y=0x3000000,
             ldy=32, m=4, n=32, k=64, dtype=cc3d.BF16, act=0, xs=None, x_scale=0.0, ws=None)
    a.update(kw)
    return lib.cc3d_linear(P(a["x"]), a["ldx"], P(a["w"]), a["ldw"], P(a["bias"]), P(a["res"]),
                           a["ldr"], P(a["y"]), a["ldy"], a["m"], a["n"], a["k"], a["dtype"],
                           a["act"], P(a["xs"]), a["x_scale"], P(a["ws"]), None)


E4M3 = dict(dtype=cc3d.FP8_E4M3, ws=0x5000000, x_scale=0.5)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), cc3d.ERR_INVALID_ARG), (dict(w=None), cc3d.ERR_INVALID_ARG),
    (dict(y=None), cc3d.ERR_INVALID_ARG), (dict(m=-1), cc3d.ERR_INVALID_ARG),
    (dict(n=0), cc3d.ERR_INVALID_ARG), (dict(k=0), cc3d.ERR_INVALID_ARG),
    (dict(ldx=56), cc3d.ERR_INVALID_ARG), (dict(ldw=0), cc3d.ERR_INVALID_ARG),
    (dict(ldy=24), cc3d.ERR_INVALID_ARG), (dict(res=0x4000000, ldr=24), cc3d.ERR_INVALID_ARG),
    (dict(act=4), cc3d.ERR_INVALID_ARG), (dict(act=-1), cc3d.ERR_INVALID_ARG),
    (dict(ws=0x5000000), cc3d.ERR_INVALID_ARG), (dict(x_scale=1.0), cc3d.ERR_INVALID_ARG),
    (dict(E4M3, ws=None), cc3d.ERR_INVALID_ARG), (dict(E4M3, x_scale=0.0), cc3d.ERR_INVALID_ARG),
    (dict(E4M3, xs=0x6000000), cc3d.ERR_INVALID_ARG),
    (dict(E4M3, x_scale=float("nan")), cc3d.ERR_INVALID_ARG),
    (dict(dtype=cc3d.FP32), cc3d.ERR_UNSUPPORTED),
    (dict(k=60), cc3d.ERR_UNSUPPORTED), (dict(n=28), cc3d.ERR_UNSUPPORTED),
    (dict(ldx=68), cc3d.ERR_UNSUPPORTED), (dict(ldy=36), cc3d.ERR_UNSUPPORTED),
    (dict(E4M3, k=56), cc3d.ERR_UNSUPPORTED), (dict(E4M3, ldw=72), cc3d.ERR_UNSUPPORTED),
    (dict(m=(1 << 30) + 1), cc3d.ERR_UNSUPPORTED),
    (dict(x=0x1000008), cc3d.ERR_ALIGNMENT), (dict(w=0x2000008), cc3d.ERR_ALIGNMENT),
    (dict(y=0x3000008), cc3d.ERR_ALIGNMENT), (dict(bias=0x4000004), cc3d.ERR_ALIGNMENT),
    (dict(E4M3, ws=0x5000004), cc3d.ERR_ALIGNMENT),
    (dict(E4M3, x_scale=0.0, xs=0x6000002), cc3d.ERR_ALIGNMENT),
    (dict(y=0x1000000), cc3d.ERR_ALIAS), (dict(y=0x2000020), cc3d.ERR_ALIAS),
    (dict(y=0x3000000, res=0x3000010, ldr=32), cc3d.ERR_ALIAS),
    (dict(y=0x3000000, res=0x3000000, ldr=40), cc3d.ERR_ALIAS),
    (dict(bias=0x3000040), cc3d.ERR_ALIAS),
])
def test_linear_refusals(lib, kw, status):
    before = cc3d.cc3d_launch_count()
    assert linear(lib, **kw) == status
    assert cc3d.cc3d_launch_count() == before


def test_calls_without_rows_do_nothing(lib):
    assert norm(lib, rows=0, x=None, y=None) == cc3d.OK
    assert linear(lib, m=0, x=None, y=None) == cc3d.OK


def test_no_gpu_means_unsupported(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    assert norm(lib) == cc3d.ERR_UNSUPPORTED
    assert linear(lib) == cc3d.ERR_UNSUPPORTED


def test_wrappers_refuse_tensors_off_the_device(lib):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises((ValueError, TypeError)):
        cc3d.linear(x, x, x)
    with pytest.raises((ValueError, TypeError)):
        cc3d.add_rms_norm(x, torch.ones(64), y=x)
