"""Refusals of the transformer operators' entry points: every check runs on
the host before anything is launched, so these need no GPU (the addresses
are never followed)."""
import pytest

from video_vae_causal_implicit_b200 import build as cbuild
from video_vae_causal_implicit_b200 import cc3d


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cc3d.lib()


# the calls' fields, in the header's order (and names)
NORM = "x residual gamma beta h y q scales rows c silu eps scale".split()
LINEAR = ("x weight bias residual y x_scales w_scales ldx ldw ldr ldy m n k dtype act "
          "x_scale").split()


def norm(lib, **kw):
    a = dict(x=0x100000, residual=None, gamma=0x1000, beta=None, rows=4, c=64, eps=1e-6, silu=0,
             h=None, y=0x200000, q=None, scales=None, scale=0.0)
    a.update(kw)
    return lib.cc3d_add_rms_norm(cc3d._NORM_CALL.pack(*(a[k] or 0 for k in NORM)), None)


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
    a = dict(x=0x1000000, ldx=64, weight=0x2000000, ldw=64, bias=None, residual=None, ldr=0,
             y=0x3000000, ldy=32, m=4, n=32, k=64, dtype=cc3d.BF16, act=0, x_scales=None,
             x_scale=0.0, w_scales=None)
    a.update(kw)
    assert set(kw) <= set(a)
    return lib.cc3d_linear(cc3d._LINEAR_CALL.pack(*(a[k] or 0 for k in LINEAR)), None)


E4M3 = dict(dtype=cc3d.FP8_E4M3, w_scales=0x5000000, x_scale=0.5)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), cc3d.ERR_INVALID_ARG), (dict(weight=None), cc3d.ERR_INVALID_ARG),
    (dict(y=None), cc3d.ERR_INVALID_ARG), (dict(m=-1), cc3d.ERR_INVALID_ARG),
    (dict(n=0), cc3d.ERR_INVALID_ARG), (dict(k=0), cc3d.ERR_INVALID_ARG),
    (dict(ldx=56), cc3d.ERR_INVALID_ARG), (dict(ldw=0), cc3d.ERR_INVALID_ARG),
    (dict(ldy=24), cc3d.ERR_INVALID_ARG), (dict(residual=0x4000000, ldr=24), cc3d.ERR_INVALID_ARG),
    (dict(act=4), cc3d.ERR_INVALID_ARG), (dict(act=-1), cc3d.ERR_INVALID_ARG),
    (dict(w_scales=0x5000000), cc3d.ERR_INVALID_ARG), (dict(x_scale=1.0), cc3d.ERR_INVALID_ARG),
    (dict(E4M3, w_scales=None), cc3d.ERR_INVALID_ARG), (dict(E4M3, x_scale=0.0), cc3d.ERR_INVALID_ARG),
    (dict(E4M3, x_scales=0x6000000), cc3d.ERR_INVALID_ARG),
    (dict(E4M3, x_scale=float("nan")), cc3d.ERR_INVALID_ARG),
    (dict(dtype=cc3d.FP32), cc3d.ERR_UNSUPPORTED),
    (dict(k=60), cc3d.ERR_UNSUPPORTED), (dict(n=28), cc3d.ERR_UNSUPPORTED),
    (dict(ldx=68), cc3d.ERR_UNSUPPORTED), (dict(ldy=36), cc3d.ERR_UNSUPPORTED),
    (dict(E4M3, k=56), cc3d.ERR_UNSUPPORTED), (dict(E4M3, ldw=72), cc3d.ERR_UNSUPPORTED),
    (dict(m=(1 << 30) + 1), cc3d.ERR_UNSUPPORTED),
    (dict(x=0x1000008), cc3d.ERR_ALIGNMENT), (dict(weight=0x2000008), cc3d.ERR_ALIGNMENT),
    (dict(y=0x3000008), cc3d.ERR_ALIGNMENT), (dict(bias=0x4000004), cc3d.ERR_ALIGNMENT),
    (dict(E4M3, w_scales=0x5000004), cc3d.ERR_ALIGNMENT),
    (dict(E4M3, x_scale=0.0, x_scales=0x6000002), cc3d.ERR_ALIGNMENT),
    (dict(y=0x1000000), cc3d.ERR_ALIAS), (dict(y=0x2000020), cc3d.ERR_ALIAS),
    (dict(y=0x3000000, residual=0x3000010, ldr=32), cc3d.ERR_ALIAS),
    (dict(y=0x3000000, residual=0x3000000, ldr=40), cc3d.ERR_ALIAS),
    (dict(bias=0x3000040), cc3d.ERR_ALIAS),
])
def test_linear_refusals(lib, kw, status):
    before = cc3d.cc3d_launch_count()
    assert linear(lib, **kw) == status
    assert cc3d.cc3d_launch_count() == before


ATTN = ("n heads kv_heads d frame t slots window sinks ring total scale q_frames k_frames q k v o "
        "q_seq q_tok q_head k_seq k_tok k_head v_seq v_tok v_head o_seq o_tok o_head").split()
KV = ("n kv_heads d frame t slots sinks ring total q_frames k_frames k v k_cache v_cache "
      "k_seq k_tok k_head v_seq v_tok v_head kc_seq kc_tok kc_head vc_seq vc_tok vc_head").split()


def attn(lib, **kw):
    a = dict(n=2, heads=4, kv_heads=2, d=64, frame=1, t=8, slots=32, window=4, sinks=2, ring=0,
             total=20, scale=0.0, q_frames=0, k_frames=0, q=0x1000000, k=0x2000000, v=0x3000000,
             o=0x4000000, q_seq=8 * 256, q_tok=256, q_head=64, k_seq=32 * 128, k_tok=128,
             k_head=64, v_seq=32 * 128, v_tok=128, v_head=64, o_seq=8 * 256, o_tok=256, o_head=64)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.cc3d_attention(cc3d._ATTN_CALL.pack(*(a[k] for k in ATTN)), None)


def append(lib, **kw):
    a = dict(n=2, kv_heads=2, d=64, frame=1, t=8, slots=32, sinks=2, ring=0, total=20, q_frames=0,
             k_frames=0, k=0x1000000, v=0x2000000, k_cache=0x3000000, v_cache=0x4000000,
             k_seq=8 * 128, k_tok=128, k_head=64, v_seq=8 * 128, v_tok=128, v_head=64,
             kc_seq=32 * 128, kc_tok=128, kc_head=64, vc_seq=32 * 128, vc_tok=128, vc_head=64)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.cc3d_kv_append(cc3d._KV_CALL.pack(*(a[k] for k in KV)), None)


CACHE = [  # of both calls
    (dict(n=-1), cc3d.ERR_INVALID_ARG), (dict(kv_heads=0), cc3d.ERR_INVALID_ARG),
    (dict(d=0), cc3d.ERR_INVALID_ARG), (dict(frame=0), cc3d.ERR_INVALID_ARG),
    (dict(t=-1), cc3d.ERR_INVALID_ARG), (dict(slots=0), cc3d.ERR_INVALID_ARG),
    (dict(sinks=-1), cc3d.ERR_INVALID_ARG), (dict(ring=-1), cc3d.ERR_INVALID_ARG),
    (dict(ring=29), cc3d.ERR_INVALID_ARG),                     # slots != sinks + ring
    (dict(total=-1), cc3d.ERR_INVALID_ARG), (dict(total=33), cc3d.ERR_INVALID_ARG),
    (dict(d=60), cc3d.ERR_UNSUPPORTED), (dict(d=392), cc3d.ERR_UNSUPPORTED),
    (dict(frame=1 << 27), cc3d.ERR_UNSUPPORTED), (dict(k_tok=132), cc3d.ERR_UNSUPPORTED),
    (dict(v_head=0), cc3d.ERR_UNSUPPORTED), (dict(k_seq=-1024), cc3d.ERR_UNSUPPORTED),
    (dict(k=0x2000008), cc3d.ERR_ALIGNMENT), (dict(v=0x3000008), cc3d.ERR_ALIGNMENT),
    (dict(k_frames=0x5000002), cc3d.ERR_ALIGNMENT), (dict(q_frames=0x5000001), cc3d.ERR_ALIGNMENT),
    (dict(k=0), cc3d.ERR_INVALID_ARG), (dict(v=0), cc3d.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(heads=0), cc3d.ERR_INVALID_ARG), (dict(heads=3), cc3d.ERR_INVALID_ARG),
    (dict(window=-1), cc3d.ERR_INVALID_ARG), (dict(scale=-1.0), cc3d.ERR_INVALID_ARG),
    (dict(scale=float("nan")), cc3d.ERR_INVALID_ARG),
    (dict(scale=float("inf")), cc3d.ERR_INVALID_ARG),
    (dict(ring=30, window=0), cc3d.ERR_INVALID_ARG),           # a ring without a window
    (dict(ring=30, window=24), cc3d.ERR_INVALID_ARG),          # and one too small for it
    (dict(heads=258), cc3d.ERR_UNSUPPORTED),
    (dict(q=0), cc3d.ERR_INVALID_ARG), (dict(o=0), cc3d.ERR_INVALID_ARG),
    (dict(q=0x1000008), cc3d.ERR_ALIGNMENT), (dict(o=0x4000008), cc3d.ERR_ALIGNMENT),
    (dict(o=0x1000000), cc3d.ERR_ALIAS), (dict(o=0x2000800), cc3d.ERR_ALIAS),
    (dict(o=0x3000000), cc3d.ERR_ALIAS), (dict(k_frames=0x4000010), cc3d.ERR_ALIAS),
    (dict(o_tok=248), cc3d.ERR_ALIAS), (dict(o_head=56), cc3d.ERR_ALIAS),   # rows that meet
    (dict(o_seq=1024), cc3d.ERR_ALIAS),
])
def test_attention_refusals(lib, kw, status):
    before = cc3d.cc3d_launch_count()
    assert attn(lib, **kw) == status
    assert cc3d.cc3d_launch_count() == before


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(k_cache=0), cc3d.ERR_INVALID_ARG), (dict(v_cache=0), cc3d.ERR_INVALID_ARG),
    (dict(k_cache=0x3000008), cc3d.ERR_ALIGNMENT), (dict(vc_tok=100), cc3d.ERR_UNSUPPORTED),
    (dict(k_cache=0x1000000), cc3d.ERR_ALIAS), (dict(v_cache=0x2000100), cc3d.ERR_ALIAS),
    (dict(v_cache=0x3000000), cc3d.ERR_ALIAS), (dict(kc_head=8), cc3d.ERR_ALIAS),
    (dict(k_frames=0x3000000), cc3d.ERR_ALIAS),
])
def test_kv_append_refusals(lib, kw, status):
    before = cc3d.cc3d_launch_count()
    assert append(lib, **kw) == status
    assert cc3d.cc3d_launch_count() == before


def test_null_calls_refused(lib):
    assert lib.cc3d_add_rms_norm(None, None) == cc3d.ERR_INVALID_ARG
    assert lib.cc3d_linear(None, None) == cc3d.ERR_INVALID_ARG
    assert lib.cc3d_attention(None, None) == cc3d.ERR_INVALID_ARG
    assert lib.cc3d_kv_append(None, None) == cc3d.ERR_INVALID_ARG


def test_packed_calls_have_the_headers_layout(tmp_path):
    """The wrappers' packed arguments against what the C compiler lays out."""
    import os
    import subprocess
    names = {"cc3d_add_norm_call": NORM, "cc3d_linear_call": LINEAR, "cc3d_attn_call": ATTN,
             "cc3d_kv_call": KV}
    body = "".join(f'printf("%zu ", sizeof({t}));' +
                   "".join(f'printf("%zu ", offsetof({t}, {f}));' for f in fs)
                   for t, fs in names.items())
    src = tmp_path / "layout.c"
    src.write_text(f'#include <stdio.h>\n#include "cc3d.h"\nint main(void) {{ {body} return 0; }}\n')
    subprocess.run(["gcc", "-I", cbuild.INCLUDE, str(src), "-o", str(tmp_path / "layout")],
                   check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "layout")], capture_output=True,
                                          text=True, check=True).stdout.split()]
    want = []
    for s in (cc3d._NORM_CALL, cc3d._LINEAR_CALL, cc3d._ATTN_CALL, cc3d._KV_CALL):
        codes = [(c, int(n or 1)) for n, c in __import__("re").findall(r"(\d*)([ifPq])", s.format)]
        want.append(s.size)
        at = 0
        for c, n in codes:
            size = 4 if c in "if" else 8
            at += -at % size
            for _ in range(n):
                want.append(at)
                at += size
    assert got == want


def test_calls_without_rows_do_nothing(lib):
    assert attn(lib, n=0, q=0, k=0, v=0, o=0) == cc3d.OK
    assert attn(lib, t=0, q=0, o=0) == cc3d.OK
    assert append(lib, t=0, k=0, v=0) == cc3d.OK
    assert norm(lib, rows=0, x=None, y=None) == cc3d.OK
    assert linear(lib, m=0, x=None, y=None) == cc3d.OK


def test_no_gpu_means_unsupported(lib):
    import torch
    if pytest.importorskip("torch").cuda.is_available():
        pytest.skip("GPU present")
    assert norm(lib) == cc3d.ERR_UNSUPPORTED
    assert linear(lib) == cc3d.ERR_UNSUPPORTED
    assert attn(lib) == cc3d.ERR_UNSUPPORTED
    assert append(lib) == cc3d.ERR_UNSUPPORTED


def test_wrappers_refuse_tensors_off_the_device(lib):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises((ValueError, TypeError)):
        cc3d.linear(x, x, x)
    with pytest.raises((ValueError, TypeError)):
        cc3d.add_rms_norm(x, torch.ones(64), y=x)
    q = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises((ValueError, TypeError)):
        cc3d.attention(q, q, q, q, total=2)
    with pytest.raises((ValueError, TypeError)):
        cc3d.kv_append(q, q, q, q, total=2)


# both caches as slices of one tensor: [n, 32, 2 heads, 64] each
INTERLEAVED = {
    "within heads": dict(v_cache=0x3000000 + 2 * 64, kc_head=128, kc_tok=256, kc_seq=32 * 256),
    "within tokens": dict(v_cache=0x3000000 + 2 * 128, kc_head=64, kc_tok=256, kc_seq=32 * 256),
    "values first": dict(v_cache=0x3000000 - 2 * 128, kc_head=64, kc_tok=256, kc_seq=32 * 256),
    "within sequences": dict(v_cache=0x3000000 + 2 * 32 * 128, kc_head=64, kc_tok=128,
                             kc_seq=2 * 32 * 128),
}


@pytest.mark.parametrize("name", INTERLEAVED)
def test_interleaved_caches_pass_the_checks(lib, name):
    if pytest.importorskip("torch").cuda.is_available():
        pytest.skip("the addresses are not real")
    kw = dict(INTERLEAVED[name])
    kw.update({"vc_" + x: kw["kc_" + x] for x in ("seq", "tok", "head")})
    assert append(lib, **kw) == cc3d.ERR_UNSUPPORTED  # no device: all argument checks passed


@pytest.mark.parametrize("kw", [
    dict(v_cache=0x3000000 + 2 * 8),                            # meeting entries
    dict(v_cache=0x3000000 + 2 * 128),                          # a token further on
    dict(v_cache=0x3000000 + 2 * 32 * 128),                     # the next sequence's keys
    dict(v_cache=0x3000000 + 2 * 64, kc_head=128, kc_tok=256, kc_seq=32 * 256),  # other strides
])
def test_overlapping_caches_refused(lib, kw):
    before = cc3d.cc3d_launch_count()
    assert append(lib, **kw) == cc3d.ERR_ALIAS
    assert cc3d.cc3d_launch_count() == before


@pytest.mark.parametrize("x_scale", [-1.0, float("nan"), float("inf"), 1e-38])
def test_linear_refuses_a_second_scale_of_any_value(lib, x_scale):
    """With one scale per row the single scale is 0, as the header says."""
    assert linear(lib, **dict(E4M3, x_scales=0x6000000, x_scale=x_scale)) == cc3d.ERR_INVALID_ARG
