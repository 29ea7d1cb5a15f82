"""cc3d_linear on the GPU against the product in 64 bits.

Tolerance, from the arithmetic: the products of bf16 (or E4M3) values are
exact in fp32, the sum of k of them is off by at most (k + 8) fp32 steps
(2^-23) of the sum of their magnitudes S, the scales and the bias by a few
more, the activation changes that by its slope (at most 1.13) and adds the
hardware exponential's and reciprocal's 2^-20 of |a|, and the one rounding to
bf16 is off by at most 2^-8 of |y|."""
import math

import pytest
import torch

from video_vae_causal_implicit_b200 import cc3d

pytestmark = pytest.mark.gpu


def reference(x, w, bias, residual, act, xs=None, ws=None):
    """(y, tolerance) in 64 bits."""
    xd, wd = x.double(), w.double()
    k = x.shape[1]
    a, mag = xd @ wd.t(), xd.abs() @ wd.abs().t()
    if ws is not None:
        sc = (xs.double()[:, None] if torch.is_tensor(xs) else xs) * ws.double()
        a, mag = a * sc, mag * sc
    if bias is not None:
        a, mag = a + bias.double(), mag + bias.double().abs()
    y = {cc3d.ACT_NONE: lambda v: v, cc3d.ACT_SILU: lambda v: v * torch.sigmoid(v),
         cc3d.ACT_GELU: lambda v: 0.5 * v * torch.erfc(-v / math.sqrt(2)),
         cc3d.ACT_GELU_TANH: lambda v: v * torch.sigmoid(
             2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))}[act](a)
    tol = 1.13 * (k + 8) * 2.0 ** -23 * mag + 2.0 ** -20 * a.abs()
    if residual is not None:
        y = y + residual.double()
        tol = tol + 2.0 ** -23 * residual.double().abs()
    return y, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs() + 1e-37


def check(y, ref, tol, what):
    bad = (y.double() - ref).abs() > tol
    assert torch.isfinite(y.float()).all(), what
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           float((y.double() - ref).abs().max()))


def make(m, n, k, seed, fp8=False, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    step = 16 if fp8 else 8
    x = torch.randn(m, k + pad * step, device="cuda", generator=g)[:, :k]
    w = torch.randn(n, k + pad * step, device="cuda", generator=g)[:, :k] * k ** -0.5
    bias = torch.randn(n, device="cuda", generator=g)
    if not fp8:
        # (rows keep their padded distance)
        x = x.to(torch.bfloat16) if not pad else _strided(x, torch.bfloat16, pad * step)
        w = w.to(torch.bfloat16) if not pad else _strided(w, torch.bfloat16, pad * step)
        return x, w, bias, None, None
    xs, ws = x.abs().amax(1) / 448, w.abs().amax(1) / 448
    cast = lambda a, s: (a / s[:, None]).clamp(-448, 448)  # noqa: E731
    x, w = cast(x, xs), cast(w, ws)
    if pad:
        return (_strided(x, torch.float8_e4m3fn, pad * step),
                _strided(w, torch.float8_e4m3fn, pad * step), bias, xs, ws)
    return x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn), bias, xs, ws


def _strided(a, dtype, pad):
    out = torch.zeros(a.shape[0], a.shape[1] + pad, device="cuda").to(dtype)
    view = out[:, :a.shape[1]]
    view.copy_(a.to(dtype))
    return view


ACTS = [cc3d.ACT_NONE, cc3d.ACT_SILU, cc3d.ACT_GELU, cc3d.ACT_GELU_TANH]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("m,n,k", [
    (1, 8, 16), (1, 2056, 1008), (3, 136, 64), (16, 128, 512), (17, 1000, 496), (64, 392, 4096),
    (127, 264, 144), (128, 128, 128), (129, 72, 80), (300, 520, 2000), (513, 384, 384),
    (1560, 1152, 384), (2049, 24, 96), (4100, 1288, 240), (9000, 2048, 16)])
def test_sizes(m, n, k, fp8):
    x, w, bias, xs, ws = make(m, n, k, m + n + k, fp8)
    act = ACTS[(m + n) % 4]
    g = torch.Generator(device="cuda").manual_seed(5)
    res = torch.randn(m, n, device="cuda", generator=g).to(torch.bfloat16)
    for residual in (None, res):
        y = torch.full((m, n), float("nan"), device="cuda", dtype=torch.bfloat16)
        cc3d.linear(x, w, y, bias=bias, residual=residual, act=act, x_scales=xs, w_scales=ws)
        cc3d.sync_status()
        check(y, *reference(x, w, bias, residual, act, xs, ws), (m, n, k, fp8, act))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [5, 700])
def test_activations_over_their_range(m, act):
    """Large positive and negative arguments, zero, no bias."""
    k, n = 16, 256
    x = torch.zeros(m, k, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = 1
    w = torch.zeros(n, k, device="cuda", dtype=torch.bfloat16)
    w[:, 0] = torch.linspace(-110, 110, n, device="cuda").to(torch.bfloat16)
    y = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
    cc3d.linear(x, w, y, act=act)
    cc3d.sync_status()
    check(y, *reference(x, w, None, None, act), act)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("m", [1, 40, 777])
def test_strided_rows_and_untouched_gaps(m, fp8):
    n, k = 264, 208
    x, w, bias, xs, ws = make(m, n, k, 3, fp8, pad=3)
    y_all = torch.full((m, n + 24), 7.0, device="cuda", dtype=torch.bfloat16)
    r_all = torch.randn(m, n + 8, device="cuda").to(torch.bfloat16)
    y, r = y_all[:, :n], r_all[:, :n]
    cc3d.linear(x, w, y, bias=bias, residual=r, x_scales=xs, w_scales=ws)
    cc3d.sync_status()
    check(y, *reference(x, w, bias, r, cc3d.ACT_NONE, xs, ws), "strided")
    assert (y_all[:, n:] == 7).all()


@pytest.mark.parametrize("m", [2, 600])
def test_residual_in_place_one_scale_and_bytes(m):
    n, k = 520, 256
    x, w, _, _, ws = make(m, n, k, 9, True)
    r = torch.randn(m, n, device="cuda").to(torch.bfloat16)
    y = r.clone()
    cc3d.linear(x.view(torch.uint8), w.view(torch.uint8), y, residual=y, x_scale=0.03, w_scales=ws)
    cc3d.sync_status()
    check(y, *reference(x, w, None, r, cc3d.ACT_NONE, 0.03, ws), "in place")


@pytest.mark.parametrize("m,n,k", [(4, 1024, 4096), (1000, 640, 1024)])
def test_same_bytes_on_every_call_stream_and_replay(m, n, k):
    x, w, bias, _, _ = make(m, n, k, 11)
    first = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
    cc3d.linear(x, w, first, bias=bias, act=cc3d.ACT_GELU)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(12):  # several calls under way at once
        y = torch.zeros_like(first)
        streams[i % 3].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(streams[i % 3]):
            cc3d.linear(x, w, y, bias=bias, act=cc3d.ACT_GELU)
        outs.append(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    y = torch.zeros_like(first)
    with torch.cuda.graph(graph):
        cc3d.linear(x, w, y, bias=bias, act=cc3d.ACT_GELU)
    for _ in range(3):
        graph.replay()
    cc3d.sync_status()
    for o in outs + [y]:
        assert torch.equal(o, first)


def test_infinities_stay_in_their_row_and_column():
    m, n, k = 200, 264, 128
    x, w, bias, _, _ = make(m, n, k, 2)
    clean = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
    cc3d.linear(x, w, clean, bias=bias)
    x2, w2 = x.clone(), w.clone()
    x2[7, 5] = float("inf")
    w2[100, 9] = float("nan")
    y = torch.empty_like(clean)
    cc3d.linear(x2, w2, y, bias=bias)
    cc3d.sync_status()
    assert not torch.isfinite(y[7]).any() and torch.isnan(y[:, 100]).all()
    keep = torch.ones(m, n, device="cuda", dtype=torch.bool)
    keep[7], keep[:, 100] = False, False
    assert torch.equal(y[keep], clean[keep])


def test_no_rows():
    x, w, _, _, _ = make(4, 16, 16, 1)
    y = torch.ones(4, 16, device="cuda", dtype=torch.bfloat16)
    before = cc3d.cc3d_launch_count()
    cc3d.linear(x[:0], w, y[:0])
    assert cc3d.cc3d_launch_count() == before and (y == 1).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [3, 700])
def test_activation_over_its_whole_range(m, act):
    """The bias alone through the activation: small and large values of both
    signs, infinities (their limits: -inf gives 0, also where the formula in
    floating point has no value) and NaN, whose neighbours keep theirs."""
    n, k = 4096, 64
    x = torch.zeros(m, k, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(n, k, device="cuda", dtype=torch.bfloat16)
    size = torch.logspace(-30, 30, n // 4, dtype=torch.float64)
    near = torch.linspace(0, 150, n // 4, dtype=torch.float64)
    bias = torch.stack([size, -size, near, -near], 1).flatten().float()
    inf = float("inf")
    odd = {0: inf, 3: -inf, 6: inf, 7: inf, 10: -inf, 11: -inf, 12: float("nan"),
           17: float("nan"), 20: inf, 21: float("nan"), 24: -inf, 25: float("nan")}
    for i, v in odd.items():
        bias[i] = v
    plain = torch.tensor([i not in odd for i in range(n)], device="cuda")
    bias = bias.cuda()
    y = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
    cc3d.linear(x, w, y, bias=bias, act=act)
    cc3d.sync_status()
    ref, tol = reference(x, w, bias, None, act)
    check(y[:, plain], ref[:, plain], tol[:, plain], "finite")
    for i, v in odd.items():
        got = y[:, i].float()
        if v != v:
            assert torch.isnan(got).all(), i
        elif v == inf or act == cc3d.ACT_NONE:
            assert (got == v).all(), i
        else:
            assert (got.abs() <= 2.0 ** -55).all(), i


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("m", [3, 700])
def test_negative_tails_keep_their_relative_error(m, act, fp8):
    """The activations' values left of zero, down to bf16's least numbers.

    With 2^z the exponential in the formula, z is off by at most six fp32 half
    steps of itself (constants and products, no cancellation), so its power by
    2^-21 |z| of itself; the hardware's exponential (twice), reciprocal and a few
    products add 2^-20, the erf form's fit 2^-20, the rounding 2^-8.  Absolutely,
    half a step of bf16's least numbers (2^-134), and for the erf form, whose
    exponential is flushed below 2^-126, that times |a| h (< 1 there)."""
    n, k = 8192, 64
    x = torch.zeros(m, k, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(n, k, device="cuda", dtype=torch.bfloat16)
    a = -torch.cat([torch.linspace(0, 130, n - 64, dtype=torch.float64),
                    torch.logspace(2, 38, 64, dtype=torch.float64)])
    bias = a[torch.randperm(n, generator=torch.Generator().manual_seed(1))].float().cuda()
    scales = {}
    if fp8:
        x, w = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
        scales = dict(x_scale=1.0, w_scales=torch.ones(n, device="cuda"))
    y = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
    cc3d.linear(x, w, y, bias=bias, act=act, **scales)
    cc3d.sync_status()
    ref, _ = reference(x[:1].float(), w.float(), bias, None, act)
    a = bias.double()
    z = {cc3d.ACT_SILU: a, cc3d.ACT_GELU: a * a / 2, cc3d.ACT_GELU_TANH:
         2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)}[act].abs() / math.log(2)
    ref = torch.where(z > 1000, torch.zeros_like(ref), ref)  # (also where 64 bits overflow)
    least = 2.0 ** -126 if act == cc3d.ACT_GELU else 2.0 ** -133
    tol = ref.abs() * (2.0 ** -8 + 2.0 ** -19 + 2.0 ** -21 * z.clamp_max(1000)) + least
    bad = ~((y.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bias[bad[0].nonzero()[:3].flatten()].tolist(),
                           y[bad][:3].tolist(), ref.expand_as(y)[bad][:3].tolist())


# Sizes for each of the tiles and splits; tests/test_ops_choice.py checks on the
# CPU that they do take them all.
CHOICES = [
    (700, 520, 96), (1000, 12288, 64), (4000, 2056, 512), (7800, 264, 1024), (7800, 264, 2048),
    (2500, 1032, 4096), (1, 8, 64), (1, 8192, 384), (5, 4104, 1008), (2, 264, 2064), (17, 2056, 2048),
    (33, 4096, 384), (33, 1000, 2000), (60, 2056, 512), (200, 1160, 512), (65, 2048, 528),
    (80, 264, 2064), (90, 264, 1040), (100, 2048, 2048), (112, 136, 4096), (200, 2048, 4096),
    (300, 1000, 4096), (512, 264, 8192), (128, 12288, 144), (100, 8, 64)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("m,n,k", CHOICES)
def test_every_tile_and_split(m, n, k, fp8):
    x, w, bias, xs, ws = make(m, n, k, m + n + k, fp8)
    res = torch.randn(m, n, device="cuda").to(torch.bfloat16)
    for residual in (res, None):
        y = torch.full((m, n), float("nan"), device="cuda", dtype=torch.bfloat16)
        cc3d.linear(x, w, y, bias=bias, residual=residual, act=cc3d.ACT_GELU_TANH, x_scales=xs,
                    w_scales=ws)
        cc3d.sync_status()
        check(y, *reference(x, w, bias, residual, cc3d.ACT_GELU_TANH, xs, ws), (m, n, k, fp8))
