"""The transformer operators as they are used together: the VAE's mid-block
(RMS_norm, q / k / v product, attention within each frame, output product
onto the input), once whole and once streamed frame by frame over a ring of
frames, a block of a transformer over streamed latents with its
feed-forward in 8 bits, and an RMS norm whose codes feed an FP8 conv plan.
References are compositions in 64 bits in which every tensor that the
operators hand on in 16 or 8 bits is rounded as they round it, so that only
the last operator's own error counts beside the handed-on roundings that
flip (each at most one step of its type, met by the weights' sizes)."""
import math

import pytest
import torch

import oracle
from tests.parity import assert_close_bf16, ncthw_np, to_dev
from video_vae_causal_implicit_b200 import cc3d, synth

pytestmark = pytest.mark.gpu


def rnd(*shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(torch.bfloat16)


def close(got, ref, what, frac=2e-2, mean=4e-3):
    """The library's parity: 2e-2 of the largest, and in the mean 4e-3 (two
    16-bit hand-overs of 2^-8 each, averaged over their rounding errors)."""
    d = (got.double() - ref).abs()
    assert torch.isfinite(got.float()).all(), what
    assert d.max() <= frac * ref.abs().max(), (what, float(d.max()), float(ref.abs().max()))
    assert d.sum() <= mean * ref.abs().sum(), (what, float(d.sum() / ref.abs().sum()))


def b16(x):
    return x.to(torch.bfloat16).double()


def norm64(x, gamma, eps=0.0):
    c = x.shape[-1]
    return x * c ** 0.5 / (x.square().sum(-1, keepdim=True) + c * eps).sqrt().clamp_min(
        1e-12) * gamma.double()


def softmax_attention(q, k, v, frame, window, sinks):
    """[tokens, d] each, 64 bits, one head."""
    f = torch.arange(q.shape[0], device=q.device) // frame
    far = f[:, None] - f
    s = (q @ k.t() / math.sqrt(q.shape[1])).masked_fill(
        (far < 0) | ((far >= window) & (f[None] >= sinks)), -math.inf)
    return torch.softmax(s, 1) @ v


class MidBlock:
    def __init__(self, c, seed):
        self.c = c
        self.gamma = torch.rand(c, device="cuda") + 0.5
        self.w_qkv, self.b_qkv = rnd(3 * c, c, seed=seed, std=c ** -0.5), torch.randn(
            3 * c, device="cuda") * 0.1
        self.w_o, self.b_o = rnd(c, c, seed=seed + 1, std=c ** -0.5), torch.randn(
            c, device="cuda") * 0.1

    def reference(self, x, frame, window, sinks):
        xd = x.double().view(-1, self.c)
        qkv = b16(b16(norm64(xd, self.gamma)) @ self.w_qkv.double().t() + self.b_qkv.double())
        o = softmax_attention(*qkv.split(self.c, 1), frame, window, sinks)
        return b16(o) @ self.w_o.double().t() + self.b_o.double() + xd


@pytest.mark.parametrize("c,t,h,w", [(384, 3, 30, 52), (96, 5, 7, 9), (192, 2, 16, 20)])
def test_mid_block_attends_within_each_frame(c, t, h, w):
    m = MidBlock(c, 5)
    x = rnd(1, t, h, w, c, seed=1)                    # NDHWC, as the convs hand it on
    tokens, frame = t * h * w, h * w
    a = torch.empty_like(x)
    cc3d.add_rms_norm(x, m.gamma, y=a)
    qkv = torch.empty(tokens, 3 * c, device="cuda", dtype=torch.bfloat16)
    cc3d.linear(a.view(tokens, c), m.w_qkv, qkv, bias=m.b_qkv)
    q, k, v = (qkv[:, i * c:(i + 1) * c].view(1, tokens, 1, c) for i in range(3))
    o = torch.empty(1, tokens, 1, c, device="cuda", dtype=torch.bfloat16)
    cc3d.attention(q, k, v, o, frame=frame, window=1, total=t)
    y = torch.empty(tokens, c, device="cuda", dtype=torch.bfloat16)
    cc3d.linear(o.view(tokens, c), m.w_o, y, bias=m.b_o, residual=x.view(tokens, c))
    cc3d.sync_status()
    close(y, m.reference(x, frame, 1, 0), "mid-block")


def test_streamed_block_with_a_ring_equals_the_whole():
    """One frame a call, window of three frames and a sink, in a captured
    graph; against the whole sequence in 64 bits."""
    c, t, h, w, window, sinks = 128, 7, 9, 13, 3, 1
    frame, ring = h * w, 3
    m = MidBlock(c, 9)
    x = rnd(1, t, h, w, c, seed=2)
    xs = torch.empty(frame, c, device="cuda", dtype=torch.bfloat16)
    a, y, o = torch.empty_like(xs), torch.empty_like(xs), torch.empty_like(xs)
    qkv = torch.empty(frame, 3 * c, device="cuda", dtype=torch.bfloat16)
    kc = torch.full((1, (sinks + ring) * frame, 1, c), float("nan"), device="cuda",
                    dtype=torch.bfloat16)
    vc = kc.clone()
    count = torch.zeros(1, device="cuda", dtype=torch.int32)
    q, k, v = (qkv[:, i * c:(i + 1) * c].view(1, frame, 1, c) for i in range(3))
    where = dict(frame=frame, sinks=sinks, ring=ring, k_frames=count)

    def step():
        cc3d.add_rms_norm(xs, m.gamma, y=a)
        cc3d.linear(a, m.w_qkv, qkv, bias=m.b_qkv)
        cc3d.kv_append(k, v, kc, vc, **where)
        cc3d.attention(q, kc, vc, o.view(1, frame, 1, c), window=window, **where)
        cc3d.linear(o, m.w_o, y, bias=m.b_o, residual=xs)

    xs.zero_()
    count.fill_(1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kc.fill_(float("nan"))
    vc.fill_(float("nan"))
    got = []
    for i in range(t):
        xs.copy_(x[0, i].view(frame, c))
        count.fill_(i + 1)
        graph.replay()
        got.append(y.clone())
    cc3d.sync_status()
    close(torch.cat(got), m.reference(x, frame, window, sinks), "streamed block")


@pytest.mark.parametrize("tokens", [3, 300])
def test_feed_forward_in_8_bits(tokens):
    """Residual addition and norm into E4M3 with row scales, the up product
    with GELU on those codes, the down product onto the stream."""
    c, f = 256, 1024
    x, r = rnd(tokens, c, seed=3), rnd(tokens, c, seed=4, std=2.0)
    gamma = torch.rand(c, device="cuda") + 0.5
    w1, w2 = rnd(f, c, seed=5, std=c ** -0.5), rnd(c, f, seed=6, std=f ** -0.5)
    s1 = (w1.float().abs().amax(1) / 448)
    q1 = (w1.float() / s1[:, None]).to(torch.float8_e4m3fn)
    h = torch.empty_like(x)
    q = torch.empty(tokens, c, device="cuda", dtype=torch.float8_e4m3fn)
    s = torch.empty(tokens, device="cuda")
    u = torch.empty(tokens, f, device="cuda", dtype=torch.bfloat16)
    cc3d.add_rms_norm(x, gamma, residual=r, eps=1e-6, h=h, q=q, scales=s)
    cc3d.linear(q, q1, u, act=cc3d.ACT_GELU_TANH, x_scales=s, w_scales=s1)
    cc3d.linear(u, w2, h, residual=h)
    cc3d.sync_status()
    hd = b16(x.double() + r.double())
    a = norm64(hd, gamma, 1e-6)
    # the codes as the operator wrote them: theirs is a test of their own
    assert ((q.double() * s.double()[:, None] - a).abs()
            <= 2.0 ** -4 * 1.01 * a.abs() + 2.0 ** -9 * s.double()[:, None]).all()
    z = (q.double() * s.double()[:, None]) @ (q1.double() * s1.double()[:, None]).t()
    z = b16(z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    close(h, z @ w2.double().t() + hd, "feed-forward")


def test_norm_codes_feed_an_fp8_conv_plan():
    """RMS_norm + SiLU into E4M3 with one scale, into an FP8 causal conv: equal
    to quantising the codes' values, within the conv's parity."""
    c, t, h, w = 128, 2, 12, 10
    case = synth.conv_case(c, 64, t, h, w, seed_base=3)
    x = synth.ndhwc(case["x"]).to("cuda")
    gamma = torch.rand(c, device="cuda") + 0.5
    scale = 4.0 / 448
    q = torch.empty(x.shape, device="cuda", dtype=torch.uint8)
    cc3d.add_rms_norm(x, gamma, silu=True, q=q, scale=scale)
    ws = to_dev(case["w"]).float().abs().amax(dim=(1, 2, 3, 4)) / 448
    plan = cc3d.Plan(to_dev(case["w"]), to_dev(case["b"]), h=h, w=w, max_t=t, dtype=cc3d.FP8_E4M3,
                     w_scale=ws, x_scale=scale)
    y = torch.empty(1, t, h, w, 64, device="cuda", dtype=torch.bfloat16)
    plan.forward(q, y)
    cc3d.sync_status()
    codes = q.view(torch.float8_e4m3fn)
    a = norm64(x.double(), gamma)
    a = a * torch.sigmoid(a)
    a = a.clamp(-448 * scale, 448 * scale)
    assert ((codes.double() * scale - a).abs()
            <= 2.0 ** -4 * 1.01 * a.abs() + 2.0 ** -9 * scale).all()
    wq = (case["w"].to("cuda").float() / ws.view(-1, 1, 1, 1, 1)).to(torch.float8_e4m3fn)
    xv = (codes.double() * scale).cpu()
    wv = wq.double().cpu() * ws.double().cpu().view(-1, 1, 1, 1, 1)
    ref = oracle.causal_conv3d(synth.ncthw_view(xv), wv, case["b"].double().numpy())
    assert_close_bf16(ncthw_np(y), ref, "norm codes into an FP8 conv")
    plan.close()


def test_calls_on_several_streams_at_once():
    """Products, attentions and convs on streams of their own give the bytes
    that each gives alone (clusters of different kernels then share the SMs)."""
    x1, w1 = rnd(1, 2048, seed=1), rnd(12288, 2048, seed=2, std=2048 ** -0.5)
    x2, w2 = rnd(7800, 384, seed=3), rnd(1152, 384, seed=4, std=384 ** -0.5)
    qf, kf, vf = (rnd(1, 1560, 12, 128, seed=s) for s in (5, 6, 7))
    qt, kt, vt = rnd(4, 1, 32, 64, seed=8), rnd(4, 3000, 8, 64, seed=9), rnd(4, 3000, 8, 64, seed=10)
    xc = rnd(1, 5, 30, 52, 384, seed=11)
    plan = cc3d.Plan(rnd(384, 384, 3, 3, 3, seed=12, std=0.01), torch.zeros(384, device="cuda"), h=30,
                     w=52, max_t=5)

    def new(*shape):
        return torch.empty(shape, device="cuda", dtype=torch.bfloat16)

    def conv():
        y = new(1, 5, 30, 52, 384)
        plan.forward(xc, y)
        return y

    calls = [
        lambda: cc3d.linear(x1, w1, new(1, 12288), act=cc3d.ACT_SILU),
        lambda: cc3d.attention(qf, kf, vf, new(1, 1560, 12, 128), frame=1560, total=1),
        conv,
        lambda: cc3d.linear(x2, w2, new(7800, 1152)),
        lambda: cc3d.attention(qt, kt, vt, new(4, 1, 32, 64), total=3000),
    ]
    alone = [f() for f in calls]
    cc3d.sync_status()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        got = []
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                for j in (i, (i + 2) % len(calls)):
                    got.append((j, calls[j]()))
        torch.cuda.synchronize()
        for j, o in got:
            assert torch.equal(o, alone[j]), j
    cc3d.sync_status()
