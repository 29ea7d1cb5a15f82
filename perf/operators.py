"""Cases of the transformer operators that stand beside the causal conv: the
matrix product with its epilogue, the RMS norm with the residual's addition
and an 8-bit output, and attention in a sliding window of frames with sink
frames over a cache.

`run` computes a case either in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, where `own` is true, through the
library's public calls.  `exact` computes the same from the definitions in 64
bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---- cases -----------------------------------------------------------------------

def listed():
    return [
        # q, k and v of a mid-block over five 30 x 52 frames of 384 channels
        dict(name="linear_qkv", op="linear", fp8=False, m=7800, k=384, n=1152, act="none",
             residual=False),
        # the second product of a wide feed-forward, added onto the residual stream;
        # a token count that fills no tile
        dict(name="linear_down_residual", op="linear", fp8=False, m=8190, k=8192, n=2048,
             act="none", residual=True),
        # the first product of a feed-forward in 8 bits, scales per token and per channel
        dict(name="linear_up_e4m3_gelu", op="linear", fp8=True, m=7800, k=2048, n=8192,
             act="gelu_tanh", residual=False),
        # one conditioning vector through a modulation layer: latency and weight bytes
        dict(name="linear_one_row_silu", op="linear", fp8=False, m=1, k=2048, n=12288, act="silu",
             residual=False),
        # one token per channel vector of a 30 x 52 clip, into 8 bits
        dict(name="norm_mid", op="norm", rows=7800, c=384, q8="rows", residual=True, silu=False),
        # a long sequence of a wide stream
        dict(name="norm_wide", op="norm", rows=32760, c=4096, q8="rows", residual=True,
             silu=False),
        # a few new tokens: latency
        dict(name="norm_few", op="norm", rows=5, c=2048, q8="rows", residual=True, silu=False),
        # the mid-block: each 30 x 52 frame attends to itself, one head of 384 channels
        dict(name="attn_frames", op="attn", n=1, frame=1560, t=5, past=0, heads=1, kv_heads=1,
             d=384, window=1, sinks=0, ring=0, ragged=False),
        # a streamed video: one new 30 x 52 frame over a ring of six frames and a sink frame
        dict(name="attn_stream", op="attn", n=1, frame=1560, t=1, past=20, heads=12, kv_heads=12,
             d=128, window=6, sinks=1, ring=6, ragged=False),
        # a whole token sequence, shared heads, window with sinks
        dict(name="attn_prefill", op="attn", n=1, frame=1, t=8190, past=0, heads=16, kv_heads=4,
             d=128, window=2048, sinks=4, ring=0, ragged=False),
        # one new token for each of eight sequences of unlike lengths over a long ring cache
        dict(name="attn_token", op="attn", n=8, frame=1, t=1, past=20000, heads=32, kv_heads=8,
             d=128, window=8192, sinks=16, ring=8192, ragged=True),
        # one new token over a short cache: latency
        dict(name="attn_token_short", op="attn", n=1, frame=1, t=1, past=500, heads=8, kv_heads=8,
             d=64, window=1024, sinks=4, ring=1024, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "norm", "attn", "attn"))
    if op == "linear":
        fp8 = rng.random() < 0.4
        step = 16 if fp8 else 8
        k = step * max(1, _log(rng, 64, 8192) // step)
        n = 8 * max(1, _log(rng, 32, 8192) // 8)
        m = _log(rng, 1, 16384)
        m = max(1, min(m, int(1.3e11 / (k * n))))
        return dict(op=op, fp8=fp8, m=m, k=k, n=n,
                    act=rng.choice(("none", "silu", "gelu", "gelu_tanh")),
                    residual=rng.random() < 0.5)
    if op == "norm":
        c = 8 * max(1, _log(rng, 64, 8192) // 8)
        rows = max(1, min(_log(rng, 1, 65536), int(1.3e8 / c)))
        return dict(op=op, rows=rows, c=c, q8=rng.choice(("rows", "rows", "one", "no")),
                    residual=rng.random() < 0.75, silu=rng.random() < 0.25)
    kind = rng.choice(("frames", "stream", "prefill", "token", "token"))
    d = rng.choice((64, 64, 96, 128, 128, 80))
    kv = rng.choice((1, 2, 4, 8))
    heads = kv * rng.choice((1, 1, 2, 3, 4, 8))
    if kind == "frames":
        frame = _log(rng, 60, 1800)
        return dict(op="attn", n=rng.choice((1, 2)), frame=frame, t=rng.randint(1, 5), past=0,
                    heads=1, kv_heads=1, d=rng.choice((96, 192, 384)), window=rng.choice((1, 1, 2)),
                    sinks=rng.choice((0, 0, 1)), ring=0, ragged=False)
    if kind == "stream":
        frame, window, t = _log(rng, 60, 1600), rng.randint(1, 6), rng.randint(1, 2)
        return dict(op="attn", n=1, frame=frame, t=t, past=rng.randint(0, 30), heads=min(heads, 12),
                    kv_heads=min(heads, 12), d=d, window=window, sinks=rng.randint(0, 2),
                    ring=window - 1 + t, ragged=False)
    if kind == "prefill":
        t = _log(rng, 100, 6000)
        return dict(op="attn", n=1, frame=1, t=t, past=_log(rng, 1, 2000) - 1, heads=min(heads, 16),
                    kv_heads=math.gcd(kv, min(heads, 16)), d=d, window=_log(rng, 32, 8192),
                    sinks=rng.randint(0, 8), ring=0, ragged=False)
    window = _log(rng, 64, 8192)
    return dict(op="attn", n=_log(rng, 1, 16), frame=1, t=1, past=_log(rng, 1, 16384), heads=heads,
                kv_heads=kv, d=d, window=window, sinks=rng.randint(0, 16), ring=window + 3,
                ragged=True)


# ---- inputs ------------------------------------------------------------------------

def _normal(g, *shape, std=1.0):
    x = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    return x.normal_(0.0, std, generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = _normal(g, m, k)
        s["w"] = _normal(g, n, k, std=k ** -0.5)
        s["bias"] = torch.empty(n, device="cuda").normal_(0.0, 0.1, generator=g)
        s["x_scales"] = s["w_scales"] = s["res"] = None
        if case["residual"]:
            s["res"] = _normal(g, m, n)
        if case["fp8"]:
            # codes and scales as the norm (tokens) and a checkpoint (channels) give them
            for name in ("x", "w"):
                a = s[name].float()
                sc = a.abs().amax(dim=1) / E4M3_MAX
                s[name] = (a / sc[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
                s[name + "_scales"] = sc
    elif case["op"] == "norm":
        r, c = case["rows"], case["c"]
        s["x"] = _normal(g, r, c)
        s["res"] = _normal(g, r, c, std=3.0) if case["residual"] else None
        s["gamma"] = torch.empty(c, device="cuda").uniform_(0.5, 1.5, generator=g)
    else:
        n, f, t, kvh, d = case["n"], case["frame"], case["t"], case["kv_heads"], case["d"]
        total = case["past"] + t
        slots = case["sinks"] + case["ring"] if case["ring"] else total
        s["q"] = _normal(g, n, t * f, case["heads"], d)
        s["k"] = _normal(g, n, slots * f, kvh, d)
        s["v"] = _normal(g, n, slots * f, kvh, d)
        s["total"], s["k_frames"] = total, None
        if case["ragged"]:
            u = torch.rand(n, generator=g, device="cuda")
            s["k_frames"] = (t + u * case["past"]).to(torch.int32)
        if case["ring"]:
            # the chunk's keys and values, which the call writes into the ring
            s["k_new"] = _normal(g, n, t * f, kvh, d)
            s["v_new"] = _normal(g, n, t * f, kvh, d)
    return s


# ---- the plain form ------------------------------------------------------------------

def _plain_act(a, act):
    if act == "silu":
        return a / (1 + torch.exp(-a))
    if act == "gelu":
        return 0.5 * a * (1 + torch.erf(a * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))
    return a


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().t()
    if s["fp8"]:
        y = y * s["x_scales"][:, None] * s["w_scales"]
    y = _plain_act(y + s["bias"], s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(torch.bfloat16)


def _plain_norm(s):
    h = s["x"]
    if s["res"] is not None:
        h = (s["x"].float() + s["res"].float()).to(torch.bfloat16)
    a = h.float()
    a = a * torch.rsqrt((a * a).mean(dim=1, keepdim=True) + 1e-6) * s["gamma"]
    if s["silu"]:
        a = a / (1 + torch.exp(-a))
    out = {"h": h} if s["res"] is not None else {}
    if s["q8"] == "no":
        out["y"] = a.to(torch.bfloat16)
        return out
    if s["q8"] == "rows":
        amax = a.abs().amax(dim=1)
        out["scales"] = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        a = a / out["scales"][:, None]
    else:
        a = a / 0.02
    out["q"] = a.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return out


def _lengths(s):
    if s["k_frames"] is not None:
        return s["k_frames"].long()
    return torch.full((s["n"],), s["total"], device="cuda", dtype=torch.long)


def _plain_attention(s):
    n, f, t, d, sinks, ring = (s[x] for x in ("n", "frame", "t", "d", "sinks", "ring"))
    last = _lengths(s)[:, None] - 1
    token = torch.arange(t * f, device="cuda")
    qf = last - (t - 1) + token // f                                  # [n, tq]
    slots = torch.arange(s["k"].shape[1] // f, device="cuda")
    if ring:
        # the chunk into its slots, then the frame that each slot holds
        slot = torch.where(qf < sinks, qf, sinks + (qf - sinks) % ring) * f + token % f
        rows = torch.arange(n, device="cuda")[:, None]
        s["k"][rows, slot] = s["k_new"]
        s["v"][rows, slot] = s["v_new"]
        kf = torch.where(slots < sinks, slots, last - (last - slots) % ring)
        kf = torch.where(kf < torch.where(slots < sinks, 0, sinks), last + 1, kf)
    else:
        kf = slots.expand(n, -1)
    kf = kf.repeat_interleave(f, dim=1)                               # [n, tk]
    far = qf[:, :, None] - kf[:, None, :]
    seen = (far >= 0) & ((far < s["window"]) | (kf[:, None, :] < sinks))
    g = s["heads"] // s["kv_heads"]
    q = s["q"].float().view(n, t * f, s["kv_heads"], g, d).permute(0, 2, 3, 1, 4)
    q = q.reshape(n, s["kv_heads"], g * t * f, d)
    k = s["k"].float().permute(0, 2, 3, 1)
    a = (q @ k).view(n, s["kv_heads"], g, t * f, -1) * d ** -0.5
    a.masked_fill_(~seen[:, None, None], -math.inf)
    a -= a.amax(dim=-1, keepdim=True)
    a.exp_()
    a /= a.sum(dim=-1, keepdim=True)
    o = a.view(n, s["kv_heads"], g * t * f, -1) @ s["v"].float().transpose(1, 2)
    o = o.view(n, s["heads"], t * f, d).transpose(1, 2).contiguous().to(torch.bfloat16)
    return {"o": o, "k": s["k"], "v": s["v"]} if ring else {"o": o}


# ---- one pass --------------------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return {"linear": _plain_linear, "norm": _plain_norm, "attn": _plain_attention}[s["op"]](s)
    from video_vae_causal_implicit_b200 import cc3d
    if s["op"] == "linear":
        y = torch.empty((s["m"], s["n"]), device="cuda", dtype=torch.bfloat16)
        act = {"none": cc3d.ACT_NONE, "silu": cc3d.ACT_SILU, "gelu": cc3d.ACT_GELU,
               "gelu_tanh": cc3d.ACT_GELU_TANH}[s["act"]]
        return cc3d.linear(s["x"], s["w"], y, bias=s["bias"], residual=s["res"], act=act,
                           x_scales=s["x_scales"], w_scales=s["w_scales"])
    if s["op"] == "norm":
        out = {"h": torch.empty_like(s["x"])} if s["res"] is not None else {}
        if s["q8"] == "no":
            out["y"] = torch.empty_like(s["x"])
        else:
            out["q"] = torch.empty_like(s["x"], dtype=torch.float8_e4m3fn)
        if s["q8"] == "rows":
            out["scales"] = torch.empty(s["rows"], device="cuda")
        cc3d.add_rms_norm(s["x"], s["gamma"], residual=s["res"], eps=1e-6, silu=s["silu"],
                          scale=0.02 if s["q8"] == "one" else 0.0, **out)
        return out
    o = torch.empty_like(s["q"])
    where = dict(frame=s["frame"], sinks=s["sinks"], ring=s["ring"], total=s["total"],
                 k_frames=s["k_frames"])
    if s["ring"]:
        cc3d.kv_append(s["k_new"], s["v_new"], s["k"], s["v"], **where)
    cc3d.attention(s["q"], s["k"], s["v"], o, window=s["window"], **where)
    return {"o": o, "k": s["k"], "v": s["v"]} if s["ring"] else {"o": o}


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        item = 1 if case["fp8"] else 2
        b = item * (m * k + n * k) + 2 * m * n * (2 if case["residual"] else 1) + 4 * n
        return {"bytes": b + (4 * (m + n) if case["fp8"] else 0), "flops": 2 * m * k * n}
    if case["op"] == "norm":
        r, c = case["rows"], case["c"]
        b = r * c * (2 + (4 if case["residual"] else 0) + (2 if case["q8"] == "no" else 1)) + 4 * c
        return {"bytes": b + (4 * r if case["q8"] == "rows" else 0), "flops": 8 * r * c}
    n, f, t, d, kvh = (case[x] for x in ("n", "frame", "t", "d", "kv_heads"))
    # a ragged case's sequences hold half of the drawn past on average
    total = t + (case["past"] // 2 if case["ragged"] else case["past"])
    pairs, lo = 0, total
    for i in range(total - t, total):
        first = max(0, i - case["window"] + 1)
        pairs += i + 1 - first + min(case["sinks"], first)
        lo = min(lo, first)
    keys = total - lo + min(case["sinks"], lo)
    b = 2 * n * f * d * (2 * t * case["heads"] + 2 * keys * kvh)
    if case["ring"]:
        b += 2 * n * f * d * kvh * t * 2  # the chunk, read once and written into the ring
    return {"bytes": b, "flops": 4 * n * case["heads"] * d * f * f * pairs}


# ---- in 64 bits, from the definitions -----------------------------------------------------

def _exact_linear(s):
    n = s["n"]
    y = torch.empty((s["m"], n), device="cuda", dtype=torch.float64)
    x = s["x"].double()
    if s["fp8"]:
        x = x * s["x_scales"].double()[:, None]
    for c in range(0, n, 1024):
        w = s["w"][c:c + 1024].double()
        if s["fp8"]:
            w = w * s["w_scales"][c:c + 1024].double()[:, None]
        y[:, c:c + 1024] = torch.nn.functional.linear(x, w, s["bias"][c:c + 1024].double())
    if s["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif s["act"] == "gelu":
        y = y * 0.5 * torch.erfc(-y / math.sqrt(2.0))
    elif s["act"] == "gelu_tanh":
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    return y if s["res"] is None else y + s["res"].double()


def _exact_norm(s):
    out = {}
    h = s["x"].double()
    if s["res"] is not None:
        out["h"] = h + s["res"].double()
        h = out["h"].to(torch.bfloat16).double()  # the stream is held in 16 bits
    a = h / torch.sqrt((h ** 2).sum(dim=1, keepdim=True) / s["c"] + 1e-6) * s["gamma"].double()
    if s["silu"]:
        a = a * torch.sigmoid(a)
    if s["q8"] == "no":
        out["y"] = a
    elif s["q8"] == "one":
        out["q"] = torch.clamp(a / 0.02, -E4M3_MAX, E4M3_MAX)
    else:
        top = torch.amax(a.abs(), dim=1)
        out["scales"] = torch.where(top == 0, 1.0, top / E4M3_MAX)
        out["q"] = a / out["scales"][:, None]
    return out


def _exact_attention(s):
    f, t, d, sinks, ring, window = (s[x] for x in ("frame", "t", "d", "sinks", "ring", "window"))
    g = s["heads"] // s["kv_heads"]
    lengths = _lengths(s).tolist()
    k, v = s["k"].clone(), s["v"].clone()
    o = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)

    def slot(p):
        return p if not ring or p < sinks else sinks + (p - sinks) % ring

    for b, total in enumerate(lengths):
        if ring:
            for i in range(t):
                at = slot(total - t + i) * f
                k[b, at:at + f] = s["k_new"][b, i * f:(i + 1) * f]
                v[b, at:at + f] = s["v_new"][b, i * f:(i + 1) * f]
        # runs of query frames, so that a long sequence takes few steps
        run_of = 1 if f > 1 else 512
        for i0 in range(0, t, run_of):
            i1 = min(t, i0 + run_of)
            first, final = total - t + i0, total - t + i1 - 1
            lo = max(0, first - window + 1)
            frames = list(range(min(sinks, lo))) + list(range(lo, final + 1))
            at = torch.tensor([slot(p) for p in frames], device="cuda")
            at = (at[:, None] * f + torch.arange(f, device="cuda")).reshape(-1)
            pk = torch.tensor(frames, device="cuda").repeat_interleave(f)
            pq = torch.arange(first, final + 1, device="cuda").repeat_interleave(f)
            hidden = (pk > pq[:, None]) | ((pk <= pq[:, None] - window) & (pk >= sinks))
            for h in range(s["heads"]):
                q = s["q"][b, i0 * f:i1 * f, h].double()
                e = q @ k[b, at, h // g].double().t() / math.sqrt(d)
                e = torch.softmax(e.masked_fill(hidden, -math.inf), dim=1)
                o[b, i0 * f:i1 * f, h] = e @ v[b, at, h // g].double()
    return {"o": o, "k": k.double(), "v": v.double()} if ring else {"o": o}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(s)
    return _exact_norm(s) if case["op"] == "norm" else _exact_attention(s)
