"""cc3d_attention and cc3d_kv_append on the GPU against the definition in 64
bits.

Tolerance, from the arithmetic.  A score is a sum of d exact products in fp32
(off by (d + 8) 2^-23 of the sum of their magnitudes) and enters the exponent
with two roundings of its own size (2^-23 |s|) beside the hardware
exponential's 2^-21; a weight is rounded to bf16 (2^-8) before the second
product while the weights' sum takes it unrounded; that product sums K terms
in fp32.  With A = sum p |v| / sum p an output is off by at most
A (2^-8 + 4 e + (K + 8) 2^-22), e the largest score error, and by its own
rounding, 2^-8 |o|.

That does not show one key too many or too few among thousands, so the masks
are tested apart, with equal scores (q = 0: every weight is exactly 1) and
values that are 1 at one token per channel: an output is then 1 / (keys seen)
if the query sees that token (exact but for the division and the rounding),
and exactly 0 if not."""
import math

import pytest
import torch

from video_vae_causal_implicit_b200 import cc3d

pytestmark = pytest.mark.gpu


def slot_of(p, sinks, ring):
    return p if not ring or p < sinks else sinks + (p - sinks) % ring


class Case:
    """Logical sequences (every frame's k and v) and the caches made of them."""

    def __init__(self, *, n=1, frame=1, t=1, total=1, heads=1, kv=1, d=64, window=0, sinks=0,
                 ring=0, slots=None, k_frames=None, q_frames=None, seed=0, fill=float("nan")):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.f, self.t, self.heads, self.kv, self.d = n, frame, t, heads, kv, d
        self.window, self.sinks, self.ring = window, sinks, ring
        self.all = list(k_frames) if k_frames is not None else [total] * n
        self.chunk = list(q_frames) if q_frames is not None else [t] * n
        self.total = total
        self.dev_all = None if k_frames is None else torch.tensor(k_frames, device="cuda",
                                                                  dtype=torch.int32)
        self.dev_chunk = None if q_frames is None else torch.tensor(q_frames, device="cuda",
                                                                    dtype=torch.int32)
        most = max(max(self.all), 1)
        self.slots = slots or (sinks + ring if ring else most)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
        self.q = rnd(n, t * frame, heads, d)
        self.lk, self.lv = rnd(n, most * frame, kv, d), rnd(n, most * frame, kv, d)
        self.fill = fill

    def caches(self):
        """The caches as the frames before the chunk and the chunk itself leave them."""
        f = self.f
        shape = (self.n, self.slots * f, self.kv, self.d)
        k, v = (torch.full(shape, self.fill, device="cuda", dtype=torch.bfloat16)
                for _ in range(2))
        for b in range(self.n):
            for p in range(self.all[b]):
                s = slot_of(p, self.sinks, self.ring)
                if s < self.slots:
                    k[b, s * f:(s + 1) * f] = self.lk[b, p * f:(p + 1) * f]
                    v[b, s * f:(s + 1) * f] = self.lv[b, p * f:(p + 1) * f]
        return k, v

    def args(self):
        return dict(frame=self.f, window=self.window, sinks=self.sinks, ring=self.ring,
                    total=self.total, k_frames=self.dev_all, q_frames=self.dev_chunk)

    def run(self, q=None, k=None, v=None, o=None, **kw):
        if k is None:
            k, v = self.caches()
        q = self.q if q is None else q
        if o is None:
            o = torch.full(q.shape, 7.0, device="cuda", dtype=torch.bfloat16)
        cc3d.attention(q, k, v, o, **self.args(), **kw)
        cc3d.sync_status()
        return o

    def seen(self, b):
        """[chunk tokens, all tokens] which keys each query sees."""
        a, c, f = self.all[b], self.chunk[b], self.f
        pq = a - c + torch.arange(c * f, device="cuda") // f
        pk = torch.arange(a * f, device="cuda") // f
        far = pq[:, None] - pk
        near = far < self.window if self.window else torch.ones_like(far, dtype=torch.bool)
        return (far >= 0) & (near | (pk < self.sinks))

    def reference(self, b, scale=None):
        """(o, tolerance) of sequence b's chunk, in 64 bits: [tokens, heads, d]."""
        a, c, f, d = self.all[b], self.chunk[b], self.f, self.d
        seen, g = self.seen(b), self.heads // self.kv
        scale = scale or d ** -0.5
        o = torch.zeros(c * f, self.heads, d, device="cuda", dtype=torch.float64)
        tol = torch.zeros_like(o)
        for h in range(self.heads if a and c else 0):
            q = self.q[b, :c * f, h].double()
            k, v = self.lk[b, :a * f, h // g].double(), self.lv[b, :a * f, h // g].double()
            s = q @ k.t() * scale
            mag = (q.abs() @ k.abs().t()) * scale
            hid = ~seen
            s = s.masked_fill(hid, -math.inf)
            p = torch.exp(s - s.amax(1, keepdim=True).clamp_min(-1e300))
            p = p.masked_fill(hid, 0)
            l = p.sum(1, keepdim=True)
            p = torch.where(l > 0, p / l.clamp_min(1e-300), p)
            o[:, h] = p @ v
            big = p @ v.abs()
            err = ((d + 8) * 2.0 ** -23 * mag + 2.0 ** -22 * mag + 2.0 ** -21).masked_fill(hid, 0)
            e = err.amax(1, keepdim=True)
            tol[:, h] = (big * (2.0 ** -8 + 4 * e + (a * f + 8) * 2.0 ** -22) +
                         2.0 ** -8 * o[:, h].abs()) * 1.01 + 1e-30
        return o, tol

    def check(self, o, scale=None):
        for b in range(self.n):
            c = self.chunk[b] * self.f
            ref, tol = self.reference(b, scale)
            got = o[b, :c].double()
            bad = ~((got - ref).abs() <= tol)
            assert not bad.any(), (b, int(bad.sum()), bad.nonzero()[:3].tolist(),
                                   float((got - ref).abs().nan_to_num(9e9).max()))
            assert (o[b, c:] == 7).all(), "rows behind the chunk"


CASES = {
    # one token, growing lengths, head sizes, shared heads
    "one key": dict(total=1, d=64),
    "short": dict(total=37, d=8, heads=2, kv=2),
    "token": dict(total=300, d=128, heads=8, kv=2, n=3),
    "token mha": dict(total=515, d=80, heads=4, kv=4),
    "token mqa": dict(total=1000, d=96, heads=32, kv=1),
    "token wide group": dict(total=130, d=64, heads=128, kv=1),
    "token odd group": dict(total=700, d=64, heads=6, kv=2),
    "token long": dict(total=9000, d=128, heads=4, kv=1),
    "token wide head": dict(total=260, d=384, heads=2, kv=1),
    # a whole sequence
    "prefill": dict(t=257, total=257, d=64, heads=3, kv=3),
    "prefill window": dict(t=700, total=700, d=128, heads=4, kv=2, window=100, sinks=3),
    "prefill many": dict(t=1500, total=1500, d=128, heads=48, kv=16, window=333, sinks=5),
    "prefill after past": dict(t=300, total=811, d=72, heads=16, kv=16, window=200, sinks=130),
    "prefill two": dict(n=2, t=640, total=700, d=96, heads=64, kv=32, window=64),
    # frames
    "frames": dict(frame=70, t=3, total=3, d=384, window=1),
    "frames 200": dict(frame=130, t=2, total=4, d=200, window=2, sinks=1, heads=2, kv=2),
    "frame of one tile": dict(frame=128, t=2, total=5, d=128, window=2, sinks=1, heads=2, kv=1),
    "frame large": dict(frame=1560, t=1, total=2, d=384, window=1),
    "frames many": dict(frame=200, t=4, total=6, d=64, heads=20, kv=20, window=3, sinks=1),
    # rings, not full, full, wrapped
    "ring young": dict(total=5, d=64, window=20, sinks=4, ring=20),
    "ring": dict(total=1003, d=64, window=250, sinks=4, ring=256, heads=2, kv=1),
    "ring exact": dict(total=777, d=128, window=100, sinks=0, ring=100),
    "ring chunk": dict(t=40, total=533, d=64, window=200, sinks=7, ring=239, heads=4, kv=2),
    "ring frames": dict(frame=100, t=2, total=11, d=128, window=3, sinks=1, ring=4, heads=3, kv=3),
    "ring frames many": dict(frame=330, t=1, total=20, d=64, window=4, sinks=1, ring=4, heads=40,
                             kv=40),
    # lengths per sequence, padded chunks, sequences without frames
    "ragged": dict(n=4, t=1, d=64, heads=4, kv=2, window=50, sinks=2, ring=60,
                   k_frames=[1, 3, 61, 400]),
    "padded": dict(n=3, t=50, d=64, heads=2, kv=2, window=30, sinks=1, k_frames=[50, 77, 10],
                   q_frames=[50, 20, 0]),
    "empty sequence": dict(n=3, t=2, d=64, heads=2, kv=2, k_frames=[0, 5, 2], q_frames=[0, 2, 2]),
    "before the start": dict(n=2, t=6, d=64, k_frames=[3, 0], window=4, q_frames=[6, 6]),
}


@pytest.mark.parametrize("name", CASES)
def test_against_the_definition(name):
    c = Case(**CASES[name], seed=len(name))
    # (the reference's chunk of a sequence shorter than it starts before frame 0)
    if name == "before the start":
        o = c.run()
        assert (o[0, :3] == 0).all() and (o[1] == 0).all()
        short = Case(**dict(CASES[name], q_frames=[3, 0]), seed=len(name))
        short.q = c.q[:, 3:]
        short.q = torch.cat([short.q, short.q], 1)
        ref, tol = short.reference(0)
        assert ((o[0, 3:].double() - ref).abs() <= tol).all()
        return
    c.check(c.run())


MASKS = {
    "tokens": dict(t=400, total=400, d=128, heads=2, kv=2, window=0),
    "tokens window": dict(t=500, total=500, d=128, heads=2, kv=1, window=129, sinks=2),
    "tokens window 1": dict(t=300, total=300, d=64, heads=1, kv=1, window=1, sinks=0),
    "tokens many": dict(t=900, total=1000, d=64, heads=40, kv=20, window=128, sinks=128),
    "one token": dict(t=1, total=2100, d=128, heads=8, kv=8, window=2000, sinks=8),
    "ring": dict(t=1, total=3333, d=128, heads=4, kv=1, window=1000, sinks=8, ring=1003),
    "ring chunk": dict(t=90, total=1234, d=128, heads=2, kv=2, window=311, sinks=3, ring=400),
    "frames": dict(frame=77, t=4, total=4, d=384, window=2, sinks=1),
    "frames ring": dict(frame=129, t=2, total=13, d=64, heads=20, kv=20, window=3, sinks=2, ring=4),
}


@pytest.mark.parametrize("name", MASKS)
def test_masks_key_by_key(name):
    for seed in range(3):
        c = Case(**MASKS[name], seed=seed)
        c.q.zero_()
        c.lk.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        g = torch.Generator(device="cuda").manual_seed(100 + seed)
        most = max(c.all) * c.f
        # marked tokens: anywhere, and at the edges of what some queries see
        edges = torch.tensor([0, c.f - 1, c.f, c.sinks * c.f - 1, c.sinks * c.f, most - 1,
                              most - c.f, (max(c.all) - c.window) * c.f,
                              (max(c.all) - c.window) * c.f - 1], device="cuda").clamp(0, most - 1)
        at = torch.randint(0, most, (c.d,), device="cuda", generator=g)
        at[:len(edges)] = edges[:c.d]
        c.lv.zero_()
        c.lv[:, at, :, torch.arange(c.d, device="cuda")] = 1
        o = c.run()
        for b in range(c.n):
            seen = c.seen(b)
            keys = seen.sum(1).double()
            want = seen[:, at].double() / keys[:, None].clamp_min(1)
            got = o[b, :c.chunk[b] * c.f].double()
            for h in range(c.heads):
                diff = (got[:, h] - want).abs() > want * 2.0 ** -8 * 1.001
                assert not diff.any(), (name, seed, h, diff.nonzero()[:4].tolist())


@pytest.mark.parametrize("name", ["token", "prefill window", "frames", "ring chunk"])
def test_slices_of_a_fused_product(name):
    """q, k and v as slices of one buffer, o with gaps, a given scale."""
    kw = dict(CASES[name], ring=0, slots=None, k_frames=None)
    kw["t"] = kw["total"]  # the chunk is the whole sequence
    c = Case(**kw, seed=3)
    hq, hk, tok = c.heads * c.d, c.kv * c.d, c.t * c.f
    fused = torch.empty(c.n, tok, hq + 2 * hk + 8, device="cuda", dtype=torch.bfloat16)
    q = fused[..., :hq].view(c.n, tok, c.heads, c.d)
    k = fused[..., hq:hq + hk].view(c.n, tok, c.kv, c.d)
    v = fused[..., hq + hk:hq + 2 * hk].view(c.n, tok, c.kv, c.d)
    q.copy_(c.q)
    k.copy_(c.lk)
    v.copy_(c.lv)
    wide = torch.full((c.n, tok, c.heads, c.d + 16), 5.0, device="cuda", dtype=torch.bfloat16)
    o = wide[..., :c.d]
    c.run(q, k, v, o, scale=0.21)
    c.check(o, 0.21)
    assert (wide[..., c.d:] == 5).all()
    # heads before tokens
    qt, kt, vt = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v))
    o2 = c.run(qt, kt, vt, scale=0.21)
    assert torch.equal(o2, o)


def test_large_scores_and_growing_maxima():
    """Scores that grow along the keys, so that the running maximum moves."""
    for t, d in ((1, 64), (300, 128), (200, 384)):
        c = Case(t=t, total=1000, d=d, heads=2, kv=2, seed=4)
        ramp = torch.linspace(0.1, 12, 1000, device="cuda").view(1, 1000, 1, 1)
        c.lk = (c.lk.float() * ramp).to(torch.bfloat16)
        c.check(c.run())
        c.lk = c.lk.flip(1)
        c.check(c.run())


def test_infinite_key_and_nan_value_are_as_in_the_definition():
    c = Case(t=1, total=200, d=64, heads=1, kv=1, window=50, seed=2)
    clean = c.run()
    # outside the window: no influence, whatever stands there
    c.lk[0, 100] = float("inf")
    c.lv[0, 120] = float("nan")
    assert torch.equal(c.run(), clean)
    c.lv[0, 180, 0, 5] = float("nan")
    o = c.run()
    assert torch.isnan(o[0, 0, 0, 5]) and torch.isfinite(o[0, 0, 0, :5].float()).all()


HIDDEN = {
    "tokens": dict(t=200, total=200, d=64, heads=4, kv=2, window=50),
    "tokens sinks": dict(t=300, total=700, d=128, heads=2, kv=1, window=100, sinks=2),
    "no window": dict(t=70, total=70, d=40, heads=1, kv=1),
    "many rows": dict(t=2000, total=2000, d=128, heads=8, kv=8, window=300),
    "shared heads": dict(t=500, total=900, d=64, heads=32, kv=4, window=0),
    "split keys": dict(t=4, total=3001, d=128, heads=8, kv=2, window=0),
    "wide frames": dict(frame=10, t=20, total=30, d=384, window=3),
    "wide": dict(frame=7, t=9, total=40, d=200, window=5, sinks=1, heads=2, kv=2),
    "ring": dict(frame=16, t=6, total=40, d=64, heads=2, kv=2, window=6, sinks=1, ring=12),
    "lengths": dict(n=3, t=40, d=128, heads=4, kv=2, window=30, k_frames=[60, 40, 130],
                    q_frames=[40, 17, 33]),
}


@pytest.mark.parametrize("name", list(HIDDEN))
def test_values_that_are_not_finite_reach_the_queries_that_see_them_alone(name):
    """Infinities and NaN in values that some queries of the chunk see and
    others, in the same tile of rows, do not."""
    c = Case(**HIDDEN[name], seed=8)
    kinds = [float("inf"), float("nan"), -float("inf")]
    put = []  # sequence, key, kv head, channel, value; a channel is used once
    for b in range(c.n):
        keys = c.all[b] * c.f
        first = max(0, (c.all[b] - c.chunk[b]) * c.f)
        at = sorted({0, 1, first, first + 1, first + 3, (first + keys) // 2, keys - 2, keys - 1,
                     max(0, first - 7), keys // 2})
        for i, key in enumerate(x for x in at if 0 <= x < keys):
            put.append((b, key, i % c.kv, (5 * i + 3) % c.d, kinds[i % 3]))
    for b, key, h, ch, value in put:
        c.lv[b, key, h, ch] = value
    o = c.run()
    for b, key, h, ch, _ in put:
        c.lv[b, key, h, ch] = 0
    group = c.heads // c.kv
    for b in range(c.n):
        rows = c.chunk[b] * c.f
        ref, tol = c.reference(b)
        got = o[b, :rows].double()
        good = (got - ref).abs() <= tol
        seen = c.seen(b)
        for _, key, h, ch, value in [x for x in put if x[0] == b]:
            for head in range(h * group, (h + 1) * group):
                mine = got[:, head, ch][seen[:, key]]
                assert (torch.isnan(mine) if value != value else mine == value).all(), (key, ch)
                good[:, head, ch] |= seen[:, key]
        assert good.all(), (b, int((~good).sum()), (~good).nonzero()[:3].tolist())
        assert (o[b, rows:] == 7).all()


@pytest.mark.parametrize("name", ["token", "prefill window", "ring chunk", "frame large",
                                  "ring frames many"])
def test_same_bytes_on_every_call_stream_and_replay(name):
    c = Case(**CASES[name], seed=1)
    k, v = c.caches()
    first = c.run(k=k, v=v)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(9):
        o = torch.full_like(first, 7)
        streams[i % 3].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(streams[i % 3]):
            cc3d.attention(c.q, k, v, o, **c.args())
        outs.append(o)
    torch.cuda.synchronize()
    o = torch.full_like(first, 7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cc3d.attention(c.q, k, v, o, **c.args())
    graph.replay()
    graph.replay()
    cc3d.sync_status()
    for x in outs + [o]:
        assert torch.equal(x, first)


APPEND = {
    "plain": dict(t=3, total=10, d=64, heads=2, kv=2),
    "ring": dict(t=2, total=47, d=128, heads=2, kv=2, window=9, sinks=2, ring=10),
    "into sinks": dict(t=4, total=5, d=64, heads=1, kv=1, window=3, sinks=3, ring=6),
    "chunk longer than the ring": dict(t=30, total=60, d=64, window=1, sinks=2, ring=7),
    "frames": dict(frame=50, t=2, total=9, d=96, heads=3, kv=3, window=2, sinks=1, ring=3),
    "ragged": dict(n=4, t=2, d=64, window=4, sinks=1, ring=5, k_frames=[2, 0, 9, 33],
                   q_frames=[2, 0, 1, 2]),
}


@pytest.mark.parametrize("name", APPEND)
def test_append(name):
    c = Case(**APPEND[name], fill=3.0)
    want_k, want_v = c.caches()
    # the caches before the chunk: the frames up to it (later ones of the
    # chunk's slots still hold what was there)
    before = Case(**dict(APPEND[name]), fill=3.0)
    before.lk, before.lv = c.lk, c.lv
    before.all = [a - q for a, q in zip(c.all, c.chunk)]
    k, v = before.caches()
    f = c.f
    shape = (c.n, c.t * f, 2, c.kv, c.d)
    new = torch.full(shape, float("nan"), device="cuda", dtype=torch.bfloat16)
    for b in range(c.n):
        a, q = c.all[b] * f, c.chunk[b] * f
        new[b, :q, 0], new[b, :q, 1] = c.lk[b, a - q:a], c.lv[b, a - q:a]
    args = c.args()
    args.pop("window")
    cc3d.kv_append(new[:, :, 0], new[:, :, 1], k, v, **args)
    cc3d.sync_status()
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


def test_streaming_token_by_token_equals_the_whole_sequence():
    """Append and attend, one frame a call, over a ring, against one call over
    the whole sequence; the calls of a step captured once and replayed."""
    n, frame, steps, heads, kv, d, window, sinks = 2, 24, 12, 4, 2, 64, 3, 1
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda h: torch.randn(n, steps * frame, h, d, device="cuda", generator=g).to(  # noqa: E731
        torch.bfloat16)
    q, k, v = rnd(heads), rnd(kv), rnd(kv)
    whole = torch.empty_like(q)
    cc3d.attention(q, k, v, whole, frame=frame, window=window, sinks=sinks, total=steps)
    ring = window
    kc = torch.full((n, (sinks + ring) * frame, kv, d), float("nan"), device="cuda",
                    dtype=torch.bfloat16)
    vc = kc.clone()
    qs, ks, vs = (x[:, :frame].clone() for x in (q, k, v))
    o = torch.empty_like(qs)
    count = torch.zeros(n, device="cuda", dtype=torch.int32)

    def step():
        cc3d.kv_append(ks, vs, kc, vc, frame=frame, sinks=sinks, ring=ring, k_frames=count)
        cc3d.attention(qs, kc, vc, o, frame=frame, window=window, sinks=sinks, ring=ring,
                       k_frames=count)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kc.fill_(float("nan"))
    vc.fill_(float("nan"))
    for i in range(steps):
        for dst, src in ((qs, q), (ks, k), (vs, v)):
            dst.copy_(src[:, i * frame:(i + 1) * frame])
        count.fill_(i + 1)
        graph.replay()
        a, b = o.double(), whole[:, i * frame:(i + 1) * frame].double()
        # the same sums in another order: bf16 steps of the weights and outputs
        assert ((a - b).abs() <= 2.0 ** -6 * (1 + b.abs())).all()
    cc3d.sync_status()


def test_long_cache_offsets_past_32_bits():
    """A cache of more than 2^31 elements: 9 sequences of a million tokens, of
    which the last ones and the sinks are read."""
    n, slots, kv, d = 9, 1 << 20, 2, 128
    assert n * slots * kv * d > 1 << 31
    k = torch.zeros(n, slots, kv, d, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    c = Case(n=n, t=1, total=600, d=d, heads=4, kv=kv, window=500, sinks=2, seed=7)
    q = c.q
    # the last 498 tokens of a sequence of `slots`, and the two sinks
    keep = torch.cat([torch.arange(2), torch.arange(slots - 500, slots)]).cuda()
    k[:, keep], v[:, keep] = c.lk[:, 98:], c.lv[:, 98:]
    o = torch.empty_like(q)
    cc3d.attention(q, k, v, o, window=500, sinks=2, total=slots)
    small = torch.empty_like(q)
    cc3d.attention(q, c.lk[:, 98:].contiguous(), c.lv[:, 98:].contiguous(), small, total=502)
    cc3d.sync_status()
    assert ((o.double() - small.double()).abs() <= 2.0 ** -6 * (1 + small.double().abs())).all()
    assert o[n - 1].abs().max() > 0


def test_no_sequences_and_no_chunk():
    c = Case(total=4, t=1, d=64)
    k, v = c.caches()
    before = cc3d.cc3d_launch_count()
    cc3d.attention(c.q[:0], k[:0], v[:0], c.q[:0].clone(), total=4)
    cc3d.attention(c.q[:, :0], k, v, c.q[:, :0].clone(), total=4)
    cc3d.kv_append(c.q[:, :0], c.q[:, :0], k, v, total=4)
    assert cc3d.cc3d_launch_count() == before


@pytest.mark.parametrize("ring", [0, 5])
def test_append_with_counts_out_of_range_writes_nothing(ring):
    """Negative counts are empty sequences, the least one among them; a frame
    past the last slot of a plain cache has no place."""
    counts = [-2 ** 31, -2 ** 31 + 1, -1, 0] + ([] if ring else [2 ** 31 - 1, 9])
    n = len(counts)
    k_frames = torch.tensor(counts, dtype=torch.int32, device="cuda")
    new = torch.ones(n, 2, 2, 64, device="cuda", dtype=torch.bfloat16)
    kc, vc = (torch.zeros(n, 7, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cc3d.kv_append(new, new.clone(), kc, vc, sinks=2, ring=ring, k_frames=k_frames)
    cc3d.sync_status()
    assert not kc.any() and not vc.any()


# One frame a call, long enough for whole waves of full row tiles and a second
# launch for what is left: (least launches, the case)
LONG_FRAMES = {
    "ring with sink": (2, dict(frame=1560, total=9, d=128, heads=12, kv=12, window=6, sinks=1,
                               ring=6)),
    "many heads": (2, dict(frame=1560, total=9, d=128, heads=24, kv=24, window=4, sinks=1,
                           ring=4)),
    "shared heads": (1, dict(frame=1301, total=7, d=64, heads=24, kv=8, window=5, sinks=1)),
    "odd head size": (1, dict(frame=1811, total=6, d=200, heads=6, kv=6)),
    "lengths and padding": (1, dict(n=3, frame=1560, d=128, heads=12, kv=12, window=4, sinks=2,
                                    ring=4, k_frames=[9, 1, 4], q_frames=[1, 1, 0])),
}


@pytest.mark.parametrize("name", LONG_FRAMES)
def test_long_frame_in_two_launches(name):
    launches, kw = LONG_FRAMES[name]
    c = Case(**kw, seed=len(name))
    k, v = c.caches()
    before = cc3d.cc3d_launch_count()
    o = c.run(k=k, v=v)
    assert launches <= cc3d.cc3d_launch_count() - before <= 2
    c.check(o)
    again = torch.full_like(o, 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cc3d.attention(c.q, k, v, again, **c.args())
    graph.replay()
    cc3d.sync_status()
    assert torch.equal(o, again)


def test_more_tiles_than_a_grid_holds_are_refused():
    """2^32 heads of all sequences: refused before an address is looked at."""
    n = 65535
    seq, far = n * 8, 1 << 40
    names = ("n heads kv_heads d frame t slots window sinks ring total scale q_frames k_frames q k v "
             "o").split()
    a = dict(zip(names, (n, n, n, 8, 1, 1, 1, 0, 0, 0, 1, 0.0, 0, 0, far, 2 * far, 3 * far, 4 * far)))
    before = cc3d.cc3d_launch_count()
    call = cc3d._ATTN_CALL.pack(*a.values(), *(4 * (seq, seq, 8)))
    assert cc3d.lib().cc3d_attention(call, None) == cc3d.ERR_UNSUPPORTED
    assert cc3d.cc3d_launch_count() == before


@pytest.mark.parametrize("heads,kv,total", [(8, 1, 4000), (16, 2, 9000), (4, 4, 130)])
@pytest.mark.parametrize("spread", [1.0, 30.0, 4000.0])
def test_one_token_with_scores_over_the_whole_range(heads, kv, total, spread):
    """Weights from 1 down to below the least number (scores apart by more than
    2^7 and 2^12), and a NaN score in every place of a key tile in turn."""
    c = Case(total=total, d=64, heads=heads, kv=kv, seed=total)
    c.check(c.run(scale=spread * 64 ** -0.5), spread * 64 ** -0.5)
    if spread == 1.0:
        k, v = c.caches()
        for key in list(range(total - 128, total)):
            kn = k.clone()
            kn[0, key, 0, 3] = float("nan")
            o = c.run(k=kn, v=v)
            mine = o[0, 0, :heads // kv].float()
            assert torch.isnan(mine).all(), key
            assert torch.isfinite(o[0, 0, heads // kv:].float()).all(), key


def test_counts_out_of_range_count_as_the_nearest():
    """Frame counts below 0 or above the slots, chunk counts below 0 or above
    t; in a ring, the largest count there is."""
    top = 2 ** 31 - 1
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    ints = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)  # noqa: E731
    q, k, v = rnd(4, 2, 4, 64), rnd(4, 12, 2, 64), rnd(4, 12, 2, 64)

    def run(counts, chunks, **kw):
        o = torch.full_like(q, 7.0)
        cc3d.attention(q, k, v, o, k_frames=ints(*counts), q_frames=ints(*chunks), **kw)
        cc3d.sync_status()
        return o
    o = run((-2 ** 31, -1, top, 13), (2, 99, top, -3), window=5, sinks=1)
    assert torch.equal(o, run((0, 0, 12, 12), (2, 2, 2, 0), window=5, sinks=1))
    assert (o[:2] == 0).all() and (o[3] == 7).all()
    # of frames 2, 3, ... one in ten has the same slot
    ring = dict(window=8, sinks=2, ring=10)
    same = [2 + (x - 2) % 10 + 20 for x in (top, top - 1, top - 9)]
    o = run((top, top - 1, top - 9, -7), (2, 2, 1, 2), **ring)
    assert torch.equal(o, run((*same, 0), (2, 2, 1, 2), **ring))


# Few query rows over many keys (their keys are split over a cluster), and many
# rows, whose keys are not: NaN has to come out of both alike.
NAN_SCORES = {
    "token long": dict(total=9000, d=128, heads=4, kv=1),
    "token": dict(n=3, total=2100, d=64, heads=8, kv=2),
    "token odd head size": dict(total=4100, d=80, heads=4, kv=4),
    "tokens": dict(t=4, total=3001, d=128, heads=8, kv=2),
    "ring": dict(total=9003, d=128, heads=8, kv=2, window=2000, sinks=5, ring=2000),
    "frames": dict(frame=1560, t=5, total=5, d=384, window=1),
    "wide frame": dict(frame=700, t=1, total=3, d=200, heads=2, kv=2),
    "stream": dict(frame=500, t=1, total=9, d=128, heads=2, kv=2, window=6, sinks=1, ring=6),
    "unsplit": dict(t=1500, total=1500, d=128, heads=48, kv=16, window=333, sinks=5),
    "unsplit frames": dict(frame=200, t=4, total=6, d=64, heads=20, kv=20, window=3, sinks=1),
}


@pytest.mark.parametrize("name", NAN_SCORES)
def test_nan_queries_and_runs_of_nan_keys_are_as_in_the_definition(name):
    """A query with a NaN has no finite output, and neither has one that sees a
    NaN key, also where every key of a long run of keys (longer than what one
    of eight CTAs may take) is NaN; all other outputs stay."""
    c = Case(**NAN_SCORES[name], seed=5)
    nan = float("nan")
    c.check(c.run())
    # NaN queries: one row of a head, and a whole token
    rows = c.q.shape[1]
    c.q[0, 0, c.heads - 1, 3] = nan
    c.q[c.n - 1, rows - 1, :, c.d - 1] = nan
    assert _check_with_nan(c, c.run()) > 0
    c.q.nan_to_num_(0.5)
    # runs of NaN keys of one kv head: short, a third, all but the last and all
    most, odd = c.all[0] * c.f, 0
    for lo, hi in ((most // 2, most // 2 + 1), (most // 3, 2 * most // 3), (0, most - 1),
                   (1, most), (0, most)):
        kept = c.lk[0, lo:hi, c.kv - 1].clone()
        c.lk[0, lo:hi, c.kv - 1, 1] = nan
        odd += _check_with_nan(c, c.run())
        c.lk[0, lo:hi, c.kv - 1] = kept
    assert odd > 0  # (a window may hide some of the runs)


def _check_with_nan(c, o):
    odd = 0
    for b in range(c.n):
        ref, tol = c.reference(b)
        got = o[b, :ref.shape[0]].double()
        odd += int(torch.isnan(ref).sum())
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), (
            b, (torch.isnan(got) != torch.isnan(ref)).nonzero()[:4].tolist())
        good = torch.isnan(ref) | ((got - ref).abs() <= tol)
        assert good.all(), (b, (~good).nonzero()[:3].tolist())
    return odd


@pytest.mark.parametrize("name", NAN_SCORES)
def test_scores_of_minus_infinity(name):
    """Keys with a score of -inf have no weight; a query that sees only such keys
    has no value (NaN), unlike one that sees nothing (zeros)."""
    c = Case(**NAN_SCORES[name], seed=6)
    c.q[..., 2] = c.q[..., 2].abs() + 0.5
    most, group, plain, odd = c.all[0] * c.f, c.heads // c.kv, c.seen, 0
    for lo, hi in ((most // 3, 2 * most // 3), (0, most - 1), (1, most), (0, most)):
        kept = c.lk[0, lo:hi, c.kv - 1].clone()
        c.lk[0, lo:hi, c.kv - 1, 2] = -math.inf
        o = c.run()[0, :c.chunk[0] * c.f].double()
        run = torch.zeros(most, device="cuda", dtype=torch.bool)
        run[lo:hi] = True
        c.seen = lambda b: plain(b) & ~run
        left, seen = c.seen(0), plain(0)
        none = seen.any(1) & ~left.any(1)
        odd += int(none.sum())
        ref, tol = c.reference(0)
        c.seen = plain
        mine = slice((c.kv - 1) * group, c.heads)  # the heads that read these keys
        assert torch.isnan(o[none][:, mine]).all(), (lo, hi)
        assert ((o - ref).abs() <= tol)[~none][:, mine].all(), (lo, hi)
        c.lk[0, lo:hi, c.kv - 1] = kept
    assert odd > 0
    blank = Case(**dict(NAN_SCORES[name], k_frames=[0] * c.n), seed=6)
    assert (blank.run() == 0).all()


@pytest.mark.parametrize("name", ["token", "token wide head", "prefill many", "frames 200",
                                  "frame large", "ring", "ring frames", "prefill window"])
def test_no_frames_at_all_gives_zeros(name):
    """total = 0: the whole chunk lies before the sequence and sees nothing, as
    with counts of 0 on the device."""
    kw = dict(CASES[name], total=0)
    c = Case(**kw)
    assert (c.run() == 0).all()
    assert (Case(**dict(kw, k_frames=[0] * c.n)).run() == 0).all()
    k, v = c.caches()
    nothing = k.clone()
    cc3d.kv_append(torch.ones_like(k[:, :c.f]), torch.ones_like(k[:, :c.f]), k, v, frame=c.f,
                   sinks=c.sinks, ring=c.ring, total=0)
    cc3d.sync_status()
    assert torch.equal(k.view(torch.int16), nothing.view(torch.int16))


@pytest.mark.parametrize("name", ["ring", "frames", "ragged", "into sinks"])
@pytest.mark.parametrize("level", ["heads", "tokens", "sequences"])
def test_append_and_attention_over_interleaved_caches(name, level):
    """Both caches as slices of one tensor: an entry's keys beside its values,
    token by token, or sequence by sequence."""
    c = Case(**dict(APPEND[name]), fill=3.0)
    want_k, want_v = c.caches()
    c.all = [a - q for a, q in zip(c.all, c.chunk)]
    old_k, old_v = c.caches()
    c.all = [a + q for a, q in zip(c.all, c.chunk)]
    n, tok, kv, d = old_k.shape
    at = {"heads": 3, "tokens": 2, "sequences": 1}[level]
    both = torch.stack([old_k, old_v], at)
    k, v = both.unbind(at)
    assert not k.is_contiguous() or level == "sequences" and n == 1
    new = torch.zeros(2, n, c.t * c.f, kv, d, device="cuda", dtype=torch.bfloat16)
    for b in range(n):
        a, q = c.all[b] * c.f, c.chunk[b] * c.f
        new[0, b, :q], new[1, b, :q] = c.lk[b, a - q:a], c.lv[b, a - q:a]
    args = c.args()
    args.pop("window")
    cc3d.kv_append(new[0], new[1], k, v, **args)
    cc3d.sync_status()
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    c.check(c.run(k=k, v=v))


# Cases for each of the kernels, with its keys in one CTA and split over a
# cluster: (kernel, CTAs, the case).  tests/test_ops_choice.py checks on the CPU
# that they do take them.
_PADDED = dict(n=2, t=300, heads=32, kv=16, window=500, sinks=4, ring=800, k_frames=[2000, 900],
               q_frames=[300, 250])
_LONG = dict(t=300, total=4300, heads=16, kv=2, window=4000, sinks=1)
_FRAMES = dict(n=2, frame=500, t=5, total=5, heads=2, kv=1, window=3)
_SMALL = dict(frame=50, t=3, total=9, window=4, sinks=3)
_TOKENS = dict(t=1111, total=2500, heads=32, kv=8, window=700, sinks=5)
KERNELS = {
    "two row tiles, 64": (0, 1, dict(_TOKENS, d=64)),
    "two row tiles, 56, split": (0, 6, dict(_LONG, d=56)),
    "two row tiles, 64, frames split": (0, 3, dict(_FRAMES, d=64)),
    "two row tiles, 128": (1, 1, dict(_TOKENS, d=128)),
    "two row tiles, 120, split": (1, 2, dict(n=4, t=40, total=4040, d=120, heads=48, kv=12, sinks=3)),
    "two row tiles, 128, frames split": (1, 3, dict(_FRAMES, d=128)),
    "two CTAs, 64": (2, 1, dict(_PADDED, d=64)),
    "two CTAs, 64, split": (2, 8, dict(_SMALL, d=64)),
    "two CTAs, 128": (3, 1, dict(_PADDED, d=128)),
    "two CTAs, 120, split": (3, 8, dict(_SMALL, d=120)),
    "128 keys, 64": (4, 1, dict(t=130, total=700, d=64, heads=32, kv=32, window=100, sinks=3)),
    "128 keys, 64, split": (4, 4, dict(t=300, total=2300, d=64, heads=8, kv=8, window=300, sinks=2)),
    "128 keys, 128": (5, 1, dict(t=130, total=700, d=128, heads=32, kv=32, window=100, sinks=3)),
    "128 keys, 128, split": (5, 3, dict(_LONG, d=128)),
    "200 channels": (6, 1, dict(t=300, total=700, d=200, heads=24, kv=24, window=100, sinks=2)),
    "136 channels, split": (6, 3, dict(_LONG, d=136)),
    "384 channels": (7, 1, dict(t=300, total=700, d=384, heads=24, kv=24, window=100, sinks=2)),
    "264 channels, split": (7, 2, dict(frame=200, t=2, total=5, d=264, heads=12, kv=12, window=3,
                                       sinks=3)),
}


@pytest.mark.parametrize("name", KERNELS)
def test_every_kernel_and_split(name, monkeypatch):
    kw = KERNELS[name][2]
    c = Case(**kw, seed=len(name))
    first = c.run()
    c.check(first)
    assert torch.equal(c.run(), first)
    for cases in (MASKS, HIDDEN, NAN_SCORES):
        monkeypatch.setitem(cases, name, kw)
    test_values_that_are_not_finite_reach_the_queries_that_see_them_alone(name)
    test_nan_queries_and_runs_of_nan_keys_are_as_in_the_definition(name)
    if "k_frames" not in kw:  # (these two take sequences of one length)
        test_masks_key_by_key(name)
        test_scores_of_minus_infinity(name)
