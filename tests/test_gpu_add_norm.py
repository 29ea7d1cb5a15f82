"""cc3d_add_rms_norm on the GPU against the norm in 64 bits.

Tolerance, from the arithmetic: h is one fp32 addition rounded to bf16 (equal
bits).  The sum of c squares is off by at most c fp32 half steps (2^-24), its
root by half of that, and a few more roundings follow: |a| is off by at most
e = (c / 2 + 16) 2^-24 of its terms' magnitude (and 2^-20 |a| with SiLU's
hardware exponential and reciprocal).  y adds bf16's 2^-8 |a|; a code's value
q s is off by E4M3's half step, 2^-4 |a| (or 2^-10 s among its subnormals)."""
import pytest
import torch

from video_vae_causal_implicit_b200 import cc3d

pytestmark = pytest.mark.gpu


def make(rows, c, seed, beta=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, c, device="cuda", generator=g).to(torch.bfloat16)
    r = (3 * torch.randn(rows, c, device="cuda", generator=g)).to(torch.bfloat16)
    gamma = torch.rand(c, device="cuda", generator=g) + 0.5
    return x, r, gamma, torch.randn(c, device="cuda", generator=g) if beta else None


def reference(h, gamma, beta, eps, silu):
    """(a, tolerance) in 64 bits."""
    c = h.shape[-1]
    hd = h.double()
    root = (hd.square().sum(-1, keepdim=True) + c * eps).sqrt().clamp_min(1e-12)
    a = hd * c ** 0.5 / root * gamma.double()
    mag = a.abs()
    if beta is not None:
        a, mag = a + beta.double(), mag + beta.double().abs()
    tol = (c / 2 + 16) * 2.0 ** -24 * mag
    if silu:
        tol = 1.1 * tol + 2.0 ** -20 * a.abs()
        a = a * torch.sigmoid(a)
    return a, tol


def check_outputs(x, residual, gamma, beta, eps, silu, kind, what):
    out = {"h": torch.empty_like(x)}
    if kind != "q":
        out["y"] = torch.empty_like(x)
    if kind != "y":
        out["q"] = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        if kind != "one":
            out["scales"] = torch.empty(x.shape[:-1], device="cuda")
    scale = 0.02 if kind == "one" else 0.0
    cc3d.add_rms_norm(x, gamma, residual=residual, beta=beta, eps=eps, silu=silu, scale=scale,
                      **out)
    cc3d.sync_status()
    h = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    assert torch.equal(out["h"], h), what
    a, tol = reference(h, gamma, beta, eps, silu)
    if "y" in out:
        assert ((out["y"].double() - a).abs() <= tol * 1.01 + 2.0 ** -8 * a.abs()).all(), what
    if "q" in out:
        if kind == "one":
            s = torch.full(x.shape[:-1], scale, device="cuda", dtype=torch.float64)
        else:
            top = a.abs().amax(-1)
            s = out["scales"].double()
            want = torch.where(top > 0, (top / 448).clamp_min(1e-36), torch.ones_like(top))
            assert ((s - want).abs() <= (tol.amax(-1) / 448) + 2.0 ** -22 * want).all(), what
        v = out["q"].double() * s[..., None]
        a = torch.maximum(torch.minimum(a, 448 * s[..., None]), -448 * s[..., None])
        lim = tol + 2.0 ** -4 * a.abs() * (1 + 2.0 ** -20) + 2.0 ** -10 * s[..., None]
        assert ((v - a).abs() <= lim).all(), (what, float(((v - a).abs() - lim).max()))


@pytest.mark.parametrize("c", [8, 40, 96, 384, 512, 520, 1024, 1032, 2048, 4096, 4104, 8192, 8200,
                               16384])
@pytest.mark.parametrize("rows", [1, 3, 37])
def test_sizes(rows, c):
    x, r, gamma, beta = make(rows, c, rows + c, beta=c % 16 == 8)
    check_outputs(x, r, gamma, beta, 1e-6, False, "both", (rows, c))
    check_outputs(x, None, gamma, beta, 0.0, True, "q", (rows, c))


@pytest.mark.parametrize("rows,c", [(7800, 384), (5000, 192), (2500, 4096), (70000, 64)])
@pytest.mark.parametrize("kind", ["y", "q", "one", "both"])
def test_many_rows(rows, c, kind):
    x, r, gamma, _ = make(rows, c, 4)
    check_outputs(x, r, gamma, None, 1e-5, False, kind, (rows, c, kind))


def test_rows_of_zeros_tiny_and_huge_values():
    x, _, gamma, _ = make(6, 64, 1)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4] = 0
    x[4, 3] = 1
    for eps in (0.0, 1e-6):
        check_outputs(x, None, gamma, None, eps, False, "both", eps)


def test_tiny_gamma_keeps_codes_finite():
    x, _, _, _ = make(3, 64, 1)
    gamma = torch.full((64,), 1e-38, device="cuda")
    q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    s = torch.empty(3, device="cuda")
    cc3d.add_rms_norm(x, gamma, q=q, scales=s)
    cc3d.sync_status()
    assert (s == torch.tensor(1e-36, device="cuda")).all()
    assert torch.isfinite(q.float()).all() and (q.float().abs() < 448).all()


def test_in_place_and_leading_dimensions():
    x, r, gamma, _ = make(30, 192, 8)
    want = (x.float() + r.float()).to(torch.bfloat16)
    x4, r4 = x.view(2, 3, 5, 192), r.view(2, 3, 5, 192)
    y = torch.empty_like(x4)
    stream = r4.clone()
    cc3d.add_rms_norm(x4, gamma, residual=stream, h=stream, y=y)
    ref = torch.empty_like(x4)
    cc3d.add_rms_norm(want.view(2, 3, 5, 192), gamma, y=ref)
    cc3d.sync_status()
    assert torch.equal(stream.view(30, 192), want) and torch.equal(y, ref)
    cc3d.add_rms_norm(x4, gamma, y=x4)  # y over x
    plain = torch.empty_like(x)
    cc3d.add_rms_norm(make(30, 192, 8)[0], gamma, y=plain)
    cc3d.sync_status()
    assert torch.equal(x4.view(30, 192), plain)


def test_agrees_with_rms_norm():
    """eps = 0 without a residual is the library's RMS_norm."""
    x, _, gamma, _ = make(300, 192, 3)
    y, z = torch.empty_like(x), torch.empty_like(x)
    cc3d.add_rms_norm(x, gamma, y=y)
    cc3d.rms(x.view(1, 1, 15, 20, 192), gamma, z.view(1, 1, 15, 20, 192))
    cc3d.sync_status()
    a, tol = reference(x, gamma, None, 0.0, False)
    for o in (y, z):
        assert ((o.double() - a).abs() <= tol * 1.01 + 2.0 ** -8 * a.abs()).all()


def test_nan_stays_in_its_row():
    x, r, gamma, _ = make(9, 384, 5)
    q, q2 = (torch.empty_like(x, dtype=torch.float8_e4m3fn) for _ in range(2))
    s, s2 = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    cc3d.add_rms_norm(x, gamma, residual=r, q=q, scales=s)
    r[4, 10] = float("nan")
    cc3d.add_rms_norm(x, gamma, residual=r, q=q2, scales=s2)
    cc3d.sync_status()
    keep = torch.arange(9, device="cuda") != 4
    assert torch.equal(q.view(torch.uint8)[keep], q2.view(torch.uint8)[keep])
    assert torch.equal(s[keep], s2[keep]) and torch.isnan(q2[4].float()).any()


@pytest.mark.parametrize("c", [64, 384, 1024, 2048, 8192])
def test_nan_and_infinities_are_as_in_the_definition(c):
    """A NaN makes its whole row NaN (its sum of squares is); an infinity makes
    itself NaN and the rest of its row 0.  Codes of such rows: scale 1."""
    x, _, gamma, _ = make(6, c, 9)
    x[1, c // 2], x[3, 5], x[4, 0] = float("nan"), float("inf"), -float("inf")
    y, q = torch.empty_like(x), torch.empty_like(x, dtype=torch.float8_e4m3fn)
    s = torch.empty(6, device="cuda")
    cc3d.add_rms_norm(x, gamma, y=y, q=q, scales=s)
    cc3d.sync_status()
    a, _ = reference(x, gamma, None, 0.0, False)
    assert torch.equal(torch.isnan(y), torch.isnan(a)) and torch.isnan(y[1]).all()
    assert torch.equal(torch.isnan(q.float()), torch.isnan(a))
    rest = ~torch.isnan(a[[3, 4]])
    assert (y[[3, 4]][rest] == 0).all() and (q.float()[[3, 4]][rest] == 0).all()
    assert (s[[1, 3, 4]] == 1).all() and (s[[0, 2, 5]] < 1).all()
