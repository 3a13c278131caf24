"""Layer norm on the GPU against its 64-bit definition, element by element.

Tolerances.  The kernels compute in fp32.  A row's sums have fewer than 80 roundings on any path (at
most 64 terms in sequence, a tree over the rest), so the mean is within 80 2^-24 < 5e-6 of mean|x|, and the
other row means within 5e-6 of the means of their terms' magnitudes; C = 1e-5 covers those with the few
roundings of the element's own arithmetic.  The mean's error e_m = C mean|x| enters y as rstd |g| e_m
and the variance as e_m^2 (the sum about any centre c is that about the mean plus (c - mean)^2).  The
result is rounded once more: half a step, 2^-8 of the value in bf16 and 2^-24 in fp32.
A column's sums run over T rows in blocks of at most 64, then over the blocks: (64 + T / 64 + 8) 2^-24
of the sum of the magnitudes."""

import numpy as np
import pytest
import torch

import fp8_absmax_reduce_gb300 as fq
from tests import _head_ref as ref
from tests.test_gpu_guard import Guarded

pytestmark = pytest.mark.gpu

C = 1e-5
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SHAPES = [(1, 1), (3, 2), (5, 8), (37, 16), (1, 2048), (2, 5120), (129, 257), (300, 1000), (65, 1409), (77, 4096), (33, 8192),
          (9, 10007), (17, 16384), (5000, 72), (1031, 3584), (401, 4104), (613, 5552),
          (60001, 776), (20000, 520), (80000, 264), (160000, 24), (3000, 1024), (2500, 768), (5, 512), (700, 1408),
          (333, 2560), (333, 2816), (77, 2056), (200, 1280), (200, 1792), (450, 2048), (5000, 4096), (10100, 3584)]


def make(T, d, dtype, seed=0, offset=0.5):
    g = torch.Generator().manual_seed(seed + 1000 * T + d)
    n = lambda *s: torch.randn(*s, generator=g)
    wide = torch.where(torch.rand(d, generator=g) < 0.02, 20.0, 1.0)
    x = (n(T, d) * wide + offset * n(T, 1)).to(dtype).cuda()
    return dict(x=x, g=(1 + 0.1 * n(d)).to(dtype).cuda(), b=(0.1 * n(d)).to(dtype).cuda(),
                dY=(0.01 * n(T, d)).to(dtype).cuda(), dres=(0.01 * n(T, d)).to(dtype).cuda())


def near(got, want, slack, dtype):
    err = (got.double() - want).abs()
    bound = (slack + want.abs() * HALF[dtype]) * (1 + 2.0 ** -7) + 1e-38
    assert bool((err <= bound).all()), float((err / bound).max())


def check_fwd(t, out, eps, bias=True):
    y, mean, rstd = out
    x, g = t["x"].double(), t["g"].double()
    b = t["b"].double() if bias else torch.zeros_like(g)
    wy, wm, wr = ref.layernorm(x, g, b, eps)
    em = C * x.abs().mean(1)
    near(mean, wm, em, torch.float32)
    rel = C + 0.5 * (em * wr) ** 2
    near(rstd, wr, wr * rel, torch.float32)
    xh = ((x - wm[:, None]) * wr[:, None]).abs()
    near(y, wy, g.abs() * (wr * em)[:, None] + (xh * g.abs()) * rel[:, None] + C * b.abs(), y.dtype)


def check_bwd(t, mean, rstd, out, dres):
    dX, dg, db = out
    x, g, dY = t["x"].double(), t["g"].double(), t["dY"].double()
    m, r = mean.double(), rstd.double()
    wX, wg, wb = ref.layernorm_bwd(dY, x, g, m, r, t["dres"].double() if dres else None)
    xh = (x - m[:, None]) * r[:, None]
    u = (dY * g).abs()
    slack = C * r[:, None] * (u + u.mean(1, keepdim=True) + xh.abs() * (u * xh.abs()).mean(1, keepdim=True))
    near(dX, wX, slack + (C * t["dres"].double().abs() if dres else 0.0), dX.dtype)
    c = (72 + x.shape[0] / 64) * 2.0 ** -24
    near(dg, wg, c * (dY * xh).abs().sum(0), torch.float32)
    near(db, wb, c * dY.abs().sum(0), torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_and_backward(T, d, dtype):
    t = make(T, d, dtype)
    out = fq.layernorm_fwd(t["x"], t["g"], t["b"], eps=1e-5)
    check_fwd(t, out, 1e-5)
    for dres in (False, True):
        grads = fq.layernorm_bwd(t["dY"], t["x"], t["g"], out[1], out[2], dres=t["dres"] if dres else None)
        check_bwd(t, out[1], out[2], grads, dres)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_mean_constant_rows_and_no_bias(dtype):
    """A mean 1000 times the deviation; rows of equal values (variance 0); no bias."""
    t = make(64, 1000, dtype, seed=3)
    t["x"] = (t["x"].float() + 1000.0 * torch.randn(64, 1, device="cuda")).to(dtype)
    t["x"][5] = 3.0
    t["x"][6] = 0.0
    out = fq.layernorm_fwd(t["x"], t["g"], eps=1e-5)
    check_fwd(t, out, 1e-5, bias=False)
    assert torch.equal(out[0][6].float(), torch.zeros(1000, device="cuda"))


def test_non_finite_rows_stay_in_their_rows():
    t = make(40, 520, torch.float32)
    t["x"][3, 7], t["x"][9, 0] = float("nan"), float("inf")
    y, mean, rstd = fq.layernorm_fwd(t["x"], t["g"], t["b"])
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[3, 9]] = True
    assert torch.equal(~torch.isfinite(y).all(1), bad) and torch.equal(torch.isnan(y).all(1), bad)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(50, 2048), (31, 1409), (700, 1000), (401, 5120), (600, 3584), (9000, 200), (45, 768), (300, 512)])
def test_in_place_guard_bands_and_repeats(T, d, dtype):
    t = make(T, d, dtype, seed=7)
    y, mean, rstd = fq.layernorm_fwd(t["x"], t["g"], t["b"])
    dX, dg, db = fq.layernorm_bwd(t["dY"], t["x"], t["g"], mean, rstd, dres=t["dres"])
    for name in ("dY", "x", "dres"):
        c = {k: v.clone() for k, v in t.items()}
        a = fq.layernorm_bwd(c["dY"], c["x"], c["g"], mean, rstd, dres=c["dres"], dX=c[name])
        assert torch.equal(a[0], dX) and torch.equal(a[1], dg) and torch.equal(a[2], db)
    x2 = t["x"].clone()
    assert torch.equal(fq.layernorm_fwd(x2, t["g"], t["b"], y=x2)[0], y)
    gy, gx = Guarded((T, d), dtype), Guarded((T, d), dtype)
    gm, gr, gg, gb = (Guarded((n,), torch.float32) for n in (T, T, d, d))
    fq.layernorm_fwd(t["x"], t["g"], t["b"], y=gy.t, mean=gm.t, rstd=gr.t)
    fq.layernorm_bwd(t["dY"], t["x"], t["g"], mean, rstd, dres=t["dres"], dX=gx.t, dg=gg.t, db=gb.t)
    torch.cuda.synchronize()
    assert all(v.intact() for v in (gy, gx, gm, gr, gg, gb))
    assert torch.equal(gy.t, y) and torch.equal(gx.t, dX) and torch.equal(gg.t, dg) and torch.equal(gb.t, db)


@pytest.mark.parametrize("d", [8192, 8191, 1024])
def test_offsets_past_32_bits(d):
    """More than 2^31 elements: the last rows' results are those of the same rows alone."""
    T = 2 ** 31 // d + 600
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    t = make(40, d, torch.bfloat16, seed=4)
    x[-40:] = t["x"]
    y, mean, rstd = fq.layernorm_fwd(x, t["g"], t["b"])
    y2, m2, r2 = fq.layernorm_fwd(t["x"], t["g"], t["b"])
    assert torch.equal(y[-40:], y2) and torch.equal(mean[-40:], m2) and torch.equal(rstd[-40:], r2)
    assert torch.equal(y[5], t["b"])
    y.zero_()
    y[-40:] = t["dY"]
    dX, dg, db = fq.layernorm_bwd(y, x, t["g"], mean, rstd)
    w = fq.layernorm_bwd(t["dY"], t["x"], t["g"], m2, r2)
    assert torch.equal(dX[-40:], w[0]) and bool((dX[:100] == 0).all())
    for got, want in ((dg, w[1]), (db, w[2])):  # other blocks, so another order of the same 40 terms
        assert float((got - want).abs().max()) <= 40 * 2.0 ** -23 * float(want.abs().max()) + 40 * 2.0 ** -23


def test_refusals():
    t = make(8, 64, torch.bfloat16)
    m = torch.zeros(8, device="cuda")
    for call in (lambda: fq.layernorm_fwd(t["x"].t(), t["g"]), lambda: fq.layernorm_fwd(t["x"][:, ::2], t["g"][:32]),
                 lambda: fq.layernorm_fwd(t["x"], t["g"][:32]), lambda: fq.layernorm_bwd(t["dY"][:4], t["x"], t["g"], m, m),
                 lambda: fq.layernorm_bwd(t["dY"], t["x"], t["g"], m[:4], m),
                 lambda: fq.layernorm_bwd(t["dY"], t["x"], t["g"], m, m, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fq.layernorm_fwd(t["x"].half(), t["g"].half()), lambda: fq.layernorm_fwd(t["x"], t["g"].float()),
                 lambda: fq.layernorm_bwd(t["dY"].float(), t["x"], t["g"], m, m)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(fq.Fp8qError):
        fq.layernorm_fwd(t["x"][:0], t["g"])
    with pytest.raises(fq.Fp8qError):
        fq.layernorm_fwd(t["x"].view(-1)[1:65].view(1, 64), t["g"])  # two bytes off a 16-byte boundary


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [1, 7, 72, 257, 768, 1000, 1409, 2048, 2056, 2560, 3584, 4104, 5120, 5552, 8192, 10007, 16384])
def test_rows_of_equal_values_have_variance_zero(d, dtype):
    """Whatever the value (sums within fp32's range) and the width: mean is the value, y is the bias, and rstd is eps^-1/2 to
    the reciprocal square root's 2 steps and the rounding of eps."""
    values = torch.tensor([0.0, 3.0, 0.1, -1000.3, 1e4 / 3, 123456.7, 1e20, -1.37e20, 3e33, -1e-30, 2e-38]).to(dtype).cuda()
    x = values[:, None].expand(-1, d).contiguous()
    t = make(len(values), d, dtype)
    for eps in (1e-5, 1e-12):
        y, mean, rstd = fq.layernorm_fwd(x, t["g"], t["b"], eps=eps)
        assert torch.equal(mean, values.float())
        assert torch.equal(y, t["b"].expand(len(values), d))
        assert float((rstd.double() * eps ** 0.5 - 1).abs().max()) <= 5 * 2.0 ** -24


@pytest.mark.parametrize("d", [72, 257, 1000, 2056, 5120, 10007])
def test_fp32_rows_far_from_zero(d):
    """Deviations of a hundred of the values' steps.  A warp's mean is rounded once, and so is the row's, so the mean is within
    two roundings (and 1e-5 of that for its correction).  The row's variance takes the warps' means with an error of e_m at
    most: 2 e_m sigma + e_m^2, so rstd is within e_m / sigma (1 + e_m / 2 sigma) beside the sums' own 1e-5.  y is off by the
    mean's error and four roundings of its own."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x = (torch.randn(64, 1, generator=g, device="cuda") * 1e4 + 3e4) * (1 + 1e-5 * torch.randn(64, d, generator=g, device="cuda"))
    one = torch.ones(d, device="cuda")
    y, mean, rstd = fq.layernorm_fwd(x, one, eps=1e-12)
    wy, wm, wr = ref.layernorm(x.double(), one.double(), None, 1e-12)
    em = 2.001 * 2.0 ** -24 * wm.abs()
    assert bool(((mean.double() - wm).abs() <= em).all())
    rel = 1e-5 + em * wr * (1 + em * wr)
    assert bool(((rstd.double() - wr).abs() <= wr * rel).all())
    assert bool(((y.double() - wy).abs() <= (em * wr)[:, None] + wy.abs() * (rel[:, None] + 2.0 ** -22)).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(3, 8), (700, 8), (30000, 128), (30000, 136), (30000, 256), (30000, 264), (3000, 512), (3000, 520), (2000, 1024), (1000, 4096),
                                 (1000, 4104), (500, 8192), (500, 8200), (400, 16384), (3000, 1000), (30000, 7), (5000, 1025), (1000, 4099)])
def test_backward_stays_inside_its_workspace(T, d, dtype):
    t = make(T, d, dtype)
    _, mean, rstd = fq.layernorm_fwd(t["x"], t["g"], t["b"])
    n = fq.layernorm_bwd_workspace_size(T, d)
    ws = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    out = fq.layernorm_bwd(t["dY"], t["x"], t["g"], mean, rstd, dres=t["dres"], ws=ws)
    torch.cuda.synchronize()
    assert bool((ws[n:] == 0xFF).all())
    check_bwd(t, mean, rstd, out, True)
