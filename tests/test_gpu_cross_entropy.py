"""The head's cross entropy on the GPU against its 64-bit definition, element by element.

Tolerances.  A logit is an fp32 tensor-core sum of d exact products in steps of at least 16 terms, each step within
2^-23 of the partial sums, which are at most S = sum |x w|: e_z = (d / 16 + 32) 2^-23 S, with S the row's largest.
The row's sum of exponentials has fewer than 100 roundings on any path and exponentials within 2^-21:
lse is within e_z + 1e-5 + 2^-24 |lse|, and a target's loss within twice e_z + the same.
Backward: p = e^(z - lse) is within e_z + 2^-21 (|z - lse| + 4) of itself; G is rounded to bf16, half a step 2^-8; the products
are fp32 sums in steps of 16 terms of |G W| (vocabulary) or |G x| (tokens); the result is rounded to its type.  So
an element is within 2^-8 sum|G w| + (n / 16 + 32) 2^-23 sum|G w| + e_p sum p|dloss w| + half a step.  The bound is
a worst case.  A rounding's RMS is 0.41 of the largest (uniform in the step, the step against the value averaged over
an octave), so with one dominant term the two roundings of 2^-8 give an RMS of sqrt(2) 0.41 / 2 = 0.29 of the bound,
and less with many terms: below 0.35 where the sums have 16 terms or more."""

import pytest
import torch

import fp8_absmax_reduce_gb300 as fq
from tests import _head_ref as ref
from tests.test_gpu_guard import Guarded

pytestmark = pytest.mark.gpu

IGN = -100
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SHAPES = [(1, 8, 1), (1, 16, 2), (2, 8, 300), (3, 64, 7), (127, 72, 129), (128, 128, 256), (129, 136, 257), (300, 512, 1000), (64, 256, 20001), (65, 128, 900), (33, 72, 5000), (24, 64, 25000), (127, 64, 39001), (300, 64, 9000), (257, 72, 21013), (512, 64, 32000),
          (257, 2048, 8200), (1000, 264, 5003), (513, 128, 16385), (2, 4096, 1001)]


def make(T, d, V, seed=0, lean=8.0, ignored=0.2, scale=0.05):
    g = torch.Generator(device="cuda").manual_seed(seed + T + 7 * d + 13 * V)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    W = (n(V, d) * scale).bfloat16()
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = n(T, d)
    x = (x + lean * torch.rand(T, 1, generator=g, device="cuda") * W[t].float() / (scale * d ** 0.5)).bfloat16()
    t[torch.rand(T, generator=g, device="cuda") < ignored] = IGN
    dl = torch.randn(T, generator=g, device="cuda") / T
    return x, W, t, dl


def e_z(x, W):
    S = (x.double().abs() @ W.double().abs().t()).max(1).values
    return (x.shape[1] / 16 + 32) * 2.0 ** -23 * S


def check_fwd(x, W, t, loss, lse):
    wl, we = ref.cross_entropy(x.double(), W.double(), t, IGN)
    tol = e_z(x, W) + 1e-5 + 2.0 ** -24 * we.abs()
    err = (lse.double() - we).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    err = (loss.double() - wl).abs()
    assert bool((err <= 2 * tol + 2.0 ** -24 * wl.abs()).all()), float((err / tol).max())
    assert bool((loss[t == IGN] == 0).all())


def check_bwd(x, W, t, dl, dX, dW):
    xd, Wd = x.double(), W.double()
    G = ref.cross_entropy_grad(xd, Wd, t, dl.double(), IGN)
    z = xd @ Wd.t()
    lse = torch.logsumexp(z, 1, keepdim=True)
    p = torch.exp(z - lse) * torch.where(t == IGN, 0.0, dl.double().abs())[:, None]
    ep = p * (2 * e_z(x, W)[:, None] + 2.0 ** -21 * ((z - lse).abs() + 4))
    for got, want, a, other, n in ((dX, G @ Wd, G.abs(), Wd.abs(), W.shape[0]), (dW, G.t() @ xd, G.abs().t(), xd.abs(), x.shape[0])):
        e = ep if got is dX else ep.t()
        bound = ((2.0 ** -8 + (n / 16 + 32) * 2.0 ** -23) * (a @ other) + e @ other + HALF[got.dtype] * want.abs()) * (1 + 2.0 ** -7) + 1e-30
        err = (got.double() - want).abs()
        assert bool((err <= bound).all()), float((err / bound).max())
        if n >= 16:
            assert float((err / bound).square().mean().sqrt()) < 0.35
    assert bool((dX[t == IGN] == 0).all())


@pytest.mark.parametrize("T", [30, 60, 128])
@pytest.mark.parametrize("V", [20001, 25000, 39001, 19456])
def test_few_tokens_find_their_targets_at_every_tile_edge(T, V):
    x, W, _, _ = make(T, 16, V)
    edges = torch.cat([torch.arange(e, V, 8) for e in (0, 7)])
    for i in range(0, edges.numel(), 16 * T):  # every 16th run of T edges
        t = edges[i:i + T].cuda()
        t = torch.cat([t, t.new_full((T - t.numel(),), V - 1)])
        loss, lse = fq.linear_cross_entropy_fwd(x, W, t, IGN)
        check_fwd(x, W, t, loss, lse)


@pytest.mark.parametrize("T,d,V", SHAPES)
def test_forward_and_backward(T, d, V):
    x, W, t, dl = make(T, d, V)
    fq.get_status(clear=True)
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    check_fwd(x, W, t, loss, lse)
    for dt in (torch.float32, torch.bfloat16):
        dX, dW = fq.linear_cross_entropy_bwd(x, W, t, lse, dl, dw_dtype=dt)
        assert dW.dtype == dt
        check_bwd(x, W, t, dl, dX, dW)
    torch.cuda.synchronize()
    assert fq.get_status() == 0


def test_mean_of_one_weight():
    x, W, t, _ = make(700, 256, 3000, lean=20.0)
    dl = torch.full((700,), 1.0 / float((t != IGN).sum()), device="cuda")
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    check_bwd(x, W, t, dl, *fq.linear_cross_entropy_bwd(x, W, t, lse, dl))


@pytest.mark.parametrize("T", [1, 2, 33, 64])
def test_few_tokens_lose_nothing_to_the_gradient_at_the_logits(T):
    """Up to 64 tokens G is kept in two bf16 parts: 2^-16 of the terms, so fp32 gradients show fp32-like errors."""
    x, W, t, dl = make(T, 512, 3001, lean=20.0, ignored=0.0)
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    dX, dW = fq.linear_cross_entropy_bwd(x, W, t, lse, dl)
    xd, Wd = x.double(), W.double()
    G = ref.cross_entropy_grad(xd, Wd, t, dl.double(), IGN)
    z = xd @ Wd.t()
    gap = (z - torch.logsumexp(z, 1, keepdim=True)).abs()
    ep = (G.abs() + (t[:, None] == torch.arange(3001, device="cuda")) * dl.double().abs()[:, None]) * (2 * e_z(x, W)[:, None] + 2.0 ** -21 * (gap + 4))
    terms = G.abs() * (2.0 ** -16 + (3001 / 16 + 64) * 2.0 ** -23) + ep
    assert bool(((dW.double() - G.t() @ xd).abs() <= terms.t() @ xd.abs() + 1e-30).all())
    assert bool(((dX.double() - G @ Wd).abs() <= (terms @ Wd.abs() + 2.0 ** -8 * (G @ Wd).abs()) * (1 + 2.0 ** -7)).all())


def test_sharp_rows_and_wide_logits():
    """Logits of hundreds: rows whose probabilities are 0 and 1, far from the largest logit on both sides."""
    x, W, t, dl = make(200, 128, 1500, lean=0.0, scale=4.0)
    x[50:] *= 8
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    check_fwd(x, W, t, loss, lse)
    assert bool(torch.isfinite(lse).all())
    # the gradient bound holds where the logits' own error stays small: the rows of moderate logits
    check_bwd(x[:50], W, t[:50], dl[:50], *fq.linear_cross_entropy_bwd(x[:50], W, t[:50], lse[:50], dl[:50]))


def test_every_token_ignored():
    x, W, t, dl = make(130, 64, 500, ignored=2.0)
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    check_fwd(x, W, t, loss, lse)
    dX, dW = fq.linear_cross_entropy_bwd(x, W, t, lse, dl)
    assert bool((loss == 0).all()) and bool((dX == 0).all()) and bool((dW == 0).all())


def test_zero_weights():
    x, W, t, dl = make(64, 64, 300)
    _, lse = fq.linear_cross_entropy_fwd(x, W, t)
    dX, dW = fq.linear_cross_entropy_bwd(x, W, t, lse, torch.zeros_like(dl))
    assert bool((dX == 0).all()) and bool((dW == 0).all())


def test_padded_rows_may_hold_anything():
    """Ignored tokens with NaN and Inf in x and in dloss: nothing of it leaves their rows."""
    x, W, t, dl = make(300, 128, 2000)
    t[7:40] = IGN
    xb, dlb = x.clone(), dl.clone()
    xb[7:40:2], xb[8:40:2] = float("nan"), float("inf")
    dlb[7:40] = float("nan")
    loss, lse = fq.linear_cross_entropy_fwd(xb, W, t)
    assert bool((loss[7:40] == 0).all())
    l0, e0 = fq.linear_cross_entropy_fwd(x, W, t)
    assert torch.equal(loss, l0) and torch.equal(lse[:7], e0[:7]) and torch.equal(lse[40:], e0[40:])
    a = fq.linear_cross_entropy_bwd(xb, W, t, lse, dlb)
    b = fq.linear_cross_entropy_bwd(x, W, t, e0, dl)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_non_finite_token_reaches_its_own_loss_only():
    x, W, t, dl = make(300, 128, 2000, ignored=0.0)
    l0, _ = fq.linear_cross_entropy_fwd(x, W, t)
    x[9, 3] = float("nan")
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    assert bool(torch.isnan(loss[9])) and bool(torch.isnan(lse[9]))
    loss[9] = l0[9]
    assert torch.equal(loss, l0)


def test_bad_targets_are_recorded_and_ignored():
    x, W, t, dl = make(100, 64, 500, ignored=0.0)
    good = t.clone()
    good[[3, 4, 5]] = IGN
    bad = t.clone()
    bad[3], bad[4], bad[5] = 500, -1, 2 ** 40
    fq.get_status(clear=True)
    a = fq.linear_cross_entropy_fwd(x, W, bad)
    torch.cuda.synchronize()
    assert fq.get_status(clear=True) == fq.STATUS_BAD_TARGET
    b = fq.linear_cross_entropy_fwd(x, W, good)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = fq.linear_cross_entropy_bwd(x, W, bad, a[1], dl)
    torch.cuda.synchronize()
    assert fq.get_status(clear=True) == fq.STATUS_BAD_TARGET
    gb = fq.linear_cross_entropy_bwd(x, W, good, a[1], dl)
    assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1])
    # another ignore_index, inside the vocabulary: class 7 does not count
    t[10] = 7
    torch.cuda.synchronize()
    assert fq.get_status(clear=True) == 0
    assert float(fq.linear_cross_entropy_fwd(x, W, t, ignore_index=7)[0][10]) == 0.0


def test_guard_bands_repeats_and_second_stream():
    T, d, V = 259, 136, 8321
    x, W, t, dl = make(T, d, V)
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    for dt in (torch.float32, torch.bfloat16):
        gl, ge, gx, gw = Guarded((T,), torch.float32), Guarded((T,), torch.float32), Guarded((T, d), torch.bfloat16), Guarded((V, d), dt)
        fq.linear_cross_entropy_fwd(x, W, t, loss=gl.t, lse=ge.t)
        fq.linear_cross_entropy_bwd(x, W, t, ge.t, dl, dX=gx.t, dW=gw.t)
        torch.cuda.synchronize()
        assert all(v.intact() for v in (gl, ge, gx, gw))
        assert torch.equal(gl.t, loss) and torch.equal(ge.t, lse)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = fq.linear_cross_entropy_bwd(x, W, t, lse, dl, dw_dtype=dt)
        s.synchronize()
        assert torch.equal(again[0], gx.t) and torch.equal(again[1], gw.t)


def test_workspace_bytes_past_the_need_are_left_alone():
    T, d, V = 130, 72, 9001
    x, W, t, dl = make(T, d, V)
    for size, run in ((fq.linear_cross_entropy_fwd_workspace_size(T, d, V), lambda w: fq.linear_cross_entropy_fwd(x, W, t, ws=w)),
                      (fq.linear_cross_entropy_bwd_workspace_size(T, d, V),
                       lambda w: fq.linear_cross_entropy_bwd(x, W, t, torch.zeros(T, device="cuda"), dl, ws=w))):
        ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        run(ws)
        torch.cuda.synchronize()
        assert bool((ws[size:] == 0xA5).all())


def test_dw_past_32_bit_offsets():
    """V d above 2^31: the last pieces' rows of dW and the logits against a head of those rows."""
    T, d, V = 3, 16384, 140000
    x, W, t, dl = make(T, d, 8)
    W = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    W[-5:] = (torch.randn(5, d, device="cuda") * 0.02).bfloat16()
    t[:] = torch.tensor([V - 1, V - 3, 0], device="cuda")
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    z = x.double() @ W[-5:].double().t()
    want = torch.logsumexp(torch.cat([z, torch.full((T, 1), float(torch.log(torch.tensor(V - 5.0))), device="cuda").double()], 1), 1)
    assert bool(((lse.double() - want).abs() <= e_z(x, W[-5:]) + 1e-5 + 2.0 ** -24 * want.abs()).all())
    dX, dW = fq.linear_cross_entropy_bwd(x, W, t, lse, dl, dw_dtype=torch.bfloat16)
    p = torch.exp(z - want[:, None])
    p[0, 4] -= 1
    p[1, 2] -= 1
    G = p * dl.double()[:, None]
    err = (dW[-5:].double() - G.t() @ x.double()).abs()
    assert bool((err <= 2.0 ** -7 * (G.abs().t() @ x.double().abs())).all())


@pytest.mark.parametrize("T,d,V", [(16500, 16, 26000), (40000, 8, 4500), (5000, 64, 30500), (1, 64, 100003), (4100, 24, 300)])
def test_many_pieces_and_parts(T, d, V):
    """Several pieces of the vocabulary (the last one short), products of few tiles cut along K (a last piece
    with fewer parts), against the definition on sampled rows of dX and dW."""
    x, W, t, dl = make(T, d, V)
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    dX, dW = fq.linear_cross_entropy_bwd(x, W, t, lse, dl)
    rows = sorted({r for r in (0, 1, T // 2, T - 2, T - 1) if 0 <= r < T})
    check_fwd(x[rows], W, t[rows], loss[rows], lse[rows])
    G = ref.cross_entropy_grad(x[rows].double(), W.double(), t[rows], dl[rows].double(), IGN)
    bound = (2.0 ** -8 * (1 + 2.0 ** -4) + (V / 16 + 32) * 2.0 ** -23) * (G.abs() @ W.double().abs()) + 2.0 ** -8 * (G @ W.double()).abs() + 1e-9
    assert bool(((dX[rows].double() - G @ W.double()).abs() <= bound).all())
    want, mag = torch.zeros(V, d, dtype=torch.float64, device="cuda"), torch.zeros(V, d, dtype=torch.float64, device="cuda")
    for i in range(0, T, 4096):
        s = slice(i, i + 4096)
        G = ref.cross_entropy_grad(x[s].double(), W.double(), t[s], dl[s].double(), IGN)
        want += G.t() @ x[s].double()
        mag += G.abs().t() @ x[s].double().abs()
    assert bool(((dW.double() - want).abs() <= (2.0 ** -8 * (1 + 2.0 ** -4) + (T / 16 + 32) * 2.0 ** -23) * mag + 1e-9).all())


def test_refusals():
    x, W, t, dl = make(16, 64, 100)
    lse = torch.zeros(16, device="cuda")
    for call in (lambda: fq.linear_cross_entropy_fwd(x, W[:, :32], t), lambda: fq.linear_cross_entropy_fwd(x, W.t(), t),
                 lambda: fq.linear_cross_entropy_fwd(x, W, t[:8]), lambda: fq.linear_cross_entropy_bwd(x, W, t, lse[:8], dl),
                 lambda: fq.linear_cross_entropy_bwd(x, W, t, lse, dl, dW=torch.empty(100, 32, device="cuda")),
                 lambda: fq.linear_cross_entropy_fwd(x, W, t.cpu()),
                 lambda: fq.linear_cross_entropy_fwd(x, W, t, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fq.linear_cross_entropy_fwd(x.float(), W, t), lambda: fq.linear_cross_entropy_fwd(x, W, t.int()),
                 lambda: fq.linear_cross_entropy_bwd(x, W, t, lse.double(), dl),
                 lambda: fq.linear_cross_entropy_bwd(x, W, t, lse, dl, dw_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(fq.Fp8qError):
        fq.linear_cross_entropy_fwd(x[:, :60].contiguous(), W[:, :60].contiguous(), t)
    with pytest.raises(fq.Fp8qError):
        fq.linear_cross_entropy_fwd(x[:0], W, t[:0])


@pytest.mark.parametrize("T,d,V", [(1, 8192, 3000), (5, 4656, 2476), (33, 2048, 1000), (64, 1600, 301), (100, 2048, 257), (128, 4096, 700),
                                   (3, 65536, 9)])
def test_small_heads_of_few_tokens_whose_logits_come_in_parts(T, d, V):
    x, W, t, dl = make(T, d, V, scale=0.02)
    nan = t == IGN
    xb, dlb = x.clone(), dl.clone()
    xb[nan], dlb[nan] = float("nan"), float("nan")
    nf, nb = fq.linear_cross_entropy_fwd_workspace_size(T, d, V), fq.linear_cross_entropy_bwd_workspace_size(T, d, V)
    wf, wb = (torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda") for n in (nf, nb))
    gl, ge, gx = Guarded((T,), torch.float32), Guarded((T,), torch.float32), Guarded((T, d), torch.bfloat16)
    fq.linear_cross_entropy_fwd(x, W, t, loss=gl.t, lse=ge.t, ws=wf)
    check_fwd(x, W, t, gl.t, ge.t)
    keep = ge.t.clone()
    for dt in (torch.float32, torch.bfloat16):
        gw = Guarded((V, d), dt)
        fq.linear_cross_entropy_bwd(xb, W, t, keep, dlb, dX=gx.t, dW=gw.t, ws=wb)
        torch.cuda.synchronize()
        check_bwd(x, W, t, dl, gx.t, gw.t)
        assert gw.intact()
    assert all(v.intact() for v in (gl, ge, gx))
    assert bool((wf[nf:] == 0xFF).all()) and bool((wb[nb:] == 0xFF).all())
    bad = t.clone()
    bad[0] = V
    fq.get_status(clear=True)
    again = fq.linear_cross_entropy_fwd(x, W, bad)
    torch.cuda.synchronize()
    assert fq.get_status(clear=True) == fq.STATUS_BAD_TARGET and float(again[0][0]) == 0.0 and torch.equal(again[1], keep)


@pytest.mark.parametrize("mask", [float("-inf"), torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("T,d,V,lo,hi", [(1, 64, 25000, 1, 24999), (3, 4656, 2476, 128, 2400), (24, 64, 25000, 512, 20000),
                                         (60, 64, 25000, 100, 24990), (100, 64, 25000, 512, 20000), (300, 64, 9000, 512, 7000),
                                         (257, 2048, 8200, 1, 8200)])
def test_masked_vocabulary_counts_for_nothing(T, d, V, lo, hi, mask):
    """Columns lo .. hi - 1 masked through a constant feature, by -inf and by the type's lowest value: whole tiles hold nothing
    else, and the loss and the gradients are those of the head without these rows."""
    x, W, t, dl = make(T, d, V, ignored=0.1)
    x[:, 0], W[:, 0] = 1.0, 0.0
    t[t != IGN] %= lo
    W[lo:hi] = 0.0
    W[lo:hi, 0] = mask
    kept = torch.cat([W[:lo], W[hi:]])
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    assert bool(torch.isfinite(lse).all())
    check_fwd(x, kept, t, loss, lse)
    dX, dW = fq.linear_cross_entropy_bwd(x, W, t, lse, dl)
    assert bool((dW[lo:hi] == 0).all())
    if mask == float("-inf"):
        dX[:, 0] = 0.0  # 0 times -inf there, in the definition too
    check_bwd(x, kept, t, dl, dX, torch.cat([dW[:lo], dW[hi:]]))


@pytest.mark.parametrize("T,d,V", [(1, 8, 4_200_003), (24, 16, 2_100_001), (33, 8, 2_100_003), (64, 24, 1_100_003), (65, 8, 2_100_001),
                                   (128, 16, 1_100_003)])
def test_few_tokens_over_several_pieces_of_the_vocabulary(T, d, V):
    """Up to 128 tokens and more than 256 MB of G: the pieces' shares of dX add up, each piece writes its own rows of dW, and
    targets lie in all of them."""
    x, W, t, dl = make(T, d, V)
    t[0] = V - 1
    loss, lse = fq.linear_cross_entropy_fwd(x, W, t)
    check_fwd(x, W, t, loss, lse)
    for dt in (torch.float32, torch.bfloat16):
        gx, gw = Guarded((T, d), torch.bfloat16), Guarded((V, d), dt)
        fq.linear_cross_entropy_bwd(x, W, t, lse, dl, dX=gx.t, dW=gw.t)
        assert fq.last_launch_count() > 6  # one piece: the tokens' rows, G, dX and its join, dW and its join
        torch.cuda.synchronize()
        assert gx.intact() and gw.intact()
        check_bwd(x, W, t, dl, gx.t, gw.t)


@pytest.mark.parametrize("T,d,V", [(1, 1024, 25000), (30, 1024, 25000), (64, 1024, 25000), (128, 1024, 25000), (24, 2048, 32000), (30, 2048, 9000),
                                   (100, 2048, 9000), (1, 4656, 2476)])
def test_few_tokens_keep_the_precision_of_their_logits(T, d, V):
    """One logit of about 70 whose products are all positive, the others 0: lse is that logit.  Sums that are cut at each step
    lose up to 2^-23 of the partial sum a step, in parts of 128 (8 steps) (8 + 1) / 2 2^-23 of the logit; adding up P = d / 128
    parts rounds to (P + 1) / 2 2^-24, and the way to log2 units and back is four roundings and two constants: 2 2^-23."""
    g = torch.Generator(device="cuda").manual_seed(T + d + V)
    u = lambda *s: torch.rand(*s, generator=g, device="cuda") + 0.1
    x, W = u(T, d).bfloat16(), torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    W[V // 2] = (u(d) * (200.0 / d)).bfloat16()
    _, lse = fq.linear_cross_entropy_fwd(x, W, torch.zeros(T, dtype=torch.int64, device="cuda"))
    z = x.double() @ W[V // 2].double()
    want = z + torch.log1p((V - 1) * torch.exp(-z))
    assert float(z.min()) > 30.0
    bound = 4.5 + (d / 128 + 1) / 4 + 2.0
    assert float(((lse.double() - want) / want).abs().max()) <= bound * 2.0 ** -23


@pytest.mark.parametrize("T,V", [(1, 300), (24, 25000), (100, 25000), (300, 9000)])
def test_small_losses_are_not_lost_in_lse(T, V):
    """Logits of two exact values, the target's of 2048 and the others' of 2048 - gap: loss = log1p((V - 1) e^-gap), down to
    2e-5, beside an lse whose step is 2.4e-4.  The target's term of the sum is within 2^-22, and the sum, a little above 1, has
    fewer than 60 roundings on any path: 64 2^-24.  The other terms are within 2^-18 of themselves: an exponent of up to 31 in log2
    units rounded to 2^-20, its constant's 2^-25 of that, the exponential's 2^-22, 60 roundings; log2 and the last product 2^-22."""
    gaps = ((torch.log(torch.tensor(float(V))) + torch.linspace(1.0, 11.0, T)) * 8).round().cuda() / 8
    x, W = torch.zeros(T, 8, device="cuda"), torch.zeros(V, 8, device="cuda")
    x[:, 0], W[:, 0] = 2048.0, 1.0
    x[:, 1], x[:, 2], W[:, 1:3] = -gaps.floor(), gaps.floor() - gaps, 1.0
    W[5, 1:3] = 0.0
    xb, Wb = x.bfloat16(), W.bfloat16()
    assert torch.equal(xb.float(), x) and torch.equal(Wb.float(), W)
    loss, _ = fq.linear_cross_entropy_fwd(xb, Wb, torch.full((T,), 5, dtype=torch.int64, device="cuda"))
    want = torch.log1p((V - 1) * torch.exp(-gaps.double()))
    err = (loss.double() - want).abs()
    assert bool((err <= 64 * 2.0 ** -24 + want * 2.0 ** -18).all()), float((err - want * 2.0 ** -18).max())
