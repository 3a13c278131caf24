"""Rotary positions on the GPU against their 64-bit definition, element by element.

Tolerances.  The phase in turns carries |pos| 2^-65 (the step of the frequency's fixed point) and
2 |angle| 2^-53 / 2 pi (its fp64 division), is cut to 32 bits (2^-32) and rounded to fp32 as a number
of half-turns up to 1 (2^-25); the sine and cosine of that are within 2 steps (2^-23).  In radians
that is below pi 2^-25 + 2^-23 + small < 2.5e-7, and A = 1e-6 of |a| + |b| covers it with the three roundings of
the rotation; |angle| 2^-51 is the reference's own angle and the division.  The result is rounded once: half a step."""

import pytest
import torch

import fp8_absmax_reduce_gb300 as fq
from tests import _head_ref as ref
from tests.test_gpu_guard import Guarded

pytestmark = pytest.mark.gpu

A = 1e-6
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def check(qkv, pos, plan, hq, hkv, out, sign):
    pos2 = pos.view(plan.n_axes, -1)
    want = ref.rope(qkv.double(), pos2, plan.inv_freq, plan.axis, plan.head_dim, hq + hkv, plan.interleaved, sign)
    T, dh, rot = qkv.shape[0], plan.head_dim, plan.rot_dim
    mag = torch.zeros(T, hq + 2 * hkv, dh, dtype=torch.float64, device="cuda")
    v = qkv.double().abs().view(T, -1, dh)
    both = (v[..., 0:rot:2] + v[..., 1:rot:2]) if plan.interleaved else (v[..., :rot // 2] + v[..., rot // 2:rot])
    ang = pos2.double().abs()[list(plan.axis)].t() * torch.tensor(plan.inv_freq, device="cuda").abs()
    both = both * (A + ang * 2.0 ** -51)[:, None]
    if plan.interleaved:
        mag[..., 0:rot:2], mag[..., 1:rot:2] = both, both
    else:
        mag[..., :rot // 2], mag[..., rot // 2:rot] = both, both
    err = (out.double() - want).abs()
    bound = (mag.view(T, -1) + want.abs() * HALF[qkv.dtype]) * (1 + 2.0 ** -8)
    assert bool((err <= bound).all()), float((err - bound).max())
    o = out.view(T, -1, dh)
    assert torch.equal(o[:, hq + hkv:], qkv.view(T, -1, dh)[:, hq + hkv:])
    assert torch.equal(o[..., rot:], qkv.view(T, -1, dh)[..., rot:])


CASES = [  # T, hq, hkv, head_dim, rot_dim, sections, interleaved
    (1, 1, 0, 8, 2, None, False), (1, 1, 0, 8, 8, None, True), (3, 2, 1, 16, 6, [1, 2], True), (17, 40, 8, 128, 128, None, False),
    (130, 5, 1, 128, 128, [16, 24, 24], False), (64, 4, 4, 64, 32, None, True), (33, 3, 1, 96, 48, [5, 19], False),
    (257, 2, 2, 256, 256, [1] * 128, True), (50, 4, 0, 40, 20, None, False), (1000, 8, 2, 72, 72, [10, 11, 12, 3], True),
    (2049, 12, 4, 128, 64, None, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rope(case, dtype):
    T, hq, hkv, dh, rot, sections, inter = case
    plan = fq.Rope.make(head_dim=dh, rot_dim=rot, sections=sections, interleaved=inter)
    g = torch.Generator(device="cuda").manual_seed(T)
    qkv = torch.randn(T, (hq + 2 * hkv) * dh, generator=g, device="cuda").to(dtype)
    for hi in (5000, 2 ** 31 - 1):
        pos = torch.randint(-hi if hi > 5000 else 0, hi, (plan.n_axes, T), generator=g, device="cuda").int()
        keep = qkv.clone()
        fwd = fq.rope_fwd(qkv, pos, plan, hq, hkv)
        check(qkv, pos, plan, hq, hkv, fwd, 1.0)
        bwd = fq.rope_bwd(qkv, pos, plan, hq, hkv)
        check(qkv, pos, plan, hq, hkv, bwd, -1.0)
        assert torch.equal(qkv, keep)
        same = qkv.clone()
        assert fq.rope_fwd(same, pos, plan, hq, hkv, out=same) is same and torch.equal(same, fwd)
        gout = Guarded(tuple(qkv.shape), dtype)
        fq.rope_bwd(qkv, pos, plan, hq, hkv, dqkv=gout.t)
        torch.cuda.synchronize()
        assert gout.intact() and torch.equal(gout.t, bwd)


def test_position_zero_and_extreme_positions():
    plan = fq.Rope.make(head_dim=64, inv_freq=[1.0] * 32, axis=[i % 2 for i in range(32)])
    x = torch.randn(4, 64, device="cuda")
    pos = torch.tensor([[0, -2 ** 31, 2 ** 31 - 1, 0], [0, 0, -1, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    out = fq.rope_fwd(x, pos, plan, 1, 0)
    assert torch.equal(out[0], x[0])
    check(x, pos, plan, 1, 0, out, 1.0)


def test_non_finite_values_stay_in_their_pairs():
    plan = fq.Rope.make(head_dim=128)
    x = torch.randn(6, 3 * 128, device="cuda").bfloat16()
    x[2, 5] = float("nan")
    out = fq.rope_fwd(x, torch.arange(6, device="cuda").int(), plan, 1, 1)
    bad = torch.isnan(out).nonzero().tolist()
    assert bad == [[2, 5], [2, 69]]


def test_long_rows_pass_32_bit_offsets():
    """2^31 elements and more in one tensor: the last rows equal the same rows alone."""
    hq, hkv, dh = 40, 8, 128
    T = 2 ** 31 // (56 * dh) + 100
    plan = fq.Rope.make(head_dim=dh)
    x = torch.empty(T, 56 * dh, dtype=torch.bfloat16, device="cuda")
    x[-50:] = torch.randn(50, 56 * dh, device="cuda").bfloat16()
    pos = torch.arange(T, device="cuda").int()
    tail = x[-50:].clone()
    fq.rope_fwd(x, pos, plan, hq, hkv, out=x)
    assert torch.equal(x[-50:], fq.rope_fwd(tail, pos[-50:].clone(), plan, hq, hkv))


def test_refusals():
    plan = fq.Rope.make(head_dim=64, sections=[16, 16])
    x = torch.zeros(8, 3 * 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    for call in (lambda: fq.rope_fwd(x, pos, plan, 2, 1), lambda: fq.rope_fwd(x, pos[:1], plan, 1, 1),
                 lambda: fq.rope_fwd(x, pos[0], plan, 1, 1), lambda: fq.rope_fwd(x[:, :128], pos, plan, 2, 0),
                 lambda: fq.rope_fwd(x, pos, plan, 1, 1, out=x[:4])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fq.rope_fwd(x, pos.long(), plan, 1, 1)
    with pytest.raises(TypeError):
        fq.rope_fwd(x.half(), pos, plan, 1, 1)
    buf = torch.zeros(8 * 192 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fq.Fp8qError):  # overlapping, but not the same
        fq.rope_fwd(buf[:8 * 192].view(8, 192), pos, plan, 1, 1, out=buf[8:].view(8, 192))


@pytest.mark.parametrize("rot", [16, 12])
def test_small_angles_keep_their_digits(rot):
    """Frequencies of both signs whose angles stay below a quarter turn, at near and far positions: cosine and sine of the angle
    itself (the pair (1, 0) turned).  The angle: |pos| 2^-65 turns for the fixed point, |angle| 2^-51 for the division and the
    reference's product, half a step of fp32; the sine 2 steps."""
    freqs = [-1e-20, 4.7e-13, -4.7e-13, -3.1e-10, 1e-10, -1e-8 / 16, 3.1e-11, -2.3e-13][:rot // 2]
    plan = fq.Rope.make(head_dim=16, rot_dim=rot, inv_freq=freqs)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 1, -1, 12345, -999999, 0], dtype=torch.int32, device="cuda")
    x = torch.zeros(7, 16, device="cuda")
    x[:, :rot // 2] = 1.0
    for sign, fn in ((1.0, fq.rope_fwd), (-1.0, fq.rope_bwd)):
        out = fn(x, pos, plan, 1, 0).double()
        ang = sign * pos.double()[:, None] * torch.tensor(freqs, dtype=torch.float64, device="cuda")
        s, c = torch.sin(ang), torch.cos(ang)
        e = ang.abs() * (2.0 ** -51 + 2.0 ** -24) + pos.double().abs()[:, None] * 2.0 ** -65 * 6.2832
        assert bool(((out[:, rot // 2:rot] - s).abs() <= e + s.abs() * 2.0 ** -22).all())
        assert bool(((out[:, :rot // 2] - c).abs() <= e * s.abs() + e * e + 2.0 ** -22).all())
