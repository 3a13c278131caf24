"""The 64-bit definitions that the GPU tests of layer norm, rotary positions and the head's cross
entropy compare with: their gradients against central differences (step 1e-5: the truncation error is
O(1e-10), the rounding error of a difference 1e-16 / 1e-5), and closed forms."""

import math

import torch

from tests import _head_ref as ref

STEP = 1e-5


def differences(f, a):
    out = torch.zeros_like(a)
    for i in range(a.numel()):
        keep = a.view(-1)[i].item()
        a.view(-1)[i] = keep + STEP
        up = f()
        a.view(-1)[i] = keep - STEP
        down = f()
        a.view(-1)[i] = keep
        out.view(-1)[i] = (up - down) / (2 * STEP)
    return out


def rnd(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_layernorm_gradients_are_differences():
    x, g, b, dY, dres = rnd(3, 7, seed=1), 1 + 0.1 * rnd(7, seed=2), rnd(7, seed=3), rnd(3, 7, seed=4), rnd(3, 7, seed=5)
    f = lambda: float((ref.layernorm(x, g, b, 1e-5)[0] * dY).sum() + (x * dres).sum())
    y, mean, rstd = ref.layernorm(x, g, b, 1e-5)
    dX, dg, db = ref.layernorm_bwd(dY, x, g, mean, rstd, dres)
    for got, a in ((dX, x), (dg, g), (db, b)):
        assert torch.allclose(differences(f, a), got, atol=1e-8)
    assert torch.allclose(((y - b) / g).mean(1), torch.zeros(3, dtype=torch.float64), atol=1e-12)


def test_rope_is_a_rotation_and_its_gradient_the_inverse():
    pos = torch.tensor([[0, 5, -7], [3, 0, 100000]], dtype=torch.int32)
    freq, axis = [1.0, 0.3, 0.01], [0, 1, 0]
    for inter in (False, True):
        x, dy = rnd(3, 4 * 8, seed=1), rnd(3, 4 * 8, seed=2)
        y = ref.rope(x, pos, freq, axis, 8, 3, inter)
        back = ref.rope(y, pos, freq, axis, 8, 3, inter, sign=-1.0)
        assert torch.allclose(back, x, atol=1e-12) and torch.equal(y[:, 24:], x[:, 24:]) and torch.equal(y[0, 6:8], x[0, 6:8])
        f = lambda: float((ref.rope(x, pos, freq, axis, 8, 3, inter) * dy).sum())
        assert torch.allclose(differences(f, x), ref.rope(dy, pos, freq, axis, 8, 3, inter, sign=-1.0), atol=1e-8)


def test_cross_entropy_gradients_are_differences():
    x, W, w = rnd(4, 5, seed=1), rnd(6, 5, seed=2), rnd(4, seed=3)
    t = torch.tensor([2, -100, 0, 5])
    f = lambda: float((ref.cross_entropy(x, W, t, -100)[0] * w).sum())
    G = ref.cross_entropy_grad(x, W, t, w, -100)
    assert torch.allclose(differences(f, x), G @ W, atol=1e-8) and torch.allclose(differences(f, W), G.t() @ x, atol=1e-8)
    loss, lse = ref.cross_entropy(torch.zeros(4, 5, dtype=torch.float64), W, t, -100)
    assert torch.allclose(lse, torch.full((4,), math.log(6), dtype=torch.float64)) and loss[1] == 0
