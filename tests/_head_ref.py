"""Plain 64-bit definitions of layer norm, rotary positions and the head's cross entropy, in torch
on whatever device the inputs are on.  They share nothing with the library; tests/test_head_ref.py
holds them against central differences."""

import torch


def layernorm(x, g, b, eps):
    """y, mean, rstd of float64 x [T, d]."""
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = (var + eps) ** -0.5
    return (x - mean[:, None]) * rstd[:, None] * g + (0.0 if b is None else b), mean, rstd


def layernorm_bwd(dY, x, g, mean, rstd, dres=None):
    xh = (x - mean[:, None]) * rstd[:, None]
    u = dY * g
    dX = rstd[:, None] * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True))
    return (dX if dres is None else dX + dres), (dY * xh).sum(0), dY.sum(0)


def rope(qkv, pos, inv_freq, axis, head_dim, rot_heads, interleaved, sign=1.0):
    """qkv [T, heads * head_dim] float64, pos [axes, T]; pair i turns by sign * pos[axis[i]] * inv_freq[i]."""
    T = qkv.shape[0]
    out = qkv.clone().view(T, -1, head_dim)
    src = qkv.view(T, -1, head_dim)
    half = len(inv_freq)
    for i, (f, a) in enumerate(zip(inv_freq, axis)):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = pos[a].double() * f * sign
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        p, q = src[:, :rot_heads, lo], src[:, :rot_heads, hi]
        out[:, :rot_heads, lo] = p * c - q * s
        out[:, :rot_heads, hi] = q * c + p * s
    return out.view(T, -1)


def cross_entropy(x, W, targets, ignore):
    """loss, lse of float64 x [T, d], W [V, d]; loss 0 where the target is ignore."""
    z = x @ W.t()
    m = z.max(1, keepdim=True).values
    lse = (m + torch.log(torch.exp(z - m).sum(1, keepdim=True)))[:, 0]
    keep = targets != ignore
    zy = z.gather(1, targets.clamp(min=0, max=W.shape[0] - 1)[:, None])[:, 0]
    return torch.where(keep, lse - zy, torch.zeros_like(lse)), lse


def cross_entropy_grad(x, W, targets, dloss, ignore):
    """The gradient at the logits, G [T, V]; dX = G W, dW = G^T x."""
    z = x @ W.t()
    p = torch.softmax(z, 1)
    keep = targets != ignore
    rows = torch.arange(x.shape[0], device=x.device)[keep]
    p[rows, targets[keep]] -= 1.0
    return p * torch.where(keep, dloss, torch.zeros_like(dloss))[:, None]
