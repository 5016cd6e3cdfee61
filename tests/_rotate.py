"""Norm and rotation of heads in 64 bits, with bounds of what FP32 arithmetic and one rounding may be off."""
from __future__ import annotations

from types import SimpleNamespace

import torch

BF16 = 2.0 ** -8       # half a step of BF16 relative to the value
F32 = 2.0 ** -24


def turn(y, pos, inv_freq, interleaved, back=False):
    """Vectors y [..., d] with their pairs turned by pos [...] * inv_freq (back: the other way)."""
    half = inv_freq.numel()
    t = pos.double()[..., None] * inv_freq
    c, s = torch.cos(t), torch.sin(t) * (-1 if back else 1)
    ia, ib = pairs(half, interleaved)
    z = y.clone()
    z[..., ia] = y[..., ia] * c - y[..., ib] * s
    z[..., ib] = y[..., ib] * c + y[..., ia] * s
    return z


def pairs(half, interleaved):
    i = torch.arange(half)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + half)


def spread(y, half, interleaved):
    """|y| of both entries of each pair, at both: what an error of a turn is relative to."""
    ia, ib = pairs(half, interleaved)
    m = y.abs().clone()
    m[..., ia] = y[..., ia].abs() + y[..., ib].abs()
    m[..., ib] = m[..., ia]
    return m


def forward(x, pos, inv_freq, weight=None, eps=1e-6, interleaved=False, norm=True):
    """z and its bound for x [..., d] (any type) at the positions pos [...].

    FP32: the sum of squares is off by at most (16 + 5) roundings relative to itself, its root by half of that,
    the products by 3 roundings and a turn by 2 and the angle's error (pi roundings for the angle, 2 for sin and cos):
    under 32 roundings of what the pair holds; the frequency comes from a double, off by 2^-52 of a turn for each
    position at most.
    """
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if weight is None else weight.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) if norm else torch.ones_like(x[..., :1])
    y = x * r * w
    half = inv_freq.numel()
    z = turn(y, pos, inv_freq, interleaved)
    far = pos.double().abs()[..., None] * 2.0 ** -52 * 6.3
    return SimpleNamespace(z=z, y=y, r=r, w=w, tol=BF16 * z.abs() + (32 * F32 + far) * spread(y, half, interleaved) + 1e-38)


def backward(x, dz, pos, inv_freq, weight=None, eps=1e-6, interleaved=False, norm=True):
    """dx, dw (summed over all vectors) and their bounds; the products and sums of dx as in forward(), twice over;
    dw is a sum whose longest chain of additions, for the tests' sizes, is under 200."""
    f = forward(x, pos, inv_freq, weight, eps, interleaved, norm)
    x, dz, d = x.double(), dz.double(), x.shape[-1]
    dy = turn(dz, pos, inv_freq, interleaved, back=True)
    g = f.w * dy
    unit = x * f.r
    mean = (unit * g).mean(-1, keepdim=True) if norm else torch.zeros_like(f.r)
    dx = f.r * (g - unit * mean)
    far = pos.double().abs()[..., None] * 2.0 ** -52 * 6.3
    sdy = spread(dz, inv_freq.numel(), interleaved)
    size = f.r * (f.w.abs() * sdy + (unit.abs() * (unit.abs() * f.w.abs() * sdy).mean(-1, keepdim=True) if norm else 0))
    dims = tuple(range(x.dim() - 1))
    dw = (dy * unit).sum(dims)
    return SimpleNamespace(dx=dx, dw=dw, dx_tol=BF16 * dx.abs() + (64 * F32 + far) * size + 1e-38,
                           dw_tol=((256 * F32 + far) * sdy * unit.abs()).sum(dims) + 1e-38)


def frequencies(rot, base=10000.0):
    return base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))


def heads(B, N, hq, hkv, d, g, std=1.7):
    """q [B, hq, N, d] and k [B, hkv, N, d] as slices of a projection, on the CPU, rows of unlike size."""
    rows = torch.randn((B, N, hq + 2 * hkv, d), generator=g) * std
    rows *= torch.exp2(torch.randint(-6, 7, (B, N, hq + 2 * hkv, 1), generator=g).float())
    rows = rows.to(torch.bfloat16)
    return rows, rows[:, :, :hq].transpose(1, 2), rows[:, :, hq:hq + hkv].transpose(1, 2)
