"""64-bit attention under a mask, with elementwise error bounds, for the windowed and paged operators.

Everything here is plain torch in float64 on the CPU.  Each function returns values and, next to
them, how far a kernel may be off that follows the library's number formats:

  * P~ is rounded to BF16 before the product with V (half a step, 2^-8 of each entry), O to BF16 on
    storing: |dO| <= 2^-8 (sum_j P_j |V_j| + |O|).
  * In the backward P and dS are rounded to BF16 (2^-8 each), and delta = rowsum(dO o O) uses the
    stored O, so |d delta| <= sum_c |dO_c| |dO error_c|; dS = P (dP - delta) is then off by
    2^-8 |dS| + P |d delta|.  The outputs are rounded to BF16 on storing.
  * FP32 sums, ex2.approx (2^-22) and the FP32 scores (|S| <= ~100 here, so scale S is off by less
    than 1e-4) stay under SLACK of these terms.
"""
from __future__ import annotations

import math

import torch

HALF = 2.0 ** -8   # BF16: half a step relative to the value
SLACK = 1.05       # FP32 parts of the arithmetic
LSE_TOL = 1e-4     # FP32 scores and sums, absolute


def window_mask(pos, keys, window=None, sinks=0):
    """[len(pos), len(keys)]: whether the query at position pos sees the key at position keys."""
    gap = pos[:, None] - keys[None, :]
    see = gap >= 0
    if window is not None:
        see &= (gap < window) | (keys[None, :] < sinks)
    return see


def forward(q, k, v, see, scale):
    """o, lse and the bound of o; a row that sees nothing gives 0 and -inf.  [..., N, d] tensors."""
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    s = (q @ k.transpose(-1, -2) * scale).masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    o = p @ v
    return dict(p=p, o=o, lse=lse, o_tol=SLACK * HALF * (p @ v.abs() + o.abs()) + 1e-6)


def backward(q, k, v, do, see, scale, fwd):
    """dq, dk, dv and their bounds."""
    q, k, v, do = (x.detach().cpu().double() for x in (q, k, v, do))
    p = fwd["p"]
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    dp = do @ t(v)
    delta = (do * fwd["o"]).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    d_delta = (do.abs() * fwd["o_tol"]).sum(-1, keepdim=True)
    ds_err = HALF * ds.abs() + p * d_delta
    out = dict(dv=t(p) @ do, dk=scale * t(ds) @ q, dq=scale * ds @ k)
    err = dict(dv=HALF * t(p) @ do.abs(), dk=scale * t(ds_err) @ q.abs(), dq=scale * ds_err @ k.abs())
    return out, {n: SLACK * (err[n] + HALF * out[n].abs()) + 1e-6 for n in out}


def assert_within(name, got, want, tol):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got - want).abs()
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bound (largest error {off.max().item():.3e})"


def assert_lse(got, want):
    got = got.detach().cpu().double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isneginf(got), torch.isneginf(want))
    assert torch.isfinite(got[fin]).all()
    if fin.any():
        assert (got[fin] - want[fin]).abs().max().item() <= LSE_TOL
