"""Accumulated attention weights and eviction in 64 bits, over the caches of tests/_paged.py."""
from __future__ import annotations

import math

import torch

from tests import _masked as M

F32 = 2.0 ** -24


def make(c, seed=0, std=1.0):
    """Weights for a cache: log-normal where its sequences' keys are, NaN elsewhere; and what sequence b's are [hkv, n]."""
    g = torch.Generator().manual_seed(seed)
    pool = torch.full((c.P, c.hkv, c.page), math.nan)
    rows = []
    for b, n in enumerate(c.lens):
        w = torch.exp(torch.randn((c.hkv, n), generator=g) * std)
        put(c, pool, b, w)
        rows.append(w)
    return pool, rows


def put(c, pool, b, w):
    t = torch.arange(w.shape[1])
    pool[c.table[b].cpu().long()[t // c.page], :, t % c.page] = w.transpose(0, 1).to(pool.dtype)


def take(c, pool, b):
    t = torch.arange(c.lens[b])
    return pool[c.table[b].cpu().long()[t // c.page], :, t % c.page].transpose(0, 1)


def log_sum_exps(c, q, new, scale, window=None, sinks=0):
    """The attention call's [T, Hq], exact and then FP32."""
    T, Hq, d = q.shape
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    for b, row, n, see in sequences(c, new, window, sinks):
        for h in range(Hq):
            s = q[row:row + n, h].double() @ c.values[b][0][h // (Hq // c.hkv)].transpose(0, 1) * scale
            lse[row:row + n, h] = s.masked_fill(~see, -math.inf).logsumexp(-1)
    return lse.float()


def sequences(c, new, window, sinks):
    row = 0
    for b, n in enumerate(new):
        kv = c.lens[b]
        if n and kv:
            yield b, row, n, M.window_mask(torch.arange(kv - n, kv), torch.arange(kv), window, sinks)
        row += n


def reference(c, rows, q, lse, new, scale, window=None, sinks=0):
    """{sequence: (weights [hkv, kv], bound)} for the sequences that have new tokens.

    FP32: q . k is summed in steps of 16 or 32 products, each step off by 2^-23 of the products' magnitudes at most (d / 8
    steps cover three vectors of E4M3 queries too), an entry of q under 2^-24 of the largest may be lost; the exponent
    scale q.k - lse takes four roundings, the exponential 2^-21; a sum of a block's columns is a chain of 32 + 3.
    """
    T, Hq, d = q.shape
    group, out = Hq // c.hkv, {}
    for b, row, n, see in sequences(c, new, window, sinks):
        kv = c.lens[b]
        w, tol = rows[b].double().clone(), torch.zeros((c.hkv, kv), dtype=torch.float64)
        w[:, max(kv - n, 0):] = 0
        seen = see.any(0)
        w[:, ~seen] = rows[b].double()[:, ~seen]
        for h in range(Hq):
            qh, k = q[row:row + n, h].double(), c.values[b][0][h // group]
            s = qh @ k.transpose(0, 1) * scale
            e = lse[row:row + n, h].double()[:, None]
            p = torch.where(see & ~torch.isinf(e), torch.exp(s - e), torch.zeros_like(s))
            off = (qh.abs() @ k.abs().transpose(0, 1)) * (d / 8 * 2 * F32) + qh.abs().amax(-1, keepdim=True) * k.abs().sum(-1) * F32
            off = off * scale + 4 * F32 * (s.abs() + e.abs().nan_to_num(posinf=0)) + 2.0 ** -21
            w[h // group] += p.sum(0)
            tol[h // group] += (p * off).sum(0)
        out[b] = w, tol + (40 + n * group / 16) * F32 * w + 1e-37
    return out


def chosen(w, keep, sinks, recent):
    """The kept positions of one head's weights [n], by sorting."""
    n = w.numel()
    if n <= keep:
        return torch.arange(n)
    order = sorted(range(sinks, n - recent), key=lambda j: (not math.isnan(w[j]), -w[j] if not math.isnan(w[j]) else 0, j))
    return torch.tensor(sorted(list(range(sinks)) + order[: keep - sinks - recent] + list(range(n - recent, n))), dtype=torch.long)
