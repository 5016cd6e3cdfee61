"""Paged caches for the tests: pages in shuffled order, everything outside the sequences poisoned."""
from __future__ import annotations

import math
from types import SimpleNamespace

import torch

from tests import _masked as M

E4M3 = torch.float8_e4m3fn


def quantize(x):
    """(codes, scale) of BF16 vectors in 64-bit arithmetic: scale = least 2^k (k >= -126) with
    max|x| <= 448 scale; codes (240 at most with scale 2^120) rounded to nearest even; a vector with NaN or Inf: code 0x7F, NaN scale."""
    x = x.detach().cpu().double()
    bad = ~torch.isfinite(x).all(-1)
    x = torch.where(bad[..., None], torch.ones_like(x), x)
    amax = x.abs().amax(-1)
    k = torch.full(amax.shape, -126.0, dtype=torch.float64)
    for e in range(-126, 121):
        k = torch.where((amax > 448 * 2.0 ** (e - 1)) & (e > -126), torch.full_like(k, e), k)
    scale = torch.where(amax > 0, torch.exp2(k), torch.ones_like(k))
    y = x / scale[..., None]
    # the spacing of E4M3 around y: 2^(floor(log2|y|) - 3), 2^-9 below 2^-6
    _, e = torch.frexp(y)
    step = torch.exp2((e.double() - 1).clamp(min=-6) - 3)
    val = torch.round(y / step) * step
    # with the largest scale a code of 256 would stand for 2^128, past the largest float: 240 is kept
    val = torch.where((k == 120)[..., None], val.clamp(-240, 240), val)
    # (y = -0 keeps its sign: round and the product keep it)
    codes = val.float().to(E4M3).view(torch.uint8)
    assert torch.equal(codes.view(E4M3).double(), val)
    codes = torch.where(bad[..., None], torch.full_like(codes, 0x7F), codes)
    return codes, torch.where(bad, torch.full_like(scale, math.nan), scale).float()


def make(lens, hkv, d, page, fmt="bf16", seed=0, std=1.5, spare=3, combined=False, max_extra=2):
    """A cache for sequences of `lens` keys.  Free pages and slots behind a sequence's end hold NaN
    (code 0x7F); table entries behind a sequence's last page point far outside the pool."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    P = sum(need) + spare
    order = torch.randperm(P, generator=g)[: sum(need)].tolist()
    table = torch.full((len(lens), max(need + [1]) + max_extra), 2 ** 30, dtype=torch.int32)
    vals = [torch.randn((n, 2, hkv, d), generator=g) for n in lens]
    kv = [(x * torch.tensor([std, 1.0])[None, :, None, None]).to(torch.bfloat16) for x in vals]
    c = SimpleNamespace(lens=list(lens), hkv=hkv, d=d, page=page, fmt=fmt, P=P)
    shape = (P, hkv, page, d)
    pool = torch.full((P, 2) + shape[1:], math.nan).to(torch.bfloat16) if fmt == "bf16" else \
        torch.full((P, 2) + shape[1:], 0x7F, dtype=torch.uint8)
    scales = torch.full((P, 2, hkv, page), math.nan)
    c.values = []    # per sequence: K and V values in float64 [hkv, n, d]
    at = 0
    for b, n in enumerate(lens):
        for i in range(need[b]):
            table[b, i] = order[at + i]
        t = torch.arange(n)
        pg, slot = table[b].long()[t // page], t % page
        out = []
        for w in range(2):
            x = kv[b][:, w]                     # [n, hkv, d]
            if fmt == "bf16":
                pool[pg, w, :, slot] = x
                out.append(x.double().transpose(0, 1))
            else:
                codes, s = quantize(x)
                pool[pg, w, :, slot] = codes
                scales[pg, w, :, slot] = s
                out.append((codes.view(E4M3).double() * s.double()[..., None]).transpose(0, 1))
        c.values.append(out)
        at += need[b]
    dev = "cuda"
    pool, scales = pool.to(dev), scales.to(dev)
    if combined:      # K and V interleaved page by page in one buffer
        c.k, c.v = pool[:, 0], pool[:, 1]
        c.ks, c.vs = scales[:, 0], scales[:, 1]
    else:
        c.k, c.v = pool[:, 0].contiguous(), pool[:, 1].contiguous()
        c.ks, c.vs = scales[:, 0].contiguous(), scales[:, 1].contiguous()
    if fmt == "bf16":
        c.ks = c.vs = None
    c.table, c.kv_len = table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    return c


def indptr(counts, dev="cuda"):
    return torch.tensor([0] + list(counts)).cumsum(0).to(torch.int32).to(dev)


def reference(c, q, new, scale, window=None, sinks=0):
    """o, lse and the bound of o for packed rows q [T, Hq, d] (CPU), in 64 bits."""
    T, Hq, d = q.shape
    group = Hq // c.hkv
    o, lse, tol = torch.zeros((T, Hq, d), dtype=torch.float64), torch.zeros((T, Hq), dtype=torch.float64), \
        torch.zeros((T, Hq, d), dtype=torch.float64)
    row = 0
    for b, n in enumerate(new):
        kv = c.lens[b]
        see = M.window_mask(torch.arange(kv - n, kv), torch.arange(kv), window, sinks)
        for h in range(Hq):
            k, v = (x[h // group] for x in c.values[b])
            if kv == 0 or n == 0:
                lse[row:row + n, h] = -math.inf
                tol[row:row + n, h] = 1e-6
                continue
            r = M.forward(q[row:row + n, h], k, v, see, scale)
            o[row:row + n, h], lse[row:row + n, h], tol[row:row + n, h] = r["o"], r["lse"], r["o_tol"]
        row += n
    return o, lse, tol
