"""Cases and plain forms of the attention operators for windows with sinks and for paged key/value caches.

Operators (the framework's entry points are called where ``own`` is true):

window   causal attention in which query i sees the keys j with i - j < window and the first ``sinks`` keys;
         the forward alone, or a training step's forward and backward
append   new tokens' keys and values written into a paged cache, as BF16 or quantised to E4M3 with one
         power-of-two scale per (token, head) vector
read     a paged cache's keys and values read back as packed BF16 rows
attend   attention of each sequence's newest tokens (one, or a chunk) over its paged cache, grouped heads,
         optionally with a window and sinks

Shapes: dense tensors [B, H, N, d]; packed rows [tokens, heads, d]; cache pages [pages, heads, page, d] with
scales [pages, heads, page]; ``kv_len`` counts the new tokens; sequence b's new tokens are the rows
q_indptr[b] .. q_indptr[b + 1] of the packed tensors and the last positions of its cache.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one tile of a short sequence: what a unit-sized step costs (latency)
        dict(name="window_step_tiny", op="window", B=1, H=2, N=128, d=64, window=33, sinks=2, backward=True),
        # a training step at the GPT-2-small attention shape with a local window
        dict(name="window_step_gpt2", op="window", B=8, H=12, N=1024, d=64, window=256, sinks=4, backward=True),
        # a training step at the long 32-head shape, window an eighth of the length
        dict(name="window_step_8k", op="window", B=1, H=32, N=8192, d=128, window=1024, sinks=4, backward=True),
        # a ragged length, a window that is no multiple of a tile, sinks over two tiles: forward alone
        dict(name="window_fwd_16k_odd", op="window", B=1, H=16, N=16001, d=128, window=4001, sinks=131, backward=False),
        # one decoding step of a batch: every sequence writes one token, BF16
        dict(name="append_step_bf16", op="append", fmt="bf16", batch=64, hkv=8, d=128, page=64, new_lo=1, new_hi=1,
             ctx_lo=200, ctx_hi=2000, lens=1),
        # prompts written at once into a quantised cache
        dict(name="append_prompt_e4m3", op="append", fmt="e4m3", batch=6, hkv=8, d=128, page=64, new_lo=1000,
             new_hi=9000, ctx_lo=0, ctx_hi=300, lens=2),
        # a quantised cache's prompts read back (moving a cache, recomputation, inspection)
        dict(name="read_e4m3", op="read", fmt="e4m3", batch=8, hkv=8, d=128, page=64, new_lo=0, new_hi=0, ctx_lo=3000,
             ctx_hi=16000, lens=3),
        # a small BF16 cache with an odd head count and small pages
        dict(name="read_bf16_small", op="read", fmt="bf16", batch=3, hkv=5, d=64, page=16, new_lo=0, new_hi=0,
             ctx_lo=1, ctx_hi=900, lens=4),
        # one sequence decoding: latency of a single token over a few thousand keys
        dict(name="attend_decode_one", op="attend", fmt="bf16", batch=1, hq=32, hkv=8, d=128, page=64, new_lo=1,
             new_hi=1, ctx_lo=4000, ctx_hi=4100, window=0, sinks=0, lens=5),
        # a serving batch of ragged lengths decoding from a quantised cache
        dict(name="attend_decode_batch_e4m3", op="attend", fmt="e4m3", batch=64, hq=32, hkv=8, d=128, page=64,
             new_lo=1, new_hi=1, ctx_lo=500, ctx_hi=16000, window=0, sinks=0, lens=6),
        # a prompt's next chunk over a long BF16 cache
        dict(name="attend_chunk_32k", op="attend", fmt="bf16", batch=1, hq=32, hkv=8, d=128, page=128, new_lo=2048,
             new_hi=2048, ctx_lo=32000, ctx_hi=32000, window=0, sinks=0, lens=7),
        # a ragged mix of chunks and single tokens, quantised, d = 64, seven heads per group, window and sinks
        dict(name="attend_mixed_window_e4m3", op="attend", fmt="e4m3", batch=12, hq=28, hkv=4, d=64, page=16,
             new_lo=1, new_hi=700, ctx_lo=10, ctx_hi=8000, window=2000, sinks=4, lens=8),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "append", "read", "attend", "attend", "attend"])
    d = rng.choice([64, 128])
    if op == "window":
        backward = rng.random() < 0.6
        n = _log_int(rng, 1, 12000)
        heads = max(1, int(1.0e9 / (n * n)))
        b = _log_int(rng, 1, min(8, heads))
        h = _log_int(rng, 1, max(1, min(32, heads // b)))
        return dict(op=op, B=b, H=h, N=n, d=d, window=_log_int(rng, 1, 4096),
                    sinks=rng.choice([0, 1, 4, _log_int(rng, 1, 300)]), backward=backward)
    fmt = rng.choice(["bf16", "e4m3"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    lens = rng.randrange(1 << 30)
    if op in ("append", "read"):
        batch = _log_int(rng, 1, 64)
        top = max(2, 40000 // batch)
        if op == "append":
            new_hi = _log_int(rng, 1, top)
            return dict(op=op, fmt=fmt, batch=batch, hkv=hkv, d=d, page=page, new_lo=_log_int(rng, 1, new_hi),
                        new_hi=new_hi, ctx_lo=0, ctx_hi=_log_int(rng, 1, top), lens=lens)
        ctx_hi = _log_int(rng, 1, top)
        return dict(op=op, fmt=fmt, batch=batch, hkv=hkv, d=d, page=page, new_lo=0, new_hi=0,
                    ctx_lo=_log_int(rng, 1, ctx_hi), ctx_hi=ctx_hi, lens=lens)
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    windowed = rng.random() < 0.4
    window = _log_int(rng, 1, 8000) if windowed else 0
    sinks = rng.choice([0, 1, 4, _log_int(rng, 1, 300)]) if windowed else 0
    if rng.random() < 0.5:  # decoding: one or a few tokens for each sequence
        batch = _log_int(rng, 1, 48)
        new_hi = rng.choice([1, 1, 1, 2, 5])
        ctx_hi = _log_int(rng, 16, min(30000, 400000 // batch))
    else:  # chunks
        batch = _log_int(rng, 1, 6)
        new_hi = _log_int(rng, 2, 1500)
        ctx_hi = _log_int(rng, 16, max(32, min(20000, int(1.0e9 / (batch * new_hi * hkv * group)))))
    return dict(op="attend", fmt=fmt, batch=batch, hq=hkv * group, hkv=hkv, d=d, page=page,
                new_lo=1 if rng.random() < 0.5 else new_hi, new_hi=new_hi, ctx_lo=_log_int(rng, 1, ctx_hi),
                ctx_hi=ctx_hi, window=window, sinks=sinks, lens=lens)


def _lengths(case):
    """(new, kv): each sequence's new tokens and its keys with them, from the case alone."""
    r = random.Random(case["lens"])
    new, kv = [], []
    for _ in range(case["batch"]):
        n = case["new_lo"] if case["new_lo"] >= case["new_hi"] else _log_int(r, max(1, case["new_lo"]), case["new_hi"])
        c = r.randint(0, case["ctx_hi"]) if case["ctx_lo"] == 0 else _log_int(r, case["ctx_lo"], case["ctx_hi"])
        new.append(n)
        kv.append(n + c)
    return new, kv


def _seen(n, window, sinks, first=0):
    """How many keys the queries at the positions first .. n - 1 see in all."""
    if window == 0:
        window = n
    total = 0
    for i in range(first, n):
        lo = max(0, i - window + 1)
        total += i + 1 - lo + min(sinks, lo)
    return total


def work(case):
    if case["op"] == "window":
        B, H, N, d = case["B"], case["H"], case["N"], case["d"]
        pairs = B * H * _seen(N, case["window"], case["sinks"])
        tensor, row = B * H * N * d * 2, B * H * N * 4
        if case["backward"]:  # q, k, v, do in; o, lse, dq, dk, dv out; two products forward, five backward
            return {"bytes": 8 * tensor + row, "flops": 14 * pairs * d}
        return {"bytes": 4 * tensor + row, "flops": 4 * pairs * d}
    new, kv = _lengths(case)
    hkv, d = case["hkv"], case["d"]
    vector = 2 * d if case["fmt"] == "bf16" else d + 4  # one head's key or value of one token in the cache
    if case["op"] == "append":
        return {"bytes": 2 * sum(new) * hkv * (2 * d + vector), "flops": 0}
    if case["op"] == "read":
        return {"bytes": 2 * sum(kv) * hkv * (2 * d + vector), "flops": 0}
    w, s, hq = case["window"], case["sinks"], case["hq"]
    pairs = sum(_seen(b, w, s, b - a) for a, b in zip(new, kv))
    lo = [max(0, b - a - w + 1) if w else 0 for a, b in zip(new, kv)]
    keys = sum(b - x + min(s, x) for b, x in zip(kv, lo))
    return {"bytes": 2 * keys * hkv * vector + sum(new) * hq * (4 * d + 4), "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------------------------------ inputs

def _normal(gen, shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 17)
    st = dict(case)
    if case["op"] == "window":
        shape = (case["B"], case["H"], case["N"], case["d"])
        st["q"], st["k"] = _normal(gen, shape, math.sqrt(3)), _normal(gen, shape, math.sqrt(3))
        st["v"], st["do"] = _normal(gen, shape), _normal(gen, shape)
        return st
    new, kv = _lengths(case)
    batch, hkv, d, page = case["batch"], case["hkv"], case["d"], case["page"]
    need = [-(-n // page) for n in kv]
    total, width = sum(need), max(need)
    # pages are handed out in a shuffled order, a few of the pool stay free
    order = torch.randperm(total + 3, generator=gen, device="cuda")[:total].to(torch.int32)
    table = torch.zeros((batch, width), device="cuda", dtype=torch.int32)
    used = torch.arange(width, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[used] = order
    shape = (total + 3, hkv, page, d)
    k, v = _normal(gen, shape, math.sqrt(3)), _normal(gen, shape)
    st["k_scale"] = st["v_scale"] = None
    if case["fmt"] == "e4m3":
        k, st["k_scale"] = _quantize(k)
        v, st["v_scale"] = _quantize(v)
    st["k_cache"], st["v_cache"], st["table"] = k, v, table
    st["kv_len"] = torch.tensor(kv, device="cuda", dtype=torch.int32)
    st["q_indptr"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    st["kv_indptr"] = torch.tensor([0] + kv, device="cuda").cumsum(0).to(torch.int32)
    st["max_new"], st["tokens"], st["rows"], st["max_kv"] = max(new), sum(new), sum(kv), max(kv)
    if case["op"] == "append":
        st["k_new"] = _normal(gen, (sum(new), hkv, d), math.sqrt(3))
        st["v_new"] = _normal(gen, (sum(new), hkv, d))
    if case["op"] == "attend":
        st["q"] = _normal(gen, (sum(new), case["hq"], d), math.sqrt(3))
    return st


# ------------------------------------------------------------------------------------- plain forms

def _quantize(x):
    """(E4M3 codes as bytes, scale): the scale is the least power of two that brings the vector within 448."""
    x = x.float()
    amax = x.abs().amax(-1)
    mant, expo = torch.frexp(amax)  # amax = mant 2^expo, mant in [0.5, 1); 448 = 0.875 * 2^9
    expo = torch.where(mant > 0.875, expo - 8, expo - 9).clamp(min=-126)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), expo), torch.ones_like(amax))
    return (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _values(cache, scale):
    """A cache's values in 32 bits."""
    if scale is None:
        return cache.float()
    return cache.view(torch.float8_e4m3fn).float() * scale[..., None]


def _visible(pos, keys, window, sinks):
    """Whether the query at position pos sees key position keys (broadcast)."""
    see = keys <= pos
    if window:
        see = see & ((pos - keys < window) | (keys < sinks))
    return see


def _softmax(s, see):
    """(probabilities, log-sum-exp) over the last axis; a row that sees nothing gives zeros and -inf."""
    s = s.masked_fill_(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)
    return p.div_(torch.where(total > 0, total, torch.ones_like(total))), lse


def _plain_window(st):
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    scale = 1.0 / math.sqrt(st["d"])
    pos = torch.arange(st["N"], device="cuda")
    see = _visible(pos[:, None], pos[None, :], st["window"], st["sinks"])
    p, lse = _softmax((q @ k.transpose(-1, -2)).mul_(scale), see)
    o = p @ v
    if not st["backward"]:
        return o.to(torch.bfloat16), lse
    do = st["do"].float()
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq, dk = (ds @ k).mul_(scale), (ds.transpose(-1, -2) @ q).mul_(scale)
    return tuple(x.to(torch.bfloat16) if x is not lse else x for x in (o, lse, dq, dk, dv))


def _slots(st):
    """(sequence, position) of each packed new token."""
    at = torch.arange(st["tokens"], device="cuda")
    seq = torch.searchsorted(st["q_indptr"][1:].long(), at, right=True)
    return seq, st["kv_len"][seq].long() - st["q_indptr"][seq + 1].long() + at


def _plain_append(st):
    seq, pos = _slots(st)
    page, slot = st["table"][seq, pos // st["page"]].long(), pos % st["page"]
    if st["k_scale"] is None:
        st["k_cache"][page, :, slot], st["v_cache"][page, :, slot] = st["k_new"], st["v_new"]
    else:
        st["k_cache"][page, :, slot], st["k_scale"][page, :, slot] = _quantize(st["k_new"])
        st["v_cache"][page, :, slot], st["v_scale"][page, :, slot] = _quantize(st["v_new"])


def _plain_read(st):
    at = torch.arange(st["rows"], device="cuda")
    seq = torch.searchsorted(st["kv_indptr"][1:].long(), at, right=True)
    pos = at - st["kv_indptr"][seq].long()
    page, slot = st["table"][seq, pos // st["page"]].long(), pos % st["page"]
    if st["k_scale"] is None:
        return st["k_cache"][page, :, slot], st["v_cache"][page, :, slot]
    return (_values(st["k_cache"][page, :, slot], st["k_scale"][page, :, slot]).to(torch.bfloat16),
            _values(st["v_cache"][page, :, slot], st["v_scale"][page, :, slot]).to(torch.bfloat16))


def _gathered(st, name):
    """Each sequence's cache in 32 bits, padded to the longest: [batch, heads, keys, d]."""
    table = st["table"].long()
    x = _values(st[name + "_cache"][table], st[name + "_scale"][table] if st[name + "_scale"] is not None else None)
    return x.permute(0, 2, 1, 3, 4).reshape(table.shape[0], st["hkv"], -1, st["d"])


def _plain_attend(st):
    batch, hq, hkv, d, longest = st["batch"], st["hq"], st["hkv"], st["d"], st["max_new"]
    seq, pos = _slots(st)
    row = torch.arange(st["tokens"], device="cuda") - st["q_indptr"][seq].long()
    q = torch.zeros((batch, longest, hq, d), device="cuda")
    q[seq, row] = st["q"].float()
    q = q.view(batch, longest, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    k, v = _gathered(st, "k"), _gathered(st, "v")
    at = torch.full((batch, longest), -1, device="cuda", dtype=torch.long)
    at[seq, row] = pos
    keys = torch.arange(k.shape[2], device="cuda")
    see = _visible(at[:, :, None], keys, st["window"], st["sinks"])[:, None, None]
    s = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(batch, hkv, hq // hkv, longest, -1)
    p, lse = _softmax(s, see)
    # what the pages hold behind a sequence's last key is not its own
    v = torch.where((keys[None, :] < st["kv_len"][:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = p.view(batch, hkv, -1, p.shape[-1]) @ v
    o = o.view(batch, hkv, hq // hkv, longest, d).permute(0, 3, 1, 2, 4).reshape(batch, longest, hq, d)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, longest, hq)
    return o[seq, row].to(torch.bfloat16), lse[seq, row]


def _cache_out(st):
    """The whole cache after a write, bytes as the E4M3 values that they are."""
    if st["k_scale"] is None:
        return {"k": st["k_cache"], "v": st["v_cache"]}
    return {"k": st["k_cache"].view(torch.float8_e4m3fn), "v": st["v_cache"].view(torch.float8_e4m3fn),
            "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def run(st):
    op = st["op"]
    if own:
        from numerics_tcgen05_tmem_gb300 import binding as fa
        if op == "window":
            o, lse = fa.forward(st["q"], st["k"], st["v"], window=st["window"], sinks=st["sinks"])
            if not st["backward"]:
                return o, lse
            return (o, lse) + fa.backward(st["q"], st["k"], st["v"], o, lse, st["do"], window=st["window"],
                                          sinks=st["sinks"])
        if op == "append":
            fa.kv_append(st["k_new"], st["v_new"], st["k_cache"], st["v_cache"], st["table"], st["kv_len"],
                         st["q_indptr"], k_scale=st["k_scale"], v_scale=st["v_scale"])
            return _cache_out(st)
        if op == "read":
            return fa.kv_read(st["k_cache"], st["v_cache"], st["table"], st["kv_len"], st["kv_indptr"], st["rows"],
                              k_scale=st["k_scale"], v_scale=st["v_scale"])
        return fa.forward_paged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["kv_len"], st["q_indptr"],
                                st["max_new"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                                window=st["window"] or None, sinks=st["sinks"])
    if op == "window":
        return _plain_window(st)
    if op == "append":
        _plain_append(st)
        return _cache_out(st)
    if op == "read":
        return _plain_read(st)
    return _plain_attend(st)


# --------------------------------------------------------------------- the definitions in 64 bits

def _exact_rows(q, k, v, scale, pos, keys, window, sinks):
    """One head's softmax attention of rows at `pos` over keys at `keys`: (probabilities, output, log-sum-exp)."""
    gap = pos[:, None] - keys[None, :]
    hidden = gap < 0
    if window > 0:
        hidden = hidden | ((gap >= window) & (keys[None, :] >= sinks))
    logits = torch.einsum("...qd,...kd->...qk", q, k) * scale
    logits = logits.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(logits, -1)
    p = torch.exp(logits - lse[..., None])
    return p, torch.einsum("...qk,...kd->...qd", p, v), lse


def _key_range(first, last, window, sinks):
    """The key positions that the queries first .. last can see, in order."""
    lo = max(0, first - window + 1) if window else 0
    return torch.cat([torch.arange(0, min(sinks, lo), device="cuda"), torch.arange(lo, last + 1, device="cuda")])


def _exact_window(st):
    n, d, window, sinks = st["N"], st["d"], st["window"], st["sinks"]
    scale = 1.0 / math.sqrt(d)
    flat = [st[x].reshape(-1, n, d) for x in ("q", "k", "v", "do")]
    heads = flat[0].shape[0]
    lse = torch.empty((heads, n), device="cuda", dtype=torch.float64)
    o, dq, dk, dv = (torch.zeros((heads, n, d), device="cuda", dtype=torch.float64) for _ in range(4))
    step = 4
    for h in range(0, heads, step):
        q, k, v, do = (x[h:h + step].double() for x in flat)
        for r in range(0, n, 512):
            end = min(n, r + 512)
            keys = _key_range(r, end - 1, window, sinks)
            p, out, stat = _exact_rows(q[:, r:end], k[:, keys], v[:, keys], scale,
                                       torch.arange(r, end, device="cuda"), keys, window, sinks)
            o[h:h + step, r:end], lse[h:h + step, r:end] = out, stat
            if not st["backward"]:
                continue
            g = do[:, r:end]
            dp = torch.einsum("hqd,hkd->hqk", g, v[:, keys])
            ds = p * (dp - torch.einsum("hqk,hqk->hq", p, dp)[..., None]) * scale
            dv[h:h + step].index_add_(1, keys, torch.einsum("hqk,hqd->hkd", p, g))
            dk[h:h + step].index_add_(1, keys, torch.einsum("hqk,hqd->hkd", ds, q[:, r:end]))
            dq[h:h + step, r:end] = torch.einsum("hqk,hkd->hqd", ds, k[:, keys])
    shape = st["q"].shape
    o, lse = o.view(shape), lse.view(shape[:3])
    return (o, lse, dq.view(shape), dk.view(shape), dv.view(shape)) if st["backward"] else (o, lse)


def _exact_codes(x):
    """(values of the nearest E4M3 codes, scale) of vectors, in 64-bit arithmetic."""
    x = x.double()
    amax = x.abs().amax(-1)
    k = torch.ceil(torch.log2(amax / E4M3_MAX))
    k = torch.where(amax > E4M3_MAX * torch.exp2(k), k + 1, k)  # log2 next to a border
    k = torch.where(amax <= E4M3_MAX * torch.exp2(k - 1), k - 1, k).clamp(min=-126)
    scale = torch.where(amax > 0, torch.exp2(k), torch.ones_like(amax))
    y = x / scale[..., None]
    _, e = torch.frexp(y)
    step = torch.exp2((e.double() - 1).clamp(min=-6) - 3)  # spacing of the codes around y
    return torch.round(y / step) * step, scale


def _exact_append(st):
    out = {}
    for name in ("k", "v"):
        cache, new = st[name + "_cache"], st[name + "_new"]
        vals = (cache if st["k_scale"] is None else cache.view(torch.float8_e4m3fn)).double()
        codes, scale = (new.double(), None) if st["k_scale"] is None else _exact_codes(new)
        scales = None if st["k_scale"] is None else st[name + "_scale"].double()
        row = 0
        for b, (n, kv) in enumerate(zip(*_lengths(st))):
            p = torch.arange(kv - n, kv, device="cuda")
            page, slot = st["table"][b].long()[p // st["page"]], p % st["page"]
            vals[page, :, slot] = codes[row:row + n]
            if scales is not None:
                scales[page, :, slot] = scale[row:row + n]
            row += n
        out[name] = vals
        if scales is not None:
            out[name + "_scale"] = scales
    return out


def _exact_sequence(st, name, b, kv):
    """Sequence b's keys or values from its pages: [heads, kv, d]."""
    pages = st["table"][b, : -(-kv // st["page"])].long()
    x = st[name + "_cache"][pages]
    if st["k_scale"] is None:
        x = x.double()
    else:
        x = x.view(torch.float8_e4m3fn).double() * st[name + "_scale"][pages].double().unsqueeze(-1)
    return x.transpose(0, 1).reshape(st["hkv"], -1, st["d"])[:, :kv]


def _exact_read(st):
    kv = _lengths(st)[1]
    return tuple(torch.cat([_exact_sequence(st, name, b, n).transpose(0, 1) for b, n in enumerate(kv)])
                 for name in ("k", "v"))


def _exact_attend(st):
    new, kv = _lengths(st)
    hkv, d, group = st["hkv"], st["d"], st["hq"] // st["hkv"]
    o = torch.zeros((st["tokens"], st["hq"], d), device="cuda", dtype=torch.float64)
    lse = torch.zeros((st["tokens"], st["hq"]), device="cuda", dtype=torch.float64)
    row = 0
    for b, (n, m) in enumerate(zip(new, kv)):
        k, v = _exact_sequence(st, "k", b, m), _exact_sequence(st, "v", b, m)
        for r in range(0, n, 256):
            end = min(n, r + 256)
            first, last = m - n + r, m - n + end - 1
            keys = _key_range(first, last, st["window"], st["sinks"])
            q = st["q"][row + r:row + end].double().view(end - r, hkv, group, d).permute(1, 2, 0, 3)
            _, out, stat = _exact_rows(q, k[:, None, keys], v[:, None, keys], 1.0 / math.sqrt(d),
                                       torch.arange(first, last + 1, device="cuda"), keys, st["window"], st["sinks"])
            o[row + r:row + end] = out.permute(2, 0, 1, 3).reshape(end - r, st["hq"], d)
            lse[row + r:row + end] = stat.permute(2, 0, 1).reshape(end - r, st["hq"])
        row += n
    return o, lse


def exact(case, seed):
    st = prepare(case, seed)
    return {"window": _exact_window, "append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](st)
