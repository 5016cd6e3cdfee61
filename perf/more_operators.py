"""Cases and plain forms of the operators around the attention calls: what makes queries and keys ready for them, and
what keeps a paged cache within a budget.

Operators (the framework's entry points are called where ``own`` is true):

rotate      queries and keys of a dense batch: a norm for each head, then the position rotation; the forward alone, or a
            training step's forward and backward (with the gradients of the norms' weights)
append      the serving form over packed rows: queries normed and rotated, keys normed, rotated and written with the
            values into a paged cache, as BF16 or as E4M3 with one power-of-two scale per (token, head) vector
accumulate  for each cached key, the attention weight that a step's new tokens give it is added to its running sum
evict       of each sequence and kv head the keys of the largest sums stay (the first and the newest ones always) and
            move, in order, to the pages of another block table

Shapes: dense tensors [B, H, N, d], as views of a projection [B, N, Hq + 2 Hkv, d]; packed rows [tokens, heads, d];
cache pages [pages, heads, page, d], their scales and sums [pages, heads, page]; ``kv_len`` counts the new tokens;
sequence b's new tokens are the rows q_indptr[b] .. q_indptr[b + 1] and the last positions of its cache.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short sequence of a small model: what a training step's two calls cost at least (latency)
        dict(name="rotate_step_tiny", op="rotate", B=1, N=128, hq=2, hkv=2, d=64, rot=64, interleaved=False, first=0,
             backward=True),
        # a training step at the GPT-2-small attention shape
        dict(name="rotate_step_gpt2", op="rotate", B=8, N=1024, hq=12, hkv=12, d=64, rot=64, interleaved=False, first=0,
             backward=True),
        # a training step at the long 32-head shape
        dict(name="rotate_step_8k", op="rotate", B=1, N=8192, hq=32, hkv=32, d=128, rot=128, interleaved=False, first=0,
             backward=True),
        # a ragged length far behind the origin, grouped heads, half of each head rotated, neighbouring pairs
        dict(name="rotate_fwd_far_odd", op="rotate", B=3, N=5001, hq=28, hkv=4, d=128, rot=64, interleaved=True,
             first=1000003, backward=False),
        # one decoding step of a batch: every sequence brings one token, BF16
        dict(name="append_decode_bf16", op="append", fmt="bf16", batch=64, hq=32, hkv=8, d=128, page=64, rot=128,
             new_lo=1, new_hi=1, ctx_lo=200, ctx_hi=2000, lens=1),
        # prompts of a few sequences into a quantised cache
        dict(name="append_prompt_e4m3", op="append", fmt="e4m3", batch=6, hq=32, hkv=8, d=128, page=64, rot=128,
             new_lo=200, new_hi=900, ctx_lo=0, ctx_hi=300, lens=2),
        # long prompts into a BF16 cache
        dict(name="append_prompt_bf16", op="append", fmt="bf16", batch=4, hq=32, hkv=8, d=128, page=64, rot=128,
             new_lo=2000, new_hi=9000, ctx_lo=0, ctx_hi=300, lens=3),
        # one sequence decoding over a few thousand keys (latency)
        dict(name="accumulate_decode_one", op="accumulate", fmt="bf16", batch=1, hq=32, hkv=8, d=128, page=64, new_lo=1,
             new_hi=1, ctx_lo=4000, ctx_hi=4100, window=0, sinks=0, lens=5),
        # a serving batch of ragged lengths decoding over a quantised cache
        dict(name="accumulate_decode_batch_e4m3", op="accumulate", fmt="e4m3", batch=64, hq=32, hkv=8, d=128, page=64,
             new_lo=1, new_hi=1, ctx_lo=500, ctx_hi=16000, window=0, sinks=0, lens=6),
        # a prompt's next chunk over a long BF16 cache
        dict(name="accumulate_chunk_32k", op="accumulate", fmt="bf16", batch=1, hq=32, hkv=8, d=128, page=128,
             new_lo=2048, new_hi=2048, ctx_lo=32000, ctx_hi=32000, window=0, sinks=0, lens=7),
        # one sequence cut to a budget
        dict(name="evict_one", op="evict", fmt="bf16", batch=1, hkv=8, d=128, page=64, ctx_lo=4500, ctx_hi=4500,
             keep=2048, sinks=4, recent=256, lens=11),
        # a serving batch of ragged lengths, quantised; some sequences are within the budget
        dict(name="evict_batch_e4m3", op="evict", fmt="e4m3", batch=64, hkv=8, d=128, page=64, ctx_lo=500, ctx_hi=16000,
             keep=2000, sinks=4, recent=200, lens=12),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "append", "append", "accumulate", "accumulate", "accumulate", "evict", "evict"])
    d = rng.choice([64, 128])
    lens = rng.randrange(1 << 30)
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    rot = rng.choice([d, d, d // 2, 48])
    if op == "rotate":
        n = _log_int(rng, 1, 30000)
        b = _log_int(rng, 1, max(1, min(16, 30000 // n)))
        h = _log_int(rng, 1, max(1, min(32, 260000 // (n * b))))
        return dict(op=op, B=b, N=n, hq=h, hkv=rng.choice([h, max(1, h // 4), 1]), d=d, rot=rot,
                    interleaved=rng.random() < 0.3, first=rng.choice([0, 0, _log_int(rng, 1, 4000000)]),
                    backward=rng.random() < 0.6)
    fmt = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        batch = _log_int(rng, 1, 64)
        new_hi = _log_int(rng, 1, max(2, (20000 if fmt == "bf16" else 4000) // batch))
        return dict(op=op, fmt=fmt, batch=batch, hq=hkv * min(group, 8), hkv=hkv, d=d, page=page, rot=rot,
                    new_lo=_log_int(rng, 1, new_hi), new_hi=new_hi, ctx_lo=0, ctx_hi=_log_int(rng, 1, 20000 // batch + 2),
                    lens=lens)
    if op == "evict":
        batch = _log_int(rng, 1, 48)
        ctx_hi = _log_int(rng, 16, min(40000, 400000 // batch))
        keep = _log_int(rng, 2, min(4000, ctx_hi))
        return dict(op=op, fmt=fmt, batch=batch, hkv=hkv, d=d, page=page, ctx_lo=_log_int(rng, 1, ctx_hi), ctx_hi=ctx_hi,
                    keep=keep, sinks=rng.choice([0, 1, min(4, keep // 2)]), recent=rng.choice([0, 1, keep // 8, keep // 2]),
                    lens=lens)
    windowed = rng.random() < 0.3
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
    return dict(op=op, fmt=fmt, batch=batch, hq=hkv * group, hkv=hkv, d=d, page=page,
                new_lo=1 if rng.random() < 0.5 else new_hi, new_hi=new_hi, ctx_lo=_log_int(rng, 1, ctx_hi), ctx_hi=ctx_hi,
                window=window, sinks=sinks, lens=lens)


def _lengths(case):
    """(new, kv): each sequence's new tokens and its keys with them, from the case alone."""
    r = random.Random(case["lens"])
    new, kv = [], []
    for _ in range(case["batch"]):
        n = 0
        if "new_hi" in case:
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
    op, d = case["op"], case["d"]
    if op == "rotate":
        heads = case["hq"] + case["hkv"]
        tensor = case["B"] * case["N"] * heads * d * 2
        if case["backward"]:  # x and dz in, z and dx out, the weights' gradients
            return {"bytes": 4 * tensor + 4 * case["N"] + 16 * d, "flops": 24 * (tensor // 2)}
        return {"bytes": 2 * tensor + 4 * case["N"] + 8 * d, "flops": 9 * (tensor // 2)}
    new, kv = _lengths(case)
    hkv = case["hkv"]
    vector = 2 * d if case["fmt"] == "bf16" else d + 4  # one head's key or value of one token in the cache
    if op == "append":
        hq = case["hq"]
        return {"bytes": sum(new) * (4 * hq * d + 2 * hkv * (2 * d + vector)), "flops": sum(new) * (hq + hkv) * d * 9}
    if op == "evict":
        kept = sum(min(n, case["keep"]) for n in kv)
        return {"bytes": hkv * (4 * sum(kv) + kept * (2 * 2 * vector + 4 + 4)), "flops": 0}
    w, s, hq = case["window"], case["sinks"], case["hq"]
    pairs = sum(_seen(b, w, s, b - a) for a, b in zip(new, kv))
    lo = [max(0, b - a - w + 1) if w else 0 for a, b in zip(new, kv)]
    keys = sum(b - x + min(s, x) for b, x in zip(kv, lo))
    return {"bytes": keys * hkv * (vector + 8) + sum(new) * hq * (2 * d + 4), "flops": 2 * pairs * hq * d}


# ------------------------------------------------------------------------------------------ inputs

def _normal(gen, shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _rotation(st, gen):
    """The frequencies (radians for each position, 64 bits) and the norms' weights."""
    i = torch.arange(st["rot"] // 2, device="cuda", dtype=torch.float64)
    st["inv_freq"] = 10000.0 ** (-2.0 * i / st["rot"])
    st["q_weight"] = 1.0 + 0.2 * torch.randn(st["d"], generator=gen, device="cuda")
    st["k_weight"] = 1.0 + 0.2 * torch.randn(st["d"], generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 29)
    st = dict(case)
    if case["op"] == "rotate":
        B, N, hq, hkv, d = (case[x] for x in ("B", "N", "hq", "hkv", "d"))
        _rotation(st, gen)
        # tokens of a projection differ in size, and so do its channels
        rows = _normal(gen, (B, N, hq + 2 * hkv, d), 1.7)
        st["q"], st["k"] = rows[:, :, :hq].transpose(1, 2), rows[:, :, hq:hq + hkv].transpose(1, 2)
        st["positions"] = torch.arange(case["first"], case["first"] + N, device="cuda", dtype=torch.int32)
        if case["backward"]:
            st["dq"], st["dk"] = _normal(gen, (B, hq, N, d)), _normal(gen, (B, hkv, N, d))
        return st
    new, kv = _lengths(case)
    batch, hkv, d, page = case["batch"], case["hkv"], case["d"], case["page"]
    need = [-(-n // page) for n in kv]
    need_out = [-(-min(n, case["keep"]) // page) for n in kv] if case["op"] == "evict" else []
    total, width = sum(need), max(need)
    # pages are handed out in a shuffled order, a few of the pool stay free
    pool = total + sum(need_out) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    st["table"] = _table(order[:total], need, width)
    shape = (pool, hkv, page, d)
    k, v = _normal(gen, shape, math.sqrt(3)), _normal(gen, shape)
    st["k_scale"] = st["v_scale"] = None
    if case["fmt"] == "e4m3":
        k, st["k_scale"] = _quantize(k)
        v, st["v_scale"] = _quantize(v)
    st["k_cache"], st["v_cache"] = k, v
    st["kv_len"] = torch.tensor(kv, device="cuda", dtype=torch.int32)
    st["q_indptr"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    st["max_new"], st["tokens"] = max(new), sum(new)
    if case["op"] == "append":
        _rotation(st, gen)
        rows = _normal(gen, (sum(new), case["hq"] + 2 * hkv, d), 1.7)
        st["q"], st["k_new"], st["v_new"] = rows.split([case["hq"], hkv, hkv], 1)
        return st
    # sums as a hundred steps over some thousand keys leave them, unevenly spread
    st["weights"] = torch.randn(shape[:3], generator=gen, device="cuda").exp_().mul_(0.02)
    if case["op"] == "evict":
        st["table_out"] = _table(order[total:total + sum(need_out)], need_out, -(-case["keep"] // page))
        return st
    st["q"] = _normal(gen, (sum(new), case["hq"], d), math.sqrt(3))
    # what the attention call over this cache hands on
    st["lse"] = _scores(st)[1]
    return st


def _table(pages, need, width):
    """A block table [batch, width]: need[b] of the pages for sequence b."""
    table = torch.zeros((len(need), width), device="cuda", dtype=torch.int32)
    used = torch.arange(width, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[used] = pages
    return table


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


def _angles(st, positions):
    """cos and sin [..., rot / 2] of positions times frequencies; the products in 64 bits."""
    a = positions.double()[..., None] * st["inv_freq"]
    return a.cos().float(), a.sin().float()


def _rotated(y, cos, sin, st):
    """y's first `rot` entries rotated pairwise; cos and sin broadcast over the heads."""
    rot = st["rot"]
    if st["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, y[..., rot:]), -1)


def _normed(x, weight):
    """(x over its root mean square, that times the weight, 1 / root mean square) in 32 bits."""
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, x * r * weight, r


def _normed_back(x, weight, dy):
    """(dx, dweight) of the norm."""
    unit, _, r = _normed(x, weight)
    g = dy * weight
    dx = r * (g - unit * (g * unit).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (dy * unit).double().sum((0, 1, 2)).float()


def _plain_rotate(st):
    cos, sin = _angles(st, st["positions"])
    q, k = (_rotated(_normed(st[x], st[x + "_weight"])[1], cos, sin, st).to(torch.bfloat16) for x in ("q", "k"))
    if not st["backward"]:
        return q, k
    dq, dqw = _normed_back(st["q"], st["q_weight"], _rotated(st["dq"].float(), cos, -sin, st))
    dk, dkw = _normed_back(st["k"], st["k_weight"], _rotated(st["dk"].float(), cos, -sin, st))
    return q, k, dq, dk, dqw, dkw


def _slots(st):
    """(sequence, position) of each packed new token."""
    at = torch.arange(st["tokens"], device="cuda")
    seq = torch.searchsorted(st["q_indptr"][1:].long(), at, right=True)
    return seq, st["kv_len"][seq].long() - st["q_indptr"][seq + 1].long() + at


def _plain_append(st):
    seq, pos = _slots(st)
    page, slot = st["table"][seq, pos // st["page"]].long(), pos % st["page"]
    cos, sin = (x[:, None] for x in _angles(st, pos))
    half = {"rot": st["rot"], "interleaved": False}
    q = _rotated(_normed(st["q"], st["q_weight"])[1], cos, sin, half).to(torch.bfloat16)
    k = _rotated(_normed(st["k_new"], st["k_weight"])[1], cos, sin, half)
    if st["k_scale"] is None:
        st["k_cache"][page, :, slot], st["v_cache"][page, :, slot] = k.to(torch.bfloat16), st["v_new"]
    else:
        st["k_cache"][page, :, slot], st["k_scale"][page, :, slot] = _quantize(k)
        st["v_cache"][page, :, slot], st["v_scale"][page, :, slot] = _quantize(st["v_new"])
    return q


def _scores(st):
    """The new tokens' scaled scores over their padded caches, with -inf where nothing is seen, and each row's log-sum-exp:
    scores [batch, hkv, group, longest, keys], lse [tokens, hq]."""
    batch, hq, hkv, d, longest = st["batch"], st["hq"], st["hkv"], st["d"], st["max_new"]
    seq, pos = _slots(st)
    row = torch.arange(st["tokens"], device="cuda") - st["q_indptr"][seq].long()
    q = torch.zeros((batch, longest, hq, d), device="cuda")
    q[seq, row] = st["q"].float()
    q = q.view(batch, longest, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    table = st["table"].long()
    k = _values(st["k_cache"][table], st["k_scale"][table] if st["k_scale"] is not None else None)
    k = k.permute(0, 2, 1, 3, 4).reshape(batch, hkv, -1, d)
    at = torch.full((batch, longest), -1, device="cuda", dtype=torch.long)
    at[seq, row] = pos
    keys = torch.arange(k.shape[2], device="cuda")
    see = keys <= at[:, :, None]
    if st["window"]:
        see = see & ((at[:, :, None] - keys < st["window"]) | (keys < st["sinks"]))
    s = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(batch, hkv, hq // hkv, longest, -1)
    s.masked_fill_(~see[:, None, None], -math.inf)
    lse = s.logsumexp(-1).permute(0, 3, 1, 2).reshape(batch, longest, hq)
    return s, lse[seq, row]


def _plain_accumulate(st):
    batch, hq, hkv, longest = st["batch"], st["hq"], st["hkv"], st["max_new"]
    s = _scores(st)[0]
    seq, pos = _slots(st)
    row = torch.arange(st["tokens"], device="cuda") - st["q_indptr"][seq].long()
    lse = torch.full((batch, longest, hq), math.inf, device="cuda")   # rows that no token fills weigh nothing
    lse[seq, row] = st["lse"]
    lse = lse.view(batch, longest, hkv, hq // hkv).permute(0, 2, 3, 1)[..., None]
    total = s.sub_(lse).exp_().sum((2, 3))   # [batch, hkv, keys]
    table = st["table"].long()
    keys = torch.arange(total.shape[2], device="cuda")
    old = st["weights"][table].permute(0, 2, 1, 3).reshape(total.shape)
    fresh = keys >= (st["kv_len"] - (st["q_indptr"][1:] - st["q_indptr"][:-1]))[:, None]
    total = total + old.masked_fill(fresh[:, None], 0.0)
    b, j = (keys < st["kv_len"][:, None]).nonzero(as_tuple=True)
    st["weights"][table[b, j // st["page"]], :, j % st["page"]] = total[b, :, j]
    return st["weights"]


def _plain_evict(st):
    batch, hkv, keep, sinks, recent = (st[x] for x in ("batch", "hkv", "keep", "sinks", "recent"))
    table, n = st["table"].long(), st["kv_len"].long()
    w = st["weights"][table].permute(0, 2, 1, 3).reshape(batch, hkv, -1)
    keys = torch.arange(w.shape[2], device="cuda")
    inside = keys < n[:, None]
    always = inside & ((keys < sinks) | (keys >= n[:, None] - recent))
    w = w.masked_fill(always[:, None], math.inf).masked_fill(~inside[:, None], -math.inf)
    order = w.sort(dim=-1, descending=True, stable=True)[1][..., :keep]
    if order.shape[2] < keep:
        order = torch.cat((order, order.new_full((batch, hkv, keep - order.shape[2]), w.shape[2])), 2)
    kept_len = n.clamp(max=keep)
    none = torch.arange(keep, device="cuda") >= kept_len[:, None]
    kept = order.masked_fill(none[:, None], 1 << 40).sort(-1)[0]
    kept = kept.masked_fill(none[:, None], -1)
    b, h, i = (kept >= 0).nonzero(as_tuple=True)
    src = kept[b, h, i]
    page, slot = table[b, src // st["page"]], src % st["page"]
    to_page, to_slot = st["table_out"].long()[b, i // st["page"]], i % st["page"]
    for name in ("k_cache", "v_cache", "k_scale", "v_scale", "weights"):
        if st[name] is not None:
            st[name][to_page, h, to_slot] = st[name][page, h, slot]
    return kept_len.to(torch.int32), kept.to(torch.int32)


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
        if op == "rotate":
            norm = dict(positions=st["positions"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                        interleaved=st["interleaved"])
            q, k = fa.norm_rotate(st["q"], st["k"], st["inv_freq"], **norm)
            if not st["backward"]:
                return q, k
            return (q, k) + fa.norm_rotate_backward(st["q"], st["k"], st["dq"], st["dk"], st["inv_freq"], **norm)
        cache = (st["k_cache"], st["v_cache"], st["table"], st["kv_len"])
        scales = dict(k_scale=st["k_scale"], v_scale=st["v_scale"])
        if op == "append":
            q = fa.qkv_append(st["q"], st["k_new"], st["v_new"], *cache, st["q_indptr"], st["inv_freq"],
                              q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS, **scales)
            return dict(_cache_out(st), q=q)
        if op == "accumulate":
            fa.kv_accumulate(st["weights"], st["q"], st["lse"], *cache, st["q_indptr"], st["max_new"],
                             window=st["window"] or None, sinks=st["sinks"], **scales)
            return st["weights"]
        kept_len, kept = fa.kv_evict(st["weights"], *cache, st["keep"], sinks=st["sinks"], recent=st["recent"],
                                     table_out=st["table_out"], **scales)
        return dict(_cache_out(st), weights=st["weights"], kept_len=kept_len, kept=kept)
    if op == "rotate":
        return _plain_rotate(st)
    if op == "append":
        q = _plain_append(st)
        return dict(_cache_out(st), q=q)
    if op == "accumulate":
        return _plain_accumulate(st)
    kept_len, kept = _plain_evict(st)
    return dict(_cache_out(st), weights=st["weights"], kept_len=kept_len, kept=kept)


# --------------------------------------------------------------------- the definitions in 64 bits

def _exact_vector(x, weight, pos, st, interleaved):
    """Normed and rotated vectors x [..., d] at the positions pos (broadcast over x's leading axes), as complex turns."""
    x = x.double()
    y = x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / st["d"] + EPS) * weight.double()
    return _exact_turn(y, pos, st, interleaved, 1.0)


def _exact_turn(y, pos, st, interleaved, sign):
    rot = st["rot"]
    turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), sign * pos.double().unsqueeze(-1) * st["inv_freq"])
    head = y[..., :rot]
    pairs = head.reshape(*head.shape[:-1], rot // 2, 2) if interleaved else \
        head.reshape(*head.shape[:-1], 2, rot // 2).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z if interleaved else z.transpose(-1, -2)
    out = y.clone()
    out[..., :rot] = z.reshape(head.shape)
    return out


def _exact_rotate(st):
    pos, il = st["positions"], st["interleaved"]
    out = [_exact_vector(st[x], st[x + "_weight"], pos, st, il) for x in ("q", "k")]
    if not st["backward"]:
        return tuple(out)
    dxs, dws = [], []
    for x in ("q", "k"):
        dy = _exact_turn(st["d" + x].double(), pos, st, il, -1.0)
        v, w = st[x].double(), st[x + "_weight"].double()
        ms = torch.sum(v * v, -1, keepdim=True) / st["d"] + EPS
        dws.append(torch.einsum("bhnd,bhnd->d", dy, v / torch.sqrt(ms)))
        g = dy * w
        dxs.append(g / torch.sqrt(ms) - v * torch.sum(v * g, -1, keepdim=True) / (st["d"] * ms * torch.sqrt(ms)))
    return tuple(out + dxs + dws)


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
    new, kv = _lengths(st)
    pos = torch.cat([torch.arange(m - n, m, device="cuda") for n, m in zip(new, kv)])
    page = torch.cat([st["table"][b].long()[torch.arange(m - n, m, device="cuda") // st["page"]]
                      for b, (n, m) in enumerate(zip(new, kv))])
    slot = pos % st["page"]
    out = {"q": _exact_vector(st["q"], st["q_weight"], pos[:, None], st, False)}
    rows = {"k": _exact_vector(st["k_new"], st["k_weight"], pos[:, None], st, False), "v": st["v_new"].double()}
    for name, x in rows.items():
        cache = st[name + "_cache"]
        if st["k_scale"] is None:
            out[name] = cache.double()
            out[name][page, :, slot] = x
        else:
            out[name], out[name + "_scale"] = cache.view(torch.float8_e4m3fn).double(), st[name + "_scale"].double()
            out[name][page, :, slot], out[name + "_scale"][page, :, slot] = _exact_codes(x)
    return out


def _exact_accumulate(st):
    new, kv = _lengths(st)
    hkv, d, group, page = st["hkv"], st["d"], st["hq"] // st["hkv"], st["page"]
    out = st["weights"].double()
    row = 0
    for b, (n, m) in enumerate(zip(new, kv)):
        pages = st["table"][b, : -(-m // page)].long()
        k = st["k_cache"][pages]
        k = k.double() if st["k_scale"] is None else \
            k.view(torch.float8_e4m3fn).double() * st["k_scale"][pages].double().unsqueeze(-1)
        k = k.transpose(0, 1).reshape(hkv, -1, d)[:, :m]
        keys = torch.arange(m, device="cuda")
        total = torch.zeros((hkv, m), device="cuda", dtype=torch.float64)
        for r in range(0, n, 128):
            end = min(n, r + 128)
            gap = torch.arange(m - n + r, m - n + end, device="cuda")[:, None] - keys
            hidden = gap < 0
            if st["window"]:
                hidden = hidden | ((gap >= st["window"]) & (keys >= st["sinks"]))
            q = st["q"][row + r:row + end].double().view(end - r, hkv, group, d)
            logits = torch.einsum("thgd,hkd->thgk", q, k) / math.sqrt(d)
            p = torch.exp(logits - st["lse"][row + r:row + end].double().view(end - r, hkv, group, 1))
            total += p.masked_fill(hidden[:, None, None], 0.0).sum((0, 2))
        where = st["table"][b].long()[keys // page]
        total[:, : m - n] += out[where[: m - n], :, keys[: m - n] % page].transpose(0, 1)
        out[where, :, keys % page] = total.transpose(0, 1)
        row += n
    return out


def _exact_evict(st):
    kv, page, keep, sinks, recent = _lengths(st)[1], st["page"], st["keep"], st["sinks"], st["recent"]
    out = _cache_out(st)
    out["weights"] = st["weights"]
    out = {name: x.double() for name, x in out.items()}
    kept = torch.full((st["batch"], st["hkv"], keep), -1, device="cuda", dtype=torch.int32)
    for b, n in enumerate(kv):
        at = torch.arange(n, device="cuda")
        pages = st["table"][b].long()
        w = st["weights"][pages[at // page], :, at % page]
        for h in range(st["hkv"]):
            chosen = at
            if n > keep:
                middle = w[sinks:n - recent, h]
                ranked = torch.argsort(middle, descending=True, stable=True)[: keep - sinks - recent] + sinks
                chosen = torch.cat((at[:sinks], ranked.sort()[0], at[n - recent:]))
            m = len(chosen)
            kept[b, h, :m] = chosen
            to = at[:m]
            to_page = st["table_out"][b].long()[to // page]
            for x in out.values():
                x[to_page, h, to % page] = x[pages[chosen // page], h, chosen % page]
    return dict(out, kept_len=None, kept=None)


def exact(case, seed):
    st = prepare(case, seed)
    return {"rotate": _exact_rotate, "append": _exact_append, "accumulate": _exact_accumulate,
            "evict": _exact_evict}[case["op"]](st)
