"""Eviction by accumulated weight (fa_kv_evict), bit for bit, and a run of the serving calls together."""
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _masked as M
from tests import _paged as P
from tests import _rotate as R
from tests import _weights as W
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def bits(x):
    return x.contiguous().view(torch.uint8).cpu()


def pools(c, w):
    return [x for x in (c.k, c.v, c.ks, c.vs, w) if x is not None]


def free_table(c, keep, extra=1):
    """A table of the pages that no sequence has, and how many keys of each sequence it holds."""
    used = {int(c.table[b, i]) for b, n in enumerate(c.lens) for i in range(-(-n // c.page))}
    free = [p for p in range(c.P) if p not in used]
    table = torch.full((len(c.lens), -(-keep // c.page) + extra), 2 ** 30, dtype=torch.int32)
    for b, n in enumerate(c.lens):
        for i in range(-(-min(n, keep) // c.page)):
            table[b, i] = free.pop()
    return table


def expected(c, w, table_out, keep, sinks, recent):
    """(pools after the call, kept_len, kept): on the CPU."""
    before = [x.cpu().clone() for x in pools(c, w)]
    after = [x.clone() for x in before]
    kept = torch.full((len(c.lens), c.hkv, keep), -1, dtype=torch.int32)
    table, to_table = c.table.cpu().long(), table_out.cpu().long()
    for b, n in enumerate(c.lens):
        rows = W.take(c, before[-1], b)
        for h in range(c.hkv):
            src = W.chosen(rows[h], keep, sinks, recent)
            m = len(src)
            kept[b, h, :m] = src.to(torch.int32)
            to = torch.arange(m)
            for x, y in zip(before, after):
                y[to_table[b, to // c.page], h, to % c.page] = x[table[b, src // c.page], h, src % c.page]
    return after, torch.tensor([min(n, keep) for n in c.lens], dtype=torch.int32), kept


CASES = [  # lens, hkv, d, page, keep, sinks, recent
    ([1], 1, 64, 16, 1, 0, 0), ([600], 8, 128, 64, 200, 4, 30), ([5, 0, 64, 65, 700, 1], 2, 64, 16, 64, 0, 0),
    ([300, 2000, 40], 3, 128, 32, 100, 100, 0), ([513, 512, 511], 1, 64, 256, 511, 0, 511), ([900], 5, 128, 128, 2, 1, 1),
    ([4500, 30], 2, 64, 64, 1025, 3, 7), ([700, 701], 1, 128, 16, 700, 0, 1), ([1200], 4, 64, 32, 3000, 10, 20), ([130, 70], 20, 64, 16, 33, 0, 33),
]


@pytest.mark.parametrize("lens,hkv,d,page,keep,sinks,recent", CASES)
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_evict(lens, hkv, d, page, keep, sinks, recent, fmt, in_place, kind):
    spare = 3 + sum(-(-min(n, keep) // page) for n in lens)
    c = P.make(lens, hkv, d, page, fmt, seed=keep, spare=spare, combined=hkv == 2)
    w = W.make(c, seed=keep, std=3.0)[0]
    if kind == "ties":           # few values: zeros of both signs, infinities, NaN, negative ones
        few = torch.tensor([0.0, -0.0, 1.0, 1.0, 1.0, 2.0, math.inf, -math.inf, math.nan, -math.nan, -1.5, 1e-42, 0.0])
        w = few[torch.randint(0, len(few), w.shape, generator=torch.Generator().manual_seed(keep))]
    w = w.cuda()
    table_out = c.table if in_place else free_table(c, keep).cuda()
    after, want_len, want_kept = expected(c, w, table_out, keep, sinks, recent)
    kv_len = c.kv_len.clone()
    kept_len, kept = binding.kv_evict(w, c.k, c.v, c.table, c.kv_len, keep, sinks=sinks, recent=recent,
                                      table_out=None if in_place else table_out, k_scale=c.ks, v_scale=c.vs)
    binding.device_status()
    assert torch.equal(kept_len.cpu(), want_len) and torch.equal(c.kv_len, kv_len)
    assert torch.equal(kept.cpu(), want_kept)
    for x, y in zip(pools(c, w), after):   # the whole pools: what is not moved to stays as it was
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("in_place", [False, True])
def test_long_sequences(in_place):
    c = P.make([40000, 17, 9000], 2, 64, 64, "e4m3", seed=1, spare=400)
    w = W.make(c, seed=1, std=0.01)[0].cuda()   # nearly equal weights: the last bits decide
    table_out = c.table if in_place else free_table(c, 8192).cuda()
    after, want_len, want_kept = expected(c, w, table_out, 8192, 4, 1000)
    kept_len, kept = binding.kv_evict(w, c.k, c.v, c.table, c.kv_len, 8192, sinks=4, recent=1000, table_out=table_out, k_scale=c.ks, v_scale=c.vs)
    binding.device_status()
    assert torch.equal(kept_len.cpu(), want_len) and torch.equal(kept.cpu(), want_kept)
    for x, y in zip(pools(c, w), after):
        assert torch.equal(bits(x), bits(y))


def test_bad_entries_are_reported_and_skipped():
    lens, keep = [200, 200, 200], 50
    for what in ("page", "page_out", "length", "negative"):
        for in_place in (False, True):
            c = P.make(lens, 2, 64, 16, "bf16", seed=5, spare=20)
            w = W.make(c, seed=5)[0].cuda()
            table_out = c.table if in_place else free_table(c, keep).cuda()
            own = c.table[1, :13].long().tolist() + ([] if in_place else table_out[1, :4].long().tolist())
            after, _, _ = expected(c, w, table_out, keep, 0, 0)
            if what == "page" or (what == "page_out" and in_place):
                c.table[1, :13] = c.P + 7
            elif what == "page_out":
                table_out[1, 2] = -3
            else:
                c.kv_len[1] = 2 ** 31 - 1 if what == "length" else -1
            binding.fa_device_report_read()
            kept_len, kept = binding.kv_evict(w, c.k, c.v, c.table, c.kv_len, keep, table_out=None if in_place else table_out)
            assert binding.fa_device_report_read()[0] == binding.FA_ERR_DEVICE_BOUNDS, what
            rest = [i for i in range(c.P) if i not in own]
            for x, y in zip(pools(c, w), after):
                assert torch.equal(bits(x[rest]), bits(y[rest])), what


def test_graph_and_stream():
    c = P.make([300, 500], 2, 64, 16, "e4m3", seed=3, spare=30)
    w = W.make(c, seed=3)[0].cuda()
    table_out = free_table(c, 100).cuda()
    call = lambda **kw: binding.kv_evict(w, c.k, c.v, c.table, c.kv_len, 100, sinks=2, recent=10, table_out=table_out, k_scale=c.ks, v_scale=c.vs, **kw)
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    w.copy_(torch.rand(w.shape, device="cuda"))
    c.kv_len[0] = 90
    graph.replay()
    want = [x.clone() for x in got] + [x.clone() for x in pools(c, w)]
    again = call()
    for a, b in zip(list(again) + pools(c, w), want):
        assert torch.equal(bits(a), bits(b))
    binding.device_status()


def test_python_refusals():
    c = P.make([300], 2, 64, 16, "bf16", seed=3, spare=30)
    w = W.make(c, seed=3)[0].cuda()
    args = (c.k, c.v, c.table, c.kv_len)
    i32 = dict(device="cuda", dtype=torch.int32)
    for bad in (dict(keep=0), dict(keep=2 ** 31), dict(keep=9, table_out=torch.zeros((2, 4), **i32)), dict(keep=9, table_out=c.table.long()),
                dict(keep=9, kept_len=torch.zeros(2, **i32)), dict(keep=9, kept=torch.zeros((1, 2, 8), **i32))):
        with pytest.raises(ValueError):
            binding.kv_evict(w, *args, **bad)
    for bad in (dict(keep=9, sinks=5, recent=5), dict(keep=9, sinks=-1), dict(keep=100, table_out=torch.zeros((1, 6), **i32)),
                dict(keep=9, kept_len=c.kv_len)):
        with pytest.raises(binding.FAError):
            binding.kv_evict(w, *args, **bad)


@pytest.mark.parametrize("in_place", [False, True])
def test_many_sequences(in_place):
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 150, (400,), generator=g).tolist()
    c = P.make(lens, 1, 64, 16, "e4m3", seed=4, spare=3 + sum(-(-min(n, 60) // 16) for n in lens))
    w = W.make(c, seed=4)[0].cuda()
    table_out = c.table if in_place else free_table(c, 60).cuda()
    after, want_len, want_kept = expected(c, w, table_out, 60, 3, 20)
    kept_len, kept = binding.kv_evict(w, c.k, c.v, c.table, c.kv_len, 60, sinks=3, recent=20, table_out=table_out, k_scale=c.ks, v_scale=c.vs)
    binding.device_status()
    assert torch.equal(kept_len.cpu(), want_len) and torch.equal(kept.cpu(), want_kept)
    for x, y in zip(pools(c, w), after):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("fmt,d,in_place", [("e4m3", 128, False), ("e4m3", 64, False), ("bf16", 64, False), ("bf16", 128, False),
                                            ("e4m3", 64, True)])
def test_more_heads_of_sequences_than_run_at_once(fmt, d, in_place):
    # more than two (sequence, kv head) pairs for each SM, the longest past what is kept on chip
    lens = [700, 8900, 64, 0, 1, 65, 101, 32] + torch.randint(0, 150, (102,), generator=torch.Generator().manual_seed(d)).tolist()
    c = P.make(lens, 3, d, 32, fmt, seed=d, spare=3 + sum(-(-min(n, 100) // 32) for n in lens))
    w = W.make(c, seed=d)[0].cuda()
    table_out = c.table if in_place else free_table(c, 100).cuda()
    after, want_len, want_kept = expected(c, w, table_out, 100, 4, 33)
    kept_len, kept = binding.kv_evict(w, c.k, c.v, c.table, c.kv_len, 100, sinks=4, recent=33, table_out=table_out, k_scale=c.ks, v_scale=c.vs)
    binding.device_status()
    assert torch.equal(kept_len.cpu(), want_len) and torch.equal(kept.cpu(), want_kept)
    for x, y in zip(pools(c, w), after):
        assert torch.equal(bits(x), bits(y))


def test_source_pages_may_be_shared():
    # two sequences over the same pages, each moved to pages of its own
    c = P.make([200, 200], 2, 64, 16, "bf16", seed=6, spare=30)
    c.table[1] = c.table[0]
    w = W.make(c, seed=6)[0].cuda()
    table_out = free_table(c, 64).cuda()
    after, _, want_kept = expected(c, w, table_out, 64, 2, 10)
    kept_len, kept = binding.kv_evict(w, c.k, c.v, c.table, c.kv_len, 64, sinks=2, recent=10, table_out=table_out)
    binding.device_status()
    assert torch.equal(kept.cpu(), want_kept) and torch.equal(kept[0], kept[1])
    for x, y in zip(pools(c, w), after):
        assert torch.equal(bits(x), bits(y))


def test_serving_with_a_budget():
    """Prompt, decoding steps and evictions, each step through the calls that a program makes; the outputs of the last step
    against 64-bit attention over the keys that were kept, rotated at their own positions."""
    B, hq, hkv, d, page, keep = 2, 4, 2, 64, 16, 40
    g = torch.Generator().manual_seed(11)
    prompts, pages = [70, 33], 12
    P_all = 2 * B * pages
    dev = dict(device="cuda")
    k, v = (torch.full((P_all, hkv, page, d), math.nan, dtype=torch.bfloat16, **dev) for _ in range(2))
    w = torch.full((P_all, hkv, page), math.nan, **dev)
    tables = [torch.arange(i, i + B * pages, **dev, dtype=torch.int32).view(B, pages) for i in (0, B * pages)]
    f = R.frequencies(d)
    qw, kw = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    norm = dict(q_weight=qw.cuda(), k_weight=kw.cuda())
    held = [[[] for _ in range(hkv)] for _ in range(B)]          # (position, token) of each kept key
    tokens = [[] for _ in range(B)]                                # each token's projected row
    kv_len, position, new = torch.zeros(B, **dev, dtype=torch.int32), [0] * B, list(prompts)
    for step in range(30):
        T = sum(new)
        rows = torch.randn((T, hq + 2 * hkv, d), generator=g).to(torch.bfloat16)
        at = torch.cat([torch.arange(p, p + n) for p, n in zip(position, new)]).to(torch.int32)
        row = 0
        for b, n in enumerate(new):
            for i in range(n):
                for h in range(hkv):
                    held[b][h].append(len(tokens[b]))
                tokens[b].append((int(at[row]), rows[row]))
                row += 1
            position[b] += n
        ip, dr = P.indptr(new), rows.cuda()
        kv_len = kv_len + torch.tensor(new, **dev, dtype=torch.int32)
        cache = (k, v, tables[0], kv_len)
        q = binding.qkv_append(dr[:, :hq], dr[:, hq:hq + hkv], dr[:, hq + hkv:], *cache, ip, f.cuda(), positions=at.cuda(), **norm)
        o, lse = binding.forward_paged(q, *cache, ip, max(new))
        binding.kv_accumulate(w, q, lse, *cache, ip, max(new))
        if step == 29:
            break
        if step % 3 == 0:        # into the other pages, and back the next time
            kv_len, kept = binding.kv_evict(w, *cache, keep, sinks=2, recent=8, table_out=tables[1])
            tables.reverse()
        else:
            kv_len, kept = binding.kv_evict(w, *cache, keep, sinks=2, recent=8)
        for b in range(B):
            for h in range(hkv):
                idx = kept[b, h].cpu()
                idx = idx[idx >= 0].tolist()
                assert idx[:2] == [0, 1] and idx[-8:] == list(range(len(held[b][h]) - 8, len(held[b][h])))
                held[b][h] = [held[b][h][i] for i in idx]
        new = [1, 1] if step % 5 else [3, 1]
    binding.device_status()
    row = 0
    for b, n in enumerate(new):
        for h in range(hq):
            kh = h // (hq // hkv)
            rows_k = torch.stack([tokens[b][i][1][hq + kh] for i in held[b][kh]])
            pos_k = torch.tensor([tokens[b][i][0] for i in held[b][kh]])
            vals = torch.stack([tokens[b][i][1][hq + hkv + kh] for i in held[b][kh]])
            keys = R.forward(rows_k, pos_k, f, kw).z
            mine = [tokens[b][len(tokens[b]) - n + i] for i in range(n)]
            qs = R.forward(torch.stack([m[1][h] for m in mine]), torch.tensor([m[0] for m in mine]), f, qw).z
            m = len(held[b][kh])
            see = M.window_mask(torch.arange(m - n, m), torch.arange(m))
            r = M.forward(qs, keys, vals, see, d ** -0.5)
            # q and k were rounded to BF16: a score is off by 2 * 2^-8 sum |q k| scale at most, an output by that times
            # 2 sum p |v| (first order, and as much again for the rest)
            off = (2 * 2.0 ** -8 * (qs.abs() @ keys.abs().t()) * d ** -0.5).amax(-1, keepdim=True)
            tol = r["o_tol"] + 4 * off * (r["p"] @ vals.double().abs())
            M.assert_within("o", o[row:row + n, h], r["o"], tol)
        row += n
