"""Accumulated attention weights (fa_kv_accumulate) against 64 bits."""
import ctypes
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding, build
from tests import _paged as P
from tests import _weights as W
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def bits(x):
    return x.contiguous().view(torch.int32).cpu()


def check(c, pool, rows, q, lse, new, scale, window=None, sinks=0, **kw):
    """One call, every weight of the pool looked at."""
    wd = pool.cuda()
    got = binding.kv_accumulate(wd, q.cuda(), lse.cuda(), c.k, c.v, c.table, c.kv_len, P.indptr(new), max(new + [1]), k_scale=c.ks,
                                v_scale=c.vs, scale=scale, window=window, sinks=sinks, **kw)
    binding.device_status()
    assert got is wd
    got = got.cpu()
    same = got.view(torch.int32) == pool.view(torch.int32)
    for b, (want, tol) in W.reference(c, rows, q, lse, new, scale, window, sinks).items():
        x = W.take(c, got, b).double()
        off = (x - want).abs()
        assert (off <= tol).all(), (b, float((off / tol).max()), x[off > tol][:4], want[off > tol][:4])
        W.put(c, same, b, torch.ones((c.hkv, c.lens[b]), dtype=torch.bool))
    assert same.all()            # nothing else was written
    return got


CASES = [  # lens, new, hq, hkv, d, page, window, sinks
    ([1], [1], 1, 1, 64, 16, None, 0), ([4100], [1], 32, 8, 128, 64, None, 0),
    ([5, 128, 129, 700, 1, 256, 257], [1] * 7, 8, 2, 128, 64, None, 0), ([90, 300], [2, 5], 7, 1, 64, 32, None, 0),
    ([40, 9, 0, 700], [3, 0, 0, 1], 16, 1, 128, 256, None, 0), ([3, 600], [5, 7], 6, 3, 64, 16, None, 0),
    ([1500], [300], 8, 2, 128, 128, None, 0), ([257, 1000, 64], [257, 100, 1], 28, 4, 64, 16, None, 0),
    ([900, 2000], [400, 3], 12, 12, 128, 64, None, 0), ([130], [130], 128, 1, 64, 64, None, 0), ([700], [9], 100, 2, 128, 32, None, 0),
    ([2100, 300], [2100, 70], 4, 1, 128, 64, None, 0), ([1030], [1030], 7, 1, 64, 16, 200, 3), ([5000], [600], 6, 1, 64, 64, None, 0),
    ([3000], [1], 8, 2, 64, 64, 500, 4), ([3000, 40], [200, 40], 4, 4, 64, 16, 300, 131), ([1200], [700], 3, 1, 128, 64, 1, 0),
    ([2000, 900], [1, 900], 14, 2, 128, 256, 129, 1), ([800], [60], 5, 1, 64, 128, 4096, 2), ([2 ** 11], [16], 4, 1, 128, 64, 17, 600),
]


@pytest.mark.parametrize("lens,new,hq,hkv,d,page,window,sinks", CASES)
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_accumulate(lens, new, hq, hkv, d, page, window, sinks, fmt):
    c = P.make(lens, hkv, d, page, fmt, seed=len(lens) + hq, combined=hkv == 2)
    g = torch.Generator().manual_seed(hq)
    T = sum(new)
    q = (torch.randn((T + 2, hq, d), generator=g) * 1.5).to(torch.bfloat16)
    q[T:] = math.nan             # rows behind the last sequence
    scale = 1 / math.sqrt(d)
    lse = torch.full((T + 2, hq), math.nan)
    lse[:T] = W.log_sum_exps(c, q[:T], new, scale, window, sinks)
    pool, rows = W.make(c, seed=hq)
    check(c, pool, rows, q, lse, new, scale, window, sinks)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_with_the_attention_calls_own_lse(fmt):
    # the weights that one step hands out sum to the number of query heads for each token
    lens, new, hq, hkv, d = [700, 33, 2100], [1, 5, 130], 8, 2, 128
    c = P.make(lens, hkv, d, 64, fmt, seed=4)
    q = torch.randn((sum(new), hq, d), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    ip = P.indptr(new)
    _, lse = binding.forward_paged(q, c.k, c.v, c.table, c.kv_len, ip, max(new), k_scale=c.ks, v_scale=c.vs)
    w = torch.zeros((c.P, hkv, 64), device="cuda")
    binding.kv_accumulate(w, q, lse, c.k, c.v, c.table, c.kv_len, ip, max(new), k_scale=c.ks, v_scale=c.vs)
    binding.device_status()
    for b, n in enumerate(new):
        total = W.take(c, w.cpu(), b).double().sum()
        assert abs(total - n * hq) <= 1e-4 * n * hq      # the attention's log-sum-exp is within 1e-4
    # a second time the old tokens' keys have the sum twice, the new ones' once
    before = w.clone()
    binding.kv_accumulate(w, q, lse, c.k, c.v, c.table, c.kv_len, ip, max(new), k_scale=c.ks, v_scale=c.vs)
    for b, n in enumerate(new):
        x, y = W.take(c, before.cpu(), b), W.take(c, w.cpu(), b)
        assert torch.equal(y[:, lens[b] - n:], x[:, lens[b] - n:]) and torch.equal(y[:, : lens[b] - n], 2 * x[:, : lens[b] - n])


def test_large_and_small_queries_over_e4m3():
    # entries of q over 2^20 and heads over 2^60 apart; keys whose scales differ by 2^40
    lens, new, hq, hkv, d = [600], [3], 4, 1, 64
    c = P.make(lens, hkv, d, 16, "e4m3", seed=7)
    g = torch.Generator().manual_seed(7)
    t = torch.arange(600)
    shift = torch.randint(-20, 21, (600,), generator=g)
    pg, slot = c.table[0].cpu().long()[t // 16], t % 16
    c.ks[pg, 0, slot] = c.ks[pg, 0, slot].cpu().mul(torch.exp2(shift.float())).cuda()
    c.values[0][0] = c.values[0][0] * torch.exp2(shift.double())[None, :, None]
    q = torch.randn((3, hq, d), generator=g) * torch.exp2(torch.randint(-20, 1, (3, hq, d), generator=g).float())
    q = (q * torch.exp2(torch.tensor([-30.0, 0.0, 3.0, 30.0]))[None, :, None] * 2.0 ** -12).to(torch.bfloat16)
    q[0, 1] = 0
    scale = 2.0 ** -4
    lse = W.log_sum_exps(c, q, new, scale)
    pool, rows = W.make(c, seed=7)
    # the largest scores are far past 2^10 here: the bound grows with them; every head's own sum still has to be right
    ref = W.reference(c, rows, q, lse, new, scale)[0]
    wd = pool.cuda()
    binding.kv_accumulate(wd, q.cuda(), lse.cuda(), c.k, c.v, c.table, c.kv_len, P.indptr(new), 3, k_scale=c.ks, v_scale=c.vs, scale=scale)
    binding.device_status()
    off = (W.take(c, wd.cpu(), 0).double() - ref[0]).abs()
    assert (off <= ref[1]).all(), float((off / ref[1]).max())


@pytest.mark.parametrize("new,hq,hkv", [([1, 3], 4, 1), ([2, 7], 8, 2), ([1, 40], 2, 2)])
def test_keys_and_queries_near_the_ends_of_the_range(new, hq, hkv):
    # keys past 2^110 with queries as small, whose products are ordinary; and the other way round
    for up in (110, -110):
        c = P.make([300, 70], hkv, 128, 16, "e4m3", seed=11)
        c.ks.mul_(2.0 ** up)
        c.values = [(k * 2.0 ** up, v) for k, v in c.values]
        q = torch.randn((sum(new), hq, 128), generator=torch.Generator().manual_seed(11)).mul(2.0 ** -up).to(torch.bfloat16)
        lse = W.log_sum_exps(c, q, new, 0.125)
        pool, rows = W.make(c, seed=11)
        check(c, pool, rows, q, lse, new, 0.125)


def test_special_values():
    # a NaN key, a NaN query, a lse of -inf and +inf: only what they reach
    lens, new, hq, hkv, d = [300, 300], [2, 1], 2, 1, 64
    for fmt in ("bf16", "e4m3"):
        c = P.make(lens, hkv, d, 16, fmt, seed=8)
        q = torch.randn((3, hq, d), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
        lse = W.log_sum_exps(c, q, new, 0.125)
        lse[0, 0], lse[1, 1] = -math.inf, math.inf
        pool, rows = W.make(c, seed=8)
        ref = W.reference(c, rows, q, lse, new, 0.125)
        page, slot = int(c.table[0, 3]), 5
        if fmt == "bf16":
            c.k[page, 0, slot, 7] = math.nan
        else:
            c.ks[page, 0, slot] = math.nan
        q[2, 1, 3] = math.nan
        wd = pool.cuda()
        binding.kv_accumulate(wd, q.cuda(), lse.cuda(), c.k, c.v, c.table, c.kv_len, P.indptr(new), 2, k_scale=c.ks, v_scale=c.vs)
        binding.device_status()
        a, b = W.take(c, wd.cpu(), 0)[0].double(), W.take(c, wd.cpu(), 1)[0]
        rest = torch.arange(300) != 53
        assert ((a - ref[0][0][0]).abs() <= ref[0][1][0])[rest].all() and torch.isnan(a[53])
        assert torch.isnan(b).all()


def test_the_same_bits_in_every_call_and_from_a_graph():
    lens, new, hq, hkv, d = [5000, 300, 1], [700, 2, 1], 8, 2, 128
    for fmt in ("bf16", "e4m3"):
        c = P.make(lens, hkv, d, 64, fmt, seed=9)
        q = torch.randn((sum(new), hq, d), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
        ip, start = P.indptr(new), W.make(c, seed=9)[0].cuda()
        _, lse = binding.forward_paged(q, c.k, c.v, c.table, c.kv_len, ip, 700, k_scale=c.ks, v_scale=c.vs)
        w = start.clone()
        call = lambda **kw: binding.kv_accumulate(w, q, lse, c.k, c.v, c.table, c.kv_len, ip, 700, k_scale=c.ks, v_scale=c.vs, **kw)
        call()
        want = bits(w)
        side = torch.cuda.Stream()
        for _ in range(3):
            w.copy_(start)
            side.wait_stream(torch.cuda.current_stream())
            call(stream=side)
            torch.cuda.current_stream().wait_stream(side)
            assert torch.equal(bits(w), want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        w.copy_(start)
        graph.replay()
        assert torch.equal(bits(w), want)
        # shorter sequences and fewer tokens: the captured call follows
        c.kv_len.copy_(torch.tensor([4000, 300, 0], dtype=torch.int32))
        ip.copy_(torch.tensor([0, 5, 5, 5], dtype=torch.int32))
        w.copy_(start)
        graph.replay()
        got = bits(w)
        w.copy_(start)
        call()
        assert torch.equal(got, bits(w)) and not torch.equal(got, want)
        binding.device_status()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_bad_entries_are_reported_and_skipped(fmt):
    lens, new, hq, hkv, d = [40, 400, 40], [1, 1, 1], 4, 2, 64
    q = torch.randn((3, hq, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    for what in ("page", "negative", "length", "rows", "indptr"):
        c = P.make(lens, hkv, d, 16, fmt, seed=5)
        pool = W.make(c, seed=5)[0]
        lse = W.log_sum_exps(c, q.cpu(), new, 0.125).cuda()
        good = pool.cuda()
        call = lambda w, ip, m=1: binding.kv_accumulate(w, q, lse, c.k, c.v, c.table, c.kv_len, ip, m, k_scale=c.ks, v_scale=c.vs)
        call(good, P.indptr(new))
        binding.device_status()
        ip, own = P.indptr(new), c.table[1, :25].long().tolist()
        if what == "page":
            c.table[1, 3] = c.P + 5
        elif what == "negative":
            c.table[1, 3] = -2 ** 31
        elif what == "length":
            c.kv_len[1] = 2 ** 31 - 1
            c.table[1, 25:] = c.table[1, 0]
        elif what == "rows":
            ip = torch.tensor([0, 1, 2, 9], dtype=torch.int32, device="cuda")
            own = c.table[2, :3].long().tolist()
        else:
            ip = torch.tensor([0, 1, 0, 1], dtype=torch.int32, device="cuda")
            own = c.table[1, :25].long().tolist() + c.table[2, :3].long().tolist()
        w = pool.cuda()
        binding.fa_device_report_read()
        call(w, ip)
        assert binding.fa_device_report_read()[0] == binding.FA_ERR_DEVICE_BOUNDS, what
        rest = [i for i in range(c.P) if i not in own]
        assert torch.equal(bits(w[rest]), bits(good[rest])), what
        # one sequence with more new tokens than max_q
    ip = torch.tensor([0, 3, 3, 3], dtype=torch.int32, device="cuda")
    call(pool.cuda(), ip, 2)
    assert binding.fa_device_report_read()[0] == binding.FA_ERR_DEVICE_BOUNDS


def test_views_and_refusals():
    lens, new, hq, hkv, d = [90, 50], [3, 1], 4, 2, 64
    c = P.make(lens, hkv, d, 16, "bf16", seed=6)
    g = torch.Generator().manual_seed(6)
    rows = torch.randn((4, hq + 4, d), generator=g).to(torch.bfloat16)
    q = rows[:, :hq]             # a slice of a projection
    lse = W.log_sum_exps(c, q, new, 0.125)
    pool, start = W.make(c, seed=6)
    wide = torch.full((c.P, 3, hkv, 16), 7.0).cuda()     # pages of a larger buffer
    wide[:, 1] = pool.cuda()
    w = wide[:, 1]
    args = (c.k, c.v, c.table, c.kv_len, P.indptr(new), 3)
    binding.kv_accumulate(w, rows.cuda()[:, :hq], lse.cuda(), *args, scale=0.125)
    for b, (want, tol) in W.reference(c, start, q, lse, new, 0.125).items():
        assert ((W.take(c, w.cpu(), b).double() - want).abs() <= tol).all()
    assert (wide[:, 0] == 7).all() and (wide[:, 2] == 7).all()
    qd, ld, ok = q.cuda(), lse.cuda(), pool.cuda()
    for bad in (lambda: binding.kv_accumulate(ok.double(), qd, ld, *args), lambda: binding.kv_accumulate(ok[:, :1], qd, ld, *args),
                lambda: binding.kv_accumulate(ok.transpose(1, 2).contiguous().transpose(1, 2), qd, ld, *args),
                lambda: binding.kv_accumulate(ok, qd, ld[:2], *args), lambda: binding.kv_accumulate(ok, qd, ld.double(), *args),
                lambda: binding.kv_accumulate(ok, qd[..., :32], ld, *args), lambda: binding.kv_accumulate(ok, qd, ld, *args, sinks=3),
                lambda: binding.kv_accumulate(ok, qd, ld, *args, window=0), lambda: binding.kv_accumulate(ok.cpu(), qd, ld, *args)):
        with pytest.raises(ValueError):
            bad()
    assert binding.kv_accumulate(ok, qd[:0], ld[:0], c.k, c.v, c.table, c.kv_len, P.indptr([0, 0]), 1) is ok


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("most", [1, 40])
def test_more_sequences_than_threads(fmt, most):
    # 900 of them, some without keys or without new tokens; one with a chunk where most = 40
    g = torch.Generator().manual_seed(most)
    lens = torch.randint(0, 20, (900,), generator=g).tolist()
    new = [min(n, 1) if i % 7 else 0 for i, n in enumerate(lens)]
    lens[500], new[500] = 600, most
    c = P.make(lens, 1, 64, 16, fmt, seed=most)
    q = torch.randn((sum(new), 4, 64), generator=g).to(torch.bfloat16)
    lse = W.log_sum_exps(c, q, new, 0.125)
    pool, rows = W.make(c, seed=1)
    check(c, pool, rows, q, lse, new, 0.125)


def test_a_program_of_captured_steps():
    # two calls captured one behind the other share a workspace, as a stream's calls do
    c = P.make([2000, 50], 2, 64, 32, "e4m3", seed=12)
    q = torch.randn((2, 8, 64), generator=torch.Generator().manual_seed(12)).to(torch.bfloat16).cuda()
    lse = W.log_sum_exps(c, q.cpu(), [1, 1], 0.125).cuda()
    ws = torch.empty(binding.fa_kv_accumulate_workspace_size(2, 1, 8, 2, 64, binding.FA_KV_E4M3), device="cuda", dtype=torch.uint8)
    a, ip = W.make(c, seed=1)[0].cuda(), P.indptr([1, 1])
    b = a.clone()
    call = lambda w, x, **kw: binding.kv_accumulate(w, x, lse, c.k, c.v, c.table, c.kv_len, ip, 1, k_scale=c.ks, v_scale=c.vs, **kw)
    q2 = q.flip(1).contiguous()
    call(b, q)
    call(b, q2)
    graph, start = torch.cuda.CUDAGraph(), a.clone()
    with torch.cuda.graph(graph):
        call(a, q, workspace=ws)
        call(a, q2, workspace=ws)
    for _ in range(2):
        a.copy_(start)
        graph.replay()
    assert torch.equal(bits(a), bits(b))
    with pytest.raises(binding.FAError):
        call(a, q, workspace=ws[:-256])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 200, 2, 30]])
def test_a_wait_that_runs_out_is_reported_and_nothing_else_breaks(monkeypatch, fmt, new):
    # test build with an injected stall (100 ms limit)
    L = ctypes.CDLL(build.build(testhooks=True))
    binding.load()
    L.fa_kv_accumulate.argtypes = binding.load().fa_kv_accumulate.argtypes
    L.fa_device_status.argtypes = [ctypes.c_void_p]
    lens, hq, d = [700, 3000, 90, 64][: len(new)], 8, 64
    c = P.make(lens, 2, d, 32, fmt, seed=2)
    q = torch.randn((sum(new), hq, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    lse, ip = W.log_sum_exps(c, q, new, 0.125), P.indptr(new)
    pool, rows = W.make(c, seed=2)
    kv = binding._paged(c.k, c.v, c.table, c.kv_len, c.ks, c.vs)
    qd, ld = q.cuda(), lse.cuda()
    n = binding.fa_kv_accumulate_workspace_size(sum(new), max(new), hq, 2, d, kv.dtype)
    ws = torch.zeros((-(-n // 256) * 256 + 512,), device="cuda", dtype=torch.uint8)
    stream = torch.cuda.current_stream().cuda_stream

    def call(w):
        assert L.fa_kv_accumulate(kv, w.data_ptr(), w.stride(0), qd.data_ptr(), hq * d, ld.data_ptr(), ip.data_ptr(), sum(new), max(new), hq,
                                  0, 0, 0.125, ws.data_ptr(), n, stream) == binding.FA_OK
        return L.fa_device_status(stream)

    w = pool.cuda()
    monkeypatch.setenv("FA_TEST_INJECT_STALL", "1")
    assert call(w) == binding.FA_ERR_TIMEOUT
    assert (ws[n:] == 0).all()
    monkeypatch.setenv("FA_TEST_INJECT_STALL", "0")
    w = pool.cuda()
    assert call(w) == binding.FA_OK
    for b, (want, tol) in W.reference(c, rows, q, lse, new, 0.125).items():
        assert ((W.take(c, w.cpu(), b).double() - want).abs() <= tol).all()
