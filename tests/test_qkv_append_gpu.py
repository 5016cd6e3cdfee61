"""Norm, rotation and the write into a paged cache in one call, against its parts and against 64 bits."""
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _paged as P
from tests import _rotate as R
from tests._parity import require_gpu
from tests.test_norm_rotate_gpu import near, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def bits(x):
    return x.contiguous().view(torch.uint8).cpu()


def places(c, new):
    """(page, slot, position) of the new tokens, on the CPU."""
    t = torch.cat([torch.arange(n - m, n) for n, m in zip(c.lens, new)])
    b = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    return c.table.cpu().long()[b, t // c.page], t % c.page, t


CASES = [  # hq, hkv, d, page, new, lens, rot, interleaved
    (1, 1, 64, 16, [1], [1], 64, False), (32, 8, 128, 64, [1] * 9, [5, 64, 65, 100, 1, 33, 700, 128, 12], 128, False),
    (7, 1, 64, 32, [40, 0, 200], [40, 9, 333], 48, True), (20, 5, 128, 256, [7, 129], [500, 129], 64, False),
    (40, 20, 64, 16, [3] * 40, list(range(3, 123, 3)), 0, False), (3, 3, 128, 128, [1] * 70, list(range(1, 71)), 128, True),
    (2, 1, 128, 64, [900, 1], [1000, 1], 112, False),
]


@pytest.mark.parametrize("hq,hkv,d,page,new,lens,rot,interleaved", CASES)
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_append(hq, hkv, d, page, new, lens, rot, interleaved, fmt):
    c = P.make(lens, hkv, d, page, fmt, seed=hq, combined=hkv == 5)
    g = torch.Generator().manual_seed(hq)
    T = sum(new)
    rows, q, k = (x[0] if i == 0 else x[0].transpose(0, 1) for i, x in enumerate(R.heads(1, T + 3, hq, hkv, d, g)))
    v = rows[:, hq + hkv:]
    w = weights(d, g)
    f = R.frequencies(rot)
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda(), eps=1e-5, interleaved=interleaved)
    dev = rows.cuda()
    out = torch.full((T + 3, hq, d), 3.0, device="cuda", dtype=torch.bfloat16)
    before = [x.clone() for x in (c.k, c.v, c.ks, c.vs) if x is not None]
    got = binding.qkv_append(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], c.k, c.v, c.table, c.kv_len, P.indptr(new),
                             f.cuda() if rot else None, k_scale=c.ks, v_scale=c.vs, out=out, **kw)
    binding.device_status()
    assert got is out and (out[T:] == 3).all()
    pg, slot, pos = places(c, new)
    # the parts: norm_rotate, then kv_append
    at = torch.zeros(T + 3, dtype=torch.int32)
    at[:T] = pos
    pq, pk = binding.norm_rotate(dev[None, :, :hq].transpose(1, 2), dev[None, :, hq:hq + hkv].transpose(1, 2),
                                 f.cuda() if rot else None, positions=at.cuda(), **kw)
    assert torch.equal(out[:T], pq[0].transpose(0, 1)[:T])
    after = [x.clone() for x in (c.k, c.v, c.ks, c.vs) if x is not None]
    for x, y in zip((c.k, c.v, c.ks, c.vs), before):
        x.copy_(y)
    binding.kv_append(pk[0].transpose(0, 1).contiguous(), dev[:, hq + hkv:].contiguous(), c.k, c.v, c.table, c.kv_len,
                      P.indptr(new), k_scale=c.ks, v_scale=c.vs)
    parts = [x for x in (c.k, c.v, c.ks, c.vs) if x is not None]
    for i, (a, b, old) in enumerate(zip(after, parts, before)):
        if fmt == "bf16" or i % 2:   # values, and BF16 keys: the same bits, in the whole pool
            assert torch.equal(bits(a), bits(b))
        else:                        # E4M3 keys are rounded once, from FP32: nothing else may have changed
            own = torch.zeros(a.shape[:3], dtype=torch.bool)
            own[pg, :, slot] = True
            assert torch.equal(bits(a)[~own.to(bool)] if a.dim() == 4 else bits(a.view(torch.uint8).view(*a.shape, 4))[~own],
                               bits(old)[~own] if a.dim() == 4 else bits(old.view(torch.uint8).view(*a.shape, 4))[~own])
    if fmt == "e4m3":
        kc, ks = after[0].cpu()[pg, :, slot], after[2].cpu()[pg, :, slot].double()
        x = rows[:T, hq:hq + hkv]
        r = R.forward(x, pos[:, None], f, w[1], 1e-5, interleaved)
        # half a step of E4M3 (2^-4 of the value, 2^-10 of the scale below its normal range) and the FP32 error
        fp32 = r.tol - R.BF16 * r.z.abs()
        near(kc.view(P.E4M3).double() * ks[..., None], r.z,
             2.0 ** -4 * (r.z.abs() + fp32) + 2.0 ** -10 * ks[..., None] + fp32)
        # the scale is the least power of two with max|z| <= 448 scale, unless max|z| is at a border
        top, slack = r.z.abs().amax(-1), fp32.amax(-1)
        assert (top - slack <= 448 * ks).all()
        assert ((top + slack > 224 * ks) | (ks == 2.0 ** -126) | (top == 0)).all()
        assert torch.equal(torch.frexp(ks)[0], torch.full_like(ks, 0.5))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_positions_that_differ_from_the_places(fmt):
    # a sequence whose cache was cut: its tokens keep their own positions
    lens, new, hq, hkv, d = [40, 300], [3, 50], 4, 2, 64
    c = P.make(lens, hkv, d, 16, fmt, seed=2)
    g = torch.Generator().manual_seed(2)
    rows, q, k = R.heads(1, 53, hq, hkv, d, g)
    f, pos = R.frequencies(d), torch.randint(0, 2 ** 31 - 1, (53,), generator=g).to(torch.int32)
    dev = rows[0].cuda()
    got = binding.qkv_append(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], c.k, c.v, c.table, c.kv_len, P.indptr(new), f.cuda(),
                             positions=pos.cuda(), k_scale=c.ks, v_scale=c.vs)
    r = R.forward(q[0], pos, f)
    near(got.transpose(0, 1), r.z, r.tol)
    kr, _ = binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr(lens), sum(lens), k_scale=c.ks, v_scale=c.vs)
    kr = torch.cat([kr[37:40], kr[40 + 250:]])
    r = R.forward(k[0], pos, f)
    tol = r.tol if fmt == "bf16" else 2.0 ** -4 * r.z.abs() + 2.0 ** -9 * r.z.abs().amax(-1, keepdim=True) * 2.0 ** -8 + r.tol
    near(kr.transpose(0, 1), r.z, tol)
    binding.device_status()


def test_without_norm_and_special_values():
    c = P.make([6], 1, 64, 16, "e4m3", seed=0)
    x = torch.zeros((6, 1, 64))
    x[0, 0, 3] = 3.3895313892515355e38
    x[1, 0, 1] = 450.0
    x[2, 0, 2] = math.nan
    x[3, 0, 2] = -math.inf
    x[4, 0, :2] = torch.tensor([1e-40, -9.2e-41])
    x = x.to(torch.bfloat16)
    binding.qkv_append(x.cuda(), x.cuda(), x.cuda(), c.k, c.v, c.table, c.kv_len, P.indptr([6]), None, norm=False, k_scale=c.ks, v_scale=c.vs)
    page = int(c.table[0, 0])
    codes, scale = P.quantize(x)
    for cache, s in ((c.k, c.ks), (c.v, c.vs)):   # without norm and rotation a key is written as a value is
        assert torch.equal(cache[page, 0, :6].cpu(), codes[:, 0])
        assert torch.equal(bits(s[page, 0, :6]), bits(scale[:, 0]))
    binding.device_status()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_bad_entries_are_reported_and_skipped(fmt):
    g = torch.Generator().manual_seed(1)
    rows, _, _ = R.heads(1, 9, 2, 2, 64, g)
    x = rows[0, :, :2].contiguous().cuda()
    f = R.frequencies(64).cuda()
    for what in ("page", "negative", "length", "short"):
        c, good = (P.make([40, 40, 40], 2, 64, 16, fmt, seed=5) for _ in range(2))
        if what == "page":
            c.table[1, 2] = c.P + 5
        elif what == "negative":
            c.table[1, 2] = -2 ** 31
        else:
            c.kv_len[1] = 2 ** 31 - 1 if what == "length" else 1
        binding.fa_device_report_read()
        a = binding.qkv_append(x, x, x, c.k, c.v, c.table, c.kv_len, P.indptr([3] * 3), f, k_scale=c.ks, v_scale=c.vs)
        assert binding.fa_device_report_read()[0] == binding.FA_ERR_DEVICE_BOUNDS
        b = binding.qkv_append(x, x, x, good.k, good.v, good.table, good.kv_len, P.indptr([3] * 3), f, k_scale=good.ks, v_scale=good.vs)
        binding.device_status()
        own = good.table[1, :3].long().tolist()
        rest = [i for i in range(c.P) if i not in own]
        assert torch.equal(bits(c.k[rest]), bits(good.k[rest])) and torch.equal(bits(c.v[rest]), bits(good.v[rest]))
        assert torch.equal(a[[0, 1, 2, 6, 7, 8]], b[[0, 1, 2, 6, 7, 8]])


def test_queries_in_place():
    lens = new = [70, 3, 200]
    c = P.make(lens, 2, 128, 64, "bf16", seed=3)
    g = torch.Generator().manual_seed(3)
    rows, _, _ = R.heads(1, 273, 8, 2, 128, g)
    q, k, v = (x.contiguous().cuda() for x in rows[0].split([8, 2, 2], 1))
    f = R.frequencies(128).cuda()
    call = lambda **kw: binding.qkv_append(q, k, v, c.k, c.v, c.table, c.kv_len, P.indptr(new), f, **kw)
    want = call()
    assert call(out=q) is q and torch.equal(q, want)


def test_graph_follows_lengths_and_tables():
    c = P.make([30, 60], 2, 128, 16, "e4m3", seed=9)
    g = torch.Generator().manual_seed(9)
    rows, _, _ = R.heads(1, 2, 4, 2, 128, g)
    dev, f, ip = rows[0].cuda(), R.frequencies(128).cuda(), P.indptr([1, 1])
    call = lambda: binding.qkv_append(dev[:, :4], dev[:, 4:6], dev[:, 6:], c.k, c.v, c.table, c.kv_len, ip, f, k_scale=c.ks, v_scale=c.vs)
    c.kv_len.sub_(1)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    c.kv_len.add_(1)
    graph.replay()
    got = [x.clone() for x in (out, c.k, c.v, c.ks, c.vs)]
    want = call()
    assert torch.equal(got[0], want)
    for a, b in zip(got[1:], (c.k, c.v, c.ks, c.vs)):
        assert torch.equal(bits(a), bits(b))
    binding.device_status()


def test_python_refusals():
    c = P.make([30], 2, 64, 16, "bf16", seed=9)
    x, f, ip = torch.zeros((3, 2, 64), device="cuda", dtype=torch.bfloat16), R.frequencies(64).cuda(), P.indptr([3])
    cache = (c.k, c.v, c.table, c.kv_len)
    for bad in (lambda: binding.qkv_append(x[:2], x, x, *cache, ip, f), lambda: binding.qkv_append(x, x, x[:2], *cache, ip, f),
                lambda: binding.qkv_append(x, x[:, :1], x, *cache, ip, f), lambda: binding.qkv_append(x, x, x, *cache, P.indptr([1, 2]), f),
                lambda: binding.qkv_append(x, x, x, *cache, ip, f, positions=ip), lambda: binding.qkv_append(x, x, x, *cache, ip, f, out=x[:2]),
                lambda: binding.qkv_append(x, x, x, *cache, ip, f, q_weight=torch.ones(64, device="cuda")),
                lambda: binding.qkv_append(x, x, x, *cache, ip, f, k_scale=c.k, v_scale=c.v)):
        with pytest.raises(ValueError):
            bad()
