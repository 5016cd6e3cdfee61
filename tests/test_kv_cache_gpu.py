"""Writing into paged caches (fa_kv_append) and reading them back (fa_kv_read), bit for bit."""
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _paged as P
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def bits(x):
    return x.contiguous().view(torch.uint8).cpu()


def place(c, pool, new, rows, w):
    """The pool [P, hkv, page, ...] (CPU) with `rows` [T, hkv, ...] written at the new tokens' slots."""
    at = 0
    for b, n in enumerate(new):
        t = torch.arange(c.lens[b] - n, c.lens[b])
        pg, slot = c.table[b].cpu().long()[t // c.page], t % c.page
        pool[pg, :, slot] = rows[at:at + n]
        at += n
    return pool


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,page,new,lens", [
    (1, 16, [1], [1]), (3, 16, [1, 1, 1], [16, 17, 300]), (8, 64, [40, 0, 200], [40, 9, 333]),
    (5, 256, [7, 129], [500, 129]), (20, 32, [3] * 40, list(range(3, 123, 3))), (2, 128, [1] * 70, list(range(1, 71)))])
def test_append(fmt, d, hkv, page, new, lens):
    c = P.make(lens, hkv, d, page, fmt, seed=hkv + d, combined=hkv == 5)
    g = torch.Generator().manual_seed(1)
    T = sum(new)
    x = (torch.randn((2, T + 3, hkv, d), generator=g) * torch.exp2(torch.randint(-20, 20, (2, T + 3, hkv, 1), generator=g).float())).to(torch.bfloat16)
    want = []
    for w, (pool, sc) in enumerate(((c.k, c.ks), (c.v, c.vs))):
        codes, s = P.quantize(x[w]) if fmt == "e4m3" else (x[w], None)
        want.append(place(c, pool.cpu().clone(), new, codes, w))
        if s is not None:
            want.append(place(c, sc.cpu().clone(), new, s, w))
    xd = x.cuda()
    binding.kv_append(xd[0], xd[1], c.k, c.v, c.table, c.kv_len, P.indptr(new), k_scale=c.ks, v_scale=c.vs)
    binding.device_status()
    got = [c.k, c.ks, c.v, c.vs] if fmt == "e4m3" else [c.k, c.v]
    for a, b in zip(got, want):     # the whole pools: nothing but the new slots has changed
        assert torch.equal(bits(a), bits(b))


def test_append_special_vectors():
    # zeros, a negative zero, subnormals, the largest values, borders of the scale rule, NaN and Inf
    d = 64
    rows = torch.zeros((12, 1, d))
    rows[1, 0, 5] = -0.0
    rows[2, 0, :3] = torch.tensor([1e-40, -3e-39, 9.2e-41])
    rows[3] = 3.3895313892515355e38
    rows[4, 0, 1] = 448.0
    rows[5, 0, 1] = 450.0
    rows[6, 0, :2] = torch.tensor([-1.75, 2.0 ** -9])
    rows[7, 0, :2] = torch.tensor([1.7578125, 1e-3])
    rows[8, 0, 3] = math.nan
    rows[9, 0, 63] = -math.inf
    rows[10, 0] = torch.linspace(-1, 1, d)
    rows[11, 0, 0] = 2.0 ** -126
    x = rows.to(torch.bfloat16)
    c = P.make([12], 1, d, 16, "e4m3", seed=0)
    binding.kv_append(x.cuda(), (-x).cuda(), c.k, c.v, c.table, c.kv_len, P.indptr([12]), k_scale=c.ks, v_scale=c.vs)
    k, v = binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr([12]), 12, k_scale=c.ks, v_scale=c.vs)
    binding.device_status()
    page = int(c.table[0, 0])
    codes, scale = P.quantize(x)
    assert torch.equal(c.k[page, 0, :12].cpu(), codes[:, 0])
    assert torch.equal(bits(c.ks[page, 0, :12]), bits(scale[:, 0]))
    want = (codes.view(P.E4M3).double() * scale.double()[..., None])
    # code * scale is a multiple of 2^-9 scale with 4 significant bits: exact in BF16 where that is at
    # least 2^-133, BF16's smallest step.  At scale = 2^-126 (row 2) the step is 2^-135, so the value
    # is rounded to BF16 once.
    exact = want.float().to(torch.bfloat16).double()
    assert torch.equal(exact[3:8], want[3:8]) and torch.equal(exact[10], want[10])
    for got, sign in ((k, 1), (v, -1)):
        fin = torch.isfinite(want)
        assert torch.equal(got.cpu().double()[fin], sign * exact[fin])
        assert torch.isnan(got.cpu()[8:10]).all() and fin[:8].all() and fin[10:].all()
    # half a step of E4M3 relative to the value, 2^-10 of the scale below its normal range
    off = (want - x.double()).abs()[torch.isfinite(x.double()) & torch.isfinite(want)]
    bound = torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * scale.double()[..., None])
    assert (off <= bound[torch.isfinite(x.double()) & torch.isfinite(want)]).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,page,lens", [(1, 16, [1]), (3, 32, [5, 0, 33, 700]), (8, 64, [64, 65, 1]), (20, 256, [300, 10])])
def test_read(fmt, d, hkv, page, lens):
    c = P.make(lens, hkv, d, page, fmt, seed=d, combined=hkv == 3)
    rows = sum(lens) + 5
    out = tuple(torch.full((rows, hkv, d), 3.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr(lens), rows, k_scale=c.ks, v_scale=c.vs, out=out)
    binding.device_status()
    for w in range(2):
        want = torch.cat([c.values[b][w].transpose(0, 1) for b in range(len(lens))])
        assert torch.equal(out[w][:sum(lens)].cpu().double(), want)
        assert (out[w][sum(lens):] == 3).all()
    # a prefix of each sequence, rows kept for more than a sequence has
    part = [n // 2 for n in lens]
    k, _ = binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr(part), sum(part), k_scale=c.ks, v_scale=c.vs)
    want = torch.cat([c.values[b][0].transpose(0, 1)[:n] for b, n in enumerate(part)])
    assert torch.equal(k.cpu().double(), want)
    wide = [n + 2 for n in lens]
    out[0].fill_(3.0)
    big = tuple(torch.full((sum(wide), hkv, d), 3.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr(wide), sum(wide), k_scale=c.ks, v_scale=c.vs, out=big)
    ends = P.indptr(wide).tolist()
    for b, n in enumerate(lens):
        assert (big[0][ends[b] + n:ends[b + 1]] == 3).all()
    binding.device_status()


def test_scales_that_are_no_powers_of_two_are_rounded_once():
    c = P.make([50], 2, 64, 16, "e4m3", seed=3)
    c.ks *= 1.37
    k, _ = binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr([50]), 50, k_scale=c.ks, v_scale=c.vs)
    t = torch.arange(50)
    pg = c.table[0].cpu().long()[t // 16]
    want = c.k.cpu()[pg, :, t % 16].view(P.E4M3).float() * c.ks.cpu()[pg, :, t % 16][..., None]
    assert torch.equal(k.cpu(), want.to(torch.bfloat16))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_bad_entries_are_reported_and_skipped(fmt):
    lens, new = [40, 40, 40], [3, 3, 3]
    g = torch.Generator().manual_seed(1)
    x = torch.randn((9, 2, 64), generator=g).to(torch.bfloat16).cuda()
    for what in ("page", "negative", "length", "short"):
        c = P.make(lens, 2, 64, 16, fmt, seed=5)
        good = P.make(lens, 2, 64, 16, fmt, seed=5)
        if what == "page":
            c.table[1, 2] = c.P + 5
        elif what == "negative":
            c.table[1, 2] = -2 ** 31
        elif what == "length":
            c.kv_len[1] = 2 ** 31 - 1
        else:
            c.kv_len[1] = 1            # two of its tokens would lie before the sequence
        binding.fa_device_report_read()
        binding.kv_append(x, x, c.k, c.v, c.table, c.kv_len, P.indptr(new), k_scale=c.ks, v_scale=c.vs)
        assert binding.fa_device_report_read()[0] == binding.FA_ERR_DEVICE_BOUNDS
        binding.kv_append(x, x, good.k, good.v, good.table, good.kv_len, P.indptr(new), k_scale=good.ks, v_scale=good.vs)
        own = good.table[1, :3].long()   # only sequence 1's pages may differ
        rest = [i for i in range(c.P) if i not in own.tolist()]
        assert torch.equal(bits(c.k[rest]), bits(good.k[rest])) and torch.equal(bits(c.v[rest]), bits(good.v[rest]))
        if what != "short":
            out = tuple(torch.full((120, 2, 64), 3.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
            binding.fa_device_report_read()
            binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr([40, 0, 40] if what == "length" else lens), 120,
                            k_scale=c.ks, v_scale=c.vs, out=out)
            rc = binding.fa_device_report_read()[0]
            assert rc == (binding.FA_OK if what == "length" else binding.FA_ERR_DEVICE_BOUNDS)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("hkv,d,page,lens", [(1, 64, 16, [39000, 1, 333]), (1, 128, 64, [20000, 4999]), (2, 64, 256, [10000]),
                                             (3, 128, 32, [2500, 77]), (40, 128, 16, [35, 2]), (130, 128, 16, [19]),
                                             (200, 64, 32, [3, 9])])
def test_append_and_read_back_at_any_number_of_heads(fmt, hkv, d, page, lens):
    # the tokens of a CTA depend on the heads and on the rows: 1 to 256
    c = P.make(lens, hkv, d, page, fmt, seed=3)
    T = sum(lens)
    g = torch.Generator().manual_seed(T)
    x = (torch.randn((2, T, hkv, d), generator=g) * torch.exp2(torch.randint(-9, 9, (2, T, hkv, 1), generator=g).float())).to(torch.bfloat16)
    k, v = x.cuda()
    ip = P.indptr(lens)
    binding.kv_append(k, v, c.k, c.v, c.table, c.kv_len, ip, k_scale=c.ks, v_scale=c.vs)
    got = binding.kv_read(c.k, c.v, c.table, c.kv_len, ip, T, k_scale=c.ks, v_scale=c.vs)
    binding.device_status()
    for a, b in zip(got, x):
        if fmt == "e4m3":
            codes, s = P.quantize(b)
            b = (codes.view(P.E4M3).double() * s.double()[..., None]).to(torch.bfloat16)   # exact
        assert torch.equal(a.cpu(), b)
