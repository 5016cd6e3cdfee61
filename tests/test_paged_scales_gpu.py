"""Attention over E4M3 caches whose vectors differ much in size, within the number formats' own bounds.

The bounds are those of the 64-bit reference, row by row and entry by entry (half a BF16 step of P~ and of
O).  A kernel whose P~ times scale is FP16 has 2^-11 of each weight, less than that half step, as long as
the weights that matter lie within FP16's normal range.
"""
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _masked as M
from tests import _paged as P
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def queries(new, hq, d, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((sum(new), hq, d), generator=g) * 1.5).to(torch.bfloat16)


def put(c, b, pos, which, x):
    """Make x [hkv, d] (BF16) the key (which = 0) or value (1) of position pos of sequence b."""
    codes, scale = P.quantize(x)
    page, slot = int(c.table[b, pos // c.page]), pos % c.page
    (c.v if which else c.k)[page, :, slot] = codes.cuda()
    (c.vs if which else c.ks)[page, :, slot] = scale.cuda()
    c.values[b][which][:, pos] = codes.view(P.E4M3).double() * scale.double()[:, None]


def check(c, new, q, window=None, sinks=0):
    o, lse = binding.forward_paged(q.cuda(), c.k, c.v, c.table, c.kv_len, P.indptr(new), max(new), k_scale=c.ks,
                                   v_scale=c.vs, window=window, sinks=sinks)
    binding.device_status()
    want, want_lse, tol = P.reference(c, q, new, 1 / math.sqrt(c.d), window, sinks)
    M.assert_within("o", o, want, tol)
    M.assert_lse(lse, want_lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,new", [(8, 1), (4, 2), (16, 1), (5, 3), (32, 1), (8, 4), (64, 1), (7, 9), (8, 40)])
@pytest.mark.parametrize("ratio", [10, 18, 20, 27, 40])
def test_a_large_value_of_no_weight(d, group, new, ratio):
    # the first key of each sequence has next to no weight (e^-60 or less) and a value 2^ratio larger than
    # the others: nothing of it may be seen in the output, for every form of the few-rows kernel (8, 16, 32
    # and 64 rows) and the chunk kernel (320)
    hkv = 2
    lens = [60, 130, 700, 1500]
    c = P.make(lens, hkv, d, 32, "e4m3", seed=group + ratio)
    q = queries([new] * len(lens), hkv * group, d, group)
    q[..., 0] = 8.0
    g = torch.Generator().manual_seed(ratio)
    for b in range(len(lens)):
        k0 = torch.zeros((hkv, d))
        k0[:, 0] = -90 * math.sqrt(d) / 8
        put(c, b, 0, 0, k0.to(torch.bfloat16))
        put(c, b, 0, 1, (torch.randn((hkv, d), generator=g) * 2.0 ** ratio).to(torch.bfloat16))
    check(c, [new] * len(lens), q)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,new", [(4, 2), (1, 5), (4, 4), (8, 4), (7, 5), (12, 5), (8, 40)])
@pytest.mark.parametrize("ratio", [16, 20, 26, 40])
def test_rows_that_do_not_see_a_large_value(d, group, new, ratio):
    # the last token's value is 2^ratio larger than all others: the tokens before it do not see it
    hkv = 2
    lens = [new, 65, 640, 2000]
    lens = [max(n, new) for n in lens]
    c = P.make(lens, hkv, d, 16, "e4m3", seed=group + ratio + 1)
    q = queries([new] * len(lens), hkv * group, d, group + 1)
    g = torch.Generator().manual_seed(ratio + 1)
    for b, n in enumerate(lens):
        put(c, b, n - 1, 1, (torch.randn((hkv, d), generator=g) * 2.0 ** ratio).to(torch.bfloat16))
    check(c, [new] * len(lens), q)
    check(c, [new] * len(lens), q, window=70, sinks=3)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,new", [(8, 1), (4, 4), (8, 4), (7, 9)])
@pytest.mark.parametrize("ratio", [-40, -20, -11, -9, 9, 11, 20, 40])
def test_a_value_of_another_size_inside_a_sequence(d, group, new, ratio):
    # like values, then one 2^ratio larger or smaller with weight of its own, then like ones again: the kernel's
    # reference for its weights changes while a piece is under way
    hkv = 2
    lens = [200, 1900]
    c = P.make(lens, hkv, d, 64, "e4m3", seed=group + ratio + 50)
    q = queries([new] * 2, hkv * group, d, group + 2)
    g = torch.Generator().manual_seed(ratio + 50)
    for b, n in enumerate(lens):
        for pos in (n // 2, n // 2 + 17):
            put(c, b, pos, 1, (torch.randn((hkv, d), generator=g) * 2.0 ** ratio).to(torch.bfloat16))
    check(c, [new] * 2, q)
    check(c, [new] * 2, q, window=150, sinks=3)


@pytest.mark.parametrize("shift", [-75, 0, 83])
@pytest.mark.parametrize("group,new", [(8, 1), (16, 1), (8, 5), (8, 90)])
def test_value_scales_over_many_binades(shift, group, new):
    # scales spread over 24 binades, and all of them moved by a power of two: the output moves with them
    c = P.make([400, 37 + new], 1, 64, 16, "e4m3", seed=4)
    g = torch.Generator().manual_seed(1)
    c.vs *= torch.exp2(torch.randint(-12, 12, c.vs.shape, generator=g).float()).cuda()
    for b, n in enumerate(c.lens):
        t = torch.arange(n)
        pg = c.table[b].cpu().long()[t // 16]
        x = c.v.cpu()[pg, :, t % 16].view(P.E4M3).double() * c.vs.cpu()[pg, :, t % 16].double()[..., None]
        c.values[b][1] = x.transpose(0, 1)
    q = queries([new] * 2, group, 64, 6)
    want, want_lse, tol = P.reference(c, q, [new] * 2, 0.125)
    o, lse = binding.forward_paged(q.cuda(), c.k, c.v, c.table, c.kv_len, P.indptr([new] * 2), new, k_scale=c.ks,
                                   v_scale=c.vs * 2.0 ** shift)
    binding.device_status()
    M.assert_within("o", o.double() * 2.0 ** -shift, want, tol)
    M.assert_lse(lse, want_lse)


@pytest.mark.parametrize("group,new", [(8, [1, 2]), (4, [5, 16]), (5, [3, 12])])
def test_any_scales_with_few_rows(group, new):
    # scales that are no powers of two, negative, zero and subnormal ones: the few-rows kernel multiplies
    # FP32 scores and weights by them, so that neither K nor V is rounded and the plain bounds hold
    c = P.make([300, 77], 1, 64, 16, "e4m3", seed=4)
    g = torch.Generator().manual_seed(9)
    c.ks *= (torch.rand(c.ks.shape, generator=g) + 0.5).cuda()
    mult = torch.rand(c.vs.shape, generator=g) + 0.5
    mult[torch.rand(c.vs.shape, generator=g) < 0.3] *= -1
    mult[torch.rand(c.vs.shape, generator=g) < 0.1] = 0
    mult[torch.rand(c.vs.shape, generator=g) < 0.1] = 2.0 ** -125   # times a scale near 2^-7: subnormal
    c.vs *= mult.cuda()
    for b, n in enumerate(c.lens):
        t = torch.arange(n)
        pg = c.table[b].cpu().long()[t // 16]
        for w, (codes, s) in enumerate(((c.k, c.ks), (c.v, c.vs))):
            x = codes.cpu()[pg, :, t % 16].view(P.E4M3).double() * s.cpu()[pg, :, t % 16].double()[..., None]
            c.values[b][w] = x.transpose(0, 1)
    check(c, new, queries(new, group, 64, 6))


def test_all_values_zero():
    # zero scales throughout: the output is zero, the log-sum-exp that of the scores
    c = P.make([300, 20], 2, 64, 16, "e4m3", seed=5)
    c.vs.fill_(0)
    c.values = [[k, torch.zeros_like(v)] for k, v in c.values]
    for new, group in (([1, 1], 4), ([3, 2], 20), ([100, 1], 4)):
        check(c, new, queries(new, 2 * group, 64, 2))
