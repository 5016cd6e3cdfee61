"""Dimensions of one entry have no stride: whatever a view carries there, the calls take it."""
import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _paged as P
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def moved(x, *strides):
    """x's values in memory of its own with these strides (of dimensions with one entry: any)."""
    y = torch.empty(1 + sum((n - 1) * s for n, s in zip(x.shape, strides)), dtype=x.dtype, device=x.device)
    y = y.as_strided(x.shape, strides)
    y.copy_(x)
    return y


def run(c, new, group):
    T = sum(new)
    g = torch.Generator().manual_seed(1)
    q, kn, vn = ((torch.randn((T, h, c.d), generator=g)).to(torch.bfloat16).cuda()
                 for h in (c.hkv * group, c.hkv, c.hkv))
    ip = P.indptr(new)
    kw = dict(k_scale=c.ks, v_scale=c.vs)
    binding.kv_append(kn, vn, c.k, c.v, c.table, c.kv_len, ip, **kw)
    o, lse = binding.forward_paged(q, c.k, c.v, c.table, c.kv_len, ip, max(new), **kw)
    rows = sum(c.lens)
    k, v = binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr(c.lens), rows, **kw)
    binding.device_status()
    return o, lse, k, v


def same(c, twin, new, group):
    for a, b in zip(run(c, new, group), run(twin, new, group)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 9])
def test_one_page(fmt, new):
    # K and V are one page each, cut from pools of different sizes
    hkv, d, page = 2, 64, 64
    c, t = (P.make([40], hkv, d, page, fmt, seed=1, spare=0) for _ in range(2))
    n = hkv * page * d
    c.k, c.v = moved(c.k, n + 64, page * d, d, 1), moved(c.v, 3 * n, page * d, d, 1)
    if fmt == "e4m3":
        c.ks, c.vs = moved(c.ks, 1, page, 1), moved(c.vs, 4 * hkv * page, page, 1)
    assert c.k.stride(0) != c.v.stride(0)
    same(c, t, [new], 4)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 9])
def test_one_head(fmt, new):
    # a cache kept as [pages, page_size, 1, d], seen with the heads in front
    d, page = 128, 32
    c, t = (P.make([100, 33], 1, d, page, fmt, seed=2) for _ in range(2))
    c.k, c.v = (x[:, 0].clone()[:, :, None].transpose(1, 2) for x in (c.k, c.v))
    assert c.k.stride(1) == d
    if fmt == "e4m3":
        c.ks, c.vs = (x[:, 0].clone()[:, :, None].transpose(1, 2) for x in (c.ks, c.vs))
    same(c, t, [new, new], 8)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_table_of_one_column(fmt):
    c, t = (P.make([20, 31, 7], 2, 64, 32, fmt, seed=3) for _ in range(2))
    c.table = torch.stack([c.table[:, 0], c.table[:, 0] * 0 - 1], 1)[:, ::2]
    t.table = t.table[:, :1].contiguous()
    assert c.table.shape == (3, 1) and c.table.stride(1) == 2
    same(c, t, [1, 5, 2], 4)


def test_what_does_not_agree_is_still_refused():
    c = P.make([100, 33], 2, 64, 32, "e4m3", seed=4)
    q = torch.zeros((2, 8, 64), device="cuda", dtype=torch.bfloat16)
    n, wide = 2 * 32 * 64, [moved(x, 2 * 2 * 32 * 64, 32 * 64, 64, 1) for x in (c.k, c.v)]
    for k, v, ks, vs, table in (
            (wide[0], c.v, c.ks, c.vs, c.table), (c.k, wide[1], c.ks, c.vs, c.table),      # page strides differ
            (c.k, c.v, c.ks, moved(c.vs, 128, 32, 1), c.table),
            (moved(c.k, n + 32 * 64, 2 * 32 * 64, 64, 1), moved(c.v, n + 32 * 64, 2 * 32 * 64, 64, 1), c.ks, c.vs, c.table),
            (c.k, c.v, moved(c.ks, 128, 64, 1), moved(c.vs, 128, 64, 1), c.table),         # heads apart
            (c.k, c.v, c.ks, c.vs, c.table.t().contiguous().t())):                         # a table by columns
        with pytest.raises(ValueError):
            binding.forward_paged(q, k, v, table, c.kv_len, P.indptr([1, 1]), 1, k_scale=ks, v_scale=vs)
