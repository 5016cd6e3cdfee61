"""Evictions that select and move, on two streams at once: each gives what it gives alone."""
import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _paged as P
from tests import _rotate as R
from tests._parity import require_gpu
from tests.test_kv_evict_gpu import bits, free_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


SIZES = {  # lens, hkv, d, keep: a few long sequences; more pairs of sequence and head than SMs; one sequence past 16384 keys
    "few": ([5000, 900, 64], 4, 64, 600), "many": ([300 + 37 * i for i in range(40)], 4, 128, 200), "long": ([20000, 700], 2, 128, 3000),
}


def program(size, fmt, in_place, stream, seed):
    """A step from append to eviction, with its cache, weights and lengths brought back before each; its outputs and pools."""
    lens, hkv, d, keep = SIZES[size]
    g = torch.Generator().manual_seed(seed)
    with torch.cuda.stream(stream):
        c = P.make(lens, hkv, d, 32, fmt, seed=seed, spare=3 + sum(-(-min(n, keep) // 32) for n in lens))
        new = [min(3, n) if i % 2 else 1 for i, n in enumerate(lens)]
        w = torch.rand((c.P, hkv, 32), generator=g).cuda()
        rows = torch.randn((sum(new), 3 * hkv, d), generator=g).to(torch.bfloat16).cuda()
        f, ip = R.frequencies(d).cuda(), P.indptr(new)
        sc = {} if c.ks is None else dict(k_scale=c.ks, v_scale=c.vs)
        cache, pools = (c.k, c.v, c.table, c.kv_len), [x for x in (c.k, c.v, c.ks, c.vs, w) if x is not None]
        start = [x.clone() for x in pools]
        table_out = None if in_place else free_table(c, keep).cuda()

    def step():
        with torch.cuda.stream(stream):
            for x, y in zip(pools, start):
                x.copy_(y)
        q = binding.qkv_append(rows[:, :hkv], rows[:, hkv:2 * hkv], rows[:, 2 * hkv:], *cache, ip, f, stream=stream, **sc)
        _, lse = binding.forward_paged(q, *cache, ip, max(new), stream=stream, **sc)
        binding.kv_accumulate(w, q, lse, *cache, ip, max(new), stream=stream, **sc)
        return [q, lse, *binding.kv_evict(w, *cache, keep, sinks=4, recent=40, table_out=table_out, stream=stream, **sc)], pools
    return step


@pytest.mark.parametrize("sizes", [("few", "few"), ("many", "long"), ("many", "many"), ("long", "few")])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("in_place", [False, True])
def test_two_streams(sizes, fmt, in_place):
    want = []
    for i, size in enumerate(sizes):
        step = program(size, fmt, in_place, torch.cuda.current_stream(), i)
        out, pools = step()
        torch.cuda.synchronize()
        want.append([bits(x) for x in out + pools])
        lens, keep = SIZES[size][0], SIZES[size][3]
        assert out[2].tolist() == [min(n, keep) for n in lens]
        b = lens.index(max(lens))                # keys go from between those that stay
        assert not torch.equal(out[3][b, 0].cpu(), torch.arange(keep, dtype=torch.int32))
    steps = [program(size, fmt, in_place, torch.cuda.Stream(), i) for i, size in enumerate(sizes)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [step() for step in steps]
    torch.cuda.synchronize()
    binding.device_status()
    for x, (out, pools) in zip(want, got):
        for a, b in zip(x, out + pools):
            assert torch.equal(a, bits(b))
