"""Eviction to pages that it may not move to."""
import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _paged as P
from tests import _weights as W
from tests._parity import require_gpu
from tests.test_kv_evict_gpu import bits, expected, free_table, pools

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("B", [2, 60])         # two launches, and one whose CTAs move their own keys
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_copy_of_the_table_is_recorded_and_nothing_moves(B, fmt):
    lens, keep = [300, 65] + [100, 20] * (B // 2 - 1), 50
    c = P.make(lens, 3, 64, 16, fmt, seed=1, spare=3 + 4 * B)
    w = W.make(c, seed=1)[0].cuda()
    before = [x.clone() for x in pools(c, w)]
    binding.fa_device_report_read()
    kept_len, kept = binding.kv_evict(w, c.k, c.v, c.table, c.kv_len, keep, sinks=2, recent=5, table_out=c.table.clone(), k_scale=c.ks, v_scale=c.vs)
    assert binding.fa_device_report_read()[0] == binding.FA_ERR_DEVICE_BOUNDS
    for x, y in zip(pools(c, w), before):
        assert torch.equal(bits(x), bits(y))
    # one sequence's row alone: the others move
    table_out = free_table(c, keep).cuda()
    after, want_len, want_kept = expected(c, w, table_out, keep, 2, 5)
    own = table_out[1, :4].long().tolist()
    table_out[1] = c.table[1, : table_out.shape[1]]
    kept_len, kept = binding.kv_evict(w, c.k, c.v, c.table, c.kv_len, keep, sinks=2, recent=5, table_out=table_out, k_scale=c.ks, v_scale=c.vs)
    assert binding.fa_device_report_read()[0] == binding.FA_ERR_DEVICE_BOUNDS
    assert torch.equal(kept_len.cpu(), want_len) and torch.equal(kept.cpu(), want_kept)
    rest = [i for i in range(c.P) if i not in own]
    for x, y in zip(pools(c, w), after):
        assert torch.equal(bits(x[rest]), bits(y[rest]))


@pytest.mark.parametrize("B", [2, 60])
def test_a_sequence_that_keeps_all_may_keep_its_pages(B):
    lens, keep = [300, 40] + [100, 50] * (B // 2 - 1), 50
    c = P.make(lens, 3, 64, 16, "e4m3", seed=2, spare=3 + 4 * B)
    w = W.make(c, seed=2)[0].cuda()
    table_out = free_table(c, keep).cuda()
    table_out[1::2] = c.table[1::2, : table_out.shape[1]]
    after, want_len, want_kept = expected(c, w, table_out, keep, 2, 5)
    kept_len, kept = binding.kv_evict(w, c.k, c.v, c.table, c.kv_len, keep, sinks=2, recent=5, table_out=table_out, k_scale=c.ks, v_scale=c.vs)
    binding.device_status()
    assert torch.equal(kept_len.cpu(), want_len) and torch.equal(kept.cpu(), want_kept)
    for x, y in zip(pools(c, w), after):
        assert torch.equal(bits(x), bits(y))
