"""Calls with windows past 32 bits and with integers that are not Python's."""
import numpy as np
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


@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("window,sinks,want", [(2 ** 32 + 5, 0, (None, 0)), (2 ** 63, 2 ** 40, (None, 0)),
                                               (50, 2 ** 32 + 1, (None, 0)), (np.int64(50), np.int32(3), (50, 3))])
def test_paged(new, window, sinks, want):
    c = P.make([300, 170], 2, 64, 16, "bf16", seed=1)
    q = torch.randn((2 * new, 8, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    o, lse = binding.forward_paged(q.cuda(), c.k, c.v, c.table, c.kv_len, P.indptr([new, new]), np.int64(new), window=window,
                                   sinks=sinks)
    ref, ref_lse, tol = P.reference(c, q, [new, new], 0.125, *want)
    M.assert_within("o", o, ref, tol)
    M.assert_lse(lse, ref_lse)
    k, v = binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr(c.lens), np.int64(470))
    assert k.shape == (470, 2, 64) and torch.equal(k, binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr(c.lens), 470)[0])
    binding.device_status()


@pytest.mark.parametrize("window,sinks,want", [(2 ** 32 + 5, 0, (300, 0)), (20, 2 ** 32 + 1, (20, 300)),
                                               (np.int64(20), torch.tensor(3), (20, 3))])
def test_windowed_step(window, sinks, want):
    g = torch.Generator().manual_seed(2)
    q, k, v, do = (torch.randn((1, 2, 300, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    o, lse = binding.forward(q, k, v, window=window, sinks=sinks)
    o2, lse2 = binding.forward(q, k, v, window=want[0], sinks=want[1])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    got = binding.backward(q, k, v, o, lse, do, window=window, sinks=sinks)
    ref = binding.backward(q, k, v, o, lse, do, window=want[0], sinks=want[1])
    assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])
    assert torch.allclose(got[0].float(), ref[0].float(), rtol=2.0 ** -6, atol=1e-4)   # (sums in any order)
    binding.device_status()
