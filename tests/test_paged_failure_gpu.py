"""Paged attention when a bounded wait runs out (test build with injected stalls, 100 ms limit).

The call must report the timeout through fa_device_status without touching memory outside its
tensors -- the joining kernels then meet a workspace whose records were never written -- and the same
context must compute correct results afterwards.
"""
import ctypes

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding, build
from tests import _masked as M
from tests import _paged as P
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    require_gpu()
    L = ctypes.CDLL(build.build(testhooks=True))
    vp, ci, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.fa_fwd_paged_workspace_size.argtypes = [ci] * 10
    L.fa_fwd_paged_workspace_size.restype = ctypes.c_size_t
    L.fa_fwd_paged.argtypes = [ctypes.POINTER(binding.PagedKV), vp, ctypes.c_int64, vp, ci, ci, ci, vp, vp, ci, ci, cf, vp,
                               ctypes.c_size_t, vp]
    L.fa_fwd_paged.restype = ci
    L.fa_device_status.argtypes = [vp]
    L.fa_device_status.restype = ci
    return L


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1, 1], [100], [1, 200, 2, 30]])
def test_a_wait_that_runs_out_is_reported_and_nothing_else_breaks(lib, monkeypatch, fmt, new):
    lens = [700, 3000, 90, 64][: len(new)] if len(new) > 1 else [3000]
    hq, d = 8, 64
    c = P.make(lens, 2, d, 32, fmt, seed=2)
    q = torch.randn((sum(new), hq, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    qd, ip = q.cuda(), P.indptr(new)
    o = torch.zeros_like(qd)
    lse = torch.zeros((sum(new), hq), device="cuda")
    kv = binding._paged(c.k, c.v, c.table, c.kv_len, c.ks, c.vs)
    n = lib.fa_fwd_paged_workspace_size(sum(new), len(new), max(new), hq, 2, d, kv.max_pages * 32, 0, 0,
                                        kv.dtype)
    stream = torch.cuda.current_stream().cuda_stream

    def call(fill):
        ws = torch.full((n + 4096,), fill, device="cuda", dtype=torch.uint8)   # + a margin that must stay as it is
        rc = lib.fa_fwd_paged(ctypes.byref(kv), qd.data_ptr(), hq * d, ip.data_ptr(), sum(new), max(new), hq,
                              o.data_ptr(), lse.data_ptr(), 0, 0, 0.125, ws.data_ptr(), n, stream)
        assert rc == binding.FA_OK
        status = lib.fa_device_status(stream)
        assert (ws[n:] == fill).all()
        return status

    for fill in (0x7F, 0xFF, 0x00, 0x01):
        monkeypatch.setenv("FA_TEST_INJECT_STALL", "1")
        assert call(fill) == binding.FA_ERR_TIMEOUT
        monkeypatch.setenv("FA_TEST_INJECT_STALL", "0")
    assert call(0x7F) == binding.FA_OK
    want, want_lse, tol = P.reference(c, q, new, 0.125)
    M.assert_within("o", o, want, tol)
    M.assert_lse(lse, want_lse)
