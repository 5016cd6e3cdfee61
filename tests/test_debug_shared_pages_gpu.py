"""The debug build records pages that two sequences of one kv_accumulate call would both add to, and no others."""
import ctypes

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding, build
from tests import _paged as P
from tests import _weights as W
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbg():
    require_gpu()
    lib = ctypes.CDLL(build.build(debug_bounds=True))
    binding.load()
    lib.fa_kv_accumulate.argtypes = binding.load().fa_kv_accumulate.argtypes
    lib.fa_device_report_read.argtypes = [ctypes.c_void_p, ctypes.POINTER(binding.DeviceReport)]
    return lib


def call(lib, c, w, q, lse, new, window=0, sinks=0):
    """(status, page) of one call."""
    kv = binding._paged(c.k, c.v, c.table, c.kv_len, c.ks, c.vs)
    hq, d = q.shape[1:]
    ip, stream = P.indptr(new), torch.cuda.current_stream().cuda_stream
    n = binding.fa_kv_accumulate_workspace_size(sum(new), max(new), hq, c.hkv, d, kv.dtype)
    ws = torch.empty(n + 256, device="cuda", dtype=torch.uint8)
    assert lib.fa_kv_accumulate(kv, w.data_ptr(), w.stride(0), q.data_ptr(), hq * d, lse.data_ptr(), ip.data_ptr(), sum(new), max(new), hq,
                                window, sinks, 0.125, ws.data_ptr(), n, stream) == binding.FA_OK
    rep = binding.DeviceReport()
    return lib.fa_device_report_read(stream, ctypes.byref(rep)), int(rep.bounds_value)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1, 1], [150, 2, 40]])
def test_shared_pages(dbg, fmt, new):
    lens, hq, d, page = [700, 90, 640], 4, 64, 32
    c = P.make(lens, 2, d, page, fmt, seed=2)
    q = torch.randn((sum(new), hq, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    lse = W.log_sum_exps(c, q, new, 0.125).cuda()
    w, q = W.make(c, seed=2)[0].cuda(), q.cuda()
    assert call(dbg, c, w, q, lse, new)[0] == binding.FA_OK
    own = c.table.clone()
    c.table[2, 5] = c.table[0, 9]                  # one page of two sequences, in the middle
    assert call(dbg, c, w, q, lse, new) == (binding.FA_ERR_DEVICE_BOUNDS, int(c.table[0, 9]))
    if max(new) == 1:                              # a window that sees it in neither, or in one
        assert call(dbg, c, w, q, lse, new, window=64)[0] == binding.FA_OK
        assert call(dbg, c, w, q, lse, new, window=64, sinks=5 * page + 1)[0] == binding.FA_OK
    assert call(dbg, c, w, q, lse, [new[0], new[1], 0])[0] == binding.FA_OK   # the second has no new tokens
    c.table.copy_(own)
    c.table[1, 3:] = c.table[0, 0]                 # behind the second sequence's last page
    assert call(dbg, c, w, q, lse, new)[0] == binding.FA_OK
