"""Windows, sinks, lengths and batches past 32 bits, and integers that are not Python's; nothing is launched here."""
import ctypes

import numpy as np
import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


HUGE = (2 ** 31, 2 ** 32 + 256, 2 ** 63 - 1, 2 ** 70)


@pytest.mark.parametrize("x", HUGE)
def test_a_window_past_32_bits_has_no_edge(x):
    size = binding.fa_bwd_window_workspace_size
    assert size(1, 8, 12000, 128, 256, 4) > size(1, 8, 12000, 128, 12000, 4)   # (a short window needs more)
    assert size(1, 8, 12000, 128, x, 4) == size(1, 8, 12000, 128, 12000, 4)
    size = binding.fa_fwd_paged_workspace_size
    a = (4096, 1, 4096, 32, 8, 128, 16000)
    e4m3 = dict(dtype=binding.FA_KV_E4M3)
    assert size(*a, 256, **e4m3) != size(*a, **e4m3)
    assert size(*a, x, **e4m3) == size(*a, **e4m3)
    assert size(*a, 256, x, **e4m3) == size(*a, 256, 16000, **e4m3)


@pytest.mark.parametrize("x", HUGE)
def test_a_negative_window_stays_negative(x):
    assert binding.fa_bwd_window_workspace_size(1, 8, 12000, 128, 256 - x, 4) == 0
    assert binding.fa_bwd_window_workspace_size(1, 8, 12000, 128, 256, -x) == 0
    assert binding.fa_fwd_paged_workspace_size(5, 5, 1, 8, 2, 64, 1000, -x) == 0


def test_integers_of_other_libraries():
    size = binding.fa_fwd_paged_workspace_size
    for as_int in (np.int64, np.int32, torch.tensor):
        assert size(9, 3, as_int(5), 8, 2, 64, as_int(1000), as_int(70), as_int(2)) == size(9, 3, 5, 8, 2, 64, 1000, 70, 2)
        assert binding.fa_bwd_window_workspace_size(1, 8, 12000, 128, as_int(256), as_int(4)) == \
            binding.fa_bwd_window_workspace_size(1, 8, 12000, 128, 256, 4)


@pytest.mark.parametrize("B,Hkv,ok", [(1 << 26, 1, True), ((1 << 27) - 1, 1, True), (1 << 27, 1, False),
                                     (1 << 24, 8, False), ((1 << 24) - 1, 8, True), (1 << 29, 1, False)])
def test_batches_past_the_largest_launch_are_refused(B, Hkv, ok):
    # the joining launch has 16 CTAs for each sequence and kv head at most, in 32 bits
    n = binding.fa_fwd_paged_workspace_size(5, B, 64, Hkv, Hkv, 64, 1000)
    assert (n > 0) == ok
    if not ok:
        assert "B*Hkv" in binding.last_error()
        at = 1 << 20   # an aligned address that is never dereferenced
        kv = binding.PagedKV(at, at, None, None, Hkv * 16 * 64, 0, at, 63, at, B, Hkv, 64, 16, 9, 63, binding.FA_KV_BF16)
        assert binding.load().fa_fwd_paged(ctypes.byref(kv), at, Hkv * 64, at, 5, 64, Hkv, at, at, 0, 0, 0.125, at, 1 << 40,
                                           None) == binding.FA_ERR_INVALID_ARG
