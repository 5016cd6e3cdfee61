"""Refusals of the windowed entry points: arguments are checked before anything touches a GPU."""
import ctypes

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


GOOD = ctypes.c_void_p(1 << 20)   # aligned, never dereferenced: validation fails first


def fwd(lib, q=GOOD, window=5, sinks=0, N=128, d=64, scale=0.125, stable=1, beta=1.25):
    return lib.fa_fwd_window(q, GOOD, GOOD, GOOD, GOOD, 1, 1, N, d, window, sinks, scale, stable, beta, None, None)


def bwd(lib, q=GOOD, window=5, sinks=0, N=128, d=64, ws=None):
    n = lib.fa_bwd_workspace_size(1, 1, N, d) if ws is None else ws
    return lib.fa_bwd_window(q, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, None, 1, 1, N, d, window, sinks,
                             0.125, GOOD, n, None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("kw,code,word", [
    (dict(window=0), binding.FA_ERR_INVALID_ARG, "window"),
    (dict(window=-3), binding.FA_ERR_INVALID_ARG, "window"),
    (dict(sinks=-1), binding.FA_ERR_INVALID_ARG, "sinks"),
    (dict(q=None), binding.FA_ERR_INVALID_ARG, "q is NULL"),
    (dict(N=0), binding.FA_ERR_INVALID_ARG, "N"),
    (dict(d=96), binding.FA_ERR_UNSUPPORTED, "96"),
])
def test_bad_arguments_are_refused(lib, call, kw, code, word):
    assert call(lib, **kw) == code
    assert word in binding.last_error()


def test_backward_workspace_is_checked(lib):
    assert bwd(lib, ws=256) == binding.FA_ERR_INVALID_ARG
    assert "workspace too small" in binding.last_error()


def test_backward_workspace_of_split_sinks(lib):
    # a long row's key tile with sinks is split over its queries: FP32 partial dK and dV per part
    plain = lib.fa_bwd_workspace_size(1, 1, 12000, 128)
    assert lib.fa_bwd_window_workspace_size(1, 1, 12000, 128, 256, 0) == plain
    part = 2 * 128 * 128 * 4
    parts, rest = divmod(lib.fa_bwd_window_workspace_size(1, 1, 12000, 128, 256, 4) - plain, part)
    assert parts >= 2 and rest == 0
    assert bwd(lib, sinks=4, N=12000, d=128, window=256, ws=plain) == binding.FA_ERR_INVALID_ARG
    assert "workspace too small" in binding.last_error()
    for bad in ((0, 1, 128, 64, 5, 0), (1, 1, 128, 96, 5, 0), (1, 1, 128, 64, 0, 0), (1, 1, 128, 64, 5, -1)):
        assert lib.fa_bwd_window_workspace_size(*bad) == 0


def test_python_helpers_refuse_a_window_without_causal():
    x = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    for kw in (dict(causal=False, window=2), dict(sinks=3)):
        with pytest.raises(ValueError):
            binding._check_window(kw.get("causal", True), kw.get("window"), kw.get("sinks", 0))
    with pytest.raises(ValueError):
        binding.forward(x, x, x, window=2)   # CPU tensors
