"""Refusals and sizes of the accumulated weights' and the eviction's entry points; nothing is launched here."""
import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding, build
from tests import _weights as W

G = 1 << 20                      # an aligned address that is never dereferenced
BAD, UNS = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def cache(**kw):
    f = dict(k=G, v=G, k_scale=G, v_scale=G, page_stride=2 * 16 * 64, scale_stride=2 * 16, block_table=G, table_stride=4,
             kv_len=G, B=3, Hkv=2, d=64, page_size=16, num_pages=9, max_pages=4, dtype=binding.FA_KV_E4M3)
    f.update(kw)
    return binding.PagedKV(*(f[n] for n, _ in binding.PagedKV._fields_))


def accumulate(lib, kv=None, w=G, w_stride=32, q=G, stride=512, lse=G, ip=G, T=5, max_q=1, Hq=8, window=0, sinks=0, scale=0.125,
               ws=1 << 21, nbytes=1 << 40):
    return lib.fa_kv_accumulate(kv or cache(), w, w_stride, q, stride, lse, ip, T, max_q, Hq, window, sinks, scale, ws, nbytes, None)


def evict(lib, kv=None, w=G, w_stride=32, out=1 << 21, out_stride=2, pages=2, keep=20, sinks=0, recent=0, kept_len=1 << 22,
          kept=1 << 23):
    return lib.fa_kv_evict(kv or cache(), w, w_stride, out, out_stride, pages, keep, sinks, recent, kept_len, kept, None)


@pytest.mark.parametrize("call", [accumulate, evict])
@pytest.mark.parametrize("kw,code,word", [
    (dict(kv=cache(d=96)), UNS, "96"), (dict(kv=cache(page_size=48)), UNS, "page_size"), (dict(kv=cache(k_scale=None)), BAD, "k_scale"),
    (dict(kv=cache(kv_len=None)), BAD, "kv_len"), (dict(w=None), BAD, "weights"), (dict(w=G + 4), BAD, "weights"),
    (dict(w_stride=31), BAD, "weight_stride"), (dict(w_stride=34), BAD, "weight_stride"),
])
def test_bad_caches_and_weights_are_refused(lib, call, kw, code, word):
    assert call(lib, **kw) == code
    assert word in binding.last_error()


@pytest.mark.parametrize("kw,code,word", [
    (dict(Hq=7), BAD, "multiple"), (dict(Hq=0), BAD, "Hq"), (dict(Hq=258, stride=258 * 64), UNS, "128"), (dict(q=None), BAD, "q is"),
    (dict(q=G + 2), BAD, "q is not"), (dict(stride=504), BAD, "q_stride"), (dict(stride=516), BAD, "q_stride"), (dict(lse=None), BAD, "lse"),
    (dict(lse=G + 1), BAD, "lse"), (dict(ip=None), BAD, "q_indptr"), (dict(T=-1), BAD, "T"), (dict(max_q=-1), BAD, "max_q"),
    (dict(scale=0.0), BAD, "scale"), (dict(scale=float("nan")), BAD, "scale"), (dict(window=-1), BAD, "window"),
    (dict(window=4, sinks=-1), BAD, "sinks"), (dict(sinks=3), BAD, "sinks"), (dict(ws=None), BAD, "workspace"),
    (dict(ws=(1 << 21) + 64), BAD, "workspace"), (dict(nbytes=100), BAD, "too small"), (dict(T=1 << 29), BAD, "2^31"),
    (dict(kv=cache(Hkv=64, page_stride=64 * 16 * 64, scale_stride=1024, max_pages=1 << 26, table_stride=1 << 26), w_stride=1024, Hq=64,
          stride=64 * 64), BAD, "2^35"), (dict(kv=cache(B=(1 << 30) + 1)), BAD, "2^30"),
])
def test_bad_accumulate_arguments_are_refused(lib, kw, code, word):
    assert accumulate(lib, **kw) == code
    assert word in binding.last_error()


def test_nothing_to_accumulate(lib):
    assert accumulate(lib, T=0) == binding.FA_OK and accumulate(lib, max_q=0) == binding.FA_OK


def test_workspace_size(lib):
    size = binding.fa_kv_accumulate_workspace_size
    # few rows over E4M3: three bytes for each entry of q and a factor for each vector
    assert size(5, 1, 8, 2, 64, binding.FA_KV_E4M3) == 3 * 5 * 8 * 64 + 256
    assert size(100, 16, 32, 8, 128, binding.FA_KV_E4M3) == 3 * 3200 * 128 + 3200 * 4
    assert size(100, 16, 32, 8, 128, binding.FA_KV_BF16) == 0
    # chunks of eight blocks of 128 rows or more: the sums of 1216 parts of 256 keys
    for dtype in (binding.FA_KV_BF16, binding.FA_KV_E4M3):
        assert size(300, 224, 32, 8, 128, dtype) == 0
        assert size(300, 225, 32, 8, 128, dtype) == size(9000, 9000, 32, 8, 64, dtype) == 1216 * 256 * 4
    for bad in (dict(d=96), dict(Hq=7), dict(Hkv=0), dict(T=-1), dict(T=0), dict(max_q=-1)):
        a = dict(T=5, max_q=1, Hq=8, Hkv=2, d=64, dtype=binding.FA_KV_E4M3)
        a.update(bad)
        assert size(**a) == 0


@pytest.mark.parametrize("kw,code,word", [
    (dict(keep=0), BAD, "keep"), (dict(sinks=-1), BAD, "sinks"), (dict(recent=-1), BAD, "recent"), (dict(sinks=12, recent=9), BAD, "at most keep"),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), BAD, "at most keep"), (dict(out=(1 << 21) + 2), BAD, "table_out"),
    (dict(pages=0), BAD, "table_out"), (dict(out_stride=1), BAD, "table_out"), (dict(pages=1), BAD, "room"),
    (dict(keep=33), BAD, "room"), (dict(kept_len=None), BAD, "kept"), (dict(kept=None), BAD, "kept"), (dict(kept=(1 << 22) + 1), BAD, "kept"),
    (dict(kept_len=G), BAD, "kv_len itself"), (dict(kept=1 << 22), BAD, "another"), (dict(kept=G), BAD, "another"),
    (dict(kept=1 << 21), BAD, "another"),
    (dict(kv=cache(B=1 << 27, Hkv=8, page_stride=8 * 16 * 64, scale_stride=128), w_stride=128), BAD, "2^31"),
])
def test_bad_evictions_are_refused(lib, kw, code, word):
    assert evict(lib, **kw) == code
    assert word in binding.last_error()


def test_python_helpers_refuse_cpu_tensors():
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    t, n, ip = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, w = torch.zeros((1, 2, 64), dtype=torch.bfloat16), torch.zeros((4, 2, 16))
    for call in (lambda: binding.kv_accumulate(w, q, torch.zeros((1, 2)), k, k, t, n, ip, 1), lambda: binding.kv_evict(w, k, k, t, n, 4)):
        with pytest.raises(ValueError):
            call()


def test_the_reference_choice():
    nan = float("nan")
    w = torch.tensor([1.0, 5.0, 2.0, 5.0, nan, 0.0, -0.0, 2.0, 9.0])
    assert W.chosen(w, 9, 0, 0).tolist() == list(range(9))
    assert W.chosen(w, 4, 0, 0).tolist() == [1, 3, 4, 8]
    assert W.chosen(w, 4, 1, 1).tolist() == [0, 1, 4, 8]
    assert W.chosen(w, 5, 0, 3).tolist() == [1, 4, 6, 7, 8]
    assert W.chosen(w, 7, 0, 0).tolist() == [0, 1, 2, 3, 4, 7, 8] and W.chosen(w, 8, 0, 0).tolist() == [0, 1, 2, 3, 4, 5, 7, 8]
    assert W.chosen(w, 2, 1, 1).tolist() == [0, 8]
