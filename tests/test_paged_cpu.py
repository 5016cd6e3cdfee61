"""Refusals and sizes of the paged-cache entry points; nothing is launched here."""
import ctypes

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


G = 1 << 20                      # an aligned address that is never dereferenced
GOOD = ctypes.c_void_p(G)


def cache(**kw):
    f = dict(k=G, v=G, k_scale=G, v_scale=G, page_stride=2 * 16 * 64, scale_stride=2 * 16, block_table=G, table_stride=4,
             kv_len=G, B=3, Hkv=2, d=64, page_size=16, num_pages=9, max_pages=4, dtype=binding.FA_KV_E4M3)
    f.update(kw)
    return ctypes.byref(binding.PagedKV(*(f[n] for n, _ in binding.PagedKV._fields_)))


def append(lib, kv=None, k=GOOD, stride=128, ip=GOOD, T=5, **kw):
    return lib.fa_kv_append(cache(**kw) if kv is None else kv, k, GOOD, stride, ip, T, None)


def read(lib, ip=GOOD, k=GOOD, rows=5, **kw):
    return lib.fa_kv_read(cache(**kw), ip, k, GOOD, rows, None)


def attend(lib, q=GOOD, stride=512, ip=GOOD, T=5, max_q=1, Hq=8, o=GOOD, lse=GOOD, window=0, sinks=0, scale=0.125,
           ws=ctypes.c_void_p(1 << 21), nbytes=1 << 40, **kw):
    return lib.fa_fwd_paged(cache(**kw), q, stride, ip, T, max_q, Hq, o, lse, window, sinks, scale, ws, nbytes, None)


BAD, UNS = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [append, read, attend])
@pytest.mark.parametrize("kw,code,word", [
    (dict(k_scale=None), BAD, "k_scale"), (dict(v_scale=G + 4), BAD, "v_scale"), (dict(v=None), BAD, "kv->v"),
    (dict(d=96), UNS, "96"), (dict(page_size=8), UNS, "page_size"), (dict(page_size=48), UNS, "page_size"),
    (dict(page_size=512), UNS, "page_size"), (dict(page_stride=2047), BAD, "page_stride"),
    (dict(page_stride=2048 + 8), BAD, "page_stride"), (dict(scale_stride=31), BAD, "scale_stride"),
    (dict(scale_stride=34), BAD, "scale_stride"), (dict(B=0), BAD, "B"), (dict(Hkv=0), BAD, "Hkv"),
    (dict(num_pages=0), BAD, "num_pages"), (dict(max_pages=0), BAD, "max_pages"), (dict(max_pages=5), BAD, "table_stride"),
    (dict(max_pages=1 << 27, table_stride=1 << 27), BAD, "2^30"), (dict(block_table=None), BAD, "block_table"),
    (dict(kv_len=G + 2), BAD, "kv_len"), (dict(dtype=2), UNS, "dtype"), (dict(ip=None), BAD, "indptr"),
])
def test_bad_caches_are_refused(lib, call, kw, code, word):
    assert call(lib, **kw) == code
    assert word in binding.last_error()


def test_bad_rows_are_refused(lib):
    assert lib.fa_kv_append(None, GOOD, GOOD, 128, GOOD, 1, None) == BAD
    assert append(lib, T=-1) == BAD
    assert append(lib, stride=120) == BAD and append(lib, stride=132) == BAD
    assert append(lib, k=ctypes.c_void_p(G + 8)) == BAD
    assert read(lib, rows=-1) == BAD and read(lib, k=None) == BAD
    # nothing to do: no launch
    assert append(lib, T=0) == binding.FA_OK and read(lib, rows=0) == binding.FA_OK
    assert attend(lib, T=0) == binding.FA_OK and attend(lib, max_q=0) == binding.FA_OK


@pytest.mark.parametrize("kw,code,word", [
    (dict(Hq=7), BAD, "multiple"), (dict(Hq=0), BAD, "Hq"), (dict(Hq=2 * 129, stride=2 * 129 * 64), UNS, "128"),
    (dict(q=ctypes.c_void_p(G + 2)), BAD, "q is not"), (dict(o=None), BAD, "o is NULL"), (dict(stride=511), BAD, "q_stride"),
    (dict(stride=516), BAD, "q_stride"), (dict(lse=ctypes.c_void_p(G + 1)), BAD, "lse"), (dict(T=-1), BAD, "T"),
    (dict(max_q=-1), BAD, "max_q"), (dict(scale=0.0), BAD, "scale"), (dict(scale=float("inf")), BAD, "scale"),
    (dict(window=-1), BAD, "window"), (dict(window=4, sinks=-1), BAD, "sinks"), (dict(sinks=3), BAD, "sinks"),
    (dict(ws=None), BAD, "workspace"), (dict(ws=ctypes.c_void_p((1 << 21) + 128)), BAD, "workspace"),
    (dict(nbytes=1000), BAD, "workspace too small"),
])
def test_bad_attention_arguments_are_refused(lib, kw, code, word):
    assert attend(lib, **kw) == code
    assert word in binding.last_error()


def test_workspace_sizes(lib):
    size = binding.fa_fwd_paged_workspace_size
    # single tokens: two slots of 8 (16, 32, 64) rows for each of 304 CTAs (FP32 outputs and
    # log-sum-exps), and 16 bytes for each sequence and kv head
    assert size(5, 5, 1, 8, 2, 64, 1000) == 2 * 304 * 8 * 64 * 4 + 2 * 304 * 8 * 4 + 256
    assert size(64, 64, 1, 32, 8, 128, 1 << 20) == 2 * 304 * 8 * 129 * 4 + 64 * 8 * 16
    assert size(64, 64, 1, 32, 2, 128, 1 << 20) == 2 * 304 * 16 * 129 * 4 + 64 * 2 * 16
    # chunks whose tiles (64 tokens by 4 heads of a group) fill whole rounds of 152 SMs need none; the
    # tiles left over are split over the keys, unless the keys are few
    assert size(152 * 64, 1, 152 * 64, 4, 1, 128, 1 << 15) == 0
    assert size(153 * 64, 1, 153 * 64, 4, 1, 128, 1 << 15) > 0
    assert size(153 * 64, 1, 153 * 64, 4, 1, 128, 256) == 0
    assert size(128, 1, 128, 1, 1, 128, 1 << 15) > 0
    assert size(128, 1, 128, 1, 1, 128, 1 << 15, 100) == 0
    # E4M3 chunks whose tiles read each key often have room for BF16 pages of 128 keys (K and V) and a
    # table: 512 tokens of 4 heads for each kv head over 16000 keys; seen keys only with a window
    copy = lambda pages, B=1: 2 * pages * B * 128 * 8 * 128 * 2 + -(-125 * B * 4 // 256) * 256
    a = (512, 1, 512, 32, 8, 128, 16000)
    assert size(*a, dtype=binding.FA_KV_E4M3) == size(*a) + copy(125)
    a = (4096, 1, 4096, 32, 8, 128, 16000, 5000)
    assert size(*a, 130, binding.FA_KV_E4M3) == size(*a, 130) + copy(2 + (5000 + 4096) // 128 + 2)
    for a in ((100, 1, 100, 32, 8, 128, 16000), (400, 40, 400, 32, 8, 128, 16000), (400, 1, 400, 32, 8, 128, 16000, 100),
              (1 << 16, 1, 1 << 16, 32, 8, 128, 1 << 23)):   # too few tiles; a copy past 2 GiB
        assert size(*a, dtype=binding.FA_KV_E4M3) == size(*a)
    for bad in (dict(d=96), dict(Hq=7), dict(sinks=-1), dict(Hkv=0), dict(T=-1), dict(T=0), dict(B=0)):
        a = dict(T=5, B=5, max_q=1, Hq=8, Hkv=2, d=64, max_kv=1000)
        a.update(bad)
        assert size(**a) == 0


def test_struct_layout_matches_the_header():
    assert ctypes.sizeof(binding.PagedKV) == 104
    assert binding.PagedKV.page_stride.offset == 32 and binding.PagedKV.dtype.offset == 96


def test_python_helpers_refuse_cpu_and_misshapen_tensors():
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    t, n, ip = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    new = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: binding.kv_append(new, new, k, k, t, n, ip), lambda: binding.kv_read(k, k, t, n, ip, 1),
                 lambda: binding.forward_paged(new, k, k, t, n, ip, 1)):
        with pytest.raises(ValueError):
            call()
