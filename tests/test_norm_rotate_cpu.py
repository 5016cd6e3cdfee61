"""Refusals of norm and rotation, and the 64-bit reference against differences; nothing is launched here."""
import ctypes

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding, build
from tests import _rotate as R

G = 1 << 20                      # an aligned address that is never dereferenced
BAD, UNS = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def rotation(**kw):
    f = dict(inv_freq=G, q_weight=G, k_weight=G, rot=64, interleaved=0, weight_bf16=0, norm=1, eps=1e-6)
    f.update(kw)
    return binding.Rotation(*(f[n] for n, _ in binding.Rotation._fields_))


def view(p=G, b=4 * 100 * 64, h=64, n=4 * 64):
    return binding.Heads(p, b, h, n)


def forward(lib, q=None, k=None, qo=None, ko=None, B=2, Hq=4, Hkv=4, N=100, d=64, pos=G, **kw):
    v = [x or view(G + (i << 24)) for i, x in enumerate((q, k, qo, ko))]
    return lib.fa_norm_rotate(rotation(**kw), *v, B, Hq, Hkv, N, d, pos, 0, None)


def backward(lib, q=None, dz=None, dx=None, k=None, dzk=None, dk=None, dw=(G, 2 * G), B=2, Hq=4, Hkv=4, N=100, d=64, pos=G, ws=1 << 21, nbytes=1 << 30, **kw):
    v = [x or view(G + (i << 24)) for i, x in enumerate((q, k, dz, dzk, dx, dk))]
    return lib.fa_norm_rotate_bwd(rotation(**kw), *v, *dw, B, Hq, Hkv, N, d, pos, 0, ws, nbytes, None)


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(binding.Rotation) == 48 and binding.Rotation.eps.offset == 40
    assert ctypes.sizeof(binding.Heads) == 32


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("kw,code,word", [
    (dict(rot=8), BAD, "rot"), (dict(rot=80), BAD, "rot"), (dict(rot=-16), BAD, "rot"), (dict(inv_freq=None), BAD, "inv_freq"),
    (dict(inv_freq=G + 4), BAD, "inv_freq"), (dict(d=96), UNS, "96"), (dict(eps=-1.0), BAD, "eps"),
    (dict(eps=float("nan")), BAD, "eps"), (dict(eps=float("inf")), BAD, "eps"), (dict(norm=0), BAD, "weights need"),
    (dict(q_weight=G + 2), BAD, "aligned"), (dict(k_weight=G + 1, weight_bf16=1), BAD, "aligned"), (dict(B=0), BAD, "B"),
    (dict(Hq=0), BAD, "Hq"), (dict(Hkv=-1), BAD, "Hkv"), (dict(N=0), BAD, "N"), (dict(N=1 << 30), BAD, "2^31"),
    (dict(pos=G + 2), BAD, "positions"), (dict(q=view(p=None)), BAD, "q is NULL"), (dict(q=view(p=G + 8)), BAD, "aligned"),
    (dict(q=view(h=4)), BAD, "strides"), (dict(q=view(n=-256)), BAD, "strides"), (dict(q=view(b=3)), BAD, "strides"),
])
def test_bad_arguments_are_refused(lib, call, kw, code, word):
    assert call(lib, **kw) == code
    assert word in binding.last_error()


def test_overlapping_outputs_are_refused(lib):
    # (only what is written: an input may have a stride of 0)
    for bad in (view(h=0), view(n=128), view(b=25600 - 8), view(h=32), view(b=0)):
        assert forward(lib, qo=bad) == BAD and "overlap" in binding.last_error()
        assert forward(lib, ko=bad) == BAD and backward(lib, dx=bad) == BAD


def test_outputs_that_are_other_tensors_are_refused(lib):
    at = [view(G + (i << 24)) for i in range(6)]
    other = view(G, h=6400, n=64)          # the queries' start, other strides
    for bad in (dict(qo=at[1]), dict(ko=at[0]), dict(qo=at[3]), dict(k=at[0], qo=at[0]), dict(qo=other)):
        assert forward(lib, **bad) == BAD and ("another tensor" in binding.last_error() or "same strides" in binding.last_error())
    for bad in (dict(dx=at[1]), dict(dx=at[3]), dict(dx=at[5]), dict(dk=at[0]), dict(dk=at[2]), dict(dx=other), dict(dz=at[3], dx=at[3]),
                dict(dw=(G, G))):
        assert backward(lib, **bad) == BAD
        assert any(w in binding.last_error() for w in ("another tensor", "same strides", "one tensor"))


def test_bad_backward_arguments_are_refused(lib):
    assert backward(lib, dw=(G, None)) == BAD and "together" in binding.last_error()
    assert backward(lib, dw=(G + 2, G)) == BAD
    assert backward(lib, norm=0, q_weight=None, k_weight=None) == BAD and "need the norm" in binding.last_error()
    assert backward(lib, ws=None) == BAD and backward(lib, ws=(1 << 21) + 128) == BAD
    assert backward(lib, nbytes=100) == BAD and "too small" in binding.last_error()


def test_workspace_size(lib):
    size = binding.fa_norm_rotate_bwd_workspace_size
    assert size(2, 4, 4, 100, 64) == 304 * 64 * 4 and size(1, 1, 1, 1, 128) == 304 * 128 * 4
    assert size(2, 4, 4, 100, 96) == 0 and size(0, 4, 4, 100, 64) == 0 and size(2, 4, 4, 1 << 30, 64) == 0


def cache(**kw):
    f = dict(k=G, v=G, k_scale=G, v_scale=G, page_stride=2 * 16 * 64, scale_stride=2 * 16, block_table=G, table_stride=4,
             kv_len=G, B=3, Hkv=2, d=64, page_size=16, num_pages=9, max_pages=4, dtype=binding.FA_KV_E4M3)
    f.update(kw)
    return binding.PagedKV(*(f[n] for n, _ in binding.PagedKV._fields_))


def append(lib, kv=None, q=G, q_stride=512, out=2 * G, Hq=8, k=3 * G, v=4 * G, stride=128, ip=G, pos=None, T=5, **kw):
    return lib.fa_qkv_append(kv or cache(), rotation(**kw), q, q_stride, out, Hq, k, v, stride, ip, pos, T, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(kv=cache(d=96)), UNS, "96"), (dict(kv=cache(page_size=8)), UNS, "page_size"), (dict(kv=cache(k_scale=None)), BAD, "k_scale"),
    (dict(rot=72), BAD, "rot"), (dict(eps=-1.0), BAD, "eps"), (dict(T=-1), BAD, "T"), (dict(Hq=0), BAD, "Hq"),
    (dict(T=1 << 30), BAD, "2^31"), (dict(q=None), BAD, "q is NULL"), (dict(out=G + 8), BAD, "q_out"), (dict(k=None), BAD, "k_new"),
    (dict(v=G + 2), BAD, "v_new"), (dict(ip=None), BAD, "q_indptr"), (dict(pos=G + 1), BAD, "positions"),
    (dict(q_stride=504), BAD, "q_stride"), (dict(q_stride=516), BAD, "q_stride"), (dict(stride=120), BAD, "new_stride"),
    (dict(stride=132), BAD, "new_stride"), (dict(out=3 * G), BAD, "q_out"), (dict(out=4 * G), BAD, "q_out"),
    (dict(out=G, q_stride=520), BAD, "q_out"), (dict(kv=cache(B=(1 << 30) + 1)), BAD, "2^30"),
])
def test_bad_append_arguments_are_refused(lib, kw, code, word):
    assert append(lib, **kw) == code
    assert word in binding.last_error()


def test_nothing_to_append(lib):
    assert append(lib, T=0) == binding.FA_OK


def test_python_helpers_refuse_cpu_and_misshapen_tensors():
    q = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    f = R.frequencies(64)
    with pytest.raises(ValueError):
        binding.norm_rotate(q, q, f)
    with pytest.raises(ValueError):
        binding.norm_rotate_backward(q, q, q, q, f)
    with pytest.raises(ValueError):
        binding._rotation(f.float(), 64, -1, None, None, 1e-6, False, True)
    w = torch.ones(64)
    for bad in ((w, None), (w, w.double()), (w[:32], w[:32]), (w, w.bfloat16())):
        with pytest.raises(ValueError):
            binding._rotation(f, 64, -1, *bad, 1e-6, False, True)
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    t, n, ip = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    new = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.qkv_append(new, new, new, k, k, t, n, ip, f)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,rot", [(True, 64), (True, 16), (True, 0), (False, 48)])
def test_reference_gradients_against_differences(interleaved, norm, rot):
    g = torch.Generator().manual_seed(rot)
    x, dz = (torch.randn((2, 3, 64), generator=g, dtype=torch.float64) for _ in range(2))
    w = None if not norm else 1 + 0.2 * torch.randn(64, generator=g, dtype=torch.float64)
    pos = torch.tensor([[0, 5, 70], [1000003, 2, 2 ** 30]])
    f = R.frequencies(rot)

    def loss(x, w):
        return (R.forward(x, pos, f, w, 1e-3, interleaved, norm).z * dz).sum()

    b = R.backward(x, dz, pos, f, w, 1e-3, interleaved, norm)
    h = 1e-6
    for at in ((0, 0, 0), (0, 2, 17), (1, 0, 63), (1, 2, 32)):
        e = torch.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - b.dx[at]) < 1e-7
    for i in (0, 15, 63) if norm else ():
        e = torch.zeros_like(w)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - b.dw[i]) < 1e-7
