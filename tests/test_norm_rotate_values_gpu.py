"""Norm and rotation of values at the ends of the range: what is not finite, sums of squares past FP32's range."""
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _paged as P
from tests import _rotate as R
from tests._parity import require_gpu
from tests.test_norm_rotate_gpu import near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (128, 48, True), (128, 0, False)])
def test_rotation_alone_turns_the_gradient_whatever_the_inputs_hold(d, rot, interleaved):
    g = torch.Generator().manual_seed(d + rot)
    B, N, hq, hkv = 2, 77, 5, 2
    _, q, k = R.heads(B, N, hq, hkv, d, g)
    dz = [torch.randn((B, h, N, d), generator=g).to(torch.bfloat16) for h in (hq, hkv)]
    f = R.frequencies(rot)
    call = lambda x, y: binding.norm_rotate_backward(x.cuda(), y.cuda(), dz[0].cuda(), dz[1].cuda(), f.cuda() if rot else None,
                                                     interleaved=interleaved, norm=False)
    want = call(q, k)
    for x, t in zip(dz, want):
        b = R.backward(x, x, torch.arange(N), f, None, 1e-6, interleaved, False)   # (its first argument has no part in dx)
        near(t, b.dx, b.dx_tol)
    for bad in (math.nan, math.inf, -math.inf):
        x, y = q.clone(), k.clone()
        x[:, ::2, 5::3] = bad
        y[..., 3] = bad
        got = call(x, y)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    binding.device_status()


SIZES = [  # powers of two of the vectors' sizes and of their gradients', eps
    ([62, 64, 90, 127, 0, 64], [0, 60, 0, 100, 0, -60], 1e-6), ([-38, -60, -64, -75, -100, -133, 3, 127], [-30, -60, 0, -60, -80, -120, 0, 100], 0.0),
    ([-50, -60, -75, -100, 70], [-40, -40, -40, -40, 0], 2.0 ** -104), ([120, 100, 0], [0, 0, 0], 3e38),
]


def extreme(sizes, n, d, g):
    """Vectors [n, d] of ordinary entries times 2^sizes[i], in turn."""
    x = torch.randn((n, d), generator=g).clamp(-1.9, 1.9).double()
    at = torch.tensor(sizes).repeat(-(-n // len(sizes)))[:n].double()
    return (x * torch.exp2(at)[:, None]).to(torch.bfloat16)


@pytest.mark.parametrize("sizes,grads,eps", SIZES)
@pytest.mark.parametrize("d,interleaved,weighted", [(64, False, True), (128, True, False), (128, False, True)])
def test_sums_of_squares_past_the_range(sizes, grads, eps, d, interleaved, weighted):
    # The factor is a power of two: the bounds of forward() and backward() hold as they are, but for results under FP32's
    # normal range (2^-149 and what BF16 keeps there, within their 1e-38).
    g = torch.Generator().manual_seed(d)
    n = 5 * len(sizes)
    q, dz = (extreme(s, n, d, g)[None, None] for s in (sizes, grads))
    k, dzk = q.flip(2), dz.flip(2)
    f, pos = R.frequencies(d), torch.arange(n)
    w = [1 + 0.3 * torch.randn(d, generator=g) for _ in range(2)] if weighted else [None, None]
    kw = dict(eps=eps, interleaved=interleaved, q_weight=w[0].cuda() if weighted else None, k_weight=w[1].cuda() if weighted else None)
    z = binding.norm_rotate(q.cuda(), k.cuda(), f.cuda(), **kw)
    dx = binding.norm_rotate_backward(q.cuda(), k.cuda(), dz.cuda(), dzk.cuda(), f.cuda(), **kw)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    for x, y, a, b, wt, dw in ((q, dz, z[0], dx[0], w[0], dx[2]), (k, dzk, z[1], dx[1], w[1], dx[3])):
        r = R.forward(x, pos, f, wt, eps, interleaved)
        near(a, r.z, r.tol, "forward")
        s = R.backward(x, y, pos, f, wt, eps, interleaved)
        fits = s.dx.abs().amax(-1) < 3e38
        assert fits.sum() > n // 2
        near(b[fits.cuda()], s.dx[fits], s.dx_tol[fits], "dx")
        if weighted:
            near(dw, s.dw, s.dw_tol, "dw")
    binding.device_status()


def test_a_vectors_result_does_not_depend_on_its_neighbours():
    # the same vectors among ordinary ones, and among ones whose squares overflow
    g = torch.Generator().manual_seed(2)
    q = torch.randn((1, 8, 60, 64), generator=g).to(torch.bfloat16)
    dz = torch.randn((1, 8, 60, 64), generator=g).to(torch.bfloat16)
    far = q.clone()
    far[:, ::3] *= 2.0 ** 100
    far[:, :, ::4] *= 2.0 ** 90
    same = torch.ones((1, 8, 60), dtype=torch.bool)
    same[:, ::3] = False
    same[:, :, ::4] = False
    f = R.frequencies(64).cuda()
    a, b = (binding.norm_rotate(x.cuda(), x.cuda(), f)[0].cpu() for x in (q, far))
    assert torch.equal(a[same], b[same])
    a, b = (binding.norm_rotate_backward(x.cuda(), x.cuda(), dz.cuda(), dz.cuda(), f)[0].cpu() for x in (q, far))
    assert torch.equal(a[same], b[same])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("sizes,grads,eps", SIZES)
def test_append_of_sums_of_squares_past_the_range(sizes, grads, eps, fmt):
    # against norm_rotate and kv_append: BF16 bit for bit; E4M3 keys are rounded once, so off by half a step of the value
    # (2^-4 of it, 2^-10 of the scale) from the 64-bit form
    d, n = 64, 5 * len(sizes)
    g = torch.Generator().manual_seed(1)
    x = extreme(sizes, n, d, g)[:, None]
    f = R.frequencies(d)
    c = P.make([n], 1, d, 16, fmt, seed=1)
    q = binding.qkv_append(x.cuda(), x.cuda(), x.cuda(), c.k, c.v, c.table, c.kv_len, P.indptr([n]), f.cuda(), eps=eps, k_scale=c.ks, v_scale=c.vs)
    kr, _ = binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr([n]), n, k_scale=c.ks, v_scale=c.vs)
    binding.device_status()
    z = binding.norm_rotate(x[None, :, 0][:, None].cuda(), x[None, :, 0][:, None].cuda(), f.cuda(), eps=eps)[0]
    assert torch.equal(q[:, 0], z[0, 0])
    if fmt == "bf16":
        assert torch.equal(kr[:, 0], z[0, 0])
    else:
        r = R.forward(x[:, 0], torch.arange(n), f, eps=float(torch.tensor(eps, dtype=torch.float32)))
        top = r.z.abs().amax(-1, keepdim=True)
        near(kr[:, 0], r.z, 2.0 ** -4 * r.z.abs() + 2.0 ** -10 * top / 224 + r.tol)
