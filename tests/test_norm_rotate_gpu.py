"""Norm and rotation of queries and keys, forward and backward, against the 64-bit form."""
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _rotate as R
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def near(got, want, tol, what=""):
    off = (got.detach().cpu().double() - want).abs()
    assert (off <= tol).all(), (what, float((off / tol).max()))


def weights(d, g, dtype=torch.float32):
    return tuple((1 + 0.3 * torch.randn(d, generator=g)).to(dtype) for _ in range(2))


SHAPES = [  # B, N, hq, hkv, d, rot, interleaved
    (1, 1, 1, 1, 64, 64, False), (1, 1, 40, 8, 128, 128, False), (2, 129, 4, 4, 64, 64, True), (3, 77, 7, 1, 128, 64, False),
    (1, 333, 5, 3, 128, 48, True), (2, 50, 33, 2, 64, 16, False), (1, 1000, 2, 1, 128, 112, False), (5, 3, 12, 12, 64, 0, False),
    (1, 65, 130, 1, 64, 32, True), (4, 31, 9, 6, 128, 128, True), (1, 700, 16, 16, 64, 48, False),
    (1, 129, 2, 2, 64, 64, False), (2, 8, 8, 1, 128, 128, False), (1, 40, 400, 1, 64, 64, False),   # (a side with one CTA)
]


@pytest.mark.parametrize("B,N,hq,hkv,d,rot,interleaved", SHAPES)
@pytest.mark.parametrize("norm,weighted", [(True, True), (True, False), (False, False)])
def test_forward_and_backward(B, N, hq, hkv, d, rot, interleaved, norm, weighted):
    g = torch.Generator().manual_seed(N + hq)
    rows, q, k = R.heads(B, N, hq, hkv, d, g)
    dq, dk = (torch.randn((B, h, N, d), generator=g).to(torch.bfloat16) for h in (hq, hkv))
    f = R.frequencies(rot)
    w = weights(d, g, torch.bfloat16 if N % 2 else torch.float32) if weighted else (None, None)
    dev = rows.cuda()
    qd, kd = dev[:, :, :hq].transpose(1, 2), dev[:, :, hq:hq + hkv].transpose(1, 2)
    kw = dict(q_weight=w[0].cuda() if weighted else None, k_weight=w[1].cuda() if weighted else None, eps=1e-5,
              interleaved=interleaved, norm=norm)
    fd = f.cuda() if rot else None
    oq, ok = binding.norm_rotate(qd, kd, fd, **kw)
    gq, gk, gqw, gkw = binding.norm_rotate_backward(qd, kd, dq.cuda(), dk.cuda(), fd, **kw)
    assert oq.is_contiguous() and ok.is_contiguous()
    assert B * N == 1 or gq.transpose(1, 2).is_contiguous()
    assert (gqw is None) == (not weighted)
    pos = torch.arange(N)
    for x, dz, z, dx, wt, dw in ((q, dq, oq, gq, w[0], gqw), (k, dk, ok, gk, w[1], gkw)):
        r = R.forward(x, pos, f, wt, 1e-5, interleaved, norm)
        near(z, r.z, r.tol, "forward")
        b = R.backward(x, dz, pos, f, wt, 1e-5, interleaved, norm)
        near(dx, b.dx, b.dx_tol, "dx")
        if weighted:
            near(dw, b.dw, b.dw_tol, "dw")
    binding.device_status()


@pytest.mark.parametrize("first", [1000003, 2 ** 31 - 40, -(2 ** 31), -5000])
@pytest.mark.parametrize("per_sequence", [False, True])
def test_positions(first, per_sequence):
    g = torch.Generator().manual_seed(3)
    B, N, d = 3, 33, 128
    rows, q, k = R.heads(B, N, 6, 2, d, g)
    pos = torch.arange(first, first + N) if first < 0 else torch.arange(first, first + N).clamp(max=2 ** 31 - 1)
    pos = pos.to(torch.int32)
    if per_sequence:
        pos = torch.stack([pos, pos.flip(0), torch.randint(-2 ** 31, 2 ** 31 - 1, (N,), generator=g).to(torch.int32)])
    wide = torch.zeros((B, N + 5), dtype=torch.int32)   # rows of a wider tensor
    wide[:, :N] = pos
    dev = wide.cuda()[:, :N] if per_sequence else pos.cuda()
    f = R.frequencies(d)
    oq, ok = binding.norm_rotate(q.cuda(), k.cuda(), f.cuda(), positions=dev)
    at = pos[:, None] if per_sequence else pos
    for x, z in ((q, oq), (k, ok)):
        r = R.forward(x, at, f)
        near(z, r.z, r.tol)


def test_frequencies_of_any_size():
    # more than a turn for each position, negative, zero: only the fraction of a turn counts
    g = torch.Generator().manual_seed(4)
    _, q, k = R.heads(1, 200, 3, 1, 64, g)
    f = torch.cat([torch.tensor([0.0, -1.0, 7.5, 2 * math.pi, 100.0, -1e-9, 1e-12, 3.0]), torch.rand(24, generator=g) * 20 - 10]).double()
    oq, _ = binding.norm_rotate(q.cuda(), k.cuda(), f.cuda(), interleaved=True)
    r = R.forward(q, torch.arange(200), f, interleaved=True)
    # a double near 100 rad for each position is itself off by 100 * 2^-53
    near(oq, r.z, r.tol + 200 * 100 * 2.0 ** -52 * R.spread(r.y, 32, True))


def test_special_vectors():
    # zeros, one large entry, tiny ones, NaN and Inf: only their own vectors are touched
    g = torch.Generator().manual_seed(5)
    x = torch.randn((1, 1, 8, 128), generator=g)
    x[0, 0, 0] = 0
    x[0, 0, 1] = 0
    x[0, 0, 1, 5] = 3e18
    x[0, 0, 2] *= 1e-20
    x[0, 0, 3, 7] = math.nan
    x[0, 0, 4, 9] = math.inf
    x = x.to(torch.bfloat16)
    f = R.frequencies(128)
    o, _ = binding.norm_rotate(x.cuda(), x.cuda(), f.cuda())
    r = R.forward(x, torch.arange(8), f)
    rest = [0, 1, 2, 5, 6, 7]
    near(o[0, 0, rest], r.z[0, 0, rest], r.tol[0, 0, rest])
    assert torch.isnan(o[0, 0, 3]).all() and not torch.isfinite(o[0, 0, 4]).all()
    dx, _, dw, _ = binding.norm_rotate_backward(x.cuda(), x.cuda(), x.cuda(), x.cuda(), f.cuda(), q_weight=torch.ones(128).cuda(),
                                                k_weight=torch.ones(128).cuda())
    b = R.backward(x, x, torch.arange(8), f)
    near(dx[0, 0, rest], b.dx[0, 0, rest], b.dx_tol[0, 0, rest])
    assert torch.isnan(dw).any()


def test_views_in_place_and_outputs_in_a_projections_gradient():
    g = torch.Generator().manual_seed(6)
    B, N, hq, hkv, d = 2, 70, 5, 3, 64
    rows, q, k = R.heads(B, N, hq, hkv, d, g)
    f, pos = R.frequencies(64).cuda(), torch.arange(N, dtype=torch.int32).cuda()
    w = [x.cuda() for x in weights(d, g)]
    kw = dict(positions=pos, q_weight=w[0], k_weight=w[1])
    want = binding.norm_rotate(q.cuda().contiguous(), k.cuda().contiguous(), f, **kw)
    dz = tuple(torch.randn(t.shape, generator=g).to(torch.bfloat16).cuda() for t in (q, k))
    want_b = binding.norm_rotate_backward(q.cuda().contiguous(), k.cuda().contiguous(), *dz, f, **kw)
    dev = rows.cuda()
    cut = lambda t: (t[:, :, :hq].transpose(1, 2), t[:, :, hq:hq + hkv].transpose(1, 2))
    grad = torch.full_like(dev, 3.0)
    got_b = binding.norm_rotate_backward(*cut(dev), *dz, f, out=cut(grad), **kw)
    for a, b in zip(got_b, want_b):
        assert torch.equal(a, b)
    assert (grad[:, :, hq + hkv:] == 3).all()
    # a gradient over its own dz
    over = tuple(t.clone() for t in dz)
    got_b = binding.norm_rotate_backward(*cut(dev), *over, f, out=over, **kw)
    assert torch.equal(got_b[0], want_b[0]) and torch.equal(over[1], want_b[1])
    binding.norm_rotate(*cut(dev), f, out=cut(dev), **kw)
    for a, b in zip(cut(dev), want):
        assert torch.equal(a, b)
    assert torch.equal(dev[:, :, hq + hkv:].cpu(), rows[:, :, hq + hkv:])
    # an expanded gradient (stride 0) and heads in front of the batch
    one = torch.ones((1, 1, 1, d), dtype=torch.bfloat16, device="cuda")
    a = binding.norm_rotate_backward(q.cuda(), k.cuda(), one.expand(B, hq, N, d), one.expand(B, hkv, N, d), f, **kw)
    b = binding.norm_rotate_backward(q.cuda(), k.cuda(), one.expand(B, hq, N, d).contiguous(), one.expand(B, hkv, N, d).contiguous(), f, **kw)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    odd = q.cuda().permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)
    assert torch.equal(binding.norm_rotate(odd, k.cuda(), f, **kw)[0], want[0])


def test_the_same_bits_in_every_call():
    g = torch.Generator().manual_seed(7)
    _, q, k = R.heads(2, 1500, 8, 2, 128, g)
    q, k, f = q.cuda(), k.cuda(), R.frequencies(128).cuda()
    w = [x.cuda() for x in weights(128, g)]
    dz = tuple(torch.randn(t.shape, generator=g).to(torch.bfloat16).cuda() for t in (q, k))
    a = binding.norm_rotate_backward(q, k, *dz, f, q_weight=w[0], k_weight=w[1])
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, binding.norm_rotate_backward(q, k, *dz, f, q_weight=w[0], k_weight=w[1])))
    # a large batch's weight gradient against 64 bits
    b = R.backward(q.cpu(), dz[0].cpu(), torch.arange(1500), R.frequencies(128), w[0].cpu(), 1e-6)
    near(a[2], b.dw, b.dw_tol)


def test_other_stream_and_graph():
    g = torch.Generator().manual_seed(8)
    _, q, k = R.heads(2, 300, 4, 2, 64, g)
    q, k, f = q.cuda(), k.cuda(), R.frequencies(64).cuda()
    w = [x.cuda() for x in weights(64, g)]
    dz = tuple(torch.randn(t.shape, generator=g).to(torch.bfloat16).cuda() for t in (q, k))
    step = lambda **s: binding.norm_rotate(q, k, f, q_weight=w[0], k_weight=w[1], **s) + \
        binding.norm_rotate_backward(q, k, *dz, f, q_weight=w[0], k_weight=w[1], **s)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    q.mul_(0.5)
    k.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_python_refusals():
    q = torch.zeros((1, 2, 8, 64), device="cuda", dtype=torch.bfloat16)
    f = R.frequencies(64).cuda()
    for bad in (lambda: binding.norm_rotate(q.float(), q, f), lambda: binding.norm_rotate(q, q[:, :, :4], f),
                lambda: binding.norm_rotate(q, q, f.float()), lambda: binding.norm_rotate(q, q, f.cpu()),
                lambda: binding.norm_rotate(q.transpose(2, 3), q.transpose(2, 3), f),
                lambda: binding.norm_rotate(q, q, f, positions=torch.zeros(8, device="cuda", dtype=torch.int64)),
                lambda: binding.norm_rotate(q, q, f, positions=torch.zeros(7, device="cuda", dtype=torch.int32)),
                lambda: binding.norm_rotate(q, q, f, out=(q, q[:, :1])),
                lambda: binding.norm_rotate_backward(q, q, q, q[:, :1], f)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.FAError):
        binding.norm_rotate(q, q, f, out=(torch.empty_like(q).expand(1, 2, 8, 64)[:, :1].expand(1, 2, 8, 64), q.clone()))
    with pytest.raises(binding.FAError):   # rotated entries past the head, and no multiple of 16
        binding.norm_rotate(q, q, R.frequencies(128).cuda())
    with pytest.raises(binding.FAError):
        binding.norm_rotate(q, q, R.frequencies(20).cuda())
