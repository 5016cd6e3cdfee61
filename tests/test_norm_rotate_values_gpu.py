"""Norm and rotation of values at the ends of the range: what is not finite, sums of squares past FP32's range."""
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
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
