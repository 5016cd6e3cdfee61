"""Attention with a sliding window and sinks (fa_fwd_window, fa_bwd_window) against 64-bit masked attention."""
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding, inputs
from tests import _masked as M
from tests._parity import require_gpu, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# N, window, sinks: a single row, windows of one key, one tile, one more than a tile; sinks inside a
# tile, past a tile, past the window; windows and sinks longer than the row; tiles hidden between
# sinks and window; N = 2200 is past the short-row rule at d = 64
SHAPES = [(1, 1, 0), (1, 5, 9), (17, 5, 3), (128, 128, 0), (129, 1, 0), (129, 1, 1), (257, 128, 1), (300, 64, 200),
          (513, 127, 129), (640, 200, 130), (700, 130, 700), (1000, 129, 4), (1000, 3, 0), (900, 5000, 7), (2200, 300, 5)]


def see(N, window, sinks):
    at = torch.arange(N)
    return M.window_mask(at, at, window, sinks)


def run(w, window, sinks, stable=1, beta=1.25, stats=False):
    q, k, v, do = to_dev(w)
    out = binding.forward(q, k, v, scale=w.scale, stable=stable, beta=beta, stats=stats, window=window, sinks=sinks)
    grads = binding.backward(q, k, v, out[0], out[1], do, scale=w.scale, window=window, sinks=sinks)
    binding.device_status()
    return out, grads


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,window,sinks", SHAPES)
def test_forward_and_gradients(N, window, sinks, d):
    B, H = (2, 3) if N <= 700 else (1, 2)
    w = inputs.random_case(B, H, N, d, True, seed=7 * N + window + d, std=1.5)
    (o, lse), grads = run(w, window, sinks, stable=(N + window) % 3)
    ref = M.forward(w.q, w.k, w.v, see(N, window, sinks), w.scale)
    M.assert_within("o", o, ref["o"], ref["o_tol"])
    M.assert_lse(lse, ref["lse"])
    want, tol = M.backward(w.q, w.k, w.v, w.do, see(N, window, sinks), w.scale, ref)
    for name, got in zip(("dq", "dk", "dv"), grads):
        M.assert_within(name, got, want[name], tol[name])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,N,window,sinks", [(4, 8, 1500, 200, 4), (5, 7, 1301, 100, 0), (8, 12, 700, 50, 140),
                                                (8, 20, 400, 30, 1), (3, 11, 1100, 540, 200)])
def test_gradients_with_more_items_than_SMs(B, H, N, window, sinks, d):
    # (key tile, head) items dealt to the SMs: several light ones each, and fewer (none, more) with sinks
    w = inputs.random_case(B, H, N, d, True, seed=B * H + N, std=1.5)
    (o, lse), grads = run(w, window, sinks)
    ref = M.forward(w.q, w.k, w.v, see(N, window, sinks), w.scale)
    M.assert_within("o", o, ref["o"], ref["o_tol"])
    want, tol = M.backward(w.q, w.k, w.v, w.do, see(N, window, sinks), w.scale, ref)
    for name, got in zip(("dq", "dk", "dv"), grads):
        M.assert_within(name, got, want[name], tol[name])


# few heads and long rows: the key tiles with sinks are split over their queries (into 2 to 8 parts),
# last tiles whole and ragged
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,N,window,sinks", [(1, 2, 4224, 100, 4), (2, 1, 6200, 1, 1), (1, 1, 8300, 64, 200),
                                                (1, 2, 8200, 300, 500), (1, 1, 7900, 2900, 257)])
def test_gradients_of_sinks_split_over_their_queries(B, H, N, window, sinks, d):
    assert binding.fa_bwd_window_workspace_size(B, H, N, d, window, sinks) > binding.fa_bwd_workspace_size(B, H, N, d)
    w = inputs.random_case(B, H, N, d, True, seed=N + window + d, std=1.2)
    (o, lse), grads = run(w, window, sinks)
    (_, _), again = run(w, window, sinks)
    assert torch.equal(grads[1], again[1]) and torch.equal(grads[2], again[2])   # parts are joined in one order
    for b in range(B):
        for h in range(H):
            one = [x[b:b + 1, h:h + 1] for x in (w.q, w.k, w.v, w.do)]
            ref = M.forward(*one[:3], see(N, window, sinks), w.scale)
            want, tol = M.backward(*one, see(N, window, sinks), w.scale, ref)
            for name, got in zip(("dq", "dk", "dv"), grads):
                M.assert_within(name, got[b:b + 1, h:h + 1], want[name], tol[name])
            del ref, want, tol


@pytest.mark.parametrize("d,N", [(64, 1000), (64, 2300), (128, 700)])
@pytest.mark.parametrize("stable", [0, 1, 2])
def test_a_window_as_long_as_the_row_is_causal_attention(N, d, stable):
    w = inputs.random_case(1, 2, N, d, True, seed=N + d, std=1.3)
    q, k, v, do = to_dev(w)
    o, lse = binding.forward(q, k, v, causal=True, scale=w.scale, stable=stable)
    want = binding.backward(q, k, v, o, lse, do, causal=True, scale=w.scale)
    for window, sinks in ((N, 0), (N + 1000, 3), (2 ** 31 - 1, 2 ** 31 - 1), (1, N)):
        (ow, lsew), got = run(w, window, sinks, stable=stable)
        assert torch.equal(ow, o) and torch.equal(lsew, lse)
        assert torch.equal(got[2], want[2])
        # dq and dk: the first rows' delta is the windowed backward's own (more exact); both within the
        # bounds of the 64-bit gradient
        ref = M.forward(w.q, w.k, w.v, see(N, N, 0), w.scale)
        exact, tol = M.backward(w.q, w.k, w.v, w.do, see(N, N, 0), w.scale, ref)
        for name, a in zip(("dq", "dk"), got):
            M.assert_within(name, a, exact[name], tol[name])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("stable", [0, 1])
def test_statistics_are_those_of_the_visible_keys(d, stable):
    # dyadic inputs: every FP32 score is exact, so maxima, ties and branches are decidable
    N, window, sinks = 1024, 200, 3
    w = inputs.tiny_ties(N=N, H=2, d=d)
    (o, lse, st), _ = run(w, window, sinks, stable=stable, stats=True)
    s = (w.q.double() @ w.k.double().transpose(-1, -2)).masked_fill(~see(N, window, sinks), -math.inf)
    rm = s.amax(-1)
    rs = (s == rm[..., None]).sum(-1)
    assert torch.equal(st["row_max_raw"].cpu().double(), rm)
    assert torch.equal(st["row_ties"].cpu().long(), rs)
    branch = torch.where((rs > 1) & (rm > 0), 1, torch.where((rs > 1) & (rm < 0), 2, 0)) * stable
    assert torch.equal(st["row_branch"].cpu().long(), branch)
    rmin = s.masked_fill(~see(N, window, sinks), math.inf).amin(-1)
    assert torch.equal(st["row_min_raw"].cpu().double(), rmin)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,window,sinks", [(2, 2, 0), (5, 5, 0), (300, 1, 1), (300, 2, 0), (300, 3, 4), (2500, 2, 0),
                                            (2500, 8, 8), (2500, 17, 0)])
def test_gradients_of_rows_with_few_keys(N, window, sinks, d):
    # P, dP and delta in FP32; dS and the results rounded to BF16: two roundings of at most half a step
    # (2^-8) each, so dq and dk are within 2^-8 sqrt(2) = 5.5e-3 in norm at worst; uniformly spread
    # rounding errors have a third of the variance of the worst case: 3.2e-3.  17 keys use the stored O.
    w = inputs.random_case(2, 4, N, d, True, seed=N + window, std=math.sqrt(3))
    _, grads = run(w, window, sinks)
    m = see(N, window, sinks)
    want, _ = M.backward(w.q, w.k, w.v, w.do, m, w.scale, M.forward(w.q, w.k, w.v, m, w.scale))
    for name, got in zip(("dq", "dk", "dv"), grads):
        off = ((got.cpu().double() - want[name]).norm() / want[name].norm()).item()
        assert off <= (3.2e-3 if window + sinks <= 16 else 5.5e-3), (name, off)


def test_gradient_against_differences():
    # directional derivatives of L = sum(dO o O) in 64 bits, by central differences
    N, d, window, sinks = 200, 64, 40, 2
    w = inputs.random_case(1, 1, N, d, True, seed=3, std=1.0)
    _, grads = run(w, window, sinks)
    m = see(N, window, sinks)
    ref = M.forward(w.q, w.k, w.v, m, w.scale)
    _, tol = M.backward(w.q, w.k, w.v, w.do, m, w.scale, ref)
    x = [t.double() for t in (w.q, w.k, w.v)]
    g = torch.Generator().manual_seed(1)
    eps = 1e-4
    for i, name in enumerate(("dq", "dk", "dv")):
        u = torch.randn(x[i].shape, generator=g, dtype=torch.float64)
        lo, hi = list(x), list(x)
        lo[i], hi[i] = x[i] - eps * u, x[i] + eps * u
        loss = [(M.forward(*y, m, w.scale)["o"] * w.do.double()).sum().item() for y in (lo, hi)]
        diff = (loss[1] - loss[0]) / (2 * eps)
        got = (grads[i].cpu().double() * u).sum().item()
        # second-order remainder of the difference: under 1e-4 here (eps^2 times third derivatives)
        assert abs(got - diff) <= (tol[name] * u.abs()).sum().item() + 1e-3, name


def test_hidden_keys_have_no_influence():
    # keys before the window and past the sinks: their K and V may be anything finite, and the
    # queries that do not see them give the same bits
    N, d, window, sinks = 700, 64, 100, 5
    w = inputs.random_case(1, 2, N, d, True, seed=11)
    q, k, v, do = to_dev(w)
    o, lse = binding.forward(q, k, v, window=window, sinks=sinks)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, sinks:200] = 3e38
    v2[:, :, sinks:200] = -3e30
    k2[:, :, sinks:200, ::2] = -3e38
    o2, lse2 = binding.forward(q, k2, v2, window=window, sinks=sinks)
    first = 200 + window - 1      # the first query that sees none of the changed keys
    assert torch.equal(o2[:, :, first:], o[:, :, first:]) and torch.equal(lse2[:, :, first:], lse[:, :, first:])
    binding.fa_device_report_read()   # the changed rows may hold Inf: clear the record


def test_capture_and_another_stream():
    w = inputs.random_case(2, 4, 640, 128, True, seed=21)
    q, k, v, do = to_dev(w)
    (o, lse), (dq, dk, dv) = run(w, 150, 4)
    ws = torch.empty(binding.fa_bwd_workspace_size(2, 4, 640, 128), device="cuda", dtype=torch.uint8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o1, lse1 = binding.forward(q, k, v, scale=w.scale, window=150, sinks=4)
        g1 = binding.backward(q, k, v, o1, lse1, do, scale=w.scale, workspace=ws, window=150, sinks=4)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o1, o) and torch.equal(g1[1], dk) and torch.equal(g1[2], dv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = binding.forward(q, k, v, scale=w.scale, window=150, sinks=4)
        g2 = binding.backward(q, k, v, o2, lse2, do, scale=w.scale, workspace=ws, window=150, sinks=4)
    for _ in range(2):
        o2.zero_()
        g2[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, o) and torch.equal(lse2, lse) and torch.equal(g2[1], dk) and torch.equal(g2[2], dv)
    binding.device_status()
