"""What accumulated attention weights are off by on average: over the attention call's log-sum-exps, and between the kernel's forms."""
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _paged as P
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def cache(n, d, fmt, seed, page=64):
    """One sequence of n keys, one kv head: the cache's tensors, its scales and the keys in 64 bits [n, d]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = ((torch.randn((n, 1, d), generator=g, device="cuda") * 1.5).to(torch.bfloat16) for _ in range(2))
    dtype = torch.bfloat16 if fmt == "bf16" else torch.uint8
    kc, vc = (torch.zeros((-(-n // page), 1, page, d), device="cuda", dtype=dtype) for _ in range(2))
    sc = {} if fmt == "bf16" else {x: torch.zeros(kc.shape[:3], device="cuda") for x in ("k_scale", "v_scale")}
    args = kc, vc, torch.arange(kc.shape[0], device="cuda", dtype=torch.int32)[None], torch.tensor([n], device="cuda", dtype=torch.int32)
    binding.kv_append(k, v, *args, P.indptr([n]), **sc)
    keys = kc.double() if fmt == "bf16" else kc.view(P.E4M3).double() * sc["k_scale"].double()[..., None]
    return args, sc, keys.reshape(-1, d)[:n]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 1024])
def test_weights_over_the_attention_calls_log_sum_exps(fmt, d, T):
    # The formula's weights of the log-sum-exps that forward_paged returned, in 64 bits.  Mean over all weights: the exponential is
    # off by 2^-22 of its value at most; q . k by half a unit of the last place on average (what is left of its cut sums), and
    # the scale in FP32 by half a unit, both of the mean score; roundings of a row's exponent (2^-21) go to either side and
    # are left by 2^-21 / sqrt(12 rows), of which four are allowed.
    n, hq = 16000, 8
    args, sc, keys = cache(n, d, fmt, d)
    g = torch.Generator(device="cuda").manual_seed(T)
    q = (torch.randn((T, hq, d), generator=g, device="cuda") * 2.5).to(torch.bfloat16)
    scale = d ** -0.5
    _, lse = binding.forward_paged(q, *args, P.indptr([T]), T, scale=scale, **sc)
    w = torch.zeros(args[0].shape[:3], device="cuda")
    binding.kv_accumulate(w, q, lse, *args, P.indptr([T]), T, scale=scale, **sc)
    binding.device_status()
    want, score = torch.zeros(n, device="cuda", dtype=torch.float64), 0.0
    hidden = torch.arange(n, device="cuda") > torch.arange(n - T, n, device="cuda")[:, None]
    for h in range(hq):
        s = (q[:, h].double() @ keys.T * scale).masked_fill_(hidden, -math.inf)
        p = torch.exp(s - lse[:, h].double()[:, None])
        want += p.sum(0)
        score += float((p * s.clamp(min=-1e3)).sum()) / (T * hq)
    off = float(w.double().sum() / want.sum()) - 1
    assert abs(off) <= 2.0 ** -22 + score * 2.0 ** -23 + 4 * 2.0 ** -21 / math.sqrt(12 * T * hq), (off * 2 ** 23, score)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("most", [(4, 17), (4, 8)])
def test_forms_over_e4m3_agree_on_average(d, one_sign, most):
    # max_q settles the form: 32, 64 or 128 columns for 8 heads of 4, 8 and 17 tokens.  They add up the same products, and none
    # may be off by more than half a unit of the last place of q . k on average, which products of one sign would show.  Two
    # hundred log-sum-exps take the roundings of the exponents (2^-21 / sqrt(12) each) out of the mean.
    n, T, hq, tries = 20000, 4, 8, 200
    (k, v, table, kv_len), sc, keys = cache(n, d, "e4m3", d)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = (torch.randn((T, hq, d), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    if one_sign:
        k, keys, q = k & 0x7F, keys.abs(), q.abs()
    scale = d ** -0.5
    s = q[-1, 3].double() @ keys.T * scale
    seen = s > s.amax() - 4
    total = []
    for m in most:
        logs = torch.zeros(n, device="cuda", dtype=torch.float64)
        for i in range(tries):
            lse = torch.full((T, hq), math.inf, device="cuda")      # one row counts
            lse[-1, 3] = s.amax() + 0.0317 * i
            w = torch.zeros(k.shape[:3], device="cuda")
            binding.kv_accumulate(w, q, lse, k, v, table, kv_len, P.indptr([T]), m, scale=scale, **sc)
            logs += w.reshape(-1)[:n].double().log()
        total.append((logs[seen] / tries).mean())
    binding.device_status()
    assert abs(float(total[0] - total[1])) <= 0.5 * 2.0 ** -23 * float(s[seen].mean()) + 4 * 2.0 ** -21 / math.sqrt(12 * tries)
