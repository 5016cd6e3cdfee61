"""Every tensor that the calls around attention allocate belongs to the stream that the call runs on; programs on two streams."""
import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _paged as P
from tests import _rotate as R
from tests import _weights as W
from tests._parity import require_gpu
from tests.test_buffers_gpu import owner, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def calls():
    g = torch.Generator().manual_seed(1)
    _, q, k = (x.cuda() for x in R.heads(2, 50, 4, 2, 64, g))
    f, w = R.frequencies(64).cuda(), torch.ones(64, device="cuda")
    c = P.make([70, 9], 2, 64, 16, "e4m3", seed=1, spare=9)
    cache, sc, ip = (c.k, c.v, c.table, c.kv_len), dict(k_scale=c.ks, v_scale=c.vs), P.indptr([1, 1])
    rows = torch.zeros((2, 2, 64), device="cuda", dtype=torch.bfloat16)
    weights = W.make(c, seed=1)[0].cuda()
    return {
        "norm_rotate": lambda s: binding.norm_rotate(q, k, f, q_weight=w, k_weight=w, stream=s),
        "norm_rotate_backward": lambda s: binding.norm_rotate_backward(q, k, q, k, f, q_weight=w, k_weight=w, stream=s),
        "qkv_append": lambda s: [binding.qkv_append(rows, rows, rows, *cache, ip, f, stream=s, **sc)],
        "kv_evict": lambda s: binding.kv_evict(weights, *cache, 20, stream=s, **sc),
    }


@pytest.mark.parametrize("name", ["norm_rotate", "norm_rotate_backward", "qkv_append", "kv_evict"])
def test_outputs_belong_to_the_calls_stream(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream, want in ((side, side.cuda_stream), (None, torch.cuda.current_stream().cuda_stream)):
        got = list(tensors(call(stream)))
        torch.cuda.synchronize()
        assert got and all(owner(t) == want for t in got)
    binding.device_status()


@pytest.mark.parametrize("formats", [("e4m3", "bf16"), ("e4m3", "e4m3")])
def test_programs_on_two_streams_at_once(formats):
    # each with a cache of its own; the sums of both are those of one program alone
    def program(i, fmt, stream):
        hkv, d, new = (2, 128, [200, 1]) if i else (4, 64, [1, 1])
        lens = [5000, 900]
        g = torch.Generator().manual_seed(i)
        with torch.cuda.stream(stream):
            c = P.make(lens, hkv, d, 32, fmt, seed=i)
            w = torch.zeros((c.P, hkv, 32), device="cuda")
            rows = torch.randn((sum(new), 3 * hkv, d), generator=g).to(torch.bfloat16).cuda()
            f, ip = R.frequencies(d).cuda(), P.indptr(new)
            sc = {} if c.ks is None else dict(k_scale=c.ks, v_scale=c.vs)
            cache = (c.k, c.v, c.table, c.kv_len)

        def step():
            q = binding.qkv_append(rows[:, :hkv], rows[:, hkv:2 * hkv], rows[:, 2 * hkv:], *cache, ip, f, stream=stream, **sc)
            _, lse = binding.forward_paged(q, *cache, ip, max(new), stream=stream, **sc)
            binding.kv_accumulate(w, q, lse, *cache, ip, max(new), stream=stream, **sc)
            left, kept = binding.kv_evict(w, *cache, 6000, stream=stream, **sc)
            return [q, lse, w, left, kept]
        return step

    alone = [program(i, fmt, torch.cuda.current_stream()) for i, fmt in enumerate(formats)]
    want = []
    for step in alone:
        for _ in range(6):
            out = step()
        torch.cuda.synchronize()
        want.append(out)
    steps = [program(i, fmt, torch.cuda.Stream()) for i, fmt in enumerate(formats)]
    torch.cuda.synchronize()
    for _ in range(6):
        got = [step() for step in steps]
    torch.cuda.synchronize()
    binding.device_status()
    for x, y in zip(want, got):
        for a, b in zip(x, y):
            assert torch.equal(a.nan_to_num(), b.nan_to_num())
