"""Every tensor that the calls around attention allocate belongs to the stream that the call runs on."""
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
