"""Every tensor that a call allocates belongs to the stream that the call runs on.

The allocator hands memory that one stream has freed to that stream's next request at once: a tensor that
belongs to another stream than the one writing it may still be in use there.
"""
import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _paged as P
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def owner(t):
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's segments")


def tensors(x):
    for t in x.values() if isinstance(x, dict) else x:
        if torch.is_tensor(t):
            yield t
        else:
            yield from tensors(t)


def calls():
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn((1, 2, 200, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    o, lse = binding.forward(q, k, v)
    q8 = torch.zeros((1, 2, 200, 64), device="cuda", dtype=torch.uint8)
    ones = torch.ones(3, device="cuda")
    c = P.make([70, 9], 2, 64, 16, "bf16", seed=1)
    cache, ip = (c.k, c.v, c.table, c.kv_len), P.indptr([1, 1])
    qp = torch.zeros((2, 4, 64), device="cuda", dtype=torch.bfloat16)
    return {
        "forward": lambda s: binding.forward(q, k, v, stats=True, stream=s),
        "forward, window": lambda s: binding.forward(q, k, v, stats=True, window=30, sinks=2, stream=s),
        "backward": lambda s: binding.backward(q, k, v, o, lse, do, want_delta=True, stream=s),
        "backward, window": lambda s: binding.backward(q, k, v, o, lse, do, want_delta=True, window=30, stream=s),
        "quantize_fp8": lambda s: binding.quantize_fp8(q, stream=s),
        "forward_fp8": lambda s: binding.forward_fp8(q8, q8, q8, ones, stats=True, stream=s),
        "kv_read": lambda s: binding.kv_read(*cache, P.indptr([70, 9]), 79, stream=s),
        "forward_paged": lambda s: binding.forward_paged(qp, *cache, ip, 1, stream=s),
    }


@pytest.mark.parametrize("name", ["forward", "forward, window", "backward", "backward, window", "quantize_fp8", "forward_fp8",
                                  "kv_read", "forward_paged"])
def test_outputs_belong_to_the_calls_stream(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream, want in ((side, side.cuda_stream), (None, torch.cuda.current_stream().cuda_stream)):
        got = list(tensors(call(stream)))
        torch.cuda.synchronize()
        assert len(got) >= 2 and all(owner(t) == want for t in got)
    binding.device_status()
