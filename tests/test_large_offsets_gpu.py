"""Offsets past 32 bits: the serving calls on the last pages of a large pool, norm and rotation of a long sequence."""
import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _paged as P
from tests import _rotate as R
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


PAGE, D, STRIDE = 16, 128, 4096


def serve(pages, first, fmt):
    """A prompt and a token through append, attention, weights and evictions, in a pool of `pages` from page `first` on."""
    dev = dict(device="cuda")
    pool = torch.zeros((pages, 2, 1, PAGE, D), dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8, **dev)
    assert pool.stride(0) == STRIDE
    side = torch.zeros(pages * STRIDE, **dev)           # scales and weights: a page's STRIDE floats apart too
    ks, vs, w = (side.as_strided((pages, 1, PAGE), (STRIDE, PAGE, 1), i * PAGE) for i in range(3))
    scales = {} if fmt == "bf16" else dict(k_scale=ks, v_scale=vs)
    lens, per = [300, 70], 24
    table, other = (first + torch.arange(i * 2 * per, (i + 1) * 2 * per, **dev, dtype=torch.int32).view(2, per) for i in (0, 1))
    g = torch.Generator().manual_seed(3)
    f = R.frequencies(D).cuda()
    out = []
    kv_len = torch.zeros(2, **dev, dtype=torch.int32)
    for new, to in ((lens, other), ([1, 1], None)):
        T = sum(new)
        q, k, v = (torch.randn((T, h, D), generator=g).to(torch.bfloat16).cuda() for h in (4, 1, 1))
        ip = P.indptr(new)
        kv_len = kv_len + torch.tensor(new, **dev, dtype=torch.int32)
        cache = (pool[:, 0], pool[:, 1], table, kv_len)
        qa = binding.qkv_append(q, k, v, *cache, ip, f, **scales)
        o, lse = binding.forward_paged(qa, *cache, ip, max(new), **scales)
        binding.kv_accumulate(w, qa, lse, *cache, ip, max(new), **scales)
        kv_len, kept = binding.kv_evict(w, *cache, 60, sinks=2, recent=9, table_out=to, **scales)
        table = table if to is None else to
        n = int(kv_len.sum())
        out += [qa, o, lse, kv_len, kept, w[table.long()][:, :3],
                *binding.kv_read(pool[:, 0], pool[:, 1], table, kv_len, P.indptr(kv_len.tolist()), n, **scales)]
    binding.device_status()
    return [x.cpu() for x in out]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_cache(fmt):
    pages = 2 ** 31 // STRIDE + 1000
    for x, y in zip(serve(100, 0, fmt), serve(pages, pages - 96, fmt)):
        assert torch.equal(x, y)


def test_keep_of_any_size():
    # what is behind the kept keys is filled up to the last of 2^31 - 1 places
    pages = torch.zeros((24, 2, 1, PAGE, D), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((24, 1, PAGE), device="cuda")
    table, kv_len = torch.arange(24, device="cuda", dtype=torch.int32)[None], torch.tensor([300], device="cuda", dtype=torch.int32)
    left, kept = binding.kv_evict(w, pages[:, 0], pages[:, 1], table, kv_len, 2 ** 31 - 1)
    binding.device_status()
    assert int(left) == 300 and kept[0, 0, :300].tolist() == list(range(300))
    assert int(kept[0, 0, 300:].max()) == -1 and int(kept[0, 0, 300:].min()) == -1


def test_norm_rotate():
    N, hq, hkv, last = 2 ** 22 + 3, 4, 1, 65
    rows = torch.randn((1, N, hq + hkv, D), device="cuda", dtype=torch.bfloat16)
    q, k = rows[:, :, :hq].transpose(1, 2), rows[:, :, hq:].transpose(1, 2)
    f, w = R.frequencies(D).cuda(), torch.linspace(0.5, 1.5, D, device="cuda")
    kw = dict(q_weight=w, k_weight=w)
    z = binding.norm_rotate(q, k, f, **kw)
    assert z[0].numel() > 2 ** 31
    dx = binding.norm_rotate_backward(q, k, *z, f, **kw)[:2]
    at = torch.arange(N - last, N, device="cuda", dtype=torch.int32)
    tail = [x[:, :, -last:] for x in (q, k)]
    zt = binding.norm_rotate(*tail, f, positions=at, **kw)
    dt = binding.norm_rotate_backward(*tail, *zt, f, positions=at, **kw)[:2]
    for x, y in zip((*z, *dx), (*zt, *dt)):
        assert torch.equal(x[:, :, -last:], y)
