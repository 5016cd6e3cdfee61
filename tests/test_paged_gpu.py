"""Attention over paged caches (fa_fwd_paged) against 64-bit attention of the cached values."""
import math

import pytest
import torch

from numerics_tcgen05_tmem_gb300 import binding
from tests import _masked as M
from tests import _paged as P
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def queries(new, hq, d, seed, std=1.5):
    g = torch.Generator().manual_seed(1000 + seed)
    return (torch.randn((sum(new), hq, d), generator=g) * std).to(torch.bfloat16)


def attend(c, q, new, max_q=None, **kw):
    out = binding.forward_paged(q.cuda() if not q.is_cuda else q, c.k, c.v, c.table, c.kv_len, P.indptr(new),
                                max(new) if max_q is None else max_q, k_scale=c.ks, v_scale=c.vs, **kw)
    return out


def check(c, new, group, seed=0, window=None, sinks=0, q=None, max_q=None, **kw):
    q = queries(new, c.hkv * group, c.d, seed) if q is None else q
    o, lse = attend(c, q, new, max_q=max_q, window=window, sinks=sinks, **kw)
    binding.device_status()
    scale = kw.get("scale", 1 / math.sqrt(c.d))
    want, want_lse, tol = P.reference(c, q.cpu(), new, scale, window, sinks)
    M.assert_within("o", o, want, tol)
    M.assert_lse(lse, want_lse)
    return o, lse


# lengths around the block, page and tile borders, a few long ones
DECODE = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1025, 3000]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,group,page", [(1, 1, 16), (2, 4, 32), (3, 7, 64), (8, 8, 128), (2, 16, 256), (1, 20, 64),
                                            (2, 33, 16), (1, 64, 32), (1, 71, 64), (1, 128, 128)])
def test_single_tokens(fmt, d, hkv, group, page):
    c = P.make(DECODE, hkv, d, page, fmt, seed=group + d)
    check(c, [1] * len(DECODE), group, seed=page)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 0), (65, 64), (100, 70), (700, 5), (5000, 2)])
def test_single_tokens_with_a_window(fmt, d, window, sinks):
    c = P.make(DECODE, 2, d, 32, fmt, seed=window + d)
    check(c, [1] * len(DECODE), 4, window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,new", [(1, 64), (2, 7), (3, 20), (4, 16), (8, 8), (5, 3)])
def test_few_tokens(fmt, d, group, new):
    c = P.make([new, new + 1, 70, 200, 1000], 2, d, 16, fmt, seed=group * new)
    check(c, [new] * 5, group)
    check(c, [new] * 5, group, window=50, sinks=3)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,group,page", [(1, 1, 16), (2, 4, 32), (2, 3, 64), (1, 7, 128), (1, 16, 256), (1, 100, 64)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (129, 1), (300, 150)])
def test_chunks(fmt, d, hkv, group, page, window, sinks):
    new = [130, 1, 257, 40, 300] if group <= 16 else [3, 9]
    lens = [130, 900, 700, 41, 1500] if group <= 16 else [40, 600]
    c = P.make(lens, hkv, d, page, fmt, seed=group + page)
    check(c, new, group, window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,kv", [(65, 65), (100, 5000), (256, 4100), (257, 2000), (700, 700)])
def test_one_sequence_split_over_its_keys(fmt, n, kv):
    # one kv head and one sequence: the tiles alone would leave most SMs idle, so the keys are split
    c = P.make([kv], 1, 128, 64, fmt, seed=n)
    check(c, [n], 1)
    check(c, [n], 1, window=1000, sinks=4)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 8])
def test_sequences_without_tokens_and_rows_without_keys(fmt, group):
    # a sequence without new tokens, lengths of zero, lengths shorter than the new tokens
    lens, new = [0, 5, 300, 3, 0, 64, 20], [1, 0, 2, 6, 0, 1, 200]
    c = P.make(lens, 2, 64, 16, fmt, seed=9)
    o, lse = check(c, new, group)
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    check(c, new, group, window=3, sinks=1)
    few = [min(n, 6) for n in new]
    check(c, few, group)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 200, 9]])
def test_strides_orders_and_padding(fmt, new):
    # K and V interleaved in one pool, q a slice of a fused projection, a padded batch
    c = P.make([77, 333, 1200], 2, 128, 32, fmt, seed=3, combined=True)
    T, hq = sum(new), 8
    g = torch.Generator().manual_seed(5)
    fused = (torch.randn((T + 4, hq + 4, 128), generator=g) * 1.5).to(torch.bfloat16).cuda()
    fused[T:] = math.nan
    q = fused[:, :hq]
    out = torch.full((T + 4, hq, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((T + 4, hq), 7.0, device="cuda")
    attend(c, q, new, out=out, lse=lse)
    binding.device_status()
    want, want_lse, tol = P.reference(c, q[:T].cpu(), new, 1 / math.sqrt(128))
    M.assert_within("o", out[:T], want, tol)
    M.assert_lse(lse[:T], want_lse)
    assert (out[T:] == 7).all() and (lse[T:] == 7).all()
    if fmt == "e4m3":   # codes as float8 tensors are the same cache
        c.k, c.v = c.k.view(P.E4M3), c.v.view(P.E4M3)
        o2, _ = attend(c, q[:T], new)
        assert torch.equal(o2, out[:T])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_std,k_std", [(1e-30, 1e30), (1e20, 1e-20), (100.0, 0.01), (1e-38, 1e-3)])
def test_extreme_magnitudes(fmt, q_std, k_std):
    # Q and K of very different size: the scores themselves stay moderate
    c = P.make([300, 17], 1, 64, 16, fmt, seed=1, std=k_std)
    for new, group in (([1, 1], 4), ([100, 3], 4)):
        q = queries(new, group, 64, 2, std=q_std)
        check(c, new, group, q=q, scale=0.125)


def test_overlapping_tensors_are_refused():
    # a stride below an entry's size (expand) would not describe the memory that the kernels address
    c = P.make([40, 40], 2, 64, 16, "e4m3", seed=1)
    q = queries([1, 1], 4, 64, 1).cuda()
    ip = P.indptr([1, 1])
    ok = dict(k_scale=c.ks, v_scale=c.vs)

    def refused(*a, **kw):
        with pytest.raises(ValueError):
            binding.forward_paged(*a, **kw)

    binding.forward_paged(q, c.k, c.v, c.table, c.kv_len, ip, 1, **ok)
    refused(q[:1].expand(2, 4, 64), c.k, c.v, c.table, c.kv_len, ip, 1, **ok)
    refused(q, c.k[:1].expand(4, 2, 16, 64), c.v[:1].expand(4, 2, 16, 64), c.table, c.kv_len, ip, 1,
            k_scale=c.ks[:4], v_scale=c.vs[:4])
    refused(q, c.k, c.v, c.table[:1].expand(2, c.table.shape[1]), c.kv_len, ip, 1, **ok)
    refused(q, c.k, c.v, c.table, c.kv_len, ip, 1, k_scale=c.ks[:1].expand(c.P, 2, 16), v_scale=c.vs[:1].expand(c.P, 2, 16))
    refused(q, c.k.transpose(1, 2), c.v.transpose(1, 2), c.table, c.kv_len, ip, 1, **ok)
    with pytest.raises(ValueError):
        binding.kv_append(q[:, :2], q[:1, :2].expand(2, 2, 64), c.k, c.v, c.table, c.kv_len, ip, **ok)
    binding.device_status()


@pytest.mark.parametrize("new,group", [([1, 2], 8), ([90, 3], 8)])
def test_scales_of_other_quantisers(new, group):
    # scales that are no powers of two, negative, zero and subnormal ones
    c = P.make([300, 77], 1, 64, 16, "e4m3", seed=4)
    g = torch.Generator().manual_seed(9)
    c.ks *= (torch.rand(c.ks.shape, generator=g) + 0.5).cuda()
    mult = torch.rand(c.vs.shape, generator=g) + 0.5
    mult[torch.rand(c.vs.shape, generator=g) < 0.3] *= -1
    mult[torch.rand(c.vs.shape, generator=g) < 0.1] = 0
    mult[torch.rand(c.vs.shape, generator=g) < 0.1] = 2.0 ** -125   # times a scale near 2^-7: subnormal
    c.vs *= mult.cuda()
    for b, n in enumerate(c.lens):
        t = torch.arange(n)
        pg = c.table[b].cpu().long()[t // 16]
        for w, (codes, s) in enumerate(((c.k, c.ks), (c.v, c.vs))):
            x = codes.cpu()[pg, :, t % 16].view(P.E4M3).double() * s.cpu()[pg, :, t % 16].double()[..., None]
            c.values[b][w] = x.transpose(0, 1)
    q = queries(new, group, 64, 6)
    o, lse = attend(c, q, new)
    binding.device_status()
    want, want_lse, tol = P.reference(c, q, new, 0.125)
    # a kernel may round K and V to BF16 (half a step each): V adds 2^-8 of |O|'s terms, as much again as
    # P~'s rounding; a score moves by at most 2^-8 sum |q_i k_i| scale, and P by that much relatively
    s_err = 0.0
    for b in range(2):
        rows = slice(0, new[0]) if b == 0 else slice(new[0], sum(new))
        s_err = max(s_err, (q[rows].double().abs() @ c.values[b][0][0].abs().T).max().item() * 0.125 * M.HALF)
    M.assert_within("o", o, want, (2 + 2 * s_err / M.HALF) * tol)
    fin = torch.isfinite(want_lse)
    assert (lse.cpu().double() - want_lse)[fin].abs().max() <= s_err + M.LSE_TOL


def test_a_side_stream_owns_its_workspace():
    # with stream=... the call's own buffers must not be handed to the current stream's next allocation
    c = P.make([20000] * 4, 2, 128, 64, "bf16", seed=3)
    q = queries([1] * 4, 8, 128, 1).cuda()
    want, _ = attend(c, q, [1] * 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ip = P.indptr([1] * 4)
    torch.cuda.synchronize()
    for _ in range(20):
        o, _ = binding.forward_paged(q, c.k, c.v, c.table, c.kv_len, ip, 1, stream=side)
        junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        del junk


def bf16_twin(c):
    """The same cache in BF16: each code times its scale (exact for the powers of two that scales are)."""
    t = P.SimpleNamespace(**vars(c))
    t.fmt, t.ks, t.vs = "bf16", None, None
    t.k, t.v = ((x.view(torch.float8_e4m3fn).float() * s[..., None]).to(torch.bfloat16)
                for x, s in ((c.k, c.ks), (c.v, c.vs)))
    return t


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("hkv,group,lens,new,window,sinks", [
    (2, 4, [1500], [500], None, 0), (3, 1, [1700], [1700], None, 0), (1, 7, [3100, 900], [450, 500], None, 0),
    (2, 16, [2000, 40, 600], [260, 1, 290], None, 0), (1, 4, [5000], [1500], 1300, 200),
    (1, 8, [2600, 3000], [700, 900], 900, 0), (2, 4, [2900], [2000], 2000, 1), (1, 2, [900, 1800], [1000, 1500], None, 0)])
def test_chunks_of_a_copied_cache(d, page, hkv, group, lens, new, window, sinks):
    # E4M3 chunks with many tiles read BF16 pages that the call writes to its workspace first: the bits of
    # the same call on a BF16 cache, whatever the workspace held, and nothing outside of it written
    c = P.make(lens, hkv, d, page, "e4m3", seed=d + page + len(new))
    cap = c.table.shape[1] * page
    args = (sum(new), len(new), max(new), hkv * group, hkv, d, cap, window or 0, sinks)
    n = binding.fa_fwd_paged_workspace_size(*args, binding.FA_KV_E4M3)
    assert n > binding.fa_fwd_paged_workspace_size(*args)
    q = queries(new, hkv * group, d, 3)
    kw = dict(window=window, sinks=sinks)
    want = attend(bf16_twin(c), q, new, **kw)
    for fill in (0xFF, 0x7F, 0x00):
        ws = torch.full((n + 4096,), fill, device="cuda", dtype=torch.uint8)
        o, lse = attend(c, q, new, workspace=ws[:n], **kw)
        torch.cuda.synchronize()
        assert (ws[n:] == fill).all()
        row = 0
        for b, m in enumerate(new):
            r = slice(row, row + m)
            # (in the last case, rows before the sequence's first key see nothing: 0 and -inf in both)
            if m * group > 16:   # the others' kernel reads the codes, and rounds elsewhere
                assert torch.equal(o[r], want[0][r]) and torch.equal(lse[r], want[1][r]), b
            row += m
    check(c, new, group, q=q, **kw)


def test_a_captured_chunk_of_a_copied_cache_follows_lengths():
    c = P.make([1500, 1300], 2, 128, 32, "e4m3", seed=5)
    new = [700, 500]
    q = queries(new, 8, 128, 2).cuda()
    kw = dict(window=1100, sinks=3)
    ip = P.indptr(new)

    def step(x):
        return binding.forward_paged(q, x.k, x.v, x.table, x.kv_len, ip, max(new), k_scale=x.ks, v_scale=x.vs, **kw)

    step(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step(c)
    for lens in ([1500, 1300], [700, 1299], [1201, 300], [900, 0]):
        c.kv_len.copy_(torch.tensor(lens))
        o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse = step(bf16_twin(c))
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
    binding.device_status()


@pytest.mark.parametrize("v_std", [1e-25, 1e25])
def test_v_scales_of_any_size(v_std):
    # E4M3 vectors whose scales differ by many powers of two, in both kernels
    c = P.make([400], 1, 64, 16, "e4m3", seed=4)
    sizes = torch.exp2(torch.randint(-12, 12, (c.P, 1, 16), generator=torch.Generator().manual_seed(1)).float())
    c.vs *= sizes.cuda() * 2.0 ** round(math.log2(v_std))
    t = torch.arange(400)
    pg = c.table[0].cpu().long()[t // 16]
    s = c.vs.cpu()[pg, :, t % 16].double()
    codes = c.v.cpu()[pg, :, t % 16].view(P.E4M3).double()
    c.values[0][1] = (codes * s[..., None]).transpose(0, 1)
    for new, group in (([1], 8), ([90], 8)):
        q = queries(new, group, 64, 6)
        o, lse = attend(c, q, new)
        binding.device_status()
        want, want_lse, tol = P.reference(c, q, new, 0.125)
        M.assert_within("o", o, want, tol + M.HALF ** 2 * want.abs().amax())
        M.assert_lse(lse, want_lse)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [5, 150, 1, 64], [100, 700, 900, 70]])
def test_bad_entries_are_reported_and_not_followed(fmt, new):
    lens = [100, 400, 900, 70]
    q = queries(new, 8, 64, 8)
    good = P.make(lens, 2, 64, 16, fmt, seed=2)
    want, want_lse, tol = P.reference(good, q, new, 0.125)
    rows = list(P.indptr(new).cpu())
    for what in ("page", "negative", "length", "indptr"):
        c = P.make(lens, 2, 64, 16, fmt, seed=2)
        kw = {}
        ip = P.indptr(new)
        if what == "page":
            c.table[1, 3] = c.P
        elif what == "negative":
            c.table[1, 3] = -1
        elif what == "length":
            c.kv_len[1] = 2 ** 31 - 1
        else:
            ip[2] = ip[1] - 1      # sequence 1 has a negative number of rows
        binding.fa_device_report_read()
        o2, lse2 = binding.forward_paged(q.cuda(), c.k, c.v, c.table, c.kv_len, ip, max(new), k_scale=c.ks, v_scale=c.vs, **kw)
        rc, rep = binding.fa_device_report_read()
        assert rc == binding.FA_ERR_DEVICE_BOUNDS and rep["flags"] & binding.FA_DEVFLAG_BOUNDS, what
        for b in (0, 3) if what == "indptr" else (0, 2, 3):
            r = slice(rows[b], rows[b + 1])
            M.assert_within(f"{what}, sequence {b}", o2[r], want[r], tol[r])
            M.assert_lse(lse2[r], want_lse[r])
    # more new tokens than max_q says: reported, and nothing past the tiles that were planned is touched
    if max(new) > 1:
        attend(good, q, new, max_q=max(new) - 1)
        assert binding.fa_device_report_read()[0] == binding.FA_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1] * 9, [300, 1, 2, 1, 40, 1, 1, 100, 1]])
def test_repeats_are_bit_identical_on_any_stream(fmt, new):
    c = P.make([300 + 211 * i for i in range(9)], 2, 128, 64, fmt, seed=6)
    q = queries(new, 8, 128, 1).cuda()
    o, lse = attend(c, q, new)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        for _ in range(3):
            o2, lse2 = attend(c, q, new, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(o2, o) and torch.equal(lse2, lse)
    binding.device_status()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("steps,max_new", [(5, 1), (3, 150)])
def test_a_captured_step_follows_lengths(fmt, steps, max_new):
    # one graph of append + attention, replayed while the sequences grow; the same steps eagerly
    lens = [250, 63, 700]
    hkv, hq, d, page = 2, 8, 64, 64
    grown = P.make([n + 1000 for n in lens], hkv, d, page, fmt, seed=12)
    table, pools = grown.table, [grown.k.clone(), grown.v.clone()]
    scales = [grown.ks.clone(), grown.vs.clone()] if fmt == "e4m3" else [None, None]
    T = 3 * max_new
    kn, vn = (torch.zeros((T, hkv, d), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.zeros((T, hq, d), device="cuda", dtype=torch.bfloat16)
    kv_len = torch.tensor(lens, device="cuda", dtype=torch.int32)
    ip = P.indptr([0, 0, 0])

    def step(k, v, ks, vs):
        binding.kv_append(kn, vn, k, v, table, kv_len, ip, k_scale=ks, v_scale=vs)
        return binding.forward_paged(q, k, v, table, kv_len, ip, max_new, k_scale=ks, v_scale=vs, window=400, sinks=2)

    mine = [x.clone() if x is not None else None for x in pools + scales]
    step(*mine)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step(*mine)
    other = [x.clone() if x is not None else None for x in pools + scales]
    g = torch.Generator().manual_seed(3)
    for i in range(steps):
        new = [1 + (i * 7 + b * 31) % max_new for b in range(3)]
        n = sum(new)
        ip.copy_(P.indptr(new))
        kv_len.add_(torch.tensor(new, device="cuda", dtype=torch.int32))
        for x in (kn, vn, q):
            x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse = step(*other)
        torch.cuda.synchronize()
        assert torch.equal(o[:n], want[:n]) and torch.equal(lse[:n], want_lse[:n])
        for a, b in zip(mine, other):
            if a is not None:   # poisoned scales are NaN: compare bits
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    binding.device_status()


def test_append_attend_read_together():
    # a prompt in two chunks, then single tokens, through a quantised cache; attention of what was
    # written equals 64-bit attention of what is read back
    hkv, group, d, page = 2, 4, 128, 16
    g = torch.Generator().manual_seed(0)
    chunks = [100, 73, 1, 1, 1]
    total = sum(chunks)
    c = P.make([total], hkv, d, page, "e4m3", seed=1)
    c.k.fill_(0x7F), c.v.fill_(0x7F), c.ks.fill_(math.nan), c.vs.fill_(math.nan)
    at = 0
    for n in chunks:
        kn, vn = ((torch.randn((n, hkv, d), generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
        q = torch.randn((n, hkv * group, d), generator=g).to(torch.bfloat16).cuda()
        at += n
        c.kv_len.fill_(at)
        ip = P.indptr([n])
        binding.kv_append(kn, vn, c.k, c.v, c.table, c.kv_len, ip, k_scale=c.ks, v_scale=c.vs)
        o, lse = binding.forward_paged(q, c.k, c.v, c.table, c.kv_len, ip, n, k_scale=c.ks, v_scale=c.vs)
        k, v = binding.kv_read(c.k, c.v, c.table, c.kv_len, P.indptr([at]), at, k_scale=c.ks, v_scale=c.vs)
        binding.device_status()
        c.lens = [at]
        c.values = [[x.cpu().double().transpose(0, 1) for x in (k, v)]]
        want, want_lse, tol = P.reference(c, q.cpu(), [n], 1 / math.sqrt(d))
        M.assert_within("o", o, want, tol)
        M.assert_lse(lse, want_lse)


def test_dense_window_and_paged_attention_agree():
    # the same tokens through fa_fwd_window and, chunk by chunk, through the cache
    N, H, d, window, sinks = 600, 4, 64, 130, 3
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((1, H, N, d), generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    od, lsed = binding.forward(q, k, v, window=window, sinks=sinks)
    c = P.make([N], H, d, 32, "bf16", seed=1)
    at = 0
    for n in (257, 1, 342):
        rows = slice(at, at + n)
        at += n
        c.kv_len.fill_(at)
        ip = P.indptr([n])
        kn, vn, qn = (x[0, :, rows].transpose(0, 1).contiguous() for x in (k, v, q))
        binding.kv_append(kn, vn, c.k, c.v, c.table, c.kv_len, ip)
        o, lse = binding.forward_paged(qn, c.k, c.v, c.table, c.kv_len, ip, n, window=window, sinks=sinks)
        want = od[0, :, rows].transpose(0, 1).cpu().double()
        # each side rounds P~ and O to BF16 once
        ref = M.forward(q[0].cpu()[:, rows], k[0].cpu(), v[0].cpu(),
                        M.window_mask(torch.arange(rows.start, rows.stop), torch.arange(N), window, sinks), d ** -0.5)
        M.assert_within("o", o, want, 2 * ref["o_tol"].transpose(0, 1))
        assert (lse.cpu() - lsed[0, :, rows].transpose(0, 1).cpu()).abs().max() <= 2 * M.LSE_TOL
    binding.device_status()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", [120, 128, 129, 256, 257, 384, 385, 513, 1300])
def test_one_tile_of_rows_over_any_number_of_blocks(fmt, d, kv):
    # 66 to 120 rows: one tile, whose blocks alternate between two chains (odd and even numbers of blocks)
    for new, group in ((66, 1), (17, 6), (120, 1)):
        c = P.make([kv], 2, d, 32, fmt, seed=kv + new)
        check(c, [new], group)
        check(c, [new], group, window=150, sinks=5)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1, 1], [70, 3, 200], [300, 280, 290]])
def test_sequences_that_share_pages(fmt, new):
    # a common prefix held once: the sequences' tables name the same pages
    page, lens = 32, [600, 500, 310]
    c = P.make(lens, 2, 64, page, fmt, seed=9)
    for b in (1, 2):
        c.table[b, :9] = c.table[0, :9]
        for w in range(2):
            c.values[b][w][:, :9 * page] = c.values[0][w][:, :9 * page]
    for kw in ({}, dict(window=260, sinks=40)):
        check(c, new, 8, **kw)
