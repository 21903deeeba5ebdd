"""The serving operators on the GPU against their plain 64-bit forms (oracle.serving): cache append,
attention of one new token over a paged cache, causal window attention of packed prompts, and the
MoE layer for a few tokens.  Rows that nothing may read hold NaN."""
import math

import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def tl():
    import communication_overlapped_gemm_gb300 as tl
    tl.lib()
    return tl


@pytest.fixture(scope="module")
def ctx(tl):
    with tl.Context(0) as c:
        yield c


def draws(seed, *shape, std=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)) * std


def f64(t):
    return t.to(torch.float32).cpu().double().numpy() if t.dtype == torch.float8_e4m3fn else t.cpu().double().numpy()


def ws(nbytes):
    return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")


def close(got, want, tol, what):
    got, want, tol = np.asarray(got, np.float64), np.asarray(want, np.float64), np.asarray(tol, np.float64)
    assert got.shape == want.shape, what
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    off = np.where(same, 0.0, np.abs(got - want))
    bad = ~(off <= np.where(same, 1.0, tol))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.nanmax(off[bad], initial=0):.3e} at {np.argwhere(bad)[0].tolist()}"


# ------------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("dtype,tokens,heads,d,page,head_major", [
    ("bf16", 1, 1, 64, 16, False), ("bf16", 13, 8, 128, 16, True), ("fp16", 257, 3, 128, 7, False), ("fp16", 40, 2, 64, 1, True),
    ("bf16", 1000, 5, 64, 64, False)])
def test_append(tl, ctx, dtype, tokens, heads, d, page, head_major, cache):
    c = dtype if cache == "same" else cache
    rng = np.random.default_rng(tokens)
    pages = tokens // page + 3
    kv = draws(tokens + 1, tokens, 2 * heads + 1, d).to(DT[dtype])
    if tokens > 4:
        kv[1, 0, :6] = torch.tensor([math.inf, -math.inf, math.nan, 0.0, 6.0e4, -1e-30]).to(DT[dtype])
    kv = kv.cuda()
    k, v = kv[:, :heads], kv[:, heads:2 * heads]           # strided views of one projection
    slots = torch.from_numpy(rng.permutation(pages * page)[:tokens].astype(np.int32))
    if tokens > 4:
        slots[3] = -1
        slots[4] = -2 ** 31
    shape = (pages, heads, page, d) if head_major else (pages, page, heads, d)
    pools = [draws(7 + i, *shape).to(DT[c]).cuda() for i in range(2)]
    pools = [p.transpose(1, 2) if head_major else p for p in pools]
    before = [f64(p) for p in pools]
    scales = [torch.rand(heads, generator=torch.Generator().manual_seed(i)) * 0.1 + 0.01 for i in range(2)] if c == "e4m3" else [None, None]
    dev = [None if s is None else s.cuda() for s in scales]
    tl.tl_kv_append(ctx, k, v, pools[0], pools[1], slots.cuda(), k_scale=dev[0], v_scale=dev[1])
    assert ctx.check() == tl.TL_OK
    for rows, pool, was, scale in zip((k, v), pools, before, scales):
        want = was
        for t, s in enumerate(slots.tolist()):
            if s < 0:
                continue
            x = rows[t].cpu().float()
            if scale is not None:  # fp32 quotient, saturated, to the nearest e4m3 (torch's own rounding on the CPU)
                x = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float()
            want[s // page, s % page] = x.double().numpy()
        assert np.array_equal(f64(pool), want, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_e4m3_rounds_every_value_as_the_quotient_does(tl, ctx, dtype):
    """Every finite 16-bit value over scales of all sizes (powers of two give exact ties), against the
    fp32 quotient rounded by torch on the CPU."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    rows = torch.where(torch.isfinite(bits), bits, torch.zeros((), dtype=DT[dtype])).view(16, 64, 64)
    for k, base in enumerate((1.0, 0.0137, 3.3e-5, 2.0 ** -20, 700.0, 1e-33, 2e32)):
        scale = torch.from_numpy(np.random.default_rng(k).uniform(0.6, 1.6, 64)).float() * base
        scale[:4] = torch.tensor([base, base * 3, base / 7, base * 1.1])
        pool = [torch.zeros((2, 16, 64, 64), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
        dev = rows.cuda()
        tl.tl_kv_append(ctx, dev, dev, *pool, torch.arange(16, dtype=torch.int32, device="cuda"), k_scale=scale.cuda(),
                        v_scale=scale.cuda())
        want = (rows.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        for p in pool:
            assert torch.equal(p[0].cpu().view(torch.uint8), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_e4m3_of_infinities_zeros_and_scales_at_the_limits(tl, ctx, dtype):
    """Infinities saturate, NaN stays NaN, zeros keep their sign; scales on both sides of 2^-60 and 2^60, where the
    quotient is taken in another way, negative ones, zero, infinity and NaN."""
    big = torch.finfo(DT[dtype]).max
    rows = torch.cat([torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, big, -big, torch.finfo(DT[dtype]).tiny]),
                      draws(7, 56).float()]).to(DT[dtype])
    scale = torch.tensor([2.0 ** -60, 2.0 ** -60 * (1 - 2.0 ** -24), 2.0 ** 60, 2.0 ** 60 * (1 + 2.0 ** -23), -0.37, -2.0 ** -70, 0.0, -0.0,
                          math.inf, math.nan, 1e-45, 3e38, 0.37, 1.0, 448.0, 2.0 ** -9])
    dev = rows.expand(1, 16, 64).contiguous().cuda()
    pool = [torch.zeros((1, 1, 16, 64), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    tl.tl_kv_append(ctx, dev, dev, *pool, torch.zeros(1, dtype=torch.int32, device="cuda"), k_scale=scale.cuda(), v_scale=scale.cuda())
    quotient = rows.float() / scale[:, None]
    want = quotient.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for p in pool:
        got = p[0, 0].cpu()
        assert torch.equal(torch.isnan(got.float()), torch.isnan(quotient))
        assert torch.equal(got.view(torch.uint8)[~torch.isnan(quotient)], want[~torch.isnan(quotient)])


def test_append_reports_slots_out_of_range_and_leaves_them_out(tl, ctx):
    k = draws(1, 4, 2, 64).bfloat16().cuda()
    guard = torch.zeros((8, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    pool = guard[2:4]                                       # pages before and after it must stay as they are
    slots = torch.tensor([5, 32, 2 ** 31 - 1, 31], dtype=torch.int32, device="cuda")
    tl.tl_kv_append(ctx, k, k, pool, pool, slots)
    assert ctx.check() == tl.TL_ERR_INDEX and ctx.check() == tl.TL_OK
    want = torch.zeros_like(guard)
    want[2, 5], want[3, 15] = k[0], k[3]
    assert torch.equal(guard, want)


# ------------------------------------------------------------------------------------------------ paged attention
def paged_case(lens, heads, kv, d, page, dtype, cache, head_major, seed=0, spare=2, spoil=True, window=0, sinks=0):
    """Sequences over shuffled pages; every row that is not visible holds NaN."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    std = 40.0 if cache == "e4m3" else 1.0
    pools = [draws(seed + 1 + i, pages, page, kv, d, std=std) for i in range(2)]
    keep = np.zeros((pages, page), bool)
    for b, n in enumerate(lens):
        for j in serving.visible(n - 1, n, window, sinks):
            keep[table[b, j // page], j % page] = True
    if spoil:
        for p in pools:
            p[torch.from_numpy(~keep)] = math.nan
    pools = [p.to(DT[cache]) for p in pools]
    dev = [(p.transpose(1, 2).contiguous().cuda().transpose(1, 2) if head_major else p.cuda()) for p in pools]
    q = draws(seed + 3, len(lens), heads + 2, d).to(DT[dtype]).cuda()[:, 1:heads + 1]   # a strided view
    return q, dev, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def run_paged(tl, ctx, q, pools, table, lengths, w=None, lse=True, **kw):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    e = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    w = ws(tl.tl_paged_attention_workspace_bytes(q.shape[0], q.shape[1], pools[0].shape[2], q.shape[2])) if w is None else w
    tl.tl_paged_attention(ctx, q, pools[0], pools[1], table, lengths, out, w, lse=e, **kw)
    return out, e


def check_paged(q, pools, table, lengths, out, e, window=0, sinks=0, k_scale=None, v_scale=None, scale=None, bad_pages=()):
    dtype = "bf16" if q.dtype == torch.bfloat16 else "fp16"
    n = lambda s: None if s is None else s.cpu().double().numpy()
    want, lse, tol, ltol = serving.paged_attention(
        f64(q), f64(pools[0]), f64(pools[1]), table.cpu().numpy(), lengths.tolist(), scale or q.shape[2] ** -0.5, window,
        sinks, n(k_scale), n(v_scale), serving.HALF_STEP[dtype],
        dtype == "fp16" or pools[0].dtype == torch.float8_e4m3fn, bad_pages)
    close(f64(out), want, tol, "out")
    if e is not None:
        close(f64(e), lse, ltol, "lse")


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300, 1025]


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (8, 2), (7, 1), (16, 1), (34, 2), (4, 4)])
@pytest.mark.parametrize("d,dtype,cache", [(64, "bf16", "bf16"), (128, "bf16", "bf16"), (64, "fp16", "fp16"), (128, "fp16", "fp16"),
                                           (64, "bf16", "e4m3"), (128, "fp16", "e4m3")])
def test_paged_attention(tl, ctx, heads, kv, d, dtype, cache):
    q, pools, table, lengths = paged_case(LENS, heads, kv, d, 16, dtype, cache, kv == 2, seed=heads)
    s = {}
    if cache == "e4m3":
        s = dict(k_scale=torch.rand(kv, device="cuda") * 0.02 + 0.01, v_scale=torch.rand(kv, device="cuda") * 0.02 + 0.01)
    out, e = run_paged(tl, ctx, q, pools, table, lengths, **s)
    assert ctx.check() == tl.TL_OK
    check_paged(q, pools, table, lengths, out, e, **s)


@pytest.mark.parametrize("page", [1, 3, 16, 33, 100, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 4), (100, 130), (64, 1000), (5000, 3)])
def test_paged_attention_windows_and_pages(tl, ctx, page, window, sinks):
    cache = "e4m3" if page == 33 else "bf16"
    q, pools, table, lengths = paged_case(LENS[:-1] + [777], 8, 2, 128, page, "bf16", cache, page == 3, seed=page,
                                          window=window, sinks=sinks)
    out, e = run_paged(tl, ctx, q, pools, table, lengths, window=window, sinks=sinks)
    assert ctx.check() == tl.TL_OK
    check_paged(q, pools, table, lengths, out, e, window, sinks)


def test_paged_attention_splits_long_sequences(tl, ctx):
    """Few rows, long sequences: split over many CTAs and joined; the result of a run is the next one's."""
    for lens in ([20011], [1, 9000, 4]):
        q, pools, table, lengths = paged_case(lens, 4, 1, 128, 16, "bf16", "bf16", False, seed=5)
        w = ws(tl.tl_paged_attention_workspace_bytes(len(lens), 4, 1, 128))
        out, e = run_paged(tl, ctx, q, pools, table, lengths, w)
        for _ in range(3):
            again, e2 = run_paged(tl, ctx, q, pools, table, lengths, w)
            assert torch.equal(out, again) and torch.equal(e, e2)
        check_paged(q, pools, table, lengths, out, e)


@pytest.mark.parametrize("heads,kv", [(4, 4), (12, 4), (64, 8), (6, 2), (16, 2)])
@pytest.mark.parametrize("d,dtype,cache", [(64, "bf16", "bf16"), (64, "fp16", "e4m3"), (128, "bf16", "e4m3")])
def test_paged_attention_heads_side_by_side(tl, ctx, heads, kv, d, dtype, cache):
    """Short rows of several kv heads that lie side by side, whole sequences and split ones, and the same
    rows in head-major pages."""
    for major in (False, True):
        q, pools, table, lengths = paged_case([3001, 1, 0, 40, 129], heads, kv, d, 16, dtype, cache, major, seed=heads)
        s = {}
        if cache == "e4m3":
            s = dict(k_scale=torch.rand(kv, device="cuda") * 0.02 + 0.01, v_scale=torch.rand(kv, device="cuda") * 0.02 + 0.01)
        for window, sinks in ((0, 0), (333, 20)):
            out, e = run_paged(tl, ctx, q, pools, table, lengths, window=window, sinks=sinks, **s)
            assert ctx.check() == tl.TL_OK
            check_paged(q, pools, table, lengths, out, e, window, sinks, **s)


def test_paged_attention_workspace_serves_calls_of_other_shapes(tl, ctx):
    w = ws(max(tl.tl_paged_attention_workspace_bytes(b, h, kv, d) for b, h, kv, d in
               ((1, 8, 1, 128), (5, 34, 2, 64), (13, 4, 4, 128))))
    for seed, (lens, h, kv, d) in enumerate((([5000], 8, 1, 128), ([1, 700, 0, 33, 4000], 34, 2, 64), (LENS, 4, 4, 128),
                                             ([5001], 8, 1, 128))):
        q, pools, table, lengths = paged_case(lens, h, kv, d, 16, "fp16", "fp16", False, seed=seed)
        out, e = run_paged(tl, ctx, q, pools, table, lengths, w)
        check_paged(q, pools, table, lengths, out, e)


def test_paged_attention_extreme_scores(tl, ctx):
    """Scores at the end of the range: one key far above the rest, one at minus infinity, a scale that
    leaves a single weight, and without lse."""
    q, pools, table, lengths = paged_case([300, 64], 4, 1, 128, 16, "bf16", "bf16", False, seed=9, spoil=False)
    q = q.abs() + 0.01
    pages = table.cpu().numpy()
    pools[0][pages[0, 3], 5, 0, 7] = -math.inf             # its score is -inf: no weight
    pools[0][pages[0, 9], 2, 0] = 60.0                     # far above
    pools[0][pages[1, 0]] = -3.3e38                        # the type's lowest values: no weight either
    for scale in (None, 3.0):
        out, e = run_paged(tl, ctx, q, pools, table, lengths, lse=scale is None, scale=scale)
        check_paged(q, pools, table, lengths, out, e, scale=scale)
        assert torch.isfinite(out).all()


def test_paged_attention_bad_pages_and_lengths_are_reported(tl, ctx):
    q, pools, table, lengths = paged_case([100, 64, 40], 8, 2, 64, 16, "bf16", "bf16", False, seed=3, spoil=False)
    good = table.clone()
    table[0, 2], table[2, 0] = 2 ** 31 - 1, -5
    table[2, 1], table[2, 2] = pools[0].shape[0], -1       # sequence 2 has no good page at all
    out, e = run_paged(tl, ctx, q, pools, table, lengths)
    assert ctx.check() == tl.TL_ERR_INDEX
    bad = (2 ** 31 - 1, -5, pools[0].shape[0], -1)
    check_paged(q, pools, table, lengths, out, e, bad_pages=bad)
    assert (out[2] == 0).all() and (e[2] == -math.inf).all()
    # a length beyond the table is cut to it, a negative one sees nothing
    longer = torch.tensor([table.shape[1] * 16 + 9, 64, -3], dtype=torch.int32, device="cuda")
    good[0, :] = good[1, 0]
    out, e = run_paged(tl, ctx, q, pools, good, longer)
    assert ctx.check() == tl.TL_ERR_INDEX
    check_paged(q, pools, good, torch.tensor([good.shape[1] * 16, 64, 0]), out, e)
    out, e = run_paged(tl, ctx, q, pools, good, lengths)   # and the workspace is still good
    assert ctx.check() == tl.TL_OK


def test_paged_attention_pages_beyond_32_bits(tl, ctx):
    """A pool of over 2^32 bytes: rows at its end."""
    pages, page = 40000, 64
    pool = torch.zeros((pages, page, 8, 128), dtype=torch.bfloat16, device="cuda")
    assert pool.numel() * 2 > 2 ** 32
    rows = draws(2, 3 * page, 8, 128).bfloat16().cuda()
    slots = torch.cat([torch.arange(p * page, p * page + page) for p in (pages - 1, 17, pages - 3)]).to(torch.int32).cuda()
    tl.tl_kv_append(ctx, rows, rows, pool, pool, slots)
    table = torch.tensor([[pages - 1, 17, pages - 3]], dtype=torch.int32, device="cuda")
    q = draws(3, 1, 16, 128).bfloat16().cuda()
    out, e = run_paged(tl, ctx, q, (pool, pool), table, torch.tensor([3 * page - 5], dtype=torch.int32, device="cuda"))
    assert ctx.check() == tl.TL_OK
    small = rows.view(3, page, 8, 128)
    check_paged(q, (small, small), torch.tensor([[0, 1, 2]]), torch.tensor([3 * page - 5]), out, e)


def test_paged_attention_on_another_stream_and_in_a_graph(tl, ctx):
    q, pools, table, lengths = paged_case([600, 33, 1], 8, 2, 128, 16, "bf16", "bf16", False, seed=4, spoil=False)
    w = ws(tl.tl_paged_attention_workspace_bytes(3, 8, 2, 128))
    out, e = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tl.tl_paged_attention(ctx, q, *pools, table, lengths, out, w, lse=e)
    torch.cuda.current_stream().wait_stream(side)
    check_paged(q, pools, table, lengths, out, e)
    new = draws(11, 3, 2, 128).bfloat16().cuda()
    slots = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.tl_kv_append(ctx, new, new, *pools, slots)
        tl.tl_paged_attention(ctx, q, *pools, table, lengths, out, w, lse=e)
    for n in ([607, 31, 16], [1, 0, 9]):
        lengths.copy_(torch.tensor(n, dtype=torch.int32))
        slots.copy_(torch.tensor([int(table[b, (m - 1) // 16]) * 16 + (m - 1) % 16 if m else -1 for b, m in enumerate(n)], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_paged(q, pools, table, lengths, out, e)
        assert torch.equal(pools[0][int(table[0, (n[0] - 1) // 16]), (n[0] - 1) % 16], new[0])


# ------------------------------------------------------------------------------------------------ window attention
def run_window(tl, ctx, q, k, v, cu_q, cu_k, **kw):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    e = torch.full(q.shape[:2], 7.0, device="cuda")
    tl.tl_window_attention(ctx, q, k, v, torch.tensor(cu_q, dtype=torch.int32).cuda(),
                           torch.tensor(cu_k, dtype=torch.int32).cuda(), out, lse=e, **kw)
    return out, e


def check_window(q, k, v, cu_q, cu_k, out, e, window=0, sinks=0, scale=None):
    dtype = "bf16" if q.dtype == torch.bfloat16 else "fp16"
    want, lse, tol, ltol = serving.window_attention(f64(q), f64(k), f64(v), cu_q, cu_k, scale or q.shape[2] ** -0.5, window,
                                                    sinks, serving.HALF_STEP[dtype], dtype == "fp16")
    n = cu_q[-1]
    close(f64(out)[:n], want[:n], tol[:n], "out")
    close(f64(e)[:n], lse[:n], ltol[:n], "lse")


def cum(lens):
    return [0] + np.cumsum(lens).tolist()


def packed(lens_q, lens_k, heads, kv, d, dtype, seed=0):
    """Views of one projection's rows where queries and keys are the same tokens, else of two."""
    if lens_q == lens_k:
        x = draws(seed, sum(lens_q), heads + 2 * kv, d).to(DT[dtype]).cuda()
        return x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    x = draws(seed + 1, sum(lens_k), 2 * kv, d).to(DT[dtype]).cuda()
    return draws(seed, sum(lens_q), heads, d).to(DT[dtype]).cuda(), x[:, :kv], x[:, kv:]


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (8, 2), (5, 1), (16, 1), (4, 4), (40, 1)])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "fp16"), (128, "fp16")])
def test_window_attention_causal(tl, ctx, heads, kv, d, dtype):
    lens = [1, 0, 2, 31, 64, 127, 129, 200]
    q, k, v = packed(lens, lens, heads, kv, d, dtype, seed=heads)
    out, e = run_window(tl, ctx, q, k, v, cum(lens), cum(lens))
    assert ctx.check() == tl.TL_OK
    check_window(q, k, v, cum(lens), cum(lens), out, e)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (7, 0), (64, 4), (128, 0), (129, 130), (200, 1), (1000, 5)])
@pytest.mark.parametrize("lens_q,lens_k", [([700], [700]), ([130, 1, 300], [130, 1, 300]), ([5, 257], [400, 600]),
                                           ([1, 1, 1], [1, 500, 129])])
def test_window_attention_windows(tl, ctx, window, sinks, lens_q, lens_k):
    q, k, v = packed(lens_q, lens_k, 4, 2, 128 if window % 2 else 64, "bf16", seed=window)
    out, e = run_window(tl, ctx, q, k, v, cum(lens_q), cum(lens_k), window=window, sinks=sinks)
    assert ctx.check() == tl.TL_OK
    check_window(q, k, v, cum(lens_q), cum(lens_k), out, e, window, sinks)


@pytest.mark.parametrize("lens,heads,kv", [([300] + [i * 7 % 6 for i in range(900)], 16, 16), ([250 + i * 37 % 150 for i in range(32)], 128, 8)])
def test_window_attention_of_more_items_than_a_list_holds(tl, ctx, lens, heads, kv):
    """More than 32 items for each CTA, so that the list of them is written anew: up to twice each half for many
    short sequences, once for 32 (which are ordered by length)."""
    q, k, v = packed(lens, lens, heads, kv, 64, "bf16", seed=len(lens))
    out, e = run_window(tl, ctx, q, k, v, cum(lens), cum(lens), window=64, sinks=1)
    assert ctx.check() == tl.TL_OK
    check_window(q, k, v, cum(lens), cum(lens), out, e, 64, 1)
    again, _ = run_window(tl, ctx, q, k, v, cum(lens), cum(lens), window=64, sinks=1)
    assert torch.equal(out, again)


def test_window_attention_queries_before_the_first_key_see_nothing(tl, ctx):
    lens_q, lens_k = [9, 200, 3], [4, 100, 0]
    q, k, v = packed(lens_q, lens_k, 4, 1, 64, "bf16", seed=1)
    for window, sinks in ((0, 0), (16, 2)):
        out, e = run_window(tl, ctx, q, k, v, cum(lens_q), cum(lens_k), window=window, sinks=sinks)
        assert ctx.check() == tl.TL_OK
        check_window(q, k, v, cum(lens_q), cum(lens_k), out, e, window, sinks)
        assert (out[:5] == 0).all() and (e[:5] == -math.inf).all() and (out[-3:] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_window_attention_nan_and_infinity_stay_with_the_rows_that_see_them(tl, ctx, d):
    """A spoilt key reaches exactly the queries it is visible to; spoilt rows between sequences none."""
    lens = [300, 70]
    q, k, v = packed([410], [410], 6, 2, d, "bf16", seed=2)
    q, k, v = q.clone(), k.clone(), v.clone()
    cu = [10, 310, 380]
    v[:10], k[:10], v[380:], k[380:] = math.nan, math.nan, math.inf, math.nan
    v[10 + 140, 0, 3], k[10 + 200, 1] = math.nan, math.nan
    v[10 + 250, 1] = -math.inf
    for window, sinks in ((0, 0), (40, 3)):
        out, e = run_window(tl, ctx, q, k, v, cu, cu, window=window, sinks=sinks)
        assert ctx.check() == tl.TL_OK
        assert (out[:10] == 7).all() and (out[380:] == 7).all()   # rows outside every sequence
        check_window(q[10:], k[10:], v[10:], cum(lens), cum(lens), out[10:], e[10:], window, sinks)
    assert torch.isnan(out).any() and not torch.isnan(out).all()


def test_window_attention_moving_maximum(tl, ctx):
    """Keys whose scores climb along the sequence (the running maximum moves at every block) and fall."""
    n = 600
    q, k, v = packed([n], [n], 2, 1, 128, "bf16", seed=3)
    q, k = q.abs(), k.clone()
    k[:, 0] = torch.linspace(-20, 20, n, device="cuda")[:, None].to(k.dtype)
    for sign in (1, -1):
        out, e = run_window(tl, ctx, q, sign * k, v, [0, n], [0, n])
        check_window(q, sign * k, v, [0, n], [0, n], out, e)


def test_window_attention_reports_bad_bounds(tl, ctx):
    q, k, v = packed([40], [40], 2, 1, 64, "bf16", seed=4)
    for cu_q, cu_k in (([0, 50], [0, 40]), ([0, 30], [0, 41]), ([-1, 20], [0, 20]), ([0, 20], [5, 4])):
        out, e = run_window(tl, ctx, q, k, v, cu_q, cu_k)
        assert ctx.check() == tl.TL_ERR_INDEX
        assert (out == 7).all() and (e == 7).all()
    out, e = run_window(tl, ctx, q, k, v, [0, 15, 10, 40], [0, 15, 10, 40])  # a good one, a bad one, a good one
    assert ctx.check() == tl.TL_ERR_INDEX
    check_window(q[:10], k[:10], v[:10], [0, 10], [0, 10], out[:10], e[:10])


def test_window_attention_matches_paged_attention_at_the_last_token(tl, ctx):
    """The last query of a prompt is the single-token form of the same mask."""
    n = 333
    q, k, v = packed([n], [n], 8, 2, 128, "bf16", seed=6)
    pool = [torch.zeros((21, 16, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    tl.tl_kv_append(ctx, k, v, *pool, torch.arange(n, dtype=torch.int32, device="cuda"))
    table = torch.arange(21, dtype=torch.int32, device="cuda")[None]
    for window, sinks in ((0, 0), (100, 4)):
        out, e = run_window(tl, ctx, q, k, v, [0, n], [0, n], window=window, sinks=sinks)
        one, e1 = run_paged(tl, ctx, q[-1:], pool, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                            window=window, sinks=sinks)
        assert (out[-1].float() - one[0].float()).abs().max() <= 2.0 ** -7 * v.float().abs().max()
        assert (e[-1] - e1[0]).abs().max() <= 1e-4


# ------------------------------------------------------------------------------------------------ MoE
def moe_case(T, H, E, F, seed, logits=None):
    x = draws(seed, T, H).bfloat16()
    w = [(draws(seed + 1 + i, E, *s, std=0.05)).bfloat16() for i, s in enumerate(((H, F), (H, F), (F, H)))]
    lg = draws(seed + 5, T, E).float() if logits is None else logits
    return x.cuda(), lg.cuda(), *[t.cuda() for t in w]


def run_moe(tl, ctx, x, lg, wg, wu, wd, topk, w=None):
    T, H = x.shape
    E, _, F = wg.shape
    out = torch.full((T, H), 7.0, device="cuda")
    ex, g = torch.empty((T, topk), dtype=torch.int32, device="cuda"), torch.empty((T, topk), device="cuda")
    w = ws(tl.tl_moe_tokens_workspace_bytes(T, H, E, F, topk)) if w is None else w
    tl.tl_moe_tokens(ctx, x, lg, topk, wg, wu, wd, out, w, experts_out=ex, gates_out=g)
    return out, ex, g


def check_moe(x, lg, wg, wu, wd, topk, out, ex, g, renorm=False):
    want, experts, gates, tol = serving.moe_tokens(*[f64(t) for t in (x, lg, wg, wu, wd)], topk, renorm)
    assert np.array_equal(ex.cpu().numpy(), experts)
    close(f64(g), gates, 2.0 ** -19 * gates, "gates")
    close(f64(out), want, tol, "out")


@pytest.mark.parametrize("T,H,E,F,topk", [(1, 256, 4, 128, 2), (1, 8, 1, 8, 1), (2, 72, 3, 40, 3), (5, 1000, 16, 712, 4),
                                          (8, 64, 8, 64, 8), (17, 128, 200, 96, 6), (33, 264, 5, 136, 1), (64, 512, 12, 200, 2),
                                          (128, 136, 9, 72, 8)])
def test_moe_tokens(tl, ctx, T, H, E, F, topk):
    case = moe_case(T, H, E, F, seed=T + H)
    got = run_moe(tl, ctx, *case, topk)
    assert ctx.check() == tl.TL_OK
    check_moe(*case, topk, *got)


@pytest.mark.parametrize("T,topk,H,F,E", [(1, 8, 256, 4096, 9), (1, 1, 8, 8192, 1), (4, 8, 264, 1000, 100), (5, 7, 520, 2000, 256),
                                          (8, 4, 256, 512, 4), (8, 6, 1032, 1000, 12)])
def test_moe_tokens_cut_into_many_pieces(tl, ctx, T, topk, H, F, E):
    """Few columns of long sums: a token's rows come in more pieces than a warp has lanes; up to and over 32
    assignments; one expert for all tokens."""
    case = moe_case(T, H, E, F, seed=100 + T)
    w = ws(tl.tl_moe_tokens_workspace_bytes(T, H, E, F, topk))
    first = run_moe(tl, ctx, *case, topk, w)
    check_moe(*case, topk, *first)
    assert all(torch.equal(a, b) for a, b in zip(first, run_moe(tl, ctx, *case, topk, w)))
    assert ctx.check() == tl.TL_OK
    assert (w[:139264] == 0).all()  # TL_SERVE_COUNTER_BYTES


def test_moe_tokens_all_to_one_expert_and_ties(tl, ctx):
    """Every token at one expert (the longest lists); equal logits go to the lower expert."""
    T, E = 100, 7
    lg = torch.zeros((T, E))
    lg[:, 5] = 9.0
    case = moe_case(T, 128, E, 96, 3, logits=lg)
    got = run_moe(tl, ctx, *case, 2)
    assert got[1].tolist() == [[5, 0]] * T
    check_moe(*case, 2, *got)
    lg = torch.full((3, E), -math.inf)
    lg[:, 2] = 0.5
    case = moe_case(3, 128, E, 96, 4, logits=lg)
    got = run_moe(tl, ctx, *case, 3)
    assert got[1].tolist() == [[2, 0, 1]] * 3
    check_moe(*case, 3, *got)


def test_moe_tokens_renormalised_and_as_tl_moe_combine(tl):
    """cfg.moe_renorm applies; at a shape both take, the layer is tl_moe_combine's (which rounds h and y to
    bf16: 2 roundings of 2^-8, and 2^-7 leaves room for what they are taken from)."""
    T, H, E, F = 128, 256, 8, 128
    case = moe_case(T, H, E, F, seed=8)
    for renorm in (0, 1):
        with tl.Context(0, moe_renorm=renorm) as c:
            got = run_moe(tl, c, *case, 2)
            check_moe(*case, 2, *got, renorm=bool(renorm))
            big = torch.empty((T, H), device="cuda")
            tl.tl_moe_combine(c, case[0], case[1], 2, *case[2:], big, ws(tl.tl_moe_workspace_bytes(T, H, E, F, 2)))
            assert c.check() == tl.TL_OK
            assert (big - got[0]).norm() <= 2.0 ** -7 * got[0].norm()


def test_moe_tokens_repeats_bit_for_bit_in_one_workspace(tl, ctx):
    w = ws(max(tl.tl_moe_tokens_workspace_bytes(T, 512, 16, 256, 2) for T in (1, 40)))
    for T in (40, 1, 40):
        case = moe_case(T, 512, 16, 256, seed=T)
        first = run_moe(tl, ctx, *case, 2, w)
        check_moe(*case, 2, *first)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, run_moe(tl, ctx, *case, 2, w)))


@pytest.mark.parametrize("T", [1, 8, 64])
def test_moe_tokens_repeats_at_the_size_of_a_layer(tl, ctx, T):
    """Every CTA has units of both products, and tiles cut between neighbours in both: no run differs."""
    H, E, F = 2048, 64, 1408
    gen = torch.Generator(device="cuda").manual_seed(T)
    w = [(torch.randn(s, generator=gen, device="cuda") * 0.02).bfloat16() for s in ((E, H, F), (E, H, F), (E, F, H))]
    x, lg = torch.randn((T, H), generator=gen, device="cuda").bfloat16(), torch.randn((T, E), generator=gen, device="cuda")
    work = ws(tl.tl_moe_tokens_workspace_bytes(T, H, E, F, 2))
    first = run_moe(tl, ctx, x, lg, *w, 2, work)
    for _ in range(60):
        again = run_moe(tl, ctx, x, lg, *w, 2, work)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert ctx.check() == tl.TL_OK
    h = torch.stack([torch.nn.functional.silu(a @ w[0][e].double()) * (a @ w[1][e].double())
                     for a, row in zip(x.double(), first[1].tolist()) for e in row])
    y = torch.stack([v @ w[2][e].double() for v, e in zip(h, first[1].flatten().tolist())]).view(T, 2, H)
    want = (torch.softmax(lg.double(), -1).gather(1, first[1].long())[:, :, None] * y).sum(1)
    # sums of 2048 and 1408 terms in fp32: a relative 2^-23 each time, at random signs sqrt(2048) of them, doubled for the chain
    assert (first[0] - want).norm() <= 2 * math.sqrt(2048) * 2.0 ** -23 * want.norm()


def test_moe_tokens_in_a_graph_on_another_stream(tl, ctx):
    x, lg, *w = moe_case(6, 256, 8, 128, seed=20)
    out, work = torch.empty((6, 256), device="cuda"), ws(tl.tl_moe_tokens_workspace_bytes(6, 256, 8, 128, 2))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tl.tl_moe_tokens(ctx, x, lg, 2, *w, out, work)
    for seed in (21, 22):
        lg.copy_(draws(seed, 6, 8).float())
        x.copy_(draws(seed + 50, 6, 256).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        want, experts, gates, tol = serving.moe_tokens(*[f64(t) for t in (x, lg, *w)], 2)
        close(f64(out), want, tol, "out")


def test_moe_tokens_nan_logits_choose_valid_experts(tl, ctx):
    lg = torch.full((2, 4), math.nan)
    lg[0, 3] = 1.0
    case = moe_case(2, 64, 4, 64, 30, logits=lg)
    out, ex, g = run_moe(tl, ctx, *case, 3)
    assert ctx.check() == tl.TL_OK
    assert ex.tolist() == [[3, 0, 1], [0, 1, 2]] and torch.isnan(g).all()
