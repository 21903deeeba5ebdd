"""Places where the plan, the norms and rotation, the 4-bit cache and the log probabilities can go wrong quietly: other
streams, graphs that share a workspace, offsets past 32 bits, kv heads read together, logits that are alike in great number."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import serving, step
from tests.test_gpu_serving import close, ctx, draws, f64, tl, ws  # noqa: F401
from tests.test_gpu_step import (E4M3, case4, check4, check_score, freqs, ints, logits, plan_case, run4,  # noqa: F401
                                 run_score, same_plan, scales)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ streams and graphs
@pytest.mark.parametrize("how", ["current", "object", "handle"])
def test_calls_on_another_stream(tl, ctx, how):
    """Work goes to the stream given (or the current one), behind what is there already: inputs that a slow copy on that
    stream still fills."""
    side = torch.cuda.Stream()
    n, d = 300, 128
    host = draws(1, n, 6, d).bfloat16()
    big = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    q, k = torch.zeros((n, 4, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, 2, d), dtype=torch.bfloat16, device="cuda")
    hq, hk = host[:, :4].contiguous().cuda(), host[:, 4:].contiguous().cuda()
    pos, f = torch.arange(n, dtype=torch.int32, device="cuda"), freqs(d).cuda()
    codes = [torch.zeros((40, 8, 2, d // 2), dtype=torch.uint8, device="cuda") for _ in "kv"]
    blocks = [torch.zeros((40, 8, 2, d // 16), device="cuda").to(E4M3) for _ in "kv"]
    kw = dict(k_blocks=blocks[0], v_blocks=blocks[1])
    back = [torch.zeros_like(k) for _ in "kv"]
    slots, cu = torch.zeros(n, dtype=torch.int32, device="cuda"), ints(0, 0)
    lens, taken, table = ints(0), ints(0), torch.full((1, 40), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(39, -1, -1, dtype=torch.int32, device="cuda")
    x, lp = logits(5, 3000, torch.float32, 1, "plain").cuda(), torch.zeros(5, device="cuda")
    w = ws(tl.tl_token_logprobs_workspace_bytes(5, 3000, 0))
    moved, count = torch.zeros_like(x), ints(n)
    torch.cuda.synchronize()
    s = dict(stream=None if how == "current" else side if how == "object" else side.cuda_stream)
    with torch.cuda.stream(side):
        for _ in range(20):
            big.add_(1)                                     # some milliseconds
        q.copy_(hq), k.copy_(hk), moved.copy_(x)
    with torch.cuda.stream(side if how == "current" else torch.cuda.current_stream()):
        tl.tl_cache_plan(ctx, lens, table, 8, free, taken, taken, lens, cu, slots, counts=count, **s)
        tl.tl_norm_rope(ctx, q, k, pos, f, q, k, **s)
        tl.tl_kv_append(ctx, k, k, *codes, slots, **kw, **s)
        tl.tl_kv_gather(ctx, *codes, slots, *back, **kw, **s)
        tl.tl_token_logprobs(ctx, moved, torch.arange(5, dtype=torch.int32, device="cuda") if how == "current" else pos[:5], lp, w, **s)
    side.synchronize()
    assert ctx.check() == tl.TL_OK
    want, tol = step.norm_rope(f64(hq), None, np.arange(n), f.double().cpu().numpy(), 0.0, False, serving.HALF_STEP["bf16"])
    close(f64(q), want, tol, "q")
    c, b = step.to_4_bits(k.cpu().float().numpy(), np.ones(2, np.float32))
    close(f64(back[0]), step.from_4_bits(c, b), 0.0 * f64(k), "rows")
    g, t, *_ = step.token_logprobs(f64(x), np.arange(5), 0, 1.0)
    close(f64(lp), g["logprob"], t["logprob"], "logprob")
    assert lens.tolist() == [n] and slots[:9].tolist() == [312 + i for i in range(8)] + [304]


def test_two_graphs_share_a_workspace(tl, ctx):
    """Replayed in turn, the attention of one and the log probabilities of the other leave each other's counters alone."""
    q, c, table, lengths = case4([5000, 33], 8, 2, 64, 16, "bf16", False, seed=6)
    x, t = logits(3, 40000, torch.bfloat16, 2, "plain").cuda(), ints(5, 6, 7)
    w = ws(max(tl.tl_token_logprobs_workspace_bytes(3, 40000, 9), tl.tl_paged_attention_workspace_bytes(2, 8, 2, 64)))
    out, e = run4(tl, ctx, q, c, table, lengths, w)
    first = run_score(tl, ctx, x, t, 9, w=w)
    graphs, kept = [], []
    for call in (lambda: run4(tl, ctx, q, c, table, lengths, w), lambda: run_score(tl, ctx, x, t, 9, w=w)):
        g = torch.cuda.CUDAGraph()
        c["scale"] = [s.cuda() for s in c["scale"]]
        with torch.cuda.graph(g):
            kept.append(call())
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        assert torch.equal(kept[0][0], out) and torch.equal(kept[0][1], e)
        assert torch.equal(kept[1][0]["logprob"], first[0]["logprob"]) and torch.equal(kept[1][1], first[1]) and torch.equal(kept[1][2], first[2])
    assert ctx.check() == tl.TL_OK


def test_plan_in_place_by_several_ctas_in_a_graph(tl, ctx):
    """Lengths that every CTA reads and one writes, tens of thousands of tokens, replayed."""
    page, batch = 16, 37
    lens, new, table, free, taken = plan_case(batch, 3000, 900, page, 3, spare=4000, room=200)
    tokens, rows = int(new.sum()) + 9, int((lens + 3 * new).sum()) + 5
    dev = [torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda() for a in (lens, new, table, free)]
    t, slots, pos, cu_q, cu_k, kv = ints(taken), *(torch.zeros(n, dtype=torch.int32, device="cuda") for n in (tokens, tokens, batch + 1, batch + 1, rows))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tl.tl_cache_plan(ctx, dev[0], dev[2], page, dev[3], t, t, dev[0], cu_q, slots, pos, counts=dev[1], cu_k=cu_k, kv_slots=kv)
    want = dict(lengths=lens, table=table, taken=np.array([taken]))
    for _ in range(3):
        g.replay()
        want, ok = step.cache_plan(want["lengths"], new, want["table"], page, free, int(want["taken"][0]), tokens, rows)
        assert ok
        same_plan(dict(table=dev[2].cpu().numpy(), slots=slots.cpu().numpy(), positions=pos.cpu().numpy(), cu_q=cu_q.cpu().numpy(),
                       cu_k=cu_k.cpu().numpy(), lengths=dev[0].cpu().numpy(), taken=t.cpu().numpy(), kv_slots=kv.cpu().numpy()), want)
    assert ctx.check() == tl.TL_OK


# ------------------------------------------------------------------------------------------------ norms and rotation
@pytest.mark.parametrize("tokens,heads,kv,d,rotary,interleaved", [(5000, 3, 1, 128, 128, False), (3000, 70, 6, 64, 32, True), (1300, 13, 13, 128, 80, False),
                                                                  (2500, 96, 8, 128, 128, True), (4000, 1, 0, 64, 16, False)])
def test_norm_rope_many_tokens(tl, ctx, tokens, heads, kv, d, rotary, interleaved):
    """CTAs that go on from token to token, with rows that do not fill their threads; some tokens against the formula."""
    x = draws(tokens, tokens, heads + kv, d).bfloat16().cuda()
    q, k = x[:, :heads], x[:, heads:]
    w = [(draws(5 + i, d) * 0.3 + 1).bfloat16().cuda() for i in range(2)]
    pos, f = torch.randint(0, 100000, (tokens,), dtype=torch.int32, device="cuda"), freqs(rotary)
    outs = [torch.full((tokens, n, d), 9.0, dtype=torch.bfloat16, device="cuda") for n in (heads, kv)]
    tl.tl_norm_rope(ctx, q, k, pos, f.cuda(), *outs, q_weight=w[0], k_weight=w[1], interleaved=interleaved)
    some = torch.cat([torch.arange(0, tokens, 173), torch.tensor([tokens - 1, tokens - 2])])
    for rows, weight, got in ((q, w[0], outs[0]), (k, w[1], outs[1])):
        want, tol = step.norm_rope(f64(rows)[some], f64(weight), pos.cpu().numpy()[some], f.double().numpy(), 1e-6, interleaved, serving.HALF_STEP["bf16"])
        close(f64(got)[some], want, tol, "rows")
        assert not (got == 9.0).all(-1).any()               # no row is left out
    tl.tl_norm_rope(ctx, q, k, pos, f.cuda(), q, k, q_weight=w[0], k_weight=w[1], interleaved=interleaved)
    assert torch.equal(q, outs[0]) and torch.equal(k, outs[1])


# ------------------------------------------------------------------------------------------------ the 4-bit cache
@pytest.mark.parametrize("batch,length,kv,d", [(3, 500, 4, 64), (32, 4090, 8, 64), (64, 4096, 8, 128), (64, 4100, 2, 128)])
def test_paged_attention_4_bits_heads_apart_and_together(tl, ctx, batch, length, kv, d):
    """Token-major rows are read by one, two or four kv heads, by the amount of work; head-major ones one by one.  The same data
    either way, and some sequences against the 64-bit form."""
    gen = torch.Generator(device="cuda").manual_seed(batch)
    page = 32
    per = -(-length // page)
    table = torch.randperm(batch * per, generator=gen, device="cuda").to(torch.int32).view(batch, per)
    lengths = torch.full((batch,), length, dtype=torch.int32, device="cuda")
    lengths[1], lengths[2] = 0, 7
    c = dict(codes=[], blocks=[], scale=[scales(kv, 1), scales(kv, 2)])
    for _ in "kv":
        c["codes"].append(torch.randint(0, 256, (batch * per, page, kv, d // 2), dtype=torch.uint8, generator=gen, device="cuda"))
        c["blocks"].append(torch.randint(0x38, 0x68, (batch * per, page, kv, d // 16), dtype=torch.uint8, generator=gen, device="cuda").view(E4M3))
    q = draws(4, batch, 3 * kv, d).bfloat16().cuda()
    out, e = run4(tl, ctx, q, c, table, lengths)
    major = dict(c, codes=[t.transpose(1, 2).contiguous().transpose(1, 2) for t in c["codes"]])
    apart, e2 = run4(tl, ctx, q, major, table, lengths)
    assert ctx.check() == tl.TL_OK
    # both are within half a step of the exact result (and the weights' fp16 roundings)
    assert float((out.float() - apart.float()).abs().max()) <= 2.0 ** -7 * float(out.float().abs().max())
    fine = torch.isfinite(e)
    assert float((e - e2)[fine].abs().max()) <= 2.0 ** -16 * float(e[fine].abs().max()) and torch.equal(fine, torch.isfinite(e2))
    some = [0, 1, 2] if batch < 5 else [0, 1, 2, batch - 1]
    used = table[some].flatten().cpu().long()
    small = dict(scale=c["scale"], values=[step.from_4_bits(t.cpu()[used].numpy(), b.view(torch.uint8).cpu()[used].numpy())
                                           for t, b in zip(c["codes"], c["blocks"])])
    at = torch.arange(len(some) * per, dtype=torch.int32).view(len(some), per)
    check4(q[some], small, at, lengths[some], out[some], e[some])


@pytest.mark.parametrize("k_scale", [[-0.001, 0.002], [0.0, 0.001], [1e-44, -1e-44]])
def test_paged_attention_4_bits_scales_of_any_sign(tl, ctx, k_scale):
    q, c, table, lengths = case4([77, 300, 0], 4, 2, 128, 16, "bf16", False, seed=4, window=100, sinks=3)
    c["scale"][0] = torch.tensor(k_scale)
    out, e = run4(tl, ctx, q, c, table, lengths, window=100, sinks=3)
    check4(q, c, table, lengths, out, e, 100, 3)


@pytest.mark.parametrize("d", [64, 128])
def test_a_4_bit_cache_past_32_bits(tl, ctx, d):
    """Pages that lie more than 4 GB from the first: the same rows as in a small cache."""
    kv, page, pages, n = 2, 16, 6, 80
    row = page * kv * (d // 2)
    far = (1 << 30) + row                                   # bytes from a page to the next: the last one 5 GB on
    hold = [torch.zeros(far * (pages - 1) + row, dtype=torch.uint8, device="cuda") for _ in "kv"]
    codes = [h.as_strided((pages, page, kv, d // 2), (far, kv * d // 2, d // 2, 1)) for h in hold]
    small = [torch.zeros((pages, page, kv, d // 2), dtype=torch.uint8, device="cuda") for _ in "kv"]
    blocks = [[torch.zeros((pages, page, kv, d // 16), device="cuda").to(E4M3) for _ in "kv"] for _ in range(2)]
    k, v = draws(1, n, kv, d).bfloat16().cuda(), draws(2, n, kv, d).bfloat16().cuda()
    slots = torch.from_numpy(np.random.default_rng(1).permutation(pages * page)[:n].astype(np.int32)).cuda()
    q, table, lengths = draws(3, 2, 4, d).bfloat16().cuda(), ints(5, 4, 3, 1, 2, 5).view(2, 3), ints(48, 35)
    got = []
    for pool, b in ((codes, blocks[0]), (small, blocks[1])):
        kw = dict(k_blocks=b[0], v_blocks=b[1])
        tl.tl_kv_append(ctx, k, v, *pool, slots, **kw)
        rows, out = [torch.zeros_like(k) for _ in "kv"], torch.zeros_like(q)
        tl.tl_kv_gather(ctx, *pool, slots, *rows, **kw)
        tl.tl_paged_attention(ctx, q, *pool, table, lengths, out, ws(tl.tl_paged_attention_workspace_bytes(2, 4, kv, d)), **kw)
        assert ctx.check() == tl.TL_OK
        got.append([*rows, out, *[p.clone() for p in pool]])
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][2].abs().max() > 0


def test_a_4_bit_cache_too_far_for_its_units_is_refused(tl, ctx):
    """Strides that only 16 divides, pages over more than 2^36 bytes: told, and nothing runs (the pages do not exist)."""
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    c = tl.PagedCache(256, 256, None, None, (1 << 36) + 16, 32, 32, tl.TL_E2M1, 3, 1, 1, 64, 256, 256, 8, 4, 4)
    work = ws(tl.tl_paged_attention_workspace_bytes(1, 2, 1, 64))
    rc = tl.lib().tl_paged_attention(ctx.handle, ctypes.byref(c), 0, q.data_ptr(), 128, 64, q.data_ptr(), 2, q.data_ptr(), q.data_ptr(), 128, 64,
                                     None, 1, 2, 0.125, 0, 0, work.data_ptr(), work.numel(), None)
    assert rc == tl.TL_ERR_INVALID


# ------------------------------------------------------------------------------------------------ log probabilities
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_token_logprobs_start_anywhere(tl, ctx, dtype):
    x = logits(9, 5003, dtype, 3, "plain").cuda()
    for part in (x[1:], x[3:, 1:], x[2:, 7:-5], x.flatten()[3:3 + 40000].view(2, 20000)):
        t = torch.arange(part.shape[0], dtype=torch.int32, device="cuda")
        out, best, ids = run_score(tl, ctx, part, t, 7)
        assert ctx.check() == tl.TL_OK
        check_score(part, t, 7, out, best, ids)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("kind", ["few threads", "few threads up", "two values", "one above", "nan among few"])
def test_token_logprobs_alike_in_great_number(tl, ctx, dtype, kind):
    """A row a CTA (there are many rows, most of them skipped), logits made so that the bound from the threads' maxima lets
    thousands through: the large ones all in the vectors of a few threads, or equal."""
    rows, vocab, top = 500, 40000, 20
    rng = np.random.default_rng(5)
    x = rng.standard_normal((6, vocab)) * 0.5
    vec = 4 if dtype == torch.float32 else 8
    few = (np.arange(vocab) // vec) % 256 < (10 if dtype == torch.float32 else 20)
    if kind == "few threads":
        x[:, few] += 10
    elif kind == "few threads up":
        x[:, few] = 10 + np.sort(rng.random((6, int(few.sum()))), -1) * 3
    elif kind == "two values":
        x[:], x[:, 100:30000] = -1.0, 2.0
    elif kind == "one above":
        x[:] = 1.0
        x[:, 39999] = 3.0
        x[2, 5:8] = 2.0
    else:
        x[:] = -np.inf
        x[:, 7] = 1.0
        x[:, 50:70] = np.nan
        x[1] = np.nan
        x[1, 35000:35004] = -np.inf
    full = torch.zeros((rows, vocab), dtype=dtype, device="cuda")
    at = torch.tensor([0, 3, 250, 251, 498, 499], device="cuda")
    full[at] = torch.from_numpy(x).to(dtype).cuda()
    t = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    t[at] = ints(0, 1, 2, 7, 39999, 300)
    out, best, ids = run_score(tl, ctx, full, t, top)
    assert ctx.check() == tl.TL_OK
    check_score(full, t, top, out, best, ids)


def test_token_logprobs_rows_past_32_bits(tl, ctx):
    vocab, stride = 3001, (1 << 30) + 77
    hold = torch.zeros(stride * 5 + vocab, dtype=torch.bfloat16, device="cuda")
    x = hold.as_strided((6, vocab), (stride, 1))
    x.copy_(logits(6, vocab, torch.bfloat16, 9, "plain"))
    t = torch.arange(6, dtype=torch.int32, device="cuda")
    out, best, ids = run_score(tl, ctx, x, t, 4)
    assert ctx.check() == tl.TL_OK
    check_score(x, t, 4, out, best, ids)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab,kind", [(1, "plain"), (40, "ties"), (515, "masked"), (2999, "plain"), (8190, "same"), (8192, "lowest"), (1200, "tail")])
def test_token_logprobs_many_short_rows(tl, ctx, vocab, kind, dtype):
    """More rows than CTAs fit: rows that start anywhere, a target for every fifth."""
    rows, top = 701, min(vocab, 32)
    x = logits(rows, vocab + 3, dtype, vocab, kind).cuda()[:, 1:vocab + 1]
    t = torch.full((rows,), -1, dtype=torch.int32)
    t[::5] = torch.from_numpy(np.random.default_rng(1).integers(0, vocab, len(t[::5])).astype(np.int32))
    t = t.cuda()
    out, best, ids = run_score(tl, ctx, x, t, top)
    assert ctx.check() == tl.TL_OK
    check_score(x, t, top, out, best, ids)
