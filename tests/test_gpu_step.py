"""What a serving step needs around its attention, on the GPU against the plain forms (oracle.step, oracle.serving): the
4-bit cache (append, gather, attention of one token), the plan, norms and rotation, log probabilities, and a step of all
of them."""
import math

import numpy as np
import pytest
import torch

from oracle import serving, step
from tests.test_gpu_serving import DT, close, ctx, draws, f64, tl, ws  # noqa: F401

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def pools4(x, scale, head_major=False):
    """Rows x [pages, page, kv, d] in 4 bits: codes and blocks on the GPU, and the values that they stand for."""
    codes, blocks = step.to_4_bits(x.float().numpy(), scale.numpy())
    lay = lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if head_major else t.cuda()  # noqa: E731
    return lay(torch.from_numpy(codes)), lay(torch.from_numpy(blocks).view(E4M3)), step.from_4_bits(codes, blocks, scale.numpy())


def scales(n, seed):
    return torch.from_numpy(np.random.default_rng(seed).uniform(0.0008, 0.0015, n)).float()


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------------------------------------ append, gather
@pytest.mark.parametrize("dtype,tokens,heads,d,page,head_major", [
    ("bf16", 1, 1, 64, 16, False), ("bf16", 13, 8, 128, 16, True), ("fp16", 257, 3, 128, 7, False), ("fp16", 40, 2, 64, 1, True),
    ("bf16", 700, 5, 64, 64, False)])
def test_append_4_bits(tl, ctx, dtype, tokens, heads, d, page, head_major):
    rng = np.random.default_rng(tokens)
    pages = tokens // page + 3
    kv = (draws(tokens + 1, tokens, 2 * heads + 1, d) * 0.5).to(DT[dtype])
    if tokens > 4:
        kv[1, 0, :6] = torch.tensor([math.inf, -1.0, 0.0, -0.0, 6.0e4, -1e-30]).to(DT[dtype])
        kv[2, 0, 16:32] = 0
        kv[2, 0, 32:48] = 1e-7                              # below the smallest block scale
        kv[3, 0, 5] = math.nan
    kv = kv.cuda()
    k, v = kv[:, :heads], kv[:, heads:2 * heads]
    slots = torch.from_numpy(rng.permutation(pages * page)[:tokens].astype(np.int32))
    if tokens > 8:
        slots[6], slots[7] = -1, -2 ** 31
    old = [pools4(draws(7 + i, pages, page, heads, d), scales(heads, i), head_major) for i in range(2)]
    dev = [scales(heads, i).cuda() for i in range(2)]
    want = [(raw(c).copy(), raw(b).copy()) for c, b, _ in old]
    kw = dict(k_scale=dev[0], v_scale=dev[1], k_blocks=old[0][1], v_blocks=old[1][1])
    tl.tl_kv_append(ctx, k, v, old[0][0], old[1][0], slots.cuda(), **kw)
    assert ctx.check() == tl.TL_OK
    outs = [torch.full((tokens, heads + 1, d), 9.0, dtype=DT[dtype], device="cuda")[:, 1:] for _ in "kv"]
    tl.tl_kv_gather(ctx, old[0][0], old[1][0], slots.cuda(), *outs, **kw)
    assert ctx.check() == tl.TL_OK
    for rows, (codes, blocks, _), (wc, wb), s, got in zip((k, v), old, want, dev, outs):
        c, b = step.to_4_bits(rows.cpu().float().numpy(), s.cpu().numpy())
        held = np.full((tokens, heads, d), 9.0)
        for t, at in enumerate(slots.tolist()):
            if at >= 0:
                wc[at // page, at % page], wb[at // page, at % page] = c[t], b[t]
                # rounded to fp32 (times the head's scale), then to the type
                x = torch.from_numpy((step.from_4_bits(c[t], b[t]).astype(np.float32) * s.cpu().numpy()[:, None]).astype(np.float32))
                held[t] = x.to(DT[dtype]).double().numpy()
        assert np.array_equal(raw(blocks), wb)
        nan = np.repeat(wb == 0x7F, 8, -1)                  # (a NaN block's codes say nothing)
        assert np.array_equal(raw(codes)[~nan], wc[~nan])
        assert np.array_equal(f64(got), held, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_4_bits_rounds_every_value_as_the_quotient_does(tl, ctx, dtype):
    """Every finite 16-bit value beside others of its size, over scales of all sizes (powers of two give exact ties)."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    rows = torch.where(torch.isfinite(bits), bits, torch.zeros((), dtype=DT[dtype]))
    order = torch.from_numpy(np.random.default_rng(3).permutation(65536).reshape(4096, 16))
    order[1::2] = torch.arange(65536).reshape(4096, 16)[1::2]                # random neighbours, and near ones
    rows = rows[order].view(16, 64, 64)
    for k, base in enumerate((1.0, 0.0137, 3.3e-5, 2.0 ** -20, 700.0, 1e-33, 2e32)):
        scale = torch.from_numpy(np.random.default_rng(k).uniform(0.6, 1.6, 64)).float() * base
        scale[:4] = torch.tensor([base, base * 3, base / 7, base * 1.1])
        codes = [torch.zeros((2, 8, 64, 32), dtype=torch.uint8, device="cuda") for _ in "kv"]
        blocks = [torch.zeros((2, 8, 64, 4), device="cuda").to(E4M3) for _ in "kv"]
        dev = rows.cuda()
        tl.tl_kv_append(ctx, dev, dev, *codes, torch.arange(16, dtype=torch.int32, device="cuda"), k_scale=scale.cuda(),
                        v_scale=scale.cuda(), k_blocks=blocks[0], v_blocks=blocks[1])
        wc, wb = step.to_4_bits(rows.float().numpy(), scale.numpy())
        for c, b in zip(codes, blocks):
            assert np.array_equal(raw(b).reshape(wb.shape), wb) and np.array_equal(raw(c).reshape(wc.shape), wc)


@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("d,page,head_major", [(64, 7, False), (128, 16, True)])
def test_gather_other_caches(tl, ctx, cache, d, page, head_major):
    dtype = "fp16" if cache == "fp16" else "bf16"
    heads, pages, n = 3, 9, 50
    pools = [draws(i, pages, page, heads, d).to(DT[cache]) for i in range(2)]
    dev = [(p.transpose(1, 2).contiguous().cuda().transpose(1, 2) if head_major else p.cuda()) for p in pools]
    slots = np.random.default_rng(1).integers(0, pages * page, n).astype(np.int32)
    slots[3], slots[4], slots[5] = -1, slots[6], -2 ** 31
    s = [scales(heads, i) if cache == "e4m3" else None for i in range(2)]
    outs = [torch.full((n, heads, d), 9.0, dtype=DT[dtype], device="cuda") for _ in "kv"]
    tl.tl_kv_gather(ctx, *dev, torch.from_numpy(slots).cuda(), *outs, **({"k_scale": s[0].cuda(), "v_scale": s[1].cuda()} if s[0] is not None else {}))
    assert ctx.check() == tl.TL_OK
    for p, scale, got in zip(pools, s, outs):
        x = p.float() if scale is None else p.float() * scale[:, None]
        want = x.to(DT[dtype])[torch.from_numpy(slots.clip(min=0) // page).long(), torch.from_numpy(slots.clip(min=0) % page).long()]
        want[torch.from_numpy(slots < 0)] = 9.0
        assert torch.equal(got.cpu(), want)


def test_gather_and_append_report_slots_out_of_range(tl, ctx):
    guard_c, guard_b = torch.zeros((8, 16, 2, 32), dtype=torch.uint8, device="cuda"), torch.zeros((8, 16, 2, 4), device="cuda").to(E4M3)
    codes, blocks = guard_c[2:4], guard_b[2:4]
    k = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = ints(5, 32, 2 ** 31 - 1, 31)
    tl.tl_kv_append(ctx, k, k, codes, codes, slots, k_blocks=blocks, v_blocks=blocks)
    assert ctx.check() == tl.TL_ERR_INDEX and ctx.check() == tl.TL_OK
    wrote = (guard_c != 0).any(-1).any(-1)
    assert wrote.nonzero().tolist() == [[2, 5], [3, 15]]
    outs = [torch.full((4, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    tl.tl_kv_gather(ctx, codes, codes, slots, *outs, k_blocks=blocks, v_blocks=blocks)
    assert ctx.check() == tl.TL_ERR_INDEX and ctx.check() == tl.TL_OK
    for o in outs:
        # (b = e4m3(1 / 6) = 11/64, 1 / b = 5.8: code 6)
        assert o[:, 0, 0].tolist() == [1.03125, 9.0, 9.0, 1.03125]


# ------------------------------------------------------------------------------------------------ attention over 4 bits
def case4(lens, heads, kv, d, page, dtype, head_major, seed=0, spare=2, window=0, sinks=0, spoil=True):
    """Sequences over shuffled pages; every row that is not visible holds NaN (its block scales) and the largest codes."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    keep = np.zeros((pages, page), bool)
    for b, n in enumerate(lens):
        for j in serving.visible(n - 1, n, window, sinks):
            keep[table[b, j // page], j % page] = True
    c = dict(values=[], codes=[], blocks=[], scale=[])
    for i in range(2):
        s = scales(kv, seed + i)
        # random codes and block scales reach every code beside every scale
        codes = torch.from_numpy(rng.integers(0, 256, (pages, page, kv, d // 2)).astype(np.uint8))
        blocks = torch.from_numpy(rng.integers(0x20, 0x7F, (pages, page, kv, d // 16)).astype(np.uint8))
        codes[:, :, :, :8] = 0x22 * (rng.random() < 2)      # a block alike in all rows
        if spoil:
            codes[torch.from_numpy(~keep)], blocks[torch.from_numpy(~keep)] = 0x7F, 0x7F
        c["values"].append(step.from_4_bits(codes.numpy(), blocks.numpy()))
        lay = lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if head_major else t.cuda()  # noqa: E731
        c["codes"].append(lay(codes))
        c["blocks"].append(lay(blocks.view(E4M3)))
        c["scale"].append(s)
    q = draws(seed + 3, len(lens), heads + 2, d).to(DT[dtype]).cuda()[:, 1:heads + 1]
    return q, c, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def run4(tl, ctx, q, c, table, lengths, w=None, scale=None, **kw):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    e = torch.full(q.shape[:2], 7.0, device="cuda")
    kv = c["codes"][0].shape[2]
    w = ws(tl.tl_paged_attention_workspace_bytes(q.shape[0], q.shape[1], kv, q.shape[2])) if w is None else w
    tl.tl_paged_attention(ctx, q, *c["codes"], table, lengths, out, w, lse=e, scale=scale, k_scale=c["scale"][0].cuda(),
                          v_scale=c["scale"][1].cuda(), k_blocks=c["blocks"][0], v_blocks=c["blocks"][1], **kw)
    return out, e


def check4(q, c, table, lengths, out, e, window=0, sinks=0, bad_pages=()):
    dtype = "bf16" if q.dtype == torch.bfloat16 else "fp16"
    want, lse, tol, ltol = serving.paged_attention(
        f64(q), *c["values"], table.cpu().numpy(), lengths.tolist(), q.shape[2] ** -0.5, window, sinks,
        c["scale"][0].double().numpy(), c["scale"][1].double().numpy(), serving.HALF_STEP[dtype], True, bad_pages)
    close(f64(out), want, tol, "out")
    close(f64(e), lse, ltol, "lse")


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300, 1025]


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (8, 2), (7, 1), (16, 1), (34, 2), (4, 4), (32, 8)])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "fp16"), (128, "fp16")])
@pytest.mark.parametrize("head_major", [False, True])
def test_paged_attention_4_bits(tl, ctx, heads, kv, d, dtype, head_major):
    q, c, table, lengths = case4(LENS, heads, kv, d, 16, dtype, head_major, seed=heads)
    out, e = run4(tl, ctx, q, c, table, lengths)
    assert ctx.check() == tl.TL_OK
    check4(q, c, table, lengths, out, e)


@pytest.mark.parametrize("page", [1, 3, 16, 33, 100, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 4), (100, 130), (64, 1000), (5000, 3)])
def test_paged_attention_4_bits_windows_and_pages(tl, ctx, page, window, sinks):
    d = 64 if page == 33 else 128
    q, c, table, lengths = case4(LENS[:-1] + [777], 8, 2, d, page, "bf16", page == 3, seed=page, window=window, sinks=sinks)
    out, e = run4(tl, ctx, q, c, table, lengths, window=window, sinks=sinks)
    assert ctx.check() == tl.TL_OK
    check4(q, c, table, lengths, out, e, window, sinks)


def test_paged_attention_4_bits_splits_long_sequences(tl, ctx):
    for lens in ([20011], [1, 9000, 4]):
        q, c, table, lengths = case4(lens, 4, 1, 128, 16, "bf16", False, seed=5)
        w = ws(tl.tl_paged_attention_workspace_bytes(len(lens), 4, 1, 128))
        out, e = run4(tl, ctx, q, c, table, lengths, w)
        for _ in range(3):
            again, e2 = run4(tl, ctx, q, c, table, lengths, w)
            assert torch.equal(out, again) and torch.equal(e, e2)
        check4(q, c, table, lengths, out, e)


def test_paged_attention_4_bits_in_one_buffer(tl, ctx):
    """Codes and block scales of a token side by side in one buffer: strides that only views have."""
    lens, heads, kv, d, page = [70, 1, 130], 8, 2, 128, 16
    q, c, table, lengths = case4(lens, heads, kv, d, page, "fp16", False, seed=8)
    one = [torch.zeros((cc.shape[0], page, kv * (d // 2 + d // 16)), dtype=torch.uint8, device="cuda") for cc in c["codes"]]
    for i in range(2):
        n = kv * d // 2
        codes = one[i][:, :, :n].unflatten(2, (kv, d // 2))
        blocks = one[i][:, :, n:].unflatten(2, (kv, d // 16))
        codes.copy_(c["codes"][i])
        blocks.copy_(c["blocks"][i].view(torch.uint8))
        c["codes"][i], c["blocks"][i] = codes, blocks.view(E4M3)
    out, e = run4(tl, ctx, q, c, table, lengths)
    assert ctx.check() == tl.TL_OK
    check4(q, c, table, lengths, out, e)


def test_paged_attention_4_bits_reports_bad_pages(tl, ctx):
    q, c, table, lengths = case4([40, 33], 4, 1, 64, 16, "bf16", False, seed=2)
    pages, table = c["codes"][0].shape[0], table.clone()
    table[0, 1], table[1, 0] = pages, -3
    out, e = run4(tl, ctx, q, c, table, lengths)
    assert ctx.check() == tl.TL_ERR_INDEX and ctx.check() == tl.TL_OK
    check4(q, c, table, lengths, out, e, bad_pages=(pages, -3))


def test_paged_attention_4_bits_small_weights(tl, ctx):
    """One key far above the rest whose value is 0, and 8191 alike whose value is 1, 2^-25 of its weight each."""
    n, kv, d, page, batch = 8192, 8, 128, 64, 64
    k, v = torch.zeros((n, kv, d)), torch.ones((n, kv, d))
    k[0, :, 0], v[0] = 16.0, 0.0
    c = dict(values=[], codes=[], blocks=[], scale=[])
    for x in (k, v):
        s = torch.full((kv,), 2.0 ** -9)
        codes, blocks, values = pools4(x.view(-1, page, kv, d), s)
        # 16 / 6 / s rounds to a block scale of which 6 makes other than 16: give its block by hand
        c["codes"].append(codes), c["blocks"].append(blocks), c["values"].append(values), c["scale"].append(s)
    q = torch.zeros((batch, kv, d), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    top = float(c["values"][0][0, 0, 0, 0])
    scale = 17.5 / top
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").expand(batch, -1).contiguous()
    out, e = run4(tl, ctx, q, c, table, torch.full((batch,), n, dtype=torch.int32, device="cuda"), scale=scale)
    assert ctx.check() == tl.TL_OK
    flat = [x.reshape(n, kv, d) for x in c["values"]]
    want, lse, tol, ltol = serving.attend(f64(q)[0, 0], flat[0][:, 0], flat[1][:, 0], scale, serving.HALF_STEP["bf16"], True)
    shape = (batch, kv, d)
    close(f64(out), np.broadcast_to(want, shape), np.broadcast_to(tol, shape), "out")
    close(f64(e), np.broadcast_to(lse, shape[:2]), np.broadcast_to(ltol, shape[:2]), "lse")


# ------------------------------------------------------------------------------------------------ plan
def plan_case(batch, longest, most_new, page, seed, spare=3, room=2):
    rng = np.random.default_rng(seed)
    lens, new = rng.integers(0, longest + 1, batch), rng.integers(0, most_new + 1, batch)
    has, needs = -(-lens // page), -(-(lens + new) // page)
    pages = rng.permutation(int(needs.sum()) + spare).astype(np.int32)
    table = np.full((batch, int(max(needs.max(), 1)) + room), -1, np.int32)
    at = 0
    for b in range(batch):
        table[b, :has[b]] = pages[at:at + has[b]]
        at += has[b]
    return lens.astype(np.int32), new.astype(np.int32), table, np.concatenate([[-9, -9], pages[at:]]).astype(np.int32), 2


def run_plan(tl, ctx, lens, new, table, page, free, taken, tokens, kv_tokens=None, in_place=False, counts=True):
    dev = [torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda() for a in (lens, new, table, free)]
    full = lambda n: torch.full((n,), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    lengths, t = dev[0], ints(taken)
    out = dict(table=dev[2], slots=full(tokens), positions=full(tokens), cu_q=full(len(lens) + 1), cu_k=full(len(lens) + 1),
               lengths=lengths if in_place else full(len(lens)), taken=t if in_place else full(1))
    if kv_tokens is not None:
        out["kv_slots"] = full(kv_tokens)
    tl.tl_cache_plan(ctx, lengths, dev[2], page, dev[3], t, out["taken"], out["lengths"], out["cu_q"], out["slots"], out["positions"],
                     counts=dev[1] if counts else None, cu_k=out["cu_k"], kv_slots=out.get("kv_slots"))
    return {w: x.cpu().numpy() for w, x in out.items()}


def same_plan(got, want):
    assert got.keys() == want.keys()
    for w in want:
        assert np.array_equal(got[w], want[w]), w


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,longest,most_new,page", [(1, 0, 1, 16), (1, 5, 3000, 1), (3, 100, 40, 7), (64, 900, 1, 16), (200, 50, 90, 64),
                                                         (513, 33, 5, 5), (1025, 20, 3, 16), (4096, 9, 2, 4), (37, 6001, 4096, 16)])
def test_plan(tl, ctx, batch, longest, most_new, page, in_place):
    lens, new, table, free, taken = plan_case(batch, longest, most_new, page, batch)
    tokens, rows = int(new.sum()) + 5, int((lens + new).sum())
    want, ok = step.cache_plan(lens, new, table, page, free, taken, tokens, rows)
    assert ok
    same_plan(run_plan(tl, ctx, lens, new, table, page, free, taken, tokens, rows, in_place), want)
    assert ctx.check() == tl.TL_OK
    if not in_place:                                        # without the optional outputs; more room than rows
        want, _ = step.cache_plan(lens, np.ones(batch, int), table, page, free, taken, batch)
        if want["slots"].min() >= 0:
            got = run_plan(tl, ctx, lens, new, table, page, free, taken, batch, counts=False)
            same_plan(got, want)


@pytest.mark.parametrize("what", ["tokens", "pages", "both", "kv", "rows", "negative", "count", "taken", "page"])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_reports_what_does_not_fit(tl, ctx, what, in_place):
    lens, new, table, free, taken = plan_case(20, 60, 30, 8, 4)
    new[7] = 0
    tokens, rows = int(new.sum()), int((lens + new).sum())
    if what in ("tokens", "both"):
        tokens -= 40
    if what in ("pages", "both"):
        free = free[:-20]
    if what == "kv":
        rows -= 9
    if what == "rows":
        lens[3], new[4], new[5], lens[6] = table.shape[1] * 8 + 1, table.shape[1] * 8, 2 ** 31 - 1, 2 ** 31 - 1
    if what == "negative":
        lens[3] = -1
        lens[9] = -2 ** 31
    if what == "count":
        new[3] = -5
    if what == "taken":
        taken = len(free) + 1
    if what == "page":
        free[4] = -2
        table[2, 0] = -1
    want, ok = step.cache_plan(lens, new, table, 8, free, taken, tokens, rows)
    assert not ok
    same_plan(run_plan(tl, ctx, lens, new, table, 8, free, taken, tokens, rows, in_place), want)
    assert ctx.check() == tl.TL_ERR_INDEX and ctx.check() == tl.TL_OK


def test_plan_of_nothing(tl, ctx):
    got = run_plan(tl, ctx, np.zeros(0), np.zeros(0), np.zeros((0, 3)), 16, np.zeros(4), 1, 6, 2)
    assert got["slots"].tolist() == [-1] * 6 and got["cu_q"].tolist() == [0] and got["cu_k"].tolist() == [0]
    assert got["taken"].tolist() == [1] and got["kv_slots"].tolist() == [-1] * 2 and got["positions"].tolist() == [0] * 6
    got = run_plan(tl, ctx, np.zeros(3), np.zeros(3), np.zeros((3, 0)), 16, np.zeros(0), 0, 0)
    assert got["cu_q"].tolist() == [0] * 4 and got["lengths"].tolist() == [0] * 3
    assert ctx.check() == tl.TL_OK


def test_plan_page_numbers_past_the_range_of_slots(tl, ctx):
    """2^31 slots are not numbered: a page number that leads there gives no slot."""
    got = run_plan(tl, ctx, np.array([0]), np.array([2]), np.full((1, 2), -1), 16, np.array([2 ** 27]), 0, 2)
    assert got["slots"].tolist() == [-1, -1] and ctx.check() == tl.TL_ERR_INDEX


def test_plan_steps_of_a_captured_graph(tl, ctx):
    """A step in place, replayed: lengths, pages taken and the table go on by themselves."""
    page, batch, n = 4, 5, 11
    lens = torch.tensor([0, 3, 4, 9, 1], dtype=torch.int32, device="cuda")
    has = -(-lens.cpu() // page)
    table = torch.full((batch, 8), -1, dtype=torch.int32)
    at = 0
    for b in range(batch):
        table[b, :has[b]] = torch.arange(at, at + int(has[b]))
        at += int(has[b])
    table, free, taken = table.cuda(), torch.arange(100, 130, dtype=torch.int32, device="cuda"), ints(0)
    slots, pos, cu = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (batch + 2, batch + 2, batch + 1))
    was = (lens.cpu().numpy().copy(), table.cpu().numpy().copy())
    call = lambda: tl.tl_cache_plan(ctx, lens, table, page, free, taken, taken, lens, cu, slots, pos)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    want = dict(lengths=was[0], table=was[1], taken=np.array([0]))
    for _ in range(n):
        graph.replay()
        want, ok = step.cache_plan(want["lengths"], [1] * batch, want["table"], page, free.tolist(), int(want["taken"][0]), batch + 2)
        assert ok and slots.tolist() == want["slots"].tolist() and pos.tolist() == want["positions"].tolist()
        assert lens.tolist() == want["lengths"].tolist() and np.array_equal(table.cpu().numpy(), want["table"])
        assert taken.tolist() == want["taken"].tolist()
    assert ctx.check() == tl.TL_OK


# ------------------------------------------------------------------------------------------------ norms and rotation
def freqs(r, base=10000.0):
    return torch.from_numpy(1.0 / base ** (np.arange(0, r, 2) / r)).float()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,heads,kv,d,rotary,interleaved,weights", [
    (1, 1, 1, 64, 64, False, "same"), (1, 32, 8, 128, 128, False, "same"), (7, 3, 1, 128, 64, True, "fp32"), (33, 28, 4, 64, 32, False, "q"),
    (500, 8, 2, 128, 128, True, "none"), (2000, 5, 5, 64, 16, True, "k"), (64, 64, 8, 128, 0, False, "same"), (3, 0, 2, 64, 64, False, "same"),
    (4, 17, 0, 128, 112, False, "fp32"), (1500, 16, 2, 128, 48, False, "same")])
def test_norm_rope(tl, ctx, dtype, tokens, heads, kv, d, rotary, interleaved, weights):
    x = (draws(tokens, tokens, heads + 2 * kv + 1, d) * 2).to(DT[dtype]).cuda()
    x[0, 0] = 0                                             # a row of zeros
    q, k = x[:, :heads], x[:, heads:heads + kv]
    w = [(draws(5 + i, d) * 0.3 + 1).to(torch.float32 if weights == "fp32" else DT[dtype]).cuda() for i in range(2)]
    w = [w[0] if weights in ("same", "fp32", "q") else None, w[1] if weights in ("same", "fp32", "k") else None]
    pos = torch.from_numpy(np.random.default_rng(1).integers(0, 1 << 20, tokens).astype(np.int32))
    pos[0] = 0
    if tokens > 2:
        pos[1], pos[2] = -5, (1 << 24) - 1
    f = freqs(rotary)
    outs = [torch.full((tokens, n + 1, d), 9.0, dtype=DT[dtype], device="cuda")[:, 1:] for n in (heads, kv)]
    kw = dict(q_weight=w[0], k_weight=w[1], eps=1e-5, interleaved=interleaved)
    args = (pos.cuda(), f.cuda()) if rotary else (None, None)
    tl.tl_norm_rope(ctx, q, k, *args, *outs, **kw)
    for rows, weight, got in ((q, w[0], outs[0]), (k, w[1], outs[1])):
        want, tol = step.norm_rope(f64(rows), None if weight is None else f64(weight), pos.numpy(), f.double().numpy() if rotary else None, 1e-5,
                                   interleaved, serving.HALF_STEP[dtype])
        close(f64(got), want, tol, "rows")
    tl.tl_norm_rope(ctx, q, k, *args, q, k, **kw)           # in place: the same bits
    assert torch.equal(q, outs[0]) and torch.equal(k, outs[1])
    assert torch.equal(x[:, heads + kv:], (draws(tokens, tokens, heads + 2 * kv + 1, d) * 2).to(DT[dtype]).cuda()[:, heads + kv:])


def test_norm_rope_far_positions(tl, ctx):
    """Angles of 2^31 turns and more; frequencies above 1, negative, 0 and the smallest."""
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 7], np.int32)
    f = freqs(128, 1e9)
    f[0], f[1], f[2], f[3], f[4], f[5] = 3.7, -0.91, 0.0, 1e-45, 1e-38, 123456.0
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    x = torch.zeros((4, 1, 128), dtype=torch.float16)
    x[:, :, :64] = 1.0                                      # (cos, sin) of each pair
    got = [torch.empty((4, 1, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    tl.tl_norm_rope(ctx, x.cuda(), x.cuda(), torch.from_numpy(pos).cuda(), f.cuda(), *got)
    for i, p in enumerate(pos.tolist()):
        for j in range(64):
            a = Fraction(p) * Fraction(float(f[j]))
            a = float(a - 2 * pi * round(a / (2 * pi)))
            # F is off by 2^-64 turns, for |f| above 1 by |f| 2^-63
            off = 2 ** -20 + abs(p) * 2.0 ** -61 * max(1.0, abs(float(f[j]))) * 2 * math.pi
            for want, at in ((math.cos(a), j), (math.sin(a), j + 64)):
                assert abs(float(got[0][i, 0, at]) - want) <= off + 2.0 ** -11 * abs(want) + 2.0 ** -24, (p, float(f[j]))
    assert torch.equal(got[0], got[1])


def test_norm_rope_large_and_infinite_rows(tl, ctx):
    """A row with a NaN or an infinity is not finite, and no other row notices; squares past fp32's range give zeros."""
    x = draws(3, 4, 3, 64).bfloat16().cuda()
    clean = torch.empty_like(x)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    pos, f = torch.arange(4, dtype=torch.int32, device="cuda"), freqs(64).cuda()
    none = x[:, :0]
    tl.tl_norm_rope(ctx, x, none, pos, f, clean, none, q_weight=w)
    y = x.clone()
    y[0, 1, 3], y[1, 2, 40], y[2, 0, 7] = math.nan, math.inf, 3e30
    out = torch.empty_like(x)
    tl.tl_norm_rope(ctx, y, none, pos, f, out, none, q_weight=w)
    assert torch.isnan(out[0, 1]).all() and not torch.isfinite(out[1, 2]).all() and (out[2, 0] == 0).all()
    keep = torch.ones((4, 3), dtype=torch.bool)
    keep[0, 1] = keep[1, 2] = keep[2, 0] = False
    assert torch.equal(out[keep], clean[keep])


# ------------------------------------------------------------------------------------------------ log probabilities
def run_score(tl, ctx, x, targets, top, scale=1.0, w=None):
    rows, vocab = x.shape
    out = {k: torch.full((rows,), 7.0, device="cuda") for k in ("logprob", "entropy", "lse")}
    best, ids = torch.full((rows, top), 7.0, device="cuda"), torch.full((rows, top), -7, dtype=torch.int32, device="cuda")
    w = ws(tl.tl_token_logprobs_workspace_bytes(rows, vocab, top)) if w is None else w
    tl.tl_token_logprobs(ctx, x, targets, out["logprob"] if targets is not None else None, w, entropy=out["entropy"], lse=out["lse"],
                         top_logprobs=best, top_ids=ids, scale=scale)
    return out, best, ids


def check_score(x, targets, top, out, best, ids, scale=1.0):
    t = None if targets is None else targets.cpu().numpy()
    live = np.arange(x.shape[0]) if t is None else np.nonzero(t >= 0)[0]
    want, tol, wid, wbest, btol = step.token_logprobs(f64(x)[live], None if t is None else t[live], top, scale)
    assert np.array_equal(ids.cpu().numpy()[live], wid)
    for w in ("entropy", "lse") if t is None else ("logprob", "entropy", "lse"):
        close(f64(out[w])[live], want[w], tol[w], w)
    close(f64(best)[live], wbest, btol, "top")
    left = np.setdiff1d(np.arange(x.shape[0]), live)
    for o in out.values():
        assert (f64(o)[left] == 7.0).all()
    assert (f64(best)[left] == 7.0).all() and (ids.cpu().numpy()[left] == -7).all()


def logits(rows, vocab, dtype, seed, kind):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, vocab)) * 3
    if kind == "masked":
        x[:, rng.random(vocab) < 0.97] = -np.inf
        x[-1] = -np.inf
    elif kind == "tail":                                    # all but the last few tokens are masked
        x[:, :max(0, vocab - 3)] = -np.inf
    elif kind == "ties":
        x = rng.integers(-2, 3, (rows, vocab)).astype(float)
    elif kind == "same":
        x[:] = rng.standard_normal((rows, 1))
    elif kind == "up":
        x.sort(-1)
    elif kind == "down":
        x[:] = -np.sort(-x)
    elif kind == "lowest":
        x[:] = np.where(rng.random((rows, vocab)) < 0.9, float(torch.finfo(dtype).min), x)
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("kind", ["plain", "masked", "tail", "ties", "same", "up", "down", "lowest"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 33, 32), (2, 1000, 5), (5, 8192, 0), (1, 20001, 20), (7, 50001, 32), (1, 131072, 1)])
def test_token_logprobs(tl, ctx, rows, vocab, top, dtype, kind):
    x = logits(rows, vocab, dtype, vocab, kind).cuda()
    t = torch.from_numpy(np.random.default_rng(2).integers(0, vocab, rows).astype(np.int32)).cuda()
    out, best, ids = run_score(tl, ctx, x, t, top, 0.8)
    assert ctx.check() == tl.TL_OK
    # (the scale is an fp32 number)
    check_score(x, t, top, out, best, ids, float(np.float32(0.8)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_token_logprobs_many_rows_skipped_rows_and_views(tl, ctx, dtype):
    """Rows that start anywhere, of a wider buffer; padding; more rows than are split."""
    for rows, vocab, top in ((300, 777, 4), (1100, 130, 2), (40, 9001, 7)):
        wide = logits(rows, vocab + 13, dtype, rows, "plain").cuda()
        x = wide[:, :vocab]
        t = torch.from_numpy(np.random.default_rng(rows).integers(0, vocab, rows).astype(np.int32))
        t[::7] = -1
        t = t.cuda()
        out, best, ids = run_score(tl, ctx, x, t, top)
        assert ctx.check() == tl.TL_OK
        check_score(x, t, top, out, best, ids)
        out, best, ids = run_score(tl, ctx, x, None, top)
        check_score(x, None, top, out, best, ids)


def test_token_logprobs_non_finite_rows(tl, ctx):
    vocab, top = 20000, 6
    x = logits(6, vocab, torch.float32, 1, "plain")
    x[0, 5], x[1, 19999], x[2, 100], x[3, 7], x[3, 9] = math.nan, math.inf, -math.inf, math.inf, math.nan
    x[4] = math.nan
    x = x.cuda()
    t = ints(1, 2, 100, 3, 0, 5)
    out, best, ids = run_score(tl, ctx, x, t, top)
    assert ctx.check() == tl.TL_OK
    check_score(x, t, top, out, best, ids)
    assert out["logprob"][2] == -math.inf


def test_token_logprobs_reports_targets_out_of_range(tl, ctx):
    x = logits(4, 30000, torch.float32, 1, "plain").cuda()
    t = ints(3, 30000, 2 ** 31 - 1, 29999)
    w = ws(tl.tl_token_logprobs_workspace_bytes(4, 30000, 3))
    out, best, ids = run_score(tl, ctx, x, t, 3, w=w)
    assert ctx.check() == tl.TL_ERR_INDEX and ctx.check() == tl.TL_OK
    skip = ints(3, -1, -1, 29999)
    check_score(x, skip, 3, out, best, ids)
    assert not w[:tl_counter_bytes].any()


tl_counter_bytes = 139264


def test_token_logprobs_shares_the_workspace_and_repeats_its_bits(tl, ctx):
    """One workspace for attention and log probabilities of several shapes, twice, and in a graph."""
    q, c, table, lengths = case4([3000, 20], 8, 2, 128, 16, "bf16", False, seed=3)
    xs = [logits(r, v, torch.float32, v, "plain").cuda() for r, v in ((1, 131072), (3, 60000), (64, 9000))]
    n = max([tl.tl_token_logprobs_workspace_bytes(*x.shape, 20) for x in xs] + [tl.tl_paged_attention_workspace_bytes(2, 8, 2, 128)])
    w, first = ws(n), None
    for _ in range(2):
        got = [run4(tl, ctx, q, c, table, lengths, w)]
        for x in xs:
            t = torch.arange(x.shape[0], dtype=torch.int32, device="cuda")
            out, best, ids = run_score(tl, ctx, x, t, 20, w=w)
            check_score(x, t, 20, out, best, ids)
            got.append((*out.values(), best, ids))
        assert first is None or all(torch.equal(a, b) for g, h in zip(first, got) for a, b in zip(g, h))
        first = got
    x, t = xs[0], ints(77)
    lp, best, ids = torch.zeros(1, device="cuda"), torch.zeros((1, 20), device="cuda"), torch.zeros((1, 20), dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.tl_token_logprobs(ctx, x, t, lp, w, top_logprobs=best, top_ids=ids)
    for seed in range(3):
        x.copy_(logits(1, 131072, torch.float32, seed, "plain"))
        graph.replay()
        want, tol, wid, wb, bt = step.token_logprobs(f64(x), [77], 20, 1.0)
        close(f64(lp), want["logprob"], tol["logprob"], "logprob")
        assert np.array_equal(ids.cpu().numpy(), wid)


# ------------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("bits", [4, 8, 16])
def test_a_turn_a_continued_turn_and_steps(tl, ctx, bits):
    """Two sequences: prompts, then a second turn whose queries see the rows read back from the cache, then captured steps, each
    through the plan, the norms and rotation, the append, and attention; everything against the 64-bit forms over the rows that the
    cache holds."""
    heads, kv, d, page, batch, dtype = 4, 2, 64, 8, 2, torch.bfloat16
    pages = 40
    if bits == 4:
        pools = [torch.zeros((pages, page, kv, d // 2), dtype=torch.uint8, device="cuda") for _ in "kv"]
        blocks = [torch.zeros((pages, page, kv, d // 16), device="cuda").to(E4M3) for _ in "kv"]
        kw = dict(k_scale=scales(kv, 0).cuda(), v_scale=scales(kv, 1).cuda(), k_blocks=blocks[0], v_blocks=blocks[1])
    else:
        pools = [torch.zeros((pages, page, kv, d), device="cuda").to(dtype if bits == 16 else E4M3) for _ in "kv"]
        kw = {} if bits == 16 else dict(k_scale=scales(kv, 0).cuda() * 16, v_scale=scales(kv, 1).cuda() * 16)
    table = torch.full((batch, 12), -1, dtype=torch.int32, device="cuda")
    free, taken, lens = torch.randperm(pages, device="cuda").to(torch.int32), ints(0), torch.zeros(batch, dtype=torch.int32, device="cuda")
    wq, wk = ((draws(5 + i, d) * 0.2 + 1).to(dtype).cuda() for i in range(2))
    f = freqs(d).cuda()
    n64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731

    def values():
        """[pages, page, kv, d]: what the cache holds, with the heads' scales."""
        if bits == 4:
            return [step.from_4_bits(raw(c), raw(b), n64(s)) for c, b, s in zip(pools, blocks, (kw["k_scale"], kw["v_scale"]))]
        return [f64(p) * (1 if bits == 16 else n64(s)[:, None]) for p, s in zip(pools, (kw.get("k_scale"), kw.get("v_scale")))]

    for turn, new in enumerate(([13, 30], [20, 1])):
        n = sum(new) + 2
        qkv = draws(turn, n, heads + 2 * kv, d).to(dtype).cuda()
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        slots, pos, rows = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (n, n, 96))
        cu_q, cu_k = ints(0, 0, 0), ints(0, 0, 0)
        tl.tl_cache_plan(ctx, lens, table, page, free, taken, taken, lens, cu_q, slots, pos, counts=ints(*new), cu_k=cu_k, kv_slots=rows)
        tl.tl_norm_rope(ctx, q, k, pos, f, q, k, q_weight=wq, k_weight=wk)
        tl.tl_kv_append(ctx, k, v, *pools, slots, **kw)
        packed = [torch.zeros((96, kv, d), dtype=dtype, device="cuda") for _ in "kv"]
        tl.tl_kv_gather(ctx, *pools, rows, *packed, **kw)
        out = torch.full((n, heads, d), 7.0, dtype=dtype, device="cuda")
        tl.tl_window_attention(ctx, q, *packed, cu_q, cu_k, out)
        assert ctx.check() == tl.TL_OK
        total = int(cu_k[-1])
        assert total == int(lens.sum()) and (slots[-2:] == -1).all()
        held = [x[rows[:total].cpu().numpy() // page, rows[:total].cpu().numpy() % page] for x in values()]
        for x, p in zip(held, packed):
            assert np.array_equal(torch.from_numpy(x.astype(np.float32)).to(dtype).double().numpy(), f64(p[:total]))
        want, _, tol, _ = serving.window_attention(f64(q), f64(packed[0][:total]), f64(packed[1][:total]), cu_q.tolist(), cu_k.tolist(), d ** -0.5)
        close(f64(out[:-2]), want[:-2], tol[:-2], "turn")
        assert (out[-2:] == 7.0).all()

    qkv = draws(9, batch, heads + 2 * kv, d).to(dtype).cuda()
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    slots, pos, cu = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (batch, batch, batch + 1))
    qr, kr, out = torch.empty_like(q), torch.empty_like(k), torch.empty((batch, heads, d), dtype=dtype, device="cuda")
    x, lp = logits(batch, 5000, torch.float32, 4, "plain").cuda(), torch.zeros(batch, device="cuda")
    best, ids = torch.zeros((batch, 3), device="cuda"), torch.zeros((batch, 3), dtype=torch.int32, device="cuda")
    w = ws(max(tl.tl_paged_attention_workspace_bytes(batch, heads, kv, d), tl.tl_token_logprobs_workspace_bytes(batch, 5000, 3)))

    def a_step():
        tl.tl_cache_plan(ctx, lens, table, page, free, taken, taken, lens, cu, slots, pos)
        tl.tl_norm_rope(ctx, q, k, pos, f, qr, kr, q_weight=wq, k_weight=wk)
        tl.tl_kv_append(ctx, kr, v, *pools, slots, **kw)
        tl.tl_paged_attention(ctx, qr, *pools, table, lens, out, w, **kw)
        tl.tl_token_logprobs(ctx, x, ids[:, 0].contiguous(), lp, w, top_logprobs=best, top_ids=ids)

    before = lens.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a_step()
    for i in range(10):                                     # over the end of a page
        graph.replay()
        assert ctx.check() == tl.TL_OK and torch.equal(lens, before + i + 1)
        want, _, tol, _ = serving.paged_attention(f64(qr), *values(), table.cpu().numpy(), lens.tolist(), d ** -0.5, u=serving.HALF_STEP["bf16"],
                                                  fp16_weights=bits < 16)
        close(f64(out), want, tol, "step")
        assert pos.tolist() == (lens - 1).tolist()
    wid = step.token_logprobs(f64(x), [0] * batch, 3, 1.0)[2]
    assert np.array_equal(ids.cpu().numpy(), wid)
