"""Calls of the step's operators that the header allows and that nothing else makes: codes that differ in every block, the plan's
largest batch in each of its forms, without its optional outputs and with one of its two numbers in place, gathers into the
other type, and the largest shapes."""
import numpy as np
import pytest
import torch

from oracle import serving, step
from tests.test_gpu_serving import DT, close, ctx, draws, f64, tl, ws  # noqa: F401
from tests.test_gpu_step import E4M3, LENS, case4, check4, freqs, ints, plan_case, raw, run4, same_plan, scales

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ the 4-bit cache
def random_codes(c, seed):
    """Every code of every row that is seen drawn anew (rows that are not keep what spoils them)."""
    rng = np.random.default_rng(seed)
    for i in range(2):
        kept = raw(c["blocks"][i])
        codes = rng.integers(0, 256, tuple(c["codes"][i].shape)).astype(np.uint8)
        codes[(kept == 0x7F).all(-1)] = 0x7F
        c["codes"][i].copy_(torch.from_numpy(codes).cuda())
        c["values"][i] = step.from_4_bits(codes, kept)
        blocks = [len(np.unique(codes[..., 8 * j:8 * j + 8])) for j in range(codes.shape[-1] // 8)]
        assert min(blocks) > 200                            # all blocks hold codes of all kinds
    return c


@pytest.mark.parametrize("heads,kv,d,dtype,head_major", [(8, 1, 64, "bf16", False), (8, 2, 128, "fp16", False), (16, 1, 64, "fp16", True),
                                                         (34, 2, 128, "bf16", False), (12, 4, 64, "bf16", False), (32, 8, 128, "bf16", True)])
def test_paged_attention_4_bits_every_code_differs(tl, ctx, heads, kv, d, dtype, head_major):
    q, c, table, lengths = case4(LENS, heads, kv, d, 16, dtype, head_major, seed=heads + d)
    c = random_codes(c, d)
    out, e = run4(tl, ctx, q, c, table, lengths)
    assert ctx.check() == tl.TL_OK
    check4(q, c, table, lengths, out, e)


@pytest.mark.parametrize("d", [64, 128])
def test_paged_attention_4_bits_every_key_by_itself(tl, ctx, d):
    """One row a sequence: the output is that row's V, dim by dim, whatever its codes and its place in a page."""
    n, kv, page = 200, 4, 8
    q, c, table, lengths = case4([1] * n, 2 * kv, kv, d, page, "fp16", False, seed=d)
    c = random_codes(c, d + 1)
    out, e = run4(tl, ctx, q, c, table, lengths)
    want = c["values"][1][table[:, 0].cpu().numpy(), 0] * c["scale"][1].double().numpy()[:, None]
    # (a weight of 1, a sum of 1: fp32's product with the scale, then fp16's rounding)
    close(f64(out), np.repeat(want, 2, 1), np.repeat(np.abs(want), 2, 1) * (2.0 ** -11 + 2.0 ** -21) + 2.0 ** -25, "out")


@pytest.mark.parametrize("d", [64, 128])
def test_paged_attention_4_bits_of_the_largest_batch(tl, ctx, d):
    lens = [int(n) for n in np.random.default_rng(d).integers(0, 40, 4096)]
    q, c, table, lengths = case4(lens, 2, 1, d, 8, "bf16", False, seed=d)
    out, e = run4(tl, ctx, q, c, table, lengths)
    assert ctx.check() == tl.TL_OK
    check4(q, c, table, lengths, out, e)


def test_gather_e4m3_rows_as_fp16(tl, ctx):
    pages, page, heads, d, n = 9, 16, 3, 128, 50
    pools = [(draws(i, pages, page, heads, d) * 40).to(E4M3) for i in range(2)]
    s = [scales(heads, i) for i in range(2)]
    slots = np.random.default_rng(1).integers(0, pages * page, n).astype(np.int32)
    outs = [torch.empty((n, heads, d), dtype=torch.float16, device="cuda") for _ in "kv"]
    tl.tl_kv_gather(ctx, *[p.cuda() for p in pools], torch.from_numpy(slots).cuda(), *outs, k_scale=s[0].cuda(), v_scale=s[1].cuda())
    assert ctx.check() == tl.TL_OK
    for p, scale, got in zip(pools, s, outs):
        want = (p.float() * scale[:, None]).half()[torch.from_numpy(slots // page).long(), torch.from_numpy(slots % page).long()]
        assert torch.equal(got.cpu(), want)


# ------------------------------------------------------------------------------------------------ plan
def planned(tl, ctx, lens, new, table, page, free, taken, tokens, kv_tokens=None, in_place=(), without=()):
    """The call with lengths, taken, both or neither in place, and without the optional outputs named."""
    dev = [torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda() for a in (lens, table, free)]
    full = lambda n: torch.full((n,), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    t = ints(taken)
    out = dict(table=dev[1], slots=full(tokens), positions=full(tokens), cu_q=full(len(lens) + 1), cu_k=full(len(lens) + 1),
               lengths=dev[0] if "lengths" in in_place else full(len(lens)), taken=t if "taken" in in_place else full(1))
    if kv_tokens is not None:
        out["kv_slots"] = full(kv_tokens)
    out = {w: None if w in without else x for w, x in out.items()}
    counts = None if new is None else torch.from_numpy(np.ascontiguousarray(new, np.int32)).cuda()
    tl.tl_cache_plan(ctx, dev[0], out["table"], page, dev[2], t, out["taken"], out["lengths"], out["cu_q"], out["slots"], out.get("positions"),
                     counts=counts, cu_k=out.get("cu_k"), kv_slots=out.get("kv_slots"))
    got = {w: x.cpu().numpy() for w, x in out.items() if x is not None}
    if "lengths" not in in_place:
        assert np.array_equal(dev[0].cpu().numpy(), lens)
    if "taken" not in in_place:
        assert t.tolist() == [taken]
    return got


@pytest.mark.parametrize("in_place", [(), ("lengths",), ("taken",), ("lengths", "taken")])
@pytest.mark.parametrize("batch,longest,page", [(2, 9, 4), (511, 70, 16), (512, 33, 5), (513, 70, 16), (3000, 20, 8), (4096, 9, 4), (4096, 100, 16)])
def test_plan_of_a_step_without_counts(tl, ctx, batch, longest, page, in_place):
    """One new token each, up to 4096 sequences: one CTA, several of a cluster (with more than 48 KB of shared memory), or plain."""
    lens, _, table, free, taken = plan_case(batch, longest, 1, page, batch, spare=batch + 3)
    want, ok = step.cache_plan(lens, np.ones(batch, int), table, page, free, taken, batch)
    assert ok
    same_plan(planned(tl, ctx, lens, None, table, page, free, taken, batch, in_place=in_place), want)
    assert ctx.check() == tl.TL_OK


@pytest.mark.parametrize("in_place", [("lengths",), ("taken",)])
@pytest.mark.parametrize("batch,longest,most_new,page", [(1, 5, 3000, 1), (64, 900, 1, 16), (1025, 20, 30, 16), (37, 6001, 4096, 16)])
def test_plan_with_one_of_its_numbers_in_place(tl, ctx, batch, longest, most_new, page, in_place):
    """By one CTA, by a cluster, and by two launches."""
    lens, new, table, free, taken = plan_case(batch, longest, most_new, page, batch)
    tokens, rows = int(new.sum()) + 5, int((lens + new).sum())
    want, ok = step.cache_plan(lens, new, table, page, free, taken, tokens, rows)
    assert ok
    same_plan(planned(tl, ctx, lens, new, table, page, free, taken, tokens, rows, in_place), want)
    assert ctx.check() == tl.TL_OK


@pytest.mark.parametrize("without", [("positions",), ("cu_k",), ("positions", "cu_k")])
@pytest.mark.parametrize("kv", [False, True])
@pytest.mark.parametrize("batch,longest,most_new,page", [(1, 5, 3000, 1), (200, 50, 90, 64), (4096, 9, 2, 4)])
def test_plan_without_its_optional_outputs(tl, ctx, batch, longest, most_new, page, kv, without):
    lens, new, table, free, taken = plan_case(batch, longest, most_new, page, batch + 1)
    tokens, rows = int(new.sum()), int((lens + new).sum()) + 4
    want, ok = step.cache_plan(lens, new, table, page, free, taken, tokens, rows if kv else None)
    assert ok
    for in_place in ((), ("lengths", "taken")):
        got = planned(tl, ctx, lens, new, table, page, free, taken, tokens, rows if kv else None, in_place, without)
        same_plan(got, {w: x for w, x in want.items() if w not in without})
    assert ctx.check() == tl.TL_OK


def test_plan_of_the_largest_step_in_a_graph(tl, ctx):
    """4096 sequences in place, replayed over the ends of pages."""
    batch, page = 4096, 4
    lens, _, table, free, taken = plan_case(batch, 9, 1, page, 5, spare=3 * batch, room=3)
    dev = [torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda() for a in (lens, table, free)]
    t, slots, pos, cu = ints(taken), *(torch.zeros(n, dtype=torch.int32, device="cuda") for n in (batch, batch, batch + 1))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tl.tl_cache_plan(ctx, dev[0], dev[1], page, dev[2], t, t, dev[0], cu, slots, pos)
    want = dict(lengths=lens, table=table, taken=np.array([taken]))
    for _ in range(6):
        g.replay()
        want, ok = step.cache_plan(want["lengths"], np.ones(batch, int), want["table"], page, free, int(want["taken"][0]), batch)
        assert ok
        same_plan(dict(table=dev[1].cpu().numpy(), slots=slots.cpu().numpy(), positions=pos.cpu().numpy(), cu_q=cu.cpu().numpy(),
                       lengths=dev[0].cpu().numpy(), taken=t.cpu().numpy()), {w: x for w, x in want.items() if w != "cu_k"})
    assert ctx.check() == tl.TL_OK


@pytest.mark.parametrize("in_place", [(), ("lengths", "taken")])
def test_plan_of_the_largest_pages(tl, ctx, in_place):
    """Lengths, slots and bounds up to the ends of 32 bits, by hand."""
    n = (1 << 30) - 1
    got = planned(tl, ctx, np.array([n - 3, 0, n]), np.array([3, 2, 0]), np.array([[0], [-1], [0]]), n, np.array([9, 1]), 1, 6, in_place=in_place)
    assert got["slots"].tolist() == [n - 3, n - 2, n - 1, n, n + 1, -1] and got["positions"].tolist() == [n - 3, n - 2, n - 1, 0, 1, 0]
    assert got["table"].tolist() == [[0], [1], [0]] and got["lengths"].tolist() == [n, 2, n] and got["taken"].tolist() == [2]
    # (2^31 rows in all: sums stop at 2^31 - 1)
    assert got["cu_q"].tolist() == [0, 3, 5, 5] and got["cu_k"].tolist() == [0, n, n + 2, 2 ** 31 - 1]
    n = 715827881
    got = planned(tl, ctx, np.array([n - 1, 2 * n - 2]), np.array([3, 2]), np.array([[0, -1], [1, 0]]), n, np.array([2]), 0, 5, in_place=in_place)
    assert got["slots"].tolist() == [n - 1, 2 * n, 2 * n + 1, n - 2, n - 1] and got["positions"].tolist() == [n - 1, n, n + 1, 2 * n - 2, 2 * n - 1]
    assert got["table"].tolist() == [[0, 2], [1, 0]] and got["lengths"].tolist() == [n + 2, 2 * n] and got["taken"].tolist() == [1]
    assert got["cu_k"].tolist() == [0, n + 2, 3 * n + 2] and 3 * n + 2 == 2 ** 31 - 3
    assert ctx.check() == tl.TL_OK


# ------------------------------------------------------------------------------------------------ norms and rotation, log probabilities
def test_norm_rope_of_the_most_heads(tl, ctx):
    tokens, heads, kv, d = 3, 65000, 536, 64
    x = draws(1, tokens, heads + kv, d).bfloat16().cuda()
    q, k = x[:, :heads], x[:, heads:]
    w = [(draws(5 + i, d) * 0.3 + 1).bfloat16().cuda() for i in range(2)]
    pos, f = ints(0, 77, 4001), freqs(d)
    outs = [torch.full((tokens, n, d), 9.0, dtype=torch.bfloat16, device="cuda") for n in (heads, kv)]
    tl.tl_norm_rope(ctx, q, k, pos, f.cuda(), *outs, q_weight=w[0], k_weight=w[1])
    for rows, weight, got, some in ((q, w[0], outs[0], [*range(0, heads, 997), heads - 1]), (k, w[1], outs[1], list(range(kv)))):
        want, tol = step.norm_rope(f64(rows[:, some]), f64(weight), pos.cpu().numpy(), f.double().numpy(), 1e-6, False, serving.HALF_STEP["bf16"])
        close(f64(got[:, some]), want, tol, "rows")
        assert not (got == 9.0).all(-1).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_token_logprobs_of_very_many_rows(tl, ctx, dtype):
    """Rows by the hundred thousand, of a few logits each, against the formula in 64 bits on the GPU."""
    rows, vocab, top = 300001, 5, 3
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randint(-20, 20, (rows, vocab), generator=gen, device="cuda") / 4.0).to(dtype)
    t = torch.randint(-1, vocab, (rows,), generator=gen, device="cuda").to(torch.int32)
    lp, ent = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    best, ids = torch.full((rows, top), 7.0, device="cuda"), torch.full((rows, top), -7, dtype=torch.int32, device="cuda")
    tl.tl_token_logprobs(ctx, x, t, lp, ws(tl.tl_token_logprobs_workspace_bytes(rows, vocab, top)), entropy=ent, top_logprobs=best, top_ids=ids)
    assert ctx.check() == tl.TL_OK
    live = t >= 0
    y = torch.log_softmax(x.double(), -1)
    order = torch.sort(x.double(), dim=-1, descending=True, stable=True).indices[:, :top]
    # |z| is at most 15 here: sums, powers of two and logarithms in fp32 are off by less than 2^-18
    for got, want in ((lp, y.gather(1, t.clamp(min=0).long()[:, None])[:, 0]), (ent, torch.special.entr(y.exp()).sum(-1))):
        assert float((got - want)[live].abs().max()) < 2.0 ** -17 and (got[~live] == 7.0).all()
    assert torch.equal(ids[live].long(), order[live]) and (ids[~live] == -7).all()
    assert float((best - y.gather(1, order))[live].abs().max()) < 2.0 ** -17
