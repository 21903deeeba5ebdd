"""Places where the serving operators can go wrong quietly: what a context reports, bits that depend on what ran
before, small weights, non-finite values, and layouts and plans of unusual sizes."""
import math

import numpy as np
import pytest
import torch

from oracle import serving
from tests.gpu_helpers import to_dev_bf16, workspace
from tests.test_gpu_serving import (DT, check_moe, check_paged, check_window, close, ctx, cum, draws, f64, moe_case,  # noqa: F401
                                    packed, paged_case, run_moe, run_paged, run_window, tl, ws)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ status
@pytest.mark.parametrize("index_first", [True, False])
def test_a_timeout_is_reported_beside_an_index_out_of_range(tl, index_first):
    """An index report leaves workspaces valid, a timeout does not: of both, the check returns the timeout."""
    from seeded_inputs import make_inputs
    inp = make_inputs("ag_gemm", 61, W=2, m_per_rank=128, n=256, k=256)
    a, b = [to_dev_bf16(x) for x in inp["a_shards"]], to_dev_bf16(inp["b"])
    c, work = torch.empty((256, 256), dtype=torch.bfloat16, device="cuda"), workspace(tl.tl_ag_gemm_workspace_bytes(2, 128, 256, 256))
    row, pool = draws(1, 1, 2, 64).bfloat16().cuda(), torch.zeros((1, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    beyond = torch.tensor([16], dtype=torch.int32, device="cuda")
    with tl.Context(0, debug_skip_chunk=3, timeout_ns=50_000_000) as c2:
        for index in (index_first, not index_first):
            if index:
                tl.tl_kv_append(c2, row, row, pool, pool, beyond)
            else:
                tl.tl_ag_gemm(c2, a, b, c, work, rank=0)   # a signal that never comes: the bounded wait runs out
            torch.cuda.synchronize()
        assert c2.check() == tl.TL_ERR_TIMEOUT
        assert c2.check() == tl.TL_OK
        tl.tl_kv_append(c2, row, row, pool, pool, beyond)
        assert c2.check() == tl.TL_ERR_INDEX and c2.check() == tl.TL_OK


# ------------------------------------------------------------------------------------------------ window attention
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [3, 5, 12])
def test_window_attention_does_not_depend_on_what_ran_before(tl, ctx, group, d):
    """Heads that do not divide a tile's 128 rows leave rows of it unused: what an earlier call left there has no
    say in the result.  The earlier call's queries are 0, then 1000 along the one dim in which the keys climb."""
    n = 600
    q, k, v = (t.clone() for t in packed([n], [n], group, 1, d, "bf16", seed=group))
    k[:, 0, 0] = (3 * torch.div(torch.arange(n, device="cuda"), 128, rounding_mode="floor")).bfloat16()
    q[:, :, 0] = 0.5
    before = torch.zeros((256, 160, d), dtype=torch.bfloat16, device="cuda")   # an item for every CTA, whole tiles
    other = draws(5, 256, 160, d).bfloat16().cuda()
    got = []
    for far in (0.0, 1000.0):
        before[:, :, 0] = far
        run_window(tl, ctx, before, other, other, [0, 256], [0, 256])
        got.append(run_window(tl, ctx, q, k, v, [0, n], [0, n]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    check_window(q, k, v, [0, n], [0, n], *got[0])


# ------------------------------------------------------------------------------------------------ small weights
def sink_and_tail(n, d, kv):
    """One key far above the rest whose value is 0, and n others alike whose value is 1: all of the result is
    their weights, 2^-25.2 each beside the first one's 1.  (As rows [n + 1, kv, d], exact in every type.)"""
    k, v = torch.zeros((n + 1, kv, d)), torch.ones((n + 1, kv, d))
    k[0, :, 0], v[0] = 16.0, 0.0
    return k, v, 17.5 / 16


@pytest.mark.parametrize("d", [64, 128])
def test_window_attention_keeps_small_fp16_weights(tl, ctx, d):
    k, v, scale = sink_and_tail(8192, d, 1)
    q = torch.zeros((1, 4, d))
    q[:, :, 0] = 1.0
    q, k, v = (t.to(torch.float16).cuda() for t in (q, k, v))
    out, e = run_window(tl, ctx, q, k, v, [0, 1], [0, k.shape[0]], scale=scale)
    assert ctx.check() == tl.TL_OK
    check_window(q, k, v, [0, 1], [0, k.shape[0]], out, e, scale=scale)
    out, e = run_window(tl, ctx, q, k, v, [0, 1], [0, k.shape[0]], scale=scale, window=8000, sinks=1)
    check_window(q, k, v, [0, 1], [0, k.shape[0]], out, e, 8000, 1, scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,cache", [("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
def test_paged_attention_keeps_small_fp16_weights(tl, ctx, dtype, cache, d):
    """Enough sequences (of the same pages) that none is split: a warp then meets a quarter of the tail with the first key."""
    kv, batch, page = 8, 64, 64
    k, v, scale = sink_and_tail(8191, d, kv)
    pools = [t.view(-1, page, kv, d).to(DT[cache]).cuda() for t in (k, v)]
    table = torch.arange(pools[0].shape[0], dtype=torch.int32, device="cuda").expand(batch, -1).contiguous()
    lengths = torch.full((batch,), 8192, dtype=torch.int32, device="cuda")
    q = torch.zeros((batch, kv, d), dtype=DT[dtype], device="cuda")
    q[:, :, 0] = 1.0
    out, e = run_paged(tl, ctx, q, pools, table, lengths, scale=scale)
    assert ctx.check() == tl.TL_OK
    u = serving.HALF_STEP[dtype]
    want, lse, tol, ltol = serving.attend(q[0, 0].cpu().double().numpy(), k[:, 0].double().numpy(), v[:, 0].double().numpy(), scale, u, True)
    shape = (batch, kv, d)
    close(f64(out), np.broadcast_to(want, shape), np.broadcast_to(tol, shape), "out")
    close(f64(e), np.broadcast_to(lse, shape[:2]), np.broadcast_to(ltol, shape[:2]), "lse")


# ------------------------------------------------------------------------------------------------ non-finite values
def check_rows(q, k, v, rows, out, e, window=0, sinks=0):
    """Some queries of one prompt against the oracle."""
    dtype = "bf16" if q.dtype == torch.bfloat16 else "fp16"
    g, n, scale = q.shape[1] // k.shape[1], q.shape[0], q.shape[2] ** -0.5
    qs, ks, vs = f64(q), f64(k), f64(v)
    for i in rows:
        seen = serving.visible(i, n, window, sinks)
        for h in range(q.shape[1]):
            with np.errstate(invalid="ignore"):
                want, lse, tol, ltol = serving.attend(qs[i, h], ks[seen, h // g], vs[seen, h // g], scale,
                                                      serving.HALF_STEP[dtype], dtype == "fp16")
            tol = np.where(np.isfinite(want), tol, 0.0)
            close(f64(out[i, h]), want, tol, f"out {i} {h}")
            close(f64(e[i, h]), lse, ltol, f"lse {i} {h}")


@pytest.mark.parametrize("heads,kv", [(4, 1), (3, 1), (2, 2)])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
def test_window_attention_non_finite_values_of_a_long_prompt(tl, ctx, heads, kv, d, dtype):
    """Values that are not finite reach the queries that see them, in their dim, as the sum has them: NaN, an infinity,
    or NaN where two infinities meet.  Every other result keeps its bits."""
    n = 2600
    q, k, v = (t.clone() for t in packed([n], [n], heads, kv, d, dtype, seed=heads))
    cu = [0, n]
    for window, sinks in ((0, 0), (500, 3), (130, 140)):
        clean, _ = run_window(tl, ctx, q, k, v, cu, cu, window=window, sinks=sinks)
        w = v.clone()
        w[2, 0, 7], w[1300, 0, 9], w[2000, 0, 9], w[1301, 0, 10] = math.nan, math.inf, -math.inf, -math.inf
        w[2590, 0, 11] = math.nan
        out, e = run_window(tl, ctx, q, k, w, cu, cu, window=window, sinks=sinks)
        assert ctx.check() == tl.TL_OK
        rows = [0, 1, 2, 3, 63, 64, 130, 499, 502, 503, 1269, 1299, 1300, 1301, 1330, 1429, 1430, 1431, 1799, 1800, 1801, 1999,
                2000, 2130, 2499, 2560, 2589, 2590, 2599]
        check_rows(q, k, w, rows, out, e, window, sinks)
        fine = torch.ones(d, dtype=torch.bool)
        fine[[7, 9, 10, 11]] = False
        assert torch.equal(out[:, :, fine], clean[:, :, fine])


def test_window_attention_an_early_nan_costs_no_wait(tl):
    """A NaN that nearly every query of a prompt sees is an answer, not a reason for a wait to run out (4 ms here)."""
    n = 8192
    q, k, v = (t.clone() for t in packed([n], [n], 8, 2, 128, "bf16", seed=12))
    out, clean = torch.empty_like(q), torch.empty_like(q)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    with tl.Context(0, timeout_ns=1_000_000) as c:
        tl.tl_window_attention(c, q, k, v, cu, cu, clean)
        assert c.check() == tl.TL_OK
        v[3, 0, 0] = math.nan
        tl.tl_window_attention(c, q, k, v, cu, cu, out)
        assert c.check() == tl.TL_OK
        assert torch.isnan(out[3:, :4, 0]).all()
        assert torch.equal(out[:3], clean[:3]) and torch.equal(out[:, :, 1:], clean[:, :, 1:]) and torch.equal(out[:, 4:], clean[:, 4:])
        k[5, 1, 0] = math.nan                                # and one in a key: the whole row is NaN
        tl.tl_window_attention(c, q, k, v, cu, cu, out)
        assert c.check() == tl.TL_OK
        assert torch.isnan(out[5:, 4:]).all() and torch.equal(out[:5, 4:], clean[:5, 4:])


def test_window_attention_values_near_the_end_of_the_range(tl, ctx):
    """A stale maximum leaves weights of up to 2^8: values whose sums pass the fp32 range that way, and back in it by
    the division, are still found."""
    n = 300
    q, k, v = (t.clone() for t in packed([n], [n], 2, 1, 64, "bf16", seed=14))
    q[:] = 0
    k[:] = 0
    q[:, :, 0], k[200, 0, 0] = 8.0, 5.0                     # its weight is 2^7.2 beside the others' 1
    v[200, 0, 3] = 3.0e38
    out, e = run_window(tl, ctx, q, k, v, [0, n], [0, n])
    assert torch.isfinite(out).all()
    check_rows(q, k, v, [0, 199, 200, 201, 299], out, e)


# ------------------------------------------------------------------------------------------------ MoE
@pytest.mark.parametrize("T", [1, 9])
def test_moe_tokens_large_hidden_values(tl, ctx, T):
    """h at the end of the range: an infinity stays one (not NaN), and a value that bf16 would round to one is carried
    in full."""
    H, E, F = 64, 2, 64
    x, lg = torch.zeros((T, H)), torch.zeros((T, E))
    x[:, 0], lg[:, 1] = 2.0 ** 62, -40.0
    for gate, up, inf in ((2.0, 8.0, True),                         # 2^63 times 2^65
                          (2 * 129 / 128, 4 * 254 / 128, False)):   # (2 - 2^-13) 2^127, over bf16's largest
        w = [torch.zeros((E, H, F)), torch.zeros((E, H, F)), torch.full((E, F, H), 2.0 ** -20)]
        w[0][:, 0, 5], w[1][:, 0, 5] = gate, up
        case = [t.cuda() for t in (x.bfloat16(), lg, *(m.bfloat16() for m in w))]
        out, ex, g = run_moe(tl, ctx, *case, 1)
        assert ctx.check() == tl.TL_OK
        if inf:
            assert (out == math.inf).all()
        else:
            check_moe(*case, 1, out, ex, g)


# ------------------------------------------------------------------------------------------------ layouts and plans
def test_strides_of_dimensions_of_one_entry_do_not_matter(tl, ctx):
    """One kv head, head-major keys and token-major values: the same addresses, other strides on paper."""
    q, pools, table, lengths = paged_case([40, 3], 4, 1, 64, 16, "bf16", "bf16", False, seed=2, spoil=False)
    major = torch.empty((pools[0].shape[0], 1, 16, 64), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    major.copy_(pools[0])
    assert major.stride() != pools[1].stride()
    want, _ = run_paged(tl, ctx, q, pools, table, lengths)
    out, e = run_paged(tl, ctx, q, (major, pools[1]), table, lengths)
    assert torch.equal(out, want)
    row = draws(1, 1, 1, 64).bfloat16().cuda()
    tl.tl_kv_append(ctx, row, row, major, pools[1], torch.tensor([5], dtype=torch.int32, device="cuda"))
    assert torch.equal(major[0, 5], row[0]) and torch.equal(pools[1][0, 5], row[0])
    with pytest.raises(ValueError, match="strides"):
        two = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
        tl.tl_kv_append(ctx, row.expand(1, 2, 64), row.expand(1, 2, 64), two, two.transpose(1, 2).contiguous().transpose(1, 2),
                        torch.tensor([5], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 2)])
def test_paged_attention_of_many_sequences(tl, ctx, window, sinks):
    """More sequences than threads of a CTA, empty ones at both ends and in runs: each thread plans several."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 90, 700)
    lens[:9], lens[128:140], lens[-20:] = 0, 0, 0
    lens[300] = 1500
    q, pools, table, lengths = paged_case(lens.tolist(), 4, 2, 64, 16, "bf16", "bf16", False, seed=700, window=window, sinks=sinks)
    out, e = run_paged(tl, ctx, q, pools, table, lengths, window=window, sinks=sinks)
    assert ctx.check() == tl.TL_OK
    check_paged(q, pools, table, lengths, out, e, window, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3)])
def test_window_attention_of_continued_prompts_ordered_by_length(tl, ctx, window, sinks):
    """More items than CTAs, of sequences that stand at different places of their keys."""
    lens_q, lens_k = [300, 257, 20], [310, 700, 400]
    q, k, v = packed(lens_q, lens_k, 48, 48, 64, "bf16", seed=21)
    out, e = run_window(tl, ctx, q, k, v, cum(lens_q), cum(lens_k), window=window, sinks=sinks)
    assert ctx.check() == tl.TL_OK
    check_window(q, k, v, cum(lens_q), cum(lens_k), out, e, window, sinks)


def test_window_attention_head_major_inputs_and_a_strided_output(tl, ctx):
    lens = [130, 77]
    n, heads, kv, d = sum(lens), 6, 2, 64
    q, k, v = (draws(31 + i, h, n, d).bfloat16().cuda().transpose(0, 1) for i, h in enumerate((heads, kv, kv)))
    room = torch.full((n, heads + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor(cum(lens), dtype=torch.int32, device="cuda")
    e = torch.empty((n, heads), device="cuda")
    for out in (room[:, 2:2 + heads], torch.full((heads, n, d), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)):
        tl.tl_window_attention(ctx, q, k, v, cu, cu, out, lse=e, window=50, sinks=1)
        assert ctx.check() == tl.TL_OK
        check_window(q, k, v, cum(lens), cum(lens), out, e, 50, 1)
    assert (room[:, :2] == 7).all() and (room[:, -1] == 7).all()


def test_paged_attention_into_a_strided_output(tl, ctx):
    q, pools, table, lengths = paged_case([3001, 0, 40], 8, 2, 128, 16, "bf16", "bf16", False, seed=6)
    room = torch.full((3, 11, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[:, 1:9]
    tl.tl_paged_attention(ctx, q, *pools, table, lengths, out, ws(tl.tl_paged_attention_workspace_bytes(3, 8, 2, 128)))
    assert ctx.check() == tl.TL_OK
    check_paged(q, pools, table, lengths, out, None)
    assert (room[:, 0] == 7).all() and (room[:, 9:] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv", [(8, 2), (12, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_paged_attention_is_off_by_its_output_rounding_alone(tl, ctx, dtype, heads, kv, d):
    """Over a 16-bit cache a weight meets V as two 16-bit terms, off by half a step of half a step: u^2 (and what fp16 cuts
    off), so that u is left for the output."""
    q, pools, table, lengths = paged_case([700, 40, 5000], heads, kv, d, 16, dtype, dtype, False, seed=heads + d, spoil=False)
    out, e = run_paged(tl, ctx, q, pools, table, lengths)
    assert ctx.check() == tl.TL_OK
    u = serving.HALF_STEP[dtype]
    args = (f64(q), f64(pools[0]), f64(pools[1]), table.cpu().numpy(), lengths.tolist(), d ** -0.5)
    want, _, tol, _ = serving.paged_attention(*args, u=0.0, fp16_weights=dtype == "fp16")
    per_unit = serving.paged_attention(*args, u=1.0, fp16_weights=dtype == "fp16")[2] - tol   # sum p |v| + |out|
    close(f64(out), want, tol + u * u * (per_unit - np.abs(want)) + u * np.abs(want), "out")


@pytest.mark.parametrize("group", [1, 4])
def test_window_attention_spoilt_values_that_a_row_walks_by(tl, ctx, group):
    """A value that shares a block with the sinks, and one before rows that see nothing: weight 0 for these rows."""
    n = 700
    q, k, v = (t.clone() for t in packed([n], [n], group, 1, 64, "bf16", seed=group))
    v[20, 0, 5], v[3, 0, 6] = math.nan, math.inf
    for window, sinks in ((100, 3), (100, 33), (300, 200)):
        out, e = run_window(tl, ctx, q, k, v, [0, n], [0, n], window=window, sinks=sinks)
        assert ctx.check() == tl.TL_OK
        check_rows(q, k, v, [0, 2, 3, 19, 20, 99, 102, 103, 119, 120, 150, 320, 500, 699], out, e, window, sinks)
    # queries of a sequence whose keys begin after them: 0, whatever V holds
    lens_q, lens_k = [200, 9], [100, 4]
    q, k, v = (t.clone() for t in packed(lens_q, lens_k, group, 1, 64, "bf16", seed=group + 7))
    v[2, 0, 1], v[101, 0, 2] = math.nan, -math.inf
    out, e = run_window(tl, ctx, q, k, v, cum(lens_q), cum(lens_k))
    assert ctx.check() == tl.TL_OK
    assert (out[:100] == 0).all() and (e[:100] == -math.inf).all() and (out[200:205] == 0).all()
    check_window(q, k, v, cum(lens_q), cum(lens_k), out, e)
