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
