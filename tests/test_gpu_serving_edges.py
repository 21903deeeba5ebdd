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
