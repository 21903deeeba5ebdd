"""How exact the step's operators are where only the output's own rounding should be left, and at the ends of the types' ranges."""
import numpy as np
import pytest
import torch

from oracle import serving, step
from tests.test_gpu_serving import close, ctx, draws, f64, tl, ws  # noqa: F401
from tests.test_gpu_step import case4, run4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv,d,dtype", [(8, 1, 128, "fp16"), (8, 2, 64, "fp16"), (16, 1, 128, "fp16"), (12, 1, 64, "fp16"), (32, 8, 128, "bf16")])
def test_paged_attention_4_bits_weights_lose_nothing(tl, ctx, heads, kv, d, dtype):
    """A weight that meets V is a sum of two fp16 terms, so it is off by half a step squared (2^-22), beside what sums and
    exponentials in fp32 are; the output is then rounded once.  Few rows a sequence, whose weights' roundings do not average
    out, and a small scale, so that the scores' own errors are small."""
    lens = list(range(10)) * 6 + [70, 300]
    q, c, table, lengths = case4(lens, heads, kv, d, 16, dtype, False, seed=21)
    scale = 2.0 ** -7
    out, e = run4(tl, ctx, q, c, table, lengths, scale=scale)
    assert ctx.check() == tl.TL_OK
    fine = 2.0 ** -22
    want, lse, tol, ltol = serving.paged_attention(f64(q), *c["values"], table.cpu().numpy(), lens, scale, 0, 0, c["scale"][0].double().numpy(),
                                                   c["scale"][1].double().numpy(), fine, True)
    close(f64(out), want, tol + serving.HALF_STEP[dtype] * (np.abs(want) + tol), "out")
    close(f64(e), lse, ltol, "lse")
