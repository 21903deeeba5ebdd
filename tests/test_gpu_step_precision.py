"""How exact the step's operators are where only the output's own rounding should be left, and at the ends of the types' ranges."""
import numpy as np
import pytest
import torch

from oracle import serving, step
from tests.test_gpu_serving import close, ctx, draws, f64, tl, ws  # noqa: F401
from tests.test_gpu_step import case4, freqs, run4

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


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-29, 1e-6])
@pytest.mark.parametrize("d,interleaved", [(64, True), (128, False)])
def test_norm_rope_small_rows(tl, ctx, d, interleaved, eps):
    """Rows of bf16 down to its smallest values, whose squares fp32 does not hold: the norm of a row does not depend on its size
    where eps leaves it alone.  Rows of every size side by side, and the tolerance of rows of ordinary size."""
    sizes = 10.0 ** np.arange(0, -41, -2, dtype=np.float64)
    x = (draws(2, 3, 2 * len(sizes), d).numpy() * np.repeat(sizes, 2)[None, :, None])
    x[:, -1] = 0.0                                          # one value at bf16's smallest among zeros
    x[:, -1, 5] = 2.0 ** -133
    x = torch.from_numpy(x).bfloat16().cuda()
    q, k = x[:, ::2].contiguous(), x[:, 1::2].contiguous()
    assert all(((r != 0).any(-1)).all() for r in (q, k))
    w = (draws(6, d) * 0.3 + 1).bfloat16().cuda()
    pos, f = torch.arange(3, dtype=torch.int32, device="cuda") * 1000, freqs(d)
    outs = [torch.empty_like(q), torch.empty_like(k)]
    tl.tl_norm_rope(ctx, q, k, pos, f.cuda(), *outs, q_weight=w, k_weight=w, eps=eps, interleaved=interleaved)
    for rows, got in ((q, outs[0]), (k, outs[1])):
        want, tol = step.norm_rope(f64(rows), f64(w), pos.cpu().numpy(), f.double().numpy(), float(np.float32(eps)), interleaved, serving.HALF_STEP["bf16"])
        close(f64(got), want, tol, "rows")
