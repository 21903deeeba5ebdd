"""Limits of the serving operators' arguments that only show at the ends of a type's range.  No GPU needed: a zeroed block
stands for a context, and calls of no rows end after the checks."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def tl():
    import communication_overlapped_gemm_gb300 as tl
    tl.build()
    tl.lib()
    return tl


# the largest fp32 number whose fp32 product with fp32's log2(e) is finite, and the next one
LOG2E = np.float32(1.4426950408889634)
LAST = np.float32(np.finfo(np.float32).max) / LOG2E
with np.errstate(over="ignore"):
    while np.isfinite(np.nextafter(LAST, np.float32(np.inf)) * LOG2E):
        LAST = np.nextafter(LAST, np.float32(np.inf))
    while not np.isfinite(LAST * LOG2E):
        LAST = np.nextafter(LAST, np.float32(0))
PAST = np.nextafter(LAST, np.float32(np.inf))


@pytest.mark.parametrize("scale,ok", [(1e-45, True), (1e38, True), (float(LAST), True), (float(PAST), False), (2.4e38, False), (3e38, False),
                                      (3.4028234e38, False)])
def test_scales_whose_product_with_log2_e_is_not_finite_are_refused(tl, scale, ok):
    """The kernels work in powers of two: 0 times an infinite factor would make every result NaN."""
    L, ctx, want = tl.lib(), ctypes.create_string_buffer(4096), tl.TL_OK if ok else tl.TL_ERR_INVALID
    assert 2.358e38 < LAST < 2.359e38
    cache = ctypes.byref(tl.PagedCache(256, 256, None, None, 16 * 2 * 64, 2 * 64, 64, 0, 4, 16, 2, 64, None, None, 0, 0, 0))
    assert L.tl_token_logprobs(ctx, 3, 256, 1000, 256, 256, None, None, None, None, 0, scale, 0, 1000, 256, 1 << 20, None) == want
    assert L.tl_paged_attention(ctx, cache, 0, 256, 256, 64, 256, 2, 256, 256, 256, 64, None, 0, 4, scale, 0, 0, 256, 1 << 30, None) == want
    assert L.tl_window_attention(ctx, 0, 256, 256, 64, 256, 128, 64, 256, 128, 64, 256, 256, 256, 256, 64, None, 0, 0, 0, 4, 2, 64, scale, 0, 0,
                                 None) == want
