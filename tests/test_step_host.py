"""Refusals of the plan, the norms and rotation, the 4-bit cache and the log probabilities: every bad argument is answered
before any CUDA call, by the C entry points and by the binding; and the 64-bit forms on cases done by hand.  No GPU
needed: a zeroed block stands for a context, which the checks do not look into."""
import ctypes
import types

import numpy as np
import pytest

from oracle import step


@pytest.fixture(scope="module")
def tl():
    import communication_overlapped_gemm_gb300 as tl
    tl.build()
    tl.lib()
    return tl


@pytest.fixture(scope="module")
def ctx():
    return ctypes.create_string_buffer(4096)


def cache(tl, **kw):
    """A 4-bit cache of 4 pages of 16 rows, 2 heads of 64."""
    f = dict(k=256, v=512, k_scale=256, v_scale=256, page_stride=16 * 2 * 32, row_stride=2 * 32, head_stride=32,
             dtype=tl.TL_E2M1, num_pages=4, page_size=16, kv_heads=2, d=64, k_blocks=256, v_blocks=256, bp=16 * 2 * 4, br=8, bh=4)
    f.update(kw)
    return tl.PagedCache(*f.values())


def test_codes(tl):
    assert (tl.TL_FP32, tl.TL_E2M1) == (3, 4)
    for name in ("tl_kv_gather", "tl_cache_plan", "tl_norm_rope", "tl_token_logprobs", "tl_token_logprobs_workspace_bytes"):
        assert name in tl.EXPORTED_SYMBOLS and name in tl.__all__


BAD = [dict(k_blocks=None), dict(v_blocks=264), dict(br=6), dict(bh=-4), dict(bp=2), dict(row_stride=40), dict(head_stride=8),
       dict(d=96), dict(page_size=0), dict(dtype=3), dict(dtype=5), dict(d=128, bh=4), dict(k=264)]


@pytest.mark.parametrize("bad", BAD)
def test_bad_4_bit_caches_are_refused(tl, ctx, bad):
    L, c = tl.lib(), ctypes.byref(cache(tl, **bad))
    assert L.tl_kv_append(ctx, c, 0, 256, 256, 128, 64, 128, 64, 256, 3, None) == tl.TL_ERR_INVALID
    assert L.tl_kv_gather(ctx, c, 0, 256, 3, 256, 256, 128, 64, 128, 64, None) == tl.TL_ERR_INVALID
    assert L.tl_paged_attention(ctx, c, 0, 256, 256, 64, 256, 2, 256, 256, 256, 64, None, 1, 4, 0.125, 0, 0, 256, 1 << 30,
                                None) == tl.TL_ERR_INVALID


def test_a_cache_without_blocks_is_not_looked_for_any(tl, ctx):
    """A tl_paged_cache as it was before block scales: what lies behind it has no say."""
    c = ctypes.byref(cache(tl, dtype=tl.TL_E4M3, page_stride=16 * 2 * 64, row_stride=2 * 64, head_stride=64, k_blocks=1, bp=-7, br=3))
    assert tl.lib().tl_kv_append(ctx, c, 0, 256, 256, 128, 64, 128, 64, 256, 0, None) == tl.TL_OK


def test_gather_refusals(tl, ctx):
    L = tl.lib()
    good = dict(ctx=ctx, cache=ctypes.byref(cache(tl)), dtype=0, slots=256, tokens=0, k=256, v=256, kt=128, kh=64, vt=128, vh=64, stream=None)
    call = lambda **kw: L.tl_kv_gather(*{**good, **kw}.values())
    assert call() == tl.TL_OK and call(tokens=3, cache=ctypes.byref(cache(tl, kv_heads=0))) == tl.TL_OK
    for bad in (dict(ctx=None), dict(cache=None), dict(dtype=2), dict(dtype=4), dict(tokens=-1), dict(kt=129), dict(vh=-64),
                dict(tokens=1, k=None), dict(tokens=1, v=264), dict(tokens=1, slots=None), dict(tokens=1 << 30)):
        assert call(**bad) == tl.TL_ERR_INVALID, bad


def test_plan_refusals(tl, ctx):
    L = tl.lib()
    good = dict(ctx=ctx, lengths=256, counts=None, batch=2, page_size=16, table=256, max_pages=4, free=256, num_free=8, taken=256,
                taken_out=256, new_lengths=256, cu_q=256, cu_k=None, slots=256, positions=None, tokens=5, kv=None, kv_tokens=0, stream=None)
    call = lambda **kw: L.tl_cache_plan(*{**good, **kw}.values())
    for bad in (dict(ctx=None), dict(lengths=None), dict(batch=-1), dict(batch=4097), dict(page_size=0), dict(table=None),
                dict(max_pages=-1), dict(max_pages=1 << 27), dict(free=None), dict(num_free=-1), dict(taken=None), dict(taken_out=None),
                dict(new_lengths=None), dict(cu_q=None), dict(slots=None), dict(tokens=-1), dict(kv_tokens=-1), dict(kv_tokens=3)):
        assert call(**bad) == tl.TL_ERR_INVALID, bad


def test_norm_rope_refusals(tl, ctx):
    L = tl.lib()
    good = dict(ctx=ctx, dtype=0, q=256, qt=256, qh=64, k=256, kt=128, kh=64, qw=256, kw=256, wdtype=0, eps=1e-6, pos=256, freq=256,
                rotary=64, inter=0, qo=256, qot=256, qoh=64, ko=256, kot=128, koh=64, tokens=0, heads=4, kv_heads=2, d=64, stream=None)
    call = lambda **kw: L.tl_norm_rope(*{**good, **kw}.values())
    assert call() == tl.TL_OK and call(tokens=3, heads=0, kv_heads=0) == tl.TL_OK
    for bad in (dict(ctx=None), dict(dtype=2), dict(dtype=3), dict(wdtype=1), dict(wdtype=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(rotary=8), dict(rotary=80), dict(rotary=-16), dict(inter=2), dict(qt=257), dict(koh=4),
                dict(kot=-64), dict(tokens=-1), dict(heads=-1), dict(d=96), dict(tokens=1, heads=65536), dict(tokens=1 << 30)):
        assert call(**bad) == tl.TL_ERR_INVALID, bad
    for bad in (dict(q=None), dict(q=264), dict(k=None), dict(qo=None), dict(ko=8), dict(pos=None), dict(freq=None)):
        assert call(tokens=1, **bad) == tl.TL_ERR_INVALID, bad


def test_token_logprobs_refusals(tl, ctx):
    L = tl.lib()
    ws = tl.tl_token_logprobs_workspace_bytes(3, 1000, 5)
    assert ws > 0
    good = dict(ctx=ctx, dtype=3, x=256, stride=1000, targets=256, lp=256, ent=None, lse=None, tlp=256, tid=256, top=5, scale=1.0,
                rows=0, vocab=1000, ws=256, n=ws, stream=None)
    call = lambda **kw: L.tl_token_logprobs(*{**good, **kw}.values())
    assert call() == tl.TL_OK
    for bad in (dict(ctx=None), dict(dtype=2), dict(dtype=4), dict(dtype=-1), dict(stride=-1), dict(top=-1), dict(top=33),
                dict(top=6, vocab=5), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 30) + 1)):
        assert call(**bad) == tl.TL_ERR_INVALID, bad
    for bad in (dict(x=None), dict(x=258), dict(targets=None), dict(tlp=None), dict(tid=None), dict(ws=None), dict(ws=264),
                dict(rows=(1 << 24) + 1)):
        assert call(**{"rows": 3, **bad}) == tl.TL_ERR_INVALID, bad
    assert call(rows=3, n=ws - 1) == tl.TL_ERR_WORKSPACE
    for bad in ((-1, 10, 1), (1, 0, 0), (1, 10, 11), (1, 100, 33), (1, 10, -1)):
        assert tl.tl_token_logprobs_workspace_bytes(*bad) == 0


def test_binding_refuses_host_tensors_and_bad_shapes(tl):
    import torch
    none = types.SimpleNamespace(handle=None, device=0)
    rows, ints = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    codes, blocks = torch.zeros((2, 16, 2, 32), dtype=torch.uint8), torch.zeros((2, 16, 2, 4), dtype=torch.float8_e4m3fn)
    f = torch.zeros(3)
    with pytest.raises(ValueError, match="4-bit cache"):
        tl.tl_kv_append(none, rows, rows, codes, codes, ints, k_blocks=blocks, v_blocks=blocks)
    with pytest.raises(ValueError, match="4-bit cache"):
        tl.tl_kv_gather(none, codes, codes, ints, rows, rows, k_blocks=blocks)
    with pytest.raises(ValueError, match="CUDA"):
        tl.tl_kv_gather(none, codes, codes, ints, rows, rows)
    with pytest.raises(ValueError, match="CUDA"):
        tl.tl_cache_plan(none, ints, ints[:, None], 16, ints, ints[:1], ints[:1], ints, torch.zeros(4, dtype=torch.int32), ints)
    with pytest.raises(ValueError, match="max_pages"):
        tl.tl_cache_plan(none, ints, ints, 16, ints, ints[:1], ints[:1], ints, ints, ints)
    with pytest.raises(ValueError, match="CUDA"):
        tl.tl_norm_rope(none, rows, rows, ints, f, rows, rows)
    with pytest.raises(ValueError, match="CUDA"):
        tl.tl_token_logprobs(none, f[:, None], ints, f, ints)


def test_formats_by_hand():
    assert step.e4m3(np.float32([0, 2 ** -10, 1.5 * 2 ** -9, 2 ** -9, 1.0, 1.0625, 1.1875, 15.5, 447.0, 464.0, 1e9, np.nan])).tolist() == \
        [0, 0, 2, 1, 0x38, 0x38, 0x3A, 0x58, 0x7E, 0x7E, 0x7E, 0x7F]
    assert step.e4m3_value([0, 1, 0x38, 0x58, 0x7E, 0xB8]).tolist() == [0, 2 ** -9, 1, 16, 448, -1]
    import torch
    every = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    assert np.array_equal(step.e4m3_value(every.numpy()), every.view(torch.float8_e4m3fn).float().numpy(), equal_nan=True)
    x = np.float32(np.linspace(0, 500, 4001))
    assert np.array_equal(step.e4m3(x), torch.from_numpy(x).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    row = np.zeros((1, 16), np.float32)
    row[0, :10] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, -3.5, 5, -0.24]      # ties to the even code
    codes, b = step.to_4_bits(row, [1.0])
    assert b.tolist() == [[0x38]]
    assert step.from_4_bits(codes, b)[0, :10].tolist() == [6, -6, 0, 1, 1, 2, 2, -4, 4, 0]
    codes, b = step.to_4_bits(row * 0.001, [2.0 ** -12])                     # 0.001 / 2^-12 = 4.096: block scale 4
    assert step.e4m3_value(b).tolist() == [[4.0]] and step.from_4_bits(codes, b, [2.0 ** -12])[0, 0] == 6 * 4 * 2.0 ** -12


def test_plan_by_hand():
    got, ok = step.cache_plan([3, 0, 4], [2, 0, 1], [[7, -1], [-1, -1], [5, -1]], 4, [9, 8, 6], 1, 4, 10)
    assert ok and got["table"].tolist() == [[7, 8], [-1, -1], [5, 6]]
    assert got["slots"].tolist() == [31, 32, 24, -1] and got["positions"].tolist() == [3, 4, 4, 0]
    assert got["cu_q"].tolist() == [0, 2, 2, 3] and got["cu_k"].tolist() == [0, 5, 5, 10] and got["taken"].tolist() == [3]
    assert got["lengths"].tolist() == [5, 0, 5]
    assert got["kv_slots"].tolist() == [28, 29, 30, 31, 32, 20, 21, 22, 23, 24]
    got, ok = step.cache_plan([4, 4], [1, 1], [[0, -1], [1, -1]], 4, [5], 0, 9)   # one page for two
    assert not ok and got["slots"].tolist() == [20, -1] + [-1] * 7 and got["lengths"].tolist() == [5, 4]


def test_norm_rope_and_logprobs_by_hand():
    x = np.zeros((1, 1, 64))
    x[0, 0, :2] = [3, 4]
    y, tol = step.norm_rope(x, np.full(64, 2.0), [2], [np.pi / 4] + [0.0] * 31, 0.0, True, 2.0 ** -8)
    assert np.allclose(y[0, 0, :3], np.array([-4, 3, 0]) * 2 * 8 / 5) and tol[0, 0, 0] < 0.1
    y, _ = step.norm_rope(x, None, [1], [np.pi / 2] + [0.0] * 31, 0.0, False, 0.0)
    assert np.allclose([y[0, 0, 0], y[0, 0, 32], y[0, 0, 1]], [0, 3, 4])
    g, _, ids, best, _ = \
        step.token_logprobs(np.array([[0.0, np.log(3.0), -np.inf, np.log(4.0)]]), [1], 3, 1.0)
    p = np.array([1, 3, 4]) / 8
    assert np.isclose(g["logprob"][0], np.log(3 / 8)) and np.isclose(g["entropy"][0], -(p * np.log(p)).sum()) and np.isclose(g["lse"][0], np.log(8))
    assert ids.tolist() == [[3, 1, 0]] and np.allclose(np.exp(best), [[0.5, 0.375, 0.125]])
    g, _, ids, best, _ = step.token_logprobs(np.full((1, 3), -np.inf), [1], 2, 1.0)
    assert g["entropy"][0] == 0 and g["lse"][0] == -np.inf and ids.tolist() == [[0, 1]] and np.all(best == -np.inf)
