"""Refusals of the serving operators (cache append, paged attention, window attention, MoE for a few
tokens): every bad argument is answered before any CUDA call, by the C entry points and by the
binding.  No GPU needed: a zeroed block stands for a context, which the checks do not look into."""
import ctypes

import numpy as np
import pytest

from oracle import serving

LL = ctypes.c_longlong


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
    f = dict(k=256, v=512, k_scale=None, v_scale=None, page_stride=16 * 2 * 64, row_stride=2 * 64, head_stride=64,
             dtype=tl.TL_BF16, num_pages=4, page_size=16, kv_heads=2, d=64)
    f.update(kw)
    return tl.PagedCache(*f.values())


BAD_CACHES = [dict(d=96), dict(d=0), dict(page_size=0), dict(num_pages=-1), dict(k=None), dict(v=264), dict(row_stride=129),
              dict(head_stride=-64), dict(dtype=1), dict(dtype=7), dict(k_scale=256), dict(num_pages=1 << 27),
              dict(dtype=2, row_stride=8)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches_are_refused(tl, ctx, bad):
    c = ctypes.byref(cache(tl, **bad))
    L = tl.lib()
    assert L.tl_kv_append(ctx, c, 0, 256, 256, 128, 64, 128, 64, 256, 3, None) == tl.TL_ERR_INVALID
    assert L.tl_paged_attention(ctx, c, 0, 256, 256, 64, 256, 2, 256, 256, 256, 64, None, 1, 4, 0.125, 0, 0, 256, 1 << 30,
                                None) == tl.TL_ERR_INVALID


def test_append_refusals(tl, ctx):
    L = tl.lib()
    good = dict(ctx=ctx, cache=ctypes.byref(cache(tl)), dtype=0, k=256, v=256, kt=128, kh=64, vt=128, vh=64, slots=256,
                tokens=0, stream=None)
    call = lambda **kw: L.tl_kv_append(*{**good, **kw}.values())
    assert call() == tl.TL_OK                                   # nothing to do
    assert call(tokens=3, cache=ctypes.byref(cache(tl, kv_heads=0))) == tl.TL_OK
    for bad in (dict(ctx=None), dict(cache=None), dict(dtype=2), dict(dtype=1), dict(tokens=-1), dict(kt=129),
                dict(vh=-64), dict(tokens=1, k=None), dict(tokens=1, v=264), dict(tokens=1, slots=None)):
        assert call(**bad) == tl.TL_ERR_INVALID, bad


def test_paged_attention_refusals(tl, ctx):
    L = tl.lib()
    ws = tl.tl_paged_attention_workspace_bytes(3, 4, 2, 64)
    assert ws > 0
    good = dict(ctx=ctx, cache=ctypes.byref(cache(tl)), dtype=0, q=256, qs=256, qh=64, table=256, max_pages=2, lengths=256,
                out=256, os=256, oh=64, lse=None, batch=0, heads=4, scale=0.125, window=0, sinks=0, ws=256, n=ws, stream=None)
    call = lambda **kw: L.tl_paged_attention(*{**good, **kw}.values())
    assert call() == tl.TL_OK and call(batch=2, heads=0) == tl.TL_OK
    for bad in (dict(ctx=None), dict(cache=None), dict(dtype=2), dict(heads=3), dict(heads=-2), dict(batch=-1),
                dict(batch=4097), dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(scale=-1.0), dict(max_pages=-1), dict(max_pages=1 << 27), dict(qs=257),
                dict(oh=-8)):
        assert call(**bad) == tl.TL_ERR_INVALID, bad
    for bad in (dict(q=None), dict(q=264), dict(out=None), dict(lengths=None), dict(table=None), dict(ws=None), dict(ws=8)):
        assert call(batch=3, **bad) == tl.TL_ERR_INVALID, bad
    assert call(batch=3, n=ws - 1) == tl.TL_ERR_WORKSPACE
    for bad in ((-1, 4, 2, 64), (4097, 4, 2, 64), (1, 3, 2, 64), (1, 4, 0, 64), (1, 4, 2, 80)):
        assert tl.tl_paged_attention_workspace_bytes(*bad) == 0


def test_window_attention_refusals(tl, ctx):
    L = tl.lib()
    good = dict(ctx=ctx, dtype=0, q=256, qt=256, qh=64, k=256, kt=128, kh=64, v=256, vt=128, vh=64, cu_q=256, cu_k=256,
                out=256, ot=256, oh=64, lse=None, batch=0, total_q=5, total_k=5, heads=4, kv_heads=2, d=64, scale=0.125,
                window=0, sinks=0, stream=None)
    call = lambda **kw: L.tl_window_attention(*{**good, **kw}.values())
    assert call() == tl.TL_OK and call(batch=1, total_q=0) == tl.TL_OK and call(batch=1, heads=0) == tl.TL_OK
    for bad in (dict(ctx=None), dict(dtype=2), dict(dtype=-1), dict(heads=3), dict(kv_heads=0), dict(d=80), dict(batch=-1),
                dict(batch=1025), dict(total_q=-1), dict(total_k=-1), dict(window=-1), dict(sinks=-1), dict(scale=0.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(heads=258, kv_heads=2), dict(qt=257), dict(kt=4),
                dict(oh=-64), dict(total_q=1 << 30)):
        assert call(**bad) == tl.TL_ERR_INVALID, bad
    for bad in (dict(q=None), dict(q=264), dict(k=None), dict(v=8), dict(out=None), dict(cu_q=None), dict(cu_k=None)):
        assert call(batch=1, **bad) == tl.TL_ERR_INVALID, bad


def test_moe_tokens_refusals(tl, ctx):
    L = tl.lib()
    ws = tl.tl_moe_tokens_workspace_bytes(3, 64, 4, 40, 2)
    assert ws > 0
    good = dict(ctx=ctx, x=256, logits=256, topk=2, wg=256, wu=256, wd=256, out=256, eo=None, go=None, ws=256, n=ws, T=3,
                H=64, E=4, F=40, stream=None)
    call = lambda **kw: L.tl_moe_tokens(*{**good, **kw}.values())
    for bad in (dict(ctx=None), dict(T=0), dict(T=129), dict(topk=0), dict(topk=5), dict(topk=9, E=16), dict(E=257),
                dict(H=60), dict(H=0), dict(F=44), dict(F=-8), dict(x=None), dict(logits=None), dict(wg=8), dict(wu=None),
                dict(wd=264), dict(out=None), dict(ws=None)):
        assert call(**bad) == tl.TL_ERR_INVALID, bad
    assert call(n=ws - 1) == tl.TL_ERR_WORKSPACE
    for bad in ((0, 64, 4, 40, 2), (129, 64, 4, 40, 2), (3, 60, 4, 40, 2), (3, 64, 4, 41, 2), (3, 64, 4, 40, 5)):
        assert tl.tl_moe_tokens_workspace_bytes(*bad) == 0


def test_binding_refuses_host_tensors_and_bad_types(tl):
    import torch
    kv = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    rows = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    ints = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        tl.tl_kv_append(None, rows, rows, kv, kv, ints)
    with pytest.raises(ValueError, match="CUDA"):
        tl.tl_paged_attention(None, rows, kv, kv, ints[:, None], ints, rows, ints)
    with pytest.raises(ValueError, match="CUDA"):
        tl.tl_window_attention(None, rows, rows, rows, ints, ints, rows)
    with pytest.raises(ValueError, match="CUDA"):
        tl.tl_moe_tokens(None, rows[0], rows[0], 1, rows, rows, rows, rows, ints)


def test_error_code_and_exports(tl):
    assert tl.TL_ERR_INDEX == -6 and b"out of range" in tl.lib().tl_strerror(tl.TL_ERR_INDEX)
    for name in ("tl_kv_append", "tl_paged_attention", "tl_window_attention", "tl_moe_tokens"):
        assert name in tl.EXPORTED_SYMBOLS and name in tl.__all__


def test_reference_by_hand():
    """The 64-bit forms on cases small enough to do by hand."""
    assert serving.visible(5, 6, 0, 0).tolist() == [0, 1, 2, 3, 4, 5]
    assert serving.visible(5, 6, 2, 1).tolist() == [0, 4, 5]
    assert serving.visible(5, 9, 2, 9).tolist() == [0, 1, 2, 3, 4, 5]
    assert serving.visible(-1, 4, 0, 2).tolist() == []
    q, k, v = np.array([1.0, 0.0]), np.array([[0.0, 7.0], [np.log(3.0), 1.0]]), np.array([[4.0, 0.0], [0.0, 8.0]])
    out, lse, _, _ = serving.attend(q, k, v, 1.0, 0.0)
    assert np.allclose(out, [1.0, 6.0]) and np.isclose(lse, np.log(4.0))
    out, lse, _, _ = serving.attend(q, k[:0], v[:0], 1.0, 0.0)
    assert out.tolist() == [0.0, 0.0] and lse == -np.inf
    x, lg = np.array([[1.0, 2.0]]), np.array([[0.0, 0.0, -50.0]])
    one = np.ones((3, 2, 2))
    out, ex, g, _ = serving.moe_tokens(x, lg, one, one, one, 2)
    assert ex.tolist() == [[0, 1]] and np.allclose(g, 0.5)
    assert np.allclose(out, 2 * 9 / (1 + np.exp(-3.0)))
