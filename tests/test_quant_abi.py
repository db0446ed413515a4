"""CPU checks of the 8-bit cache's entry points and of rotation with several axes: what their host-side checks
refuse, before anything touches a GPU."""
import ctypes

import pytest

import decode_ragged_paged_gb300 as pd
from decode_ragged_paged_gb300 import build as pdbuild

A = 0x10000  # an aligned address that is never read: every call below is refused first
INVALID, UNSUPPORTED = pd.PD_ERR_INVALID_ARG, pd.PD_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    pdbuild.build()
    return pd.load_library()


def _batch(**kw):
    b = dict(batch_size=2, qo_indptr=A, kv_len=A, page_indptr=A, page_indices=A, num_pages=4, total_qo=6,
             max_qo_len=5, max_kv_len=32)
    b.update(kw)
    return pd.Batch(**b)


def _append(lib, **kw):
    d = dict(num_kv_heads=2, head_dim=128, page_size=16, scale_block=16, dtype=pd.PD_BF16, layout=0, k_stride=0,
             v_stride=0)
    b = {}
    p = dict(k_new=A, v_new=A, k_pool=A, v_pool=A, k_scale=A, v_scale=A)
    for k, v in kw.items():
        (d if k in d else p if k in p else b)[k] = v
    desc, batch = pd.KvQuantDesc(**d), _batch(**b)
    return lib.pd_kv_append_quant(ctypes.byref(desc), ctypes.byref(batch), *p.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), INVALID),
    (dict(num_kv_heads=0), INVALID),
    (dict(head_dim=0), INVALID),
    (dict(page_size=0), INVALID),
    (dict(scale_block=0), INVALID),
    (dict(scale_block=-8), INVALID),
    (dict(scale_block=12), INVALID),          # does not divide a page
    (dict(scale_block=32), INVALID),          # nor does more than a page
    (dict(layout=2), INVALID),
    (dict(batch_size=-1), INVALID),
    (dict(total_qo=-1), INVALID),
    (dict(max_kv_len=-1), INVALID),
    (dict(head_dim=100), UNSUPPORTED),        # not whole vectors of 8
    (dict(head_dim=1032), UNSUPPORTED),
    (dict(num_kv_heads=16385), UNSUPPORTED),
    (dict(page_size=1 << 21, scale_block=1 << 21), UNSUPPORTED),
    (dict(num_pages=0), INVALID),
    (dict(qo_indptr=None), INVALID),
    (dict(kv_len=None), INVALID),
    (dict(page_indptr=None), INVALID),
    (dict(page_indices=None), INVALID),
    (dict(k_new=None), INVALID),
    (dict(v_pool=None), INVALID),
    (dict(k_scale=None), INVALID),
    (dict(k_new=A + 8), INVALID),             # not 16-byte aligned
    (dict(v_pool=A + 8), INVALID),
    (dict(v_scale=A + 2), INVALID),
    (dict(k_stride=260), INVALID),            # rows not 16-byte aligned
    (dict(v_stride=-256), INVALID),
])
def test_append_refuses(lib, kw, code):
    assert _append(lib, **kw) == code


def test_append_without_work(lib):
    none = dict(k_new=None, v_new=None, k_pool=None, v_pool=None, k_scale=None, v_scale=None)
    assert _append(lib, batch_size=0, **none) == pd.PD_OK
    assert _append(lib, total_qo=0, **none) == pd.PD_OK


def _chunk(lib, block=16, window=-1, stride=0, ws=A, ws_bytes=1 << 40, size=False, **kw):
    d = dict(num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, kv_dtype=pd.PD_BF16, o_dtype=pd.PD_BF16,
             layout=0, causal=1, sm_scale=0.0)
    b = {}
    p = dict(q=A, k_pool=A, v_pool=A, k_scale=A, v_scale=A, o=A)
    for k, v in kw.items():
        (d if k in d else p if k in p else b)[k] = v
    desc, batch = pd.AttnDesc(**d), _batch(**b)
    if size:
        return lib.pd_attn_chunk_quant_workspace_size(ctypes.byref(desc), ctypes.byref(batch), block)
    return lib.pd_attn_chunk_quant(ctypes.byref(desc), ctypes.byref(batch), block, window, stride, *p.values(), None, ws,
                                   ws_bytes, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_kv_heads=3), INVALID),
    (dict(head_dim=96), UNSUPPORTED),
    (dict(kv_dtype=5), INVALID),
    (dict(layout=2), INVALID),
    (dict(block=0), INVALID),
    (dict(block=-16), INVALID),
    (dict(block=12), INVALID),
    (dict(block=32), INVALID),
    (dict(qo_indptr=None), INVALID),
    (dict(num_pages=0), INVALID),
    (dict(total_qo=-1), INVALID),
    (dict(max_kv_len=(1 << 24) + 1), UNSUPPORTED),
    (dict(stride=1016), INVALID),             # below the 1024 elements of a row
    (dict(stride=1028), INVALID),             # rows not 16-byte aligned
    (dict(q=A + 8), INVALID),
    (dict(v_pool=A + 8), INVALID),
    (dict(k_scale=None), INVALID),
    (dict(v_scale=None), INVALID),
    (dict(k_scale=A + 2), INVALID),
    (dict(v_scale=A + 1), INVALID),
    (dict(o=None), INVALID),
    (dict(ws=None), INVALID),
    (dict(ws=A + 8), INVALID),
    (dict(ws_bytes=64), pd.PD_ERR_WORKSPACE),
    (dict(num_qo_heads=1 << 15, num_kv_heads=1 << 15, max_kv_len=1 << 24), UNSUPPORTED),  # more units than 32 bits count
])
def test_chunk_refuses(lib, kw, code):
    assert _chunk(lib, **kw) == code


def test_chunk_without_work_and_workspace(lib):
    none = dict(q=None, k_pool=None, v_pool=None, k_scale=None, v_scale=None, o=None, ws=None)
    assert _chunk(lib, batch_size=0, **none) == pd.PD_OK
    assert _chunk(lib, total_qo=0, **none) == pd.PD_OK
    assert _chunk(lib, max_qo_len=0, **none) == pd.PD_OK
    assert _chunk(lib, size=True, block=12) == 0 and _chunk(lib, size=True, block=0) == 0
    for kw in (dict(), dict(max_qo_len=1), dict(kv_dtype=pd.PD_F32), dict(block=4), dict(head_dim=64)):
        n = _chunk(lib, size=True, **kw)
        assert n > 0 and n % 256 == 0
        assert _chunk(lib, size=True, max_kv_len=1 << 20, **kw) == n  # does not grow with the cache
        assert _chunk(lib, ws_bytes=n - 1, **kw) == pd.PD_ERR_WORKSPACE


def _axes(lib, append=False, tokens=4, axes=3, stride=4, freq_axis="turns", **kw):
    d = dict(num_qo_heads=8, num_kv_heads=2, head_dim=128, rope_dim=128, interleaved=0, dtype=pd.PD_BF16, page_size=16,
             num_pages=4, layout=0, eps=1e-6, q_stride=0, k_stride=0, v_stride=0, q_out_stride=0, k_out_stride=0)
    p = dict(q=A, k=A, v=A, qw=A, kw=A, inv_freq=A, positions=A, slot_map=A, q_out=A, k_out=A, v_out=A)
    for k, v in kw.items():
        (d if k in d else p)[k] = v
    if freq_axis == "turns":
        freq_axis = bytes(i % max(1, min(axes, 4)) for i in range(256))
    desc = pd.NormRopeDesc(**d)
    head = (ctypes.byref(desc), tokens, axes, stride, freq_axis, p["q"], p["k"])
    tail = (p["qw"], p["kw"], p["inv_freq"], p["positions"])
    if append:
        return lib.pd_qk_norm_rope_axes_append(*head, p["v"], *tail, p["slot_map"], p["q_out"], p["k_out"], p["v_out"],
                                               None, None)
    return lib.pd_qk_norm_rope_axes(*head, *tail, p["q_out"], p["k_out"], None)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(axes=0), INVALID),
    (dict(axes=-1), INVALID),
    (dict(axes=5), UNSUPPORTED),
    (dict(stride=-4), INVALID),
    (dict(freq_axis=None), INVALID),
    (dict(freq_axis=bytes([0] * 63 + [3])), INVALID),  # an axis that is not there
    (dict(rope_dim=0), INVALID),
    (dict(rope_dim=130), INVALID),
    (dict(rope_dim=62), UNSUPPORTED),
    (dict(head_dim=1024, rope_dim=514), UNSUPPORTED),
    (dict(dtype=7), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(q=None), INVALID),
    (dict(positions=None), INVALID),
    (dict(inv_freq=None), INVALID),
    (dict(q_out_stride=1016), INVALID),
    (dict(q=A + 2), UNSUPPORTED),
])
def test_axes_refuse(lib, append, kw, code):
    assert _axes(lib, append=append, **kw) == code


def test_axes_append_refuses(lib):
    for kw in (dict(v=None), dict(slot_map=None), dict(v_out=None), dict(page_size=0), dict(num_pages=0), dict(layout=3)):
        assert _axes(lib, append=True, **kw) == INVALID
    assert _axes(lib, append=True, tokens=0, q=None, k=None, v=None) == pd.PD_OK


def test_binding_refuses_host_tensors():
    import torch
    t, x = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 64)
    pool, scale = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 1)
    with pytest.raises(pd.PdError):
        pd.pd_kv_append_quant(x, x, pool, pool, scale, scale, t, t, t, t, max_kv_len=4)
    with pytest.raises(pd.PdError):
        pd.pd_attn_chunk_quant(x, pool, pool, scale, scale, t, t, t, t, max_qo_len=4, max_kv_len=4)
    with pytest.raises(pd.PdError):
        pd.pd_qk_norm_rope_axes(x, x, None, None, torch.zeros(32), bytes(32), torch.zeros(1, 4, dtype=torch.int32))
    with pytest.raises(pd.PdError):
        pd.pd_qk_norm_rope_axes_append(x, x, x, None, None, torch.zeros(32), bytes(32),
                                       torch.zeros(1, 4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64), x, x)
