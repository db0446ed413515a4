"""CPU checks of the chunk-step entry points (tables, norm and rotation, chunk
attention): what their host-side checks refuse, before anything touches a GPU."""
import ctypes
import sys

import pytest

import decode_ragged_paged_gb300 as pd
from decode_ragged_paged_gb300 import build as pdbuild

A = 0x10000  # an aligned address that is never read: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    pdbuild.build()
    return pd.load_library()


def _attn(**kw):
    d = dict(num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, kv_dtype=pd.PD_BF16, o_dtype=pd.PD_BF16,
             layout=0, causal=1, sm_scale=0.0)
    d.update(kw)
    return pd.AttnDesc(**d)


def _batch(**kw):
    b = dict(batch_size=2, qo_indptr=A, kv_len=A, page_indptr=A, page_indices=A, num_pages=4, total_qo=6,
             max_qo_len=5, max_kv_len=32)
    b.update(kw)
    return pd.Batch(**b)


def _chunk(lib, d=None, b=None, window=-1, stride=0, q=A, o=A, ws=A, ws_bytes=1 << 40):
    return lib.pd_attn_chunk(ctypes.byref(d or _attn()), ctypes.byref(b or _batch()), window, stride, q, A, A, o, None,
                             ws, ws_bytes, None, None)


@pytest.mark.parametrize("d,b,kw,code", [
    (dict(num_kv_heads=3), {}, {}, pd.PD_ERR_INVALID_ARG),
    (dict(head_dim=96), {}, {}, pd.PD_ERR_UNSUPPORTED),
    (dict(kv_dtype=5), {}, {}, pd.PD_ERR_INVALID_ARG),
    (dict(layout=2), {}, {}, pd.PD_ERR_INVALID_ARG),
    ({}, dict(qo_indptr=None), {}, pd.PD_ERR_INVALID_ARG),
    ({}, dict(num_pages=0), {}, pd.PD_ERR_INVALID_ARG),
    ({}, dict(total_qo=-1), {}, pd.PD_ERR_INVALID_ARG),
    ({}, dict(max_kv_len=(1 << 26) + 1), {}, pd.PD_ERR_UNSUPPORTED),
    ({}, dict(max_kv_len=(1 << 24) + 1), {}, pd.PD_ERR_UNSUPPORTED),
    ({}, {}, dict(stride=1016), pd.PD_ERR_INVALID_ARG),       # below the 1024 elements of a row
    ({}, {}, dict(stride=1028), pd.PD_ERR_INVALID_ARG),       # rows not 16-byte aligned
    ({}, {}, dict(q=A + 8), pd.PD_ERR_INVALID_ARG),
    ({}, {}, dict(o=None), pd.PD_ERR_INVALID_ARG),
    ({}, {}, dict(ws=None), pd.PD_ERR_INVALID_ARG),
    ({}, {}, dict(ws_bytes=64), pd.PD_ERR_WORKSPACE),
])
def test_chunk_refuses(lib, d, b, kw, code):
    assert _chunk(lib, _attn(**d), _batch(**b), **kw) == code


def test_chunk_empty_and_workspace(lib):
    assert _chunk(lib, b=_batch(batch_size=0), q=None, o=None, ws=None) == pd.PD_OK
    assert _chunk(lib, b=_batch(total_qo=0), q=None, o=None, ws=None) == pd.PD_OK
    size = lambda d, b: lib.pd_attn_chunk_workspace_size(ctypes.byref(d), ctypes.byref(b))  # noqa: E731
    n = size(_attn(), _batch())
    assert n > 0 and n % 256 == 0
    assert size(_attn(num_kv_heads=3), _batch()) == 0
    # partials and plan do not grow with the cache
    assert size(_attn(), _batch(max_kv_len=1 << 20)) == n


def test_chunk_refuses_more_work_than_it_counts(lib):
    # the line holds up to about two items a CTA and a block's heads, of all their key tiles, in 32 bits
    many = dict(num_qo_heads=1 << 15, num_kv_heads=1 << 15)
    assert _chunk(lib, _attn(**many), _batch(max_kv_len=1 << 24), ws_bytes=64) == pd.PD_ERR_UNSUPPORTED
    assert _chunk(lib, _attn(**many), _batch(max_kv_len=1 << 20), ws_bytes=64) == pd.PD_ERR_WORKSPACE
    # more items than 32 bits number
    assert _chunk(lib, b=_batch(batch_size=2 ** 31 - 1, total_qo=2 ** 31 - 1, max_qo_len=2 ** 20),
                  ws_bytes=64) == pd.PD_ERR_UNSUPPORTED
    big = _batch(batch_size=2 ** 31 - 1, total_qo=2 ** 31 - 1, max_qo_len=2 ** 20)
    assert lib.pd_attn_chunk_workspace_size(ctypes.byref(_attn()), ctypes.byref(big)) == 0
    # a decode of 2^16 requests of any length is within both
    assert _chunk(lib, b=_batch(batch_size=1 << 16, total_qo=1 << 16, max_qo_len=1, max_kv_len=1 << 24),
                  ws_bytes=64) == pd.PD_ERR_WORKSPACE


def _tables(lib, rows=None, **kw):
    d = dict(batch_size=4, page_size=16, num_pages=64, table_rows=8, table_cols=8, total_qo=16, max_page_indices=32,
             free_capacity=10)
    ptrs = {k: A + 0x1000 * i for i, k in enumerate(
        ("cached_len", "new_len", "block_table", "free_pages", "free_count", "free_count_out", "qo_indptr", "kv_len",
         "page_indptr", "page_indices", "positions", "slot_map"))}
    for k, v in kw.items():
        (d if k in d else ptrs)[k] = v
    desc = pd.TablesDesc(**d)
    return lib.pd_batch_tables(ctypes.byref(desc), rows, *ptrs.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch_size=-1), pd.PD_ERR_INVALID_ARG),
    (dict(page_size=0), pd.PD_ERR_INVALID_ARG),
    (dict(num_pages=0), pd.PD_ERR_INVALID_ARG),
    (dict(table_cols=0), pd.PD_ERR_INVALID_ARG),
    (dict(batch_size=9), pd.PD_ERR_INVALID_ARG),              # more requests than rows, without a row list
    (dict(batch_size=8193, table_rows=9000), pd.PD_ERR_UNSUPPORTED),
    (dict(new_len=None), pd.PD_ERR_INVALID_ARG),
    (dict(qo_indptr=None), pd.PD_ERR_INVALID_ARG),
    (dict(page_indices=None), pd.PD_ERR_INVALID_ARG),
    (dict(slot_map=None), pd.PD_ERR_INVALID_ARG),
    (dict(slot_map=A + 0xb004), pd.PD_ERR_INVALID_ARG),       # 64-bit entries
    (dict(positions=A + 0xa002), pd.PD_ERR_INVALID_ARG),
    (dict(free_count=None), pd.PD_ERR_INVALID_ARG),
    (dict(free_count_out=None), pd.PD_ERR_INVALID_ARG),
    (dict(kv_len=A), pd.PD_ERR_INVALID_ARG),                  # kv_len on cached_len
    (dict(kv_len=A + 12), pd.PD_ERR_INVALID_ARG),             # and on its last entry
    (dict(page_indices=A + 0x3000), pd.PD_ERR_INVALID_ARG),   # the page list on the free list
    (dict(positions=A + 0x7000 - 60), pd.PD_ERR_INVALID_ARG),  # one result on another's first entry
])
def test_tables_refuse(lib, kw, code):
    assert _tables(lib, **kw) == code


def test_slot_map_refuses(lib):
    call = lambda b, page=16, pos=A, slot=A: lib.pd_slot_map(ctypes.byref(b), page, pos, slot, None, None)  # noqa: E731
    assert call(_batch(), page=0) == pd.PD_ERR_INVALID_ARG
    assert call(_batch(kv_len=None)) == pd.PD_ERR_INVALID_ARG
    assert call(_batch(), pos=None) == pd.PD_ERR_INVALID_ARG
    assert call(_batch(), slot=A + 4) == pd.PD_ERR_INVALID_ARG
    assert call(_batch(total_qo=0), pos=None, slot=None) == pd.PD_OK


def _rope(lib, tokens=4, append=False, **kw):
    d = dict(num_qo_heads=8, num_kv_heads=2, head_dim=128, rope_dim=128, interleaved=0, dtype=pd.PD_BF16, page_size=16,
             num_pages=4, layout=0, eps=1e-6, q_stride=0, k_stride=0, v_stride=0, q_out_stride=0, k_out_stride=0)
    p = dict(q=A, k=A, v=A, qw=A, kw=A, inv_freq=A, positions=A, slot_map=A, q_out=A, k_out=A, v_out=A)
    for k, v in kw.items():
        (d if k in d else p)[k] = v
    desc = pd.NormRopeDesc(**d)
    if append:
        return lib.pd_qk_norm_rope_append(ctypes.byref(desc), tokens, p["q"], p["k"], p["v"], p["qw"], p["kw"],
                                          p["inv_freq"], p["positions"], p["slot_map"], p["q_out"], p["k_out"],
                                          p["v_out"], None, None)
    return lib.pd_qk_norm_rope(ctypes.byref(desc), tokens, p["q"], p["k"], p["qw"], p["kw"], p["inv_freq"],
                               p["positions"], p["q_out"], p["k_out"], None)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), pd.PD_ERR_INVALID_ARG),
    (dict(head_dim=0), pd.PD_ERR_INVALID_ARG),
    (dict(rope_dim=130), pd.PD_ERR_INVALID_ARG),
    (dict(rope_dim=63), pd.PD_ERR_INVALID_ARG),
    (dict(rope_dim=62), pd.PD_ERR_UNSUPPORTED),               # no run of two pairs
    (dict(head_dim=250, rope_dim=0), pd.PD_ERR_UNSUPPORTED),
    (dict(head_dim=1024), pd.PD_ERR_UNSUPPORTED),             # more than 32 lanes
    (dict(eps=float("nan")), pd.PD_ERR_INVALID_ARG),
    (dict(eps=-1.0), pd.PD_ERR_INVALID_ARG),
    (dict(tokens=-1), pd.PD_ERR_INVALID_ARG),
    (dict(q=None), pd.PD_ERR_INVALID_ARG),
    (dict(k_out=None), pd.PD_ERR_INVALID_ARG),
    (dict(positions=None), pd.PD_ERR_INVALID_ARG),
    (dict(inv_freq=None), pd.PD_ERR_INVALID_ARG),
    (dict(q_out_stride=1016), pd.PD_ERR_INVALID_ARG),         # two tokens would share results
    (dict(q_stride=-1024), pd.PD_ERR_INVALID_ARG),
    (dict(q_stride=1025), pd.PD_ERR_UNSUPPORTED),             # odd rows
    (dict(q=A + 2), pd.PD_ERR_UNSUPPORTED),
])
def test_norm_rope_refuses(lib, append, kw, code):
    assert _rope(lib, append=append, **kw) == code


def test_norm_rope_append_refuses(lib):
    for kw in (dict(v=None), dict(slot_map=None), dict(v_out=None), dict(page_size=0), dict(num_pages=0),
               dict(layout=3), dict(num_kv_heads=0)):
        assert _rope(lib, append=True, **kw) == pd.PD_ERR_INVALID_ARG
    assert _rope(lib, append=True, tokens=0, q=None, k=None, v=None) == pd.PD_OK


def test_binding_refuses_host_tensors():
    import torch
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(pd.PdError):
        pd.pd_slot_map(t, t, t, t, page_size=16, num_pages=1, total_qo=4)
    with pytest.raises(pd.PdError):
        pd.pd_batch_tables(t, t, t.view(2, 2), page_size=16, num_pages=1, total_qo=4, max_page_indices=4)
    x = torch.zeros(2, 4, 64)
    with pytest.raises(pd.PdError):
        pd.pd_qk_norm_rope(x, x, None, None, None, None)


@pytest.fixture
def unloaded(lib, monkeypatch):
    """The package as it is before its first call."""
    monkeypatch.setattr(pd, "_lib", None)
    monkeypatch.setattr(pd, "_bind", None)
    return monkeypatch


def test_calls_that_do_not_use_the_binding_module_do_without_it(unloaded):
    import torch
    unloaded.setitem(sys.modules, "decode_ragged_paged_gb300._pd_bind", None)  # as if it had not been built
    unloaded.delattr(pd, "_pd_bind", raising=False)
    assert pd.load_library().pd_version() >= 100
    x = torch.zeros(2, 4, 64)
    with pytest.raises(pd.PdError, match="_pd_bind"):
        pd.pd_qk_norm_rope(x, x, None, None, None, None)


def test_the_binding_module_belongs_to_one_torch_and_one_python(unloaded):
    import sysconfig
    import torch
    assert pdbuild.BIND.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and not pdbuild._bind_stale()
    assert pd._load_bind().__file__ == pdbuild.BIND
    unloaded.setattr(torch, "__version__", "0.1")
    assert pdbuild._bind_stale()               # rebuilt by the next build()
    unloaded.setattr(pd, "_bind", None)
    with pytest.raises(pd.PdError, match="built for torch"):  # and not used before
        pd._load_bind()
