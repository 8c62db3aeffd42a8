"""Refusals of the tree calls, on the host: every call below is turned down by its
argument checks, before any CUDA call.  No GPU."""
import ctypes

import pytest
import torch

import fp8_quantized_kv_gb300 as fk
from test_step_host import INVALID, UNSUPPORTED, WORKSPACE, _cache, _paged, lib  # noqa: F401


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(batch=-1)), (INVALID, dict(rows=-1)), (INVALID, dict(words=0)), (INVALID, dict(parents=None)), (INVALID, dict(cu=None)),
    (INVALID, dict(lens=None)), (INVALID, dict(masks=None)), (INVALID, dict(pos=None)), (INVALID, dict(masks=0x10004)),
    (INVALID, dict(pos=0x11000)), (INVALID, dict(pos=0x12000)), (INVALID, dict(pos=0x13004)), (INVALID, dict(pos=0x14002)),
    (INVALID, dict(parents=0x10001)), (UNSUPPORTED, dict(words=33)), (UNSUPPORTED, dict(rows=1 << 31)),
])
def test_tables_refusals(lib, want, kw):  # noqa: F811
    a = dict(parents=0x10000, cu=0x11000, lens=0x12000, batch=4, rows=16, words=2, masks=0x13000, pos=0x14000)
    a.update(kw)
    assert lib.fp8kv_tree_tables(*a.values(), None) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(total=-1)), (INVALID, dict(q_heads=3)), (INVALID, dict(window=-1)), (INVALID, dict(sinks=-1)),
    (INVALID, dict(splits=-1)), (INVALID, dict(kernel=1)), (INVALID, dict(kernel=7)), (INVALID, dict(out_dtype=2)),
    (INVALID, dict(sm=float("inf"))), (INVALID, dict(q=None)), (INVALID, dict(lens=None)), (INVALID, dict(out=None)),
    (INVALID, dict(cu=None)), (INVALID, dict(masks=None)), (INVALID, dict(words=0)), (INVALID, dict(masks=0x22002)),
    (INVALID, dict(pos=0x23002)), (INVALID, dict(pos=None, window=16)), (INVALID, dict(masks=0x40000)), (INVALID, dict(pos=0x30000)),
    (INVALID, dict(out=0x10000)), (INVALID, dict(ws=0x30008)), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=100)),
    (UNSUPPORTED, dict(words=33)), (UNSUPPORTED, dict(q_heads=34)), (UNSUPPORTED, dict(total=1 << 31)), (UNSUPPORTED, dict(splits=5000)),
])
def test_attention_refusals(lib, want, kw):  # noqa: F811
    a = dict(q=0x10000, cu=0x20000, lens=0x21000, masks=0x22000, words=1, pos=0x23000, total=10, q_heads=4, sm=0.1, window=0, sinks=0,
             splits=2, kernel=0, ws=0x30000, ws_bytes=1 << 30, out=0x40000, out_dtype=0)
    a.update(kw)
    v = list(a.values())
    assert lib.fp8kv_tree_attention(v[0], _paged(), *v[1:], None) == want


def test_attention_refusals_by_cache(lib):  # noqa: F811
    args = (0x20000, 0x21000, 0x22000, 1, 0x23000, 10, 4, 0.1, 0, 0, 0, 0, 0x30000, 1 << 30, 0x40000, 0, None)
    turning = _cache(k_bias=0x8000, rope_cos=0x9000, rope_sin=0xA000, rope_positions=2048)
    assert lib.fp8kv_tree_attention(0x10000, turning, *args) == UNSUPPORTED
    assert lib.fp8kv_tree_attention(0x10000, None, *args) == INVALID
    assert lib.fp8kv_tree_workspace_bytes(_paged(), 10, 4, 0, 0, 2, 0) == lib.fp8kv_chunk_workspace_bytes(_paged(), 10, 4, 0, 0, 2, 0) > 0
    assert lib.fp8kv_tree_workspace_bytes(_paged(), 10, 3, 0, 0, 2, 0) == 0
    # nothing to do
    assert lib.fp8kv_tree_attention(0x10000, _paged(), *args[:5], 0, *args[6:]) == 0


def _accept(lib, caches, n=None, **kw):  # noqa: F811
    from fp8_quantized_kv_gb300._lib import CacheStruct
    refs = (ctypes.POINTER(CacheStruct) * max(1, len(caches)))(*[ctypes.pointer(c._obj) for c in caches])
    a = dict(parents=0x10000, tokens=0x11000, choices=0x12000, cu=0x13000, lens=0x14000, batch=4, rows=16, most=4, path=0x15000,
             accepted=0x16000, next=0x17000, new_lens=0x18000)
    a.update(kw)
    return lib.fp8kv_tree_accept(refs if caches else None, len(caches) if n is None else n, *a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(batch=-1)), (INVALID, dict(rows=-1)), (INVALID, dict(most=0)), (INVALID, dict(parents=None)), (INVALID, dict(tokens=None)),
    (INVALID, dict(choices=None)), (INVALID, dict(cu=None)), (INVALID, dict(lens=None)), (INVALID, dict(path=None)),
    (INVALID, dict(accepted=None)), (INVALID, dict(next=None)), (INVALID, dict(new_lens=None)), (INVALID, dict(new_lens=0x14000)),
    (INVALID, dict(path=0x11010)), (INVALID, dict(accepted=0x15004)), (INVALID, dict(next=0x17004)), (INVALID, dict(tokens=0x11004)),
    (INVALID, dict(lens=0x14001)), (UNSUPPORTED, dict(rows=1 << 31)),
])
def test_accept_refusals(lib, want, kw):  # noqa: F811
    assert _accept(lib, [], **kw) == want


def test_accept_refusals_by_caches(lib):  # noqa: F811
    big = dict(max_tokens=16, k=0x100000, v=0x200000, k_scale=0x300000, v_scale=0x400000)
    apart = dict(max_tokens=16, k=0x500000, v=0x600000, k_scale=0x700000, v_scale=0x800000)
    one = _cache(**big)
    assert _accept(lib, [], n=1) == INVALID and _accept(lib, [], n=-1) == INVALID
    assert _accept(lib, [one, one]) == INVALID                                             # the same cache twice
    assert _accept(lib, [one, _cache(**{**apart, "v": 0x100010})]) == INVALID              # shared rows
    for kw in (dict(batch=5), dict(kv_heads=4), dict(head_dim=64), dict(dtype=3, v_scale=None),
               dict(layout=1, max_tokens=0, page_size=16, num_pages=4, max_pages_per_seq=2, page_table=0x900000)):
        assert _accept(lib, [one, _cache(**{**apart, **kw})]) == INVALID
    assert _accept(lib, [_cache(**{**big, "batch": 5})]) == INVALID
    assert _accept(lib, [one], lens=0x200100) == INVALID                                   # an input among a cache's rows
    assert _accept(lib, [one], path=0x100000) == INVALID                                   # outputs in a cache, in a page table
    paged = dict(layout=1, max_tokens=0, page_size=16, num_pages=4, max_pages_per_seq=2, page_table=0x18000)
    assert _accept(lib, [_cache(**{**big, **paged})]) == INVALID
    assert _accept(lib, [_paged(max_pages_per_seq=1 << 27)]) == UNSUPPORTED
    assert _accept(lib, [one] * 513) == UNSUPPORTED
    assert _accept(lib, [], batch=0) == 0


def test_binding_refusals():
    i32 = torch.zeros(4, dtype=torch.int32)
    if torch.cuda.is_available():
        pytest.skip("the message differs with a device")
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        fk.fp8kv_tree_tables(i32, i32, i32, 32)


@pytest.mark.parametrize("want,kw", [(INVALID, dict(window=-1)), (INVALID, dict(sinks=-1)), (INVALID, dict(words=0)),
                                     (INVALID, dict(masks=0x10004)), (UNSUPPORTED, dict(words=33)), (0, dict(rows=0))])
def test_windowed_tables_refusals(lib, want, kw):  # noqa: F811
    a = dict(parents=0x10000, cu=0x11000, lens=0x12000, batch=4, rows=16, words=2, window=8, sinks=4, masks=0x13000, pos=0x14000)
    a.update(kw)
    assert lib.fp8kv_tree_tables_window(*a.values(), None) == want


def test_accept_refuses_a_page_table_among_rows(lib):  # noqa: F811
    """The table of one layer inside the rows or scales of another (or of its own cache): those are written."""
    paged = dict(layout=1, max_tokens=0, page_size=16, num_pages=4, max_pages_per_seq=2)
    a = dict(k=0x100000, v=0x200000, k_scale=0x300000, v_scale=0x400000)
    b = dict(k=0x500000, v=0x600000, k_scale=0x700000, v_scale=0x800000)
    rows = 4 * 2 * 16                                                   # of a cache: 128 bytes of codes, 4 of scales each
    for at in (0x100000, 0x200010, 0x300000 + 4 * rows - 16, 0x400000, 0x500000 + 128 * rows - 16, 0x700000 - 16 + 4 * rows, 0x800000 - 16):
        first, second = _cache(**a, **paged, page_table=0x900000), _cache(**b, **paged, page_table=at)
        assert _accept(lib, [first, second]) == INVALID and _accept(lib, [second, first]) == INVALID
        assert _accept(lib, [first, first]) == INVALID


@pytest.mark.parametrize("what", ["cu", "lens", "table", "k", "v_scale"])
@pytest.mark.parametrize("end", [0, 1])
def test_out_and_workspace_apart_from_what_is_read(lib, end, what):  # noqa: F811
    """Offsets, lengths, page table and cache rows that out or the workspace would write
    over: refused, in the tree and in the chunk call."""
    far = dict(k=0x1000000, v=0x2000000, k_scale=0x3000000, v_scale=0x4000000, page_table=0x5000000)
    out_bytes, ws_bytes = 10 * 4 * 128 * 2, 10 * 4 * 2 * 130 * 4
    for base, size in ((0x40000, out_bytes), (0x30000, ws_bytes)):
        at = base + (size - 16 if end else 0)
        a = dict(cu=0x20000, lens=0x21000)
        cache = dict(far)
        if what in a:
            a[what] = at
        else:
            cache["page_table" if what == "table" else what] = at
        tail = (10, 4, 0.1, 0, 0, 2, 0, 0x30000, 1 << 30, 0x40000, 0, None)
        assert lib.fp8kv_tree_attention(0x10000, _paged(**cache), a["cu"], a["lens"], 0x22000, 1, 0x23000, *tail) == INVALID
        assert lib.fp8kv_chunk_attention(0x10000, _paged(**cache), a["cu"], a["lens"], *tail) == INVALID


def test_plan_of_wide_trees_under_a_small_window(lib):  # noqa: F811
    """A tile of a tree sees the window and all nodes of the tree, not its own alone:
    the split count that is asked for is used, and an automatic one counts those tiles."""
    cache = _cache(batch=1, max_tokens=65536)
    share = 1024 * 4 * 130 * 4                                          # bytes of one share of every row
    for kernel in (0, 5, 2):
        assert lib.fp8kv_tree_workspace_bytes(cache, 1024, 4, 64, 0, 10, kernel) == 10 * share
        assert lib.fp8kv_tree_workspace_bytes(cache, 1024, 4, 64, 0, 100, kernel) == 18 * share      # (64 + 1,024 tokens: 17 tiles, or 18)
    assert lib.fp8kv_tree_workspace_bytes(cache, 1024, 4, 64, 0, 0, 0) >= 3 * share
    # one tree among many small ones may hold most rows
    assert lib.fp8kv_tree_workspace_bytes(_cache(batch=8, max_tokens=8192), 1031, 4, 64, 0, 10, 0) == 10 * 1031 * 4 * 130 * 4
    # a chunk call's tile sees its own 64 queries only: (64 + 64) / 64 tiles, or one more
    assert lib.fp8kv_chunk_num_splits(cache, 1024, 4, 64, 0, 10, 2) == 3
