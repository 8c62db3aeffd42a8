"""Refusals of the serving-step calls, on the host: every call below is turned
down by its argument checks, before any CUDA call.  No GPU."""
import ctypes

import pytest
import torch

import fp8_quantized_kv_gb300 as fk

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from fp8_quantized_kv_gb300 import build as kbuild
    from fp8_quantized_kv_gb300._lib import get_lib
    kbuild.build()
    return get_lib()


def _cache(**kw):
    from fp8_quantized_kv_gb300._lib import CacheStruct
    base = dict(dtype=0, layout=0, batch=4, kv_heads=2, head_dim=128, max_tokens=1024,
                k=0x1000, v=0x2000, k_scale=0x3000, v_scale=0x4000)
    base.update(kw)
    return ctypes.byref(CacheStruct(**base))


def _paged(**kw):
    return _cache(**{**dict(layout=1, max_tokens=0, page_size=16, num_pages=64, max_pages_per_seq=8, page_table=0x5000), **kw})


def _tables(lib, cache, **kw):
    a = dict(cached=0x10000, new=0x11000, free=0x12000, num_free=16, head=0x13000, rows=8, cu=0x14000, lens=0x15000,
             seq=0x16000, pos=0x17000, slots=0x18000, head_out=0x19000)
    a.update(kw)
    return lib.fp8kv_build_tables(cache, a["cached"], a["new"], a["free"], a["num_free"], a["head"], a["rows"], a["cu"], a["lens"],
                                  a["seq"], a["pos"], a["slots"], a["head_out"], None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(rows=-1)), (INVALID, dict(num_free=-1)), (INVALID, dict(cached=None)), (INVALID, dict(new=None)),
    (INVALID, dict(cu=None)), (INVALID, dict(lens=None)), (INVALID, dict(seq=None)), (INVALID, dict(slots=None)),
    (INVALID, dict(free=None)), (INVALID, dict(head=None)), (INVALID, dict(head_out=None)),
    (INVALID, dict(lens=0x10000)), (INVALID, dict(head_out=0x13000)),      # outputs over inputs
    (INVALID, dict(pos=0x16004)), (INVALID, dict(cu=0x5000)), (INVALID, dict(cached=0x5000)),
    (INVALID, dict(slots=0x18004)), (INVALID, dict(cached=0x10002)), (INVALID, dict(head=0x13001)),
    (UNSUPPORTED, dict(rows=1 << 31)),
])
def test_tables_refusals(lib, want, kw):
    assert _tables(lib, _paged(), **kw) == want


def test_tables_refusals_by_cache(lib):
    assert _tables(lib, _paged(batch=16385)) == UNSUPPORTED
    assert _tables(lib, _paged(page_size=8)) == UNSUPPORTED
    assert _tables(lib, _paged(max_pages_per_seq=1 << 27)) == UNSUPPORTED  # positions past 31 bits
    assert _tables(lib, _cache()) == INVALID                               # a free list with a contiguous cache
    assert _tables(lib, None) == INVALID


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(positions=-1)), (INVALID, dict(rot=0)), (INVALID, dict(base=0.0)), (INVALID, dict(base=float("inf"))),
    (INVALID, dict(factor=0.0)), (INVALID, dict(factor=float("nan"))), (INVALID, dict(amplitude=float("inf"))),
    (INVALID, dict(original=-1)), (INVALID, dict(original=64, lo=2.0, hi=2.0)), (INVALID, dict(original=64, lo=float("nan"))),
    (INVALID, dict(cos=None)), (INVALID, dict(sin=0x20010)), (INVALID, dict(cos=0x20002)), (UNSUPPORTED, dict(rot=7)), (UNSUPPORTED, dict(rot=258)),
    (UNSUPPORTED, dict(positions=1 << 31)),
])
def test_rope_tables_refusals(lib, want, kw):
    a = dict(positions=100, rot=64, base=1e4, factor=1.0, original=0, lo=1.0, hi=4.0, amplitude=1.0, cos=0x20000, sin=0x80000)
    a.update(kw)
    assert lib.fp8kv_rope_tables(*a.values(), None) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(n=-1)), (INVALID, dict(q_heads=0)), (INVALID, dict(rot=0)), (INVALID, dict(rot=136)), (INVALID, dict(layout=2)),
    (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(pos=None)), (INVALID, dict(slots=None)), (INVALID, dict(cos=None)),
    (INVALID, dict(q_out=None)), (INVALID, dict(q=0x100008)), (INVALID, dict(qs=512 - 8)), (INVALID, dict(ks=252)),
    (INVALID, dict(vs=260)), (INVALID, dict(q_out=0x100010)), (INVALID, dict(qs=1024, q_out=0x100000)), (INVALID, dict(q_out=0x200000)),
    (INVALID, dict(slots=0x500004)), (UNSUPPORTED, dict(rot=12)), (UNSUPPORTED, dict(n=1 << 31)),
])
def test_rope_append_refusals(lib, want, kw):
    a = dict(q=0x100000, qs=512, k=0x200000, ks=256, v=0x300000, vs=256, q_heads=4, pos=0x400000, slots=0x500000, n=16,
             cos=0x600000, sin=0x700000, positions=64, rot=64, layout=0, q_out=0x800000)
    a.update(kw)
    assert lib.fp8kv_rope_append(_cache(), *a.values(), None) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(total=-1)), (INVALID, dict(q_heads=3)), (INVALID, dict(window=-1)), (INVALID, dict(sinks=-1)),
    (INVALID, dict(splits=-1)), (INVALID, dict(kernel=1)), (INVALID, dict(kernel=7)), (INVALID, dict(out_dtype=2)),
    (INVALID, dict(sm=float("nan"))), (INVALID, dict(q=None)), (INVALID, dict(lens=None)), (INVALID, dict(out=None)),
    (INVALID, dict(q=0x10008)), (INVALID, dict(out=0x40008)), (INVALID, dict(cu=None)), (INVALID, dict(ws=0x30008)),
    (INVALID, dict(out=0x10000)), (INVALID, dict(out=0x10100)), (INVALID, dict(cu=0x20002)), (INVALID, dict(lens=0x21002)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=100)), (UNSUPPORTED, dict(q_heads=34)), (UNSUPPORTED, dict(total=1 << 31)),
    (UNSUPPORTED, dict(splits=5000)), (INVALID, dict(ws=0x3f000)), (INVALID, dict(ws=0xf000)),      # workspace over out, over q
])
def test_chunk_refusals(lib, want, kw):
    a = dict(q=0x10000, cu=0x20000, lens=0x21000, total=10, q_heads=4, sm=0.1, window=0, sinks=0, splits=2, kernel=0, ws=0x30000,
             ws_bytes=1 << 30, out=0x40000, out_dtype=0)
    a.update(kw)
    v = list(a.values())
    assert lib.fp8kv_chunk_attention(v[0], _paged(), *v[1:], None) == want


def test_chunk_refusals_by_cache(lib):
    args = (0x20000, 0x21000, 10, 4, 0.1, 0, 0, 0, 0, 0x30000, 1 << 30, 0x40000, 0, None)
    turning = _cache(k_bias=0x8000, rope_cos=0x9000, rope_sin=0xA000, rope_positions=2048)
    assert lib.fp8kv_chunk_attention(0x10000, turning, *args) == UNSUPPORTED
    assert lib.fp8kv_chunk_attention(0x10000, None, *args) == INVALID
    assert lib.fp8kv_chunk_attention(0x10000, _paged(max_pages_per_seq=1 << 27), *args) == UNSUPPORTED
    tc = args[:8] + (2,) + args[9:]
    for kw in (dict(head_dim=64), dict(dtype=4)):
        assert lib.fp8kv_chunk_attention(0x10000, _cache(**kw), *tc) == UNSUPPORTED
    # other calls do not know the chunk kernel's name
    assert lib.fp8kv_prefill_attention(0x10000, _cache(), 0x20000, 16, 4, 0.1, 5, 0x40000, 0, None) == INVALID
    assert lib.fp8kv_decode_split(0x10000, _cache(), 0x20000, 4, 0.1, 0, 5, 0x30000, 1 << 30, None) == INVALID


def test_chunk_plan(lib):
    """Splits and workspace from the sizes alone: splits for few tiles of a
    long cache, none for many tiles or a short window; never more than tiles."""
    n = lib.fp8kv_chunk_num_splits
    long = dict(batch=1, max_tokens=65536)
    assert n(_cache(**long), 1, 4, 0, 0, 0, 0) > 8
    assert n(_cache(**long), 1, 4, 128, 4, 0, 0) <= 2
    assert n(_cache(**long), 16384, 4, 0, 0, 0, 0) == 1
    assert n(_cache(max_tokens=64), 4, 4, 0, 0, 100, 0) == 2
    assert n(_cache(), 4, 3, 0, 0, 0, 0) == 0
    assert lib.fp8kv_chunk_workspace_bytes(_cache(), 4, 4, 0, 0, 3, 0) == 4 * 4 * 3 * 130 * 4
    assert lib.fp8kv_chunk_workspace_bytes(_cache(), 4, 4, 0, 0, 1, 0) == 0


def test_python_argument_checks():
    """The binding turns wrong tensors down by name."""
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="pos: expected a contiguous CUDA"):
        fk._here(t, torch.int32, "pos", 0)
    with pytest.raises(ValueError, match="free_pages and free_head"):
        cache = type("C", (), dict(layout=fk.LAYOUT_PAGED, batch=4))()
        fk.fp8kv_build_tables(cache, t, t, 4)
    with pytest.raises(ValueError, match="layout"):
        fk.fp8kv_rope_append(None, torch.zeros(1, 2, 64), None, None, t, t, t, t, layout="quarter")


def test_stride_of_one_row():
    """A single token's stride is never used: any slice of it will do."""
    t = torch.zeros(256, dtype=torch.bfloat16).as_strided((1, 2, 128), (4100, 128, 1))
    assert t.stride(0) == 4100 and fk._rows(t, 2, 128, 1, "k", -1)[1] == 256


@pytest.mark.parametrize("layout", ["contiguous", "paged"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("group", [1, 8, 9, 16])
def test_chunk_idle_step(lib, group, head_dim, layout):
    """A step without a query, and one without a sequence, plans and returns like
    any other, whatever the group's size."""
    for batch, kernels in ((4, (0, 5, 2)), (0, (0, 5))):
        kw = dict(batch=batch, kv_heads=1, head_dim=head_dim)
        cache = _paged(**kw) if layout == "paged" else _cache(**kw)
        for kernel in kernels:
            if kernel == 2 and head_dim == 64:
                continue
            for window, splits in ((0, 0), (0, 3), (128, 0)):
                assert lib.fp8kv_chunk_num_splits(cache, 0, group, window, 0, splits, kernel) >= 1
                assert lib.fp8kv_chunk_workspace_bytes(cache, 0, group, window, 0, splits, kernel) == 0
                assert lib.fp8kv_chunk_attention(None, cache, 0x20000, None, 0, group, 0.1, window, 0, splits, kernel, None, 0, None, 0,
                                                 None) == 0


@pytest.mark.parametrize("kw", [dict(base=1e-300), dict(base=1e-12, rot=2 * 128), dict(factor=1e-300), dict(factor=1e-7),
                                dict(factor=1e-310, original=4096, lo=1.0, hi=4.0), dict(amplitude=1e39), dict(amplitude=-1e300),
                                dict(base=5e-324), dict(base=1e-300, positions=0)])
def test_rope_tables_refuse_what_no_table_holds(lib, kw):
    """Frequencies that are not finite, or so high that no fraction of a turn is
    left of them, and amplitudes that overflow fp32."""
    a = dict(positions=100, rot=64, base=1e4, factor=1.0, original=0, lo=1.0, hi=4.0, amplitude=1.0, cos=0x20000, sin=0x80000)
    a.update(kw)
    assert lib.fp8kv_rope_tables(*a.values(), None) == INVALID
    # slow frequencies, down to none at all, have tables
    for base in (1.0, 0.3, 1e300):
        assert lib.fp8kv_rope_tables(0, 64, base, 1.0, 0, 1.0, 4.0, 1.0, None, None, None) == 0
