"""What the tree calls leave alone where they refuse something: cache rows of a
sequence past the capacity or on a bad page, table rows of trees with bad offsets."""
import pytest
import torch

import fp8_quantized_kv_gb300 as fk
from test_gpu_chunk import _i32, make_cache
from test_gpu_tree import cache_copy

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_device_error():
    fk.fp8kv_get_device_error(clear=True)
    yield


def moved(cache, before, moves):
    """The cache's tensors as `before` with rows moved: (sequence, from, to)."""
    span, out = cache.page_size or cache.max_tokens, []
    for o in before:
        if o is None:
            out.append(None)
            continue
        w = o.clone()
        for b, i, k in moves:
            (p0, r0), (p1, r1) = [(int(cache.page_table[b, x // span]) if cache.page_size else b, x % span) for x in (i, k)]
            w[p1, :, r1] = o[p0, :, r0]
        out.append(w)
    return out


def same(cache, want):
    return all(t is None or torch.equal(t.view(torch.uint8), w.view(torch.uint8))
               for t, w in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want))


def accept(caches, lens, cu=(0, 4, 8)):
    """Trees of four nodes whose path is 0, 2, 3: of 40 tokens, tokens 38, 39 go to 37, 38."""
    i64 = dict(dtype=torch.int64, device="cuda")
    return fk.fp8kv_tree_accept(caches, _i32([-1, 0, 0, 2] * 2), torch.tensor([1, 2, 1, 1] * 2, **i64), torch.ones(8, **i64), _i32(list(cu)),
                                _i32(lens), 8)


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("dtype", ["k8v8", "k16v16", "mxk8v8"])
def test_accept_past_the_capacity_moves_nothing(dtype, page):
    """One sequence past the capacity, beside one whose rows move; and in one of two layers only."""
    cache = make_cache(dtype, 128, 2, [40, 44], page, seed=31, poison=False)
    before = cache_copy(cache)
    got = accept([cache], [40, cache.capacity + 1])
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG and got["accepted"].tolist() == [3, 3]
    assert same(cache, moved(cache, before, [(0, 38, 37), (0, 39, 38)]))
    small, large = make_cache(dtype, 128, 2, [40, 44], page, seed=32, poison=False), make_cache(dtype, 128, 2, [40, 120], page, seed=33, poison=False)
    before = cache_copy(small), cache_copy(large)
    assert small.capacity < 100 < large.capacity
    accept([small, large], [40, 100])
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
    assert same(small, moved(small, before[0], [(0, 38, 37), (0, 39, 38)]))
    assert same(large, moved(large, before[1], [(0, 38, 37), (0, 39, 38), (1, 98, 97), (1, 99, 98)]))


@pytest.mark.parametrize("bad", [-1, 1 << 20])
@pytest.mark.parametrize("dtype", ["k8v8", "k16v16", "mxk8v8"])
def test_accept_on_a_bad_page_moves_nothing(dtype, bad):
    """A row from or to a bad page stays; page 0, which a clamped id would reach, too.  (Of
    50 tokens, the nodes are 46 to 49: 48 would go to 47, over the page's end, 49 to 48.)"""
    for gone, kept in ((47 // 16, [(1, 49, 48)]), (48 // 16, [])):
        cache = make_cache(dtype, 128, 2, [40, 50], 16, seed=34, poison=False)
        before = cache_copy(cache)
        want = moved(cache, before, [(0, 38, 37), (0, 39, 38)] + kept)
        cache.page_table[1, gone] = bad
        got = accept([cache], [40, 50])
        assert fk.fp8kv_get_device_error() == fk.DEVERR_BAD_PAGE and got["accepted"].tolist() == [3, 3]
        assert same(cache, want)


@pytest.mark.parametrize("cu,left,padding", [([0, 3, 12], [3, 4, 5, 6, 7], []), ([-2, 3, 6], [0, 1, 2], [6, 7]), ([0, 3, 1 << 30], [3, 4, 5, 6, 7], []),
                                             ([0, 9, 8], [0, 1, 2, 3, 4, 5, 6, 7], [])])
@pytest.mark.parametrize("words", [1, 3])
def test_tables_leave_rows_of_bad_offsets(cu, left, padding, words):
    """Rows of a tree whose offsets pass the rows, start below them or decrease stay as they were."""
    masks, pos = torch.full((8, words), 9, dtype=torch.int32, device="cuda"), torch.full((8,), 9, dtype=torch.int32, device="cuda")
    fk.fp8kv_tree_tables(_i32([-1, 0, 1, -1, 0, 1, -1, 0]), _i32(cu), _i32([50, 50]), 32 * words, masks=masks, pos=pos)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
    for r in range(8):
        if r in left:
            assert masks[r].tolist() == [9] * words and int(pos[r]) == 9
        elif r in padding:
            assert masks[r].tolist() == [0] * words and int(pos[r]) == -1
        else:
            assert int(pos[r]) >= 47 and int(masks[r, 0]) > 0
