"""Chunk attention at its edges: offsets that are refused, in calls with splits;
queries and keys that are not finite; positions close to 2^31; value scales far
apart."""
import pytest
import torch

import fp8_quantized_kv_gb300 as fk
from test_gpu_chunk import _i32, cache_values, definition, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_device_error():
    fk.fp8kv_get_device_error(clear=True)
    yield


# (dtype, head dim, kernel, query heads): the few-row kernel with one and two sets
# of rows, the warp-level kernel's 64-row tiles, tcgen05
FORMS = [("k8v8", 128, "warp_mma", 2), ("k16v16", 64, "warp_mma", 2), ("mxk8v8", 128, "warp_mma", 4), ("k8v16", 64, "rows64", 4),
         ("k8v8", 64, "rows64", 2), ("k8v8", 128, "tensor_cores", 2), ("k16v16", 128, "tensor_cores", 4)]


def _call(q, cache, cu, lens, kernel, **kw):
    return fk.fp8kv_chunk_attention(q, cache, _i32(cu), _i32(lens), kernel="warp_mma" if kernel == "rows64" else kernel, **kw)


# --------------------------------------------------------- refused offsets --
@pytest.mark.parametrize("splits", [1, 3, 9])
@pytest.mark.parametrize("dtype,D,kernel,Hq", FORMS)
def test_refused_offsets_leave_their_rows(dtype, D, kernel, Hq, splits):
    """Rows of a sequence whose offsets decrease or pass total_q stay as they
    were, with and without splits, whatever the workspace holds.  The others' rows
    are those of a call without it; where offsets decrease some may be left too."""
    lens, step = [700, 700, 700], 40 if kernel == "rows64" else 2
    cache = make_cache(dtype, D, 1, lens, 16, seed=60)
    total = 3 * step
    q = torch.randn(total, Hq, D, device="cuda").to(torch.bfloat16)
    good = _call(q, cache, [0, step, 2 * step, total], lens, kernel, num_splits=splits, out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == 0
    need = fk.fp8kv_chunk_workspace_bytes(cache, total, Hq, num_splits=splits, kernel="warp_mma" if kernel == "rows64" else kernel)
    for cu, kept in (([0, step, total + 3, total], slice(0, step)),           # past total_q, then back
                     ([0, step, 2 * step, total + 1], slice(0, 2 * step)),    # past total_q at the end
                     ([0, step, -1, -1], slice(0, step))):                    # below zero
        out = torch.full((total, Hq, D), 3.0, device="cuda")
        ws = torch.full((max(need, 16) // 4,), 0.5, device="cuda").view(torch.uint8)       # finite, so that it would show
        _call(q, cache, cu, lens, kernel, num_splits=splits, out=out, workspace=ws)
        assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
        same = (out[kept] == good[kept]) | ((out[kept] == 3.0) if sorted(cu) != cu else False)
        assert bool(same.all()) and bool((out[:1] == good[:1]).all())
        rest = torch.ones(total, dtype=torch.bool)
        rest[kept] = False
        assert bool((out[rest.cuda()] == 3.0).all())


def test_more_rows_than_a_step_holds():
    """fp8kv_build_tables reports more new rows than n_rows; the attention of that
    step leaves the cut sequence's rows alone, in the splits that it chooses."""
    B, D, Hq, n_rows = 3, 128, 2, 4
    cache = fk.Fp8KVCache.paged(torch.full((B, 256), -1, dtype=torch.int32), 700, 1, D, 16)
    t = fk.fp8kv_build_tables(cache, _i32([0] * B), _i32([1000, 1000, 1000]), 3000, _i32(list(range(700))), _i32([0]))
    k = torch.randn(3000, 1, D, device="cuda").to(torch.bfloat16)
    fk.fp8kv_append(cache, k, k, t["seq_idx"], t["pos"])
    t = fk.fp8kv_build_tables(cache, t["seq_lens"], _i32([1, 1, 5]), n_rows, _i32(list(range(700))), t["free_head"])
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
    # (the tokens themselves, out of this test's way: any finite values do)
    q = torch.randn(n_rows, Hq, D, device="cuda").to(torch.bfloat16)
    assert fk.fp8kv_chunk_num_splits(cache, n_rows, Hq) > 1
    ws = torch.full((fk.fp8kv_chunk_workspace_bytes(cache, n_rows, Hq) // 4,), 0.5, device="cuda").view(torch.uint8)
    out = torch.full((n_rows, Hq, D), 3.0, device="cuda")
    fk.fp8kv_chunk_attention(q, cache, t["cu_new"], t["seq_lens"], out=out, workspace=ws)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
    assert bool((out[2:] == 3.0).all()) and not bool((out[:2] == 3.0).any())


@pytest.mark.parametrize("cu", [[0, 4, 3, 8], [0, 7, 3, 8], [0, 9, 3, 8], [0, 5, 3, 3, 8], [0, 8, 0, 8], [5, 3, 4, 8],
                                [0] * 40 + [6, 5] + [6] * 40 + [8]])
@pytest.mark.parametrize("splits", [1, 5])
def test_every_decrease_is_reported(cu, splits):
    """Offsets that decrease anywhere are reported, and no row gets anything that
    this call did not write: a share of the workspace as it was would bring 1e9.
    (A row that two sequences claim can mix their shares, whose references differ
    by less than 2^16 here.)"""
    B = len(cu) - 1
    cache = make_cache("k8v8", 64, 1, [200] * B, 16, seed=61)
    q = torch.randn(8, 1, 64, device="cuda").to(torch.bfloat16)
    out = torch.full((8, 1, 64), 3.0, device="cuda")
    need = fk.fp8kv_chunk_workspace_bytes(cache, 8, 1, num_splits=splits)
    ws = torch.ones(max(need, 16) // 4, device="cuda")
    ws[:8 * splits * 64] = 1e9
    fk.fp8kv_chunk_attention(q, cache, _i32(cu), _i32([200] * B), num_splits=splits, out=out, workspace=ws.view(torch.uint8))
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
    assert out.abs().max() <= 1e6


# ------------------------------------------------ queries that are not finite --
@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("dtype,D,kernel,Hq", FORMS + [("k16v8", 128, "tensor_cores", 2), ("k8v16", 128, "tensor_cores", 2)])
def test_queries_that_are_not_finite(dtype, D, kernel, Hq, splits):
    """An infinite or NaN element makes every score of its query +-inf or NaN, and
    the softmax of such scores NaN (all -inf among them): that row is NaN on every
    kernel, the others keep their bits, and one that sees no key stays zero."""
    n = 80 if kernel == "rows64" else 7
    lens, cu = [300, n - 3], [0, n, 2 * n]               # sequence 1's first three queries see nothing
    cache = make_cache(dtype, D, 1, lens, 16, seed=62)
    q = torch.randn(2 * n, Hq, D, device="cuda").to(torch.bfloat16)
    args = dict(num_splits=splits, out_dtype=torch.float32)
    ref = _call(q, cache, cu, lens, kernel, **args)
    bad = q.clone()
    bad[0, 0, 3] = float("inf")
    bad[2, 1, D - 1] = float("-inf")
    bad[3, 0, 17] = float("nan")
    bad[n - 1, 1] = float("inf")
    bad[5, 1, 9], bad[5, 1, 40] = float("inf"), 3.0e38
    bad[n + 1, 0, 0], bad[n + 2, 1, 5] = float("inf"), float("nan")      # see nothing
    out = _call(bad, cache, cu, lens, kernel, **args)
    assert fk.fp8kv_get_device_error() == 0
    rows = [(0, 0), (2, 1), (3, 0), (n - 1, 1), (5, 1)]
    nan = torch.zeros(2 * n, Hq, dtype=torch.bool, device="cuda")
    for r, h in rows:
        nan[r, h] = True
    assert bool(torch.isnan(out[nan]).all())
    assert torch.equal(out[~nan], ref[~nan])
    assert bool((out[n:n + 3] == 0).all())


@pytest.mark.parametrize("dtype,D,kernel,Hq", FORMS + [("k16v8", 128, "tensor_cores", 2)])
def test_query_with_all_scores_below_every_number(dtype, D, kernel, Hq):
    """Keys on one side of a query's infinite element give it scores of -inf alone."""
    n = 80 if kernel == "rows64" else 5
    cache = fk.Fp8KVCache.contiguous(1, 1, D, 96, dtype)
    k = torch.randn(90, 1, D, device="cuda").abs().add(0.5).to(torch.bfloat16)
    fk.fp8kv_append(cache, k, k, _i32([0] * 90), _i32(list(range(90))))
    q = torch.zeros(n, Hq, D, device="cuda", dtype=torch.bfloat16)
    q[1, 0] = float("-inf")
    out = _call(q, cache, [0, n], [90], kernel, out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == 0
    assert bool(torch.isnan(out[1, 0]).all()) and torch.isfinite(out[:1]).all() and torch.isfinite(out[1, 1:]).all()


def test_infinite_query_with_a_score_scale_of_zero():
    """0 inf is NaN, on bf16 keys too, whose operand carries the scale's sign."""
    for dtype in ("k8v8", "k16v16"):
        cache = make_cache(dtype, 128, 1, [90], 16, seed=64)
        q = torch.randn(40, 2, 128, device="cuda").to(torch.bfloat16)
        q[7, 1, 3] = float("inf")
        for kernel in ("warp_mma", "tensor_cores"):
            out = _call(q, cache, [0, 40], [90], kernel, sm_scale=0.0, out_dtype=torch.float32)
            assert bool(torch.isnan(out[7, 1]).all()) and torch.isfinite(out[7, 0]).all() and torch.isfinite(out[8:]).all()
    assert fk.fp8kv_get_device_error() == 0


@pytest.mark.parametrize("splits", [1, 5])
@pytest.mark.parametrize("dtype,D,kernel,Hq", [f for f in FORMS if f[0] != "mxk8v8"] + [("k8v16", 128, "tensor_cores", 2)])
def test_scores_of_minus_infinity(dtype, D, kernel, Hq, splits):
    """An infinite key on the far side of a query scores -inf: it weighs nothing
    beside keys with finite scores, and a query that sees such keys alone is NaN,
    whichever share holds them; queries before the first token stay zero."""
    n, T, bad = (80, 300, (250, 251, 252, 299)) if kernel == "rows64" else (9, 300, (293, 294, 295, 299))
    cache = fk.Fp8KVCache.contiguous(2, 1, D, 304, dtype)
    g = torch.Generator(device="cuda").manual_seed(66)
    k = (torch.rand(T + 4, 1, D, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    v = torch.randn(T + 4, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    fk.fp8kv_append(cache, k, v, _i32([0] * T + [1] * 4), _i32(list(range(T)) + list(range(4))))
    q = torch.zeros(2 * n, Hq, D, device="cuda", dtype=torch.bfloat16)
    q[:, :, 0] = -1.0
    for j in bad:
        if dtype in ("k8v8", "k8v16"):
            cache.k_scale[0, 0, j] = float("inf")
        else:
            cache.k[0, 0, j, 0] = float("inf")
    args = dict(num_splits=splits, out_dtype=torch.float32)
    pos = torch.arange(T - n, T)
    for window, sinks in ((0, 0), (1, 0), (2, 0), (3, 0), (2, 1)):
        out = _call(q, cache, [0, n, 2 * n], [T, 4], kernel, window=window, sinks=sinks, **args)
        assert fk.fp8kv_get_device_error() == 0
        seen = [[j for j in range(int(p) + 1) if window == 0 or j > p - window or j < sinks] for p in pos]
        alone = torch.tensor([all(j in bad for j in s) for s in seen], device="cuda")
        assert bool(torch.isnan(out[:n][alone]).all()) and bool(torch.isfinite(out[:n][~alone]).all())
        assert bool((out[n:2 * n - 4] == 0).all()) and bool(torch.isfinite(out[2 * n - 4:]).all())
        # a weight of zero: the value of such a key does not matter
        old = cache.v[0, 0, 299].clone()
        cache.v[0, 0, 299] = cache.v[0, 0, 17]
        again = _call(q, cache, [0, n, 2 * n], [T, 4], kernel, window=window, sinks=sinks, **args)
        cache.v[0, 0, 299] = old
        assert torch.equal(again[:n][~alone], out[:n][~alone])


@pytest.mark.parametrize("dtype,D,kernel,Hq", FORMS)
def test_query_with_all_scores_below_every_number_in_splits(dtype, D, kernel, Hq):
    """As without splits, in shares that hold the query's own key and in others."""
    n = 80 if kernel == "rows64" else 5
    cache = fk.Fp8KVCache.contiguous(1, 1, D, 608, dtype)
    k = torch.randn(600, 1, D, device="cuda").abs().add(0.5).to(torch.bfloat16)
    fk.fp8kv_append(cache, k, k, _i32([0] * 600), _i32(list(range(600))))
    q = torch.zeros(n, Hq, D, device="cuda", dtype=torch.bfloat16)
    q[1, 0] = float("-inf")
    for splits in (2, 6):
        for window, sinks in ((0, 0), (100, 70)):
            out = _call(q, cache, [0, n], [600], kernel, out_dtype=torch.float32, num_splits=splits, window=window, sinks=sinks)
            assert bool(torch.isnan(out[1, 0]).all()) and torch.isfinite(out[:1]).all() and torch.isfinite(out[1, 1:]).all()
            assert torch.isfinite(out[2:]).all()
    assert fk.fp8kv_get_device_error() == 0


# --------------------------------------------------- positions close to 2^31 --
@pytest.mark.parametrize("D,kernel,new", [(128, "warp_mma", 1), (128, "tensor_cores", 40), (64, "rows64", 70)])
def test_positions_up_to_31_bits(D, kernel, new):
    """A table row for 2^31 - 16 tokens, full, under a window: the last tile's end
    is past 31 bits when rounded up.  Tiles lie as in a sequence of 112 tokens."""
    cols, window = (1 << 27) - 1, 15
    small = make_cache("k8v8", D, 1, [112], 16, seed=65, poison=False)
    q = torch.randn(new, 2, D, device="cuda").to(torch.bfloat16)
    want = _call(q, small, [0, new], [112], kernel, window=window, num_splits=1, out_dtype=torch.float32)
    big = fk.Fp8KVCache.paged(torch.full((1, cols), -1, dtype=torch.int32), small.num_pages, 1, D, 16)
    for side in ("k", "v", "k_scale", "v_scale"):
        getattr(big, side).copy_(getattr(small, side))
    big.page_table[0, cols - 7:] = small.page_table[0, :7]
    out = _call(q, big, [0, new], [cols * 16], kernel, window=window, num_splits=1, out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == 0 and torch.equal(out, want)


# ------------------------------------------------------ range of the weights --
@pytest.mark.parametrize("octaves", [10, 20, 24])
@pytest.mark.parametrize("dtype,D,kernel,Hq", [f for f in FORMS if f[0] in ("k8v8", "mxk8v8")] + [("k16v8", 128, "tensor_cores", 2)])
def test_small_value_scale_of_the_heaviest_key(dtype, D, kernel, Hq, octaves):
    """A query's weight goes to keys whose value scale is 2^-octaves of another seen
    key's, which weighs next to nothing.  The weight operand is an f16 number times
    a power of two that puts the largest seen value scale in [2^6, 2^7) (64-row
    tiles: [2^14, 2^15)).  Below 2^-14 its step is 2^-24, and half of that is, in
    values (codes up to 448, scale = max |v| / 448), 2^-31 (2^-39) of the largest
    seen |v| for each key; the sum that divides it is 1 at least.  The rest of the
    tolerance is that of the other tests."""
    n, T = (80, 84) if kernel == "rows64" else (3, 12)
    cache = fk.Fp8KVCache.contiguous(1, 1, D, 96, dtype)
    g = torch.Generator(device="cuda").manual_seed(67)
    base = torch.randn(1, 1, D, generator=g, device="cuda")
    k = (-2.0 * base).repeat(T, 1, 1)
    k[1] = 1.5 * base                                       # the heaviest key (all queries see it), and the one beside it
    k[2] = 1.5 * base + 0.01 * torch.randn(1, D, generator=g, device="cuda")
    v = torch.randn(T, 1, D, generator=g, device="cuda")
    v[1:3] *= 2.0 ** -octaves
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    fk.fp8kv_append(cache, k, v, _i32([0] * T), _i32(list(range(T))))
    # scores of about 1.5 |base|^2 sm (17 and 12 at these head dims), and -2 |base|^2 sm
    q = base.expand(n, Hq, D).contiguous().to(torch.bfloat16)
    lens, cu, sm = [T], [0, n], D ** -0.5
    out = _call(q, cache, cu, lens, kernel, out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == 0
    o, pv, qk, qs, keys, vmax = definition(q, cache_values(cache, lens), cu, lens, 0, 0, sm)
    d = D * 2.0 ** -23 * qk + 2.0 ** -19 + (2.0 ** -18 * qs if kernel == "tensor_cores" else 0)
    step = 2.0 ** (-39 if kernel == "rows64" else -31)
    tol = (2.0 ** -11 + 4 * d)[..., None] * pv + (keys[:, None] * vmax * step)[..., None]
    worst = ((out.double().cpu() - o).abs() - tol).max().item()
    assert worst <= 0, f"past the tolerance by {worst:.3e}"
