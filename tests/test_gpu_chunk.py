"""Ragged chunk attention over the cache (fp8kv_chunk_attention) against the
definition in 64 bits: every cache type, head dim and group size, lengths from
nothing to many tiles, windows with first tokens, splits, keys that must not
be seen, and a whole serving step.

Tolerance, per element, for an fp32 output (derived, not fitted).  With exact
weights p (sum 1) and values v:
  - a weight is rounded once to the 16-bit operand: u_P = 2^-11 (f16, e4m3
    values) or 2^-8 (bf16 values) of its size;
  - a score is an fp32 dot product of D exact products: at most D 2^-23
    sum |q||k| sm_scale off (the tensor core may truncate), and scaling,
    exponential and its argument add 2^-19 for the score sizes used here; a
    score error d changes a weight by a factor within 1 +- 2 d, and the sum
    that divides them as much again;
  - an f16 weight is held relative to the largest value scale, absolute step
    2^-39 of the largest value, at most one per key.
So |o - exact| <= (u_P + 4 (d + 2^-19)) sum p |v| + keys 2^-38 max |v|.  The
tcgen05 kernel's query operand adds 2^-18 max |q| sum |k| sm_scale to d ("auto"
may pick that kernel).  A bf16 output adds its rounding, 2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

import fp8_quantized_kv_gb300 as fk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_device_error():
    fk.fp8kv_get_device_error(clear=True)
    yield


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_cache(dtype, D, Hkv, lens, page, seed, poison=True, spread=0.0):
    """A cache holding lens[b] tokens a sequence, everything else NaN (codes
    0x7F, scales NaN, page ids out of range) if `poison`."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    if page:
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        perm = rng.permutation(pages).astype(np.int32)
        table = np.full((B, max([1] + need) + 1), -7 if poison else 0, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        cache = fk.Fp8KVCache.paged(torch.from_numpy(table), pages, Hkv, D, page, dtype)
    else:
        cache = fk.Fp8KVCache.contiguous(B, Hkv, D, max(16, -(-max(lens) // 16) * 16), dtype)
    if poison:
        for t in (cache.k, cache.v):
            t.fill_(0x7F if t.dtype == torch.uint8 else float("nan"))
        for t in (cache.k_scale, cache.v_scale):
            if t is not None:
                t.fill_(0xFF if t.dtype == torch.uint8 else float("nan"))
    n = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(n, Hkv, D, generator=g, device="cuda")
    v = torch.randn(n, Hkv, D, generator=g, device="cuda")
    if spread:
        v *= torch.exp2(spread * (2 * torch.rand(n, Hkv, 1, generator=g, device="cuda") - 1))
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    if n:
        seq = np.repeat(np.arange(B), lens)
        pos = np.concatenate([np.arange(x) for x in lens])
        fk.fp8kv_append(cache, k, v, _i32(seq.tolist()), _i32(pos.tolist()))
    return cache


def cache_values(cache, lens):
    """fp64 K and V of every sequence, [tokens, Hkv, D], read back from the cache."""
    span = cache.page_size or cache.max_tokens
    out = []
    for b, n in enumerate(lens):
        t = torch.arange(n)
        lead = cache.page_table[b].cpu().long()[t // span] if cache.page_size else torch.full_like(t, b)
        pair = []
        for side in ("k", "v"):
            x, sc = getattr(cache, side), getattr(cache, side + "_scale")
            rows = x[lead.cuda(), :, (t % span).cuda()].cpu()
            if x.dtype == torch.uint8:
                val = rows.view(torch.float8_e4m3fn).double()
                s = sc[lead.cuda(), :, (t % span).cuda()].cpu()
                val = val * (torch.exp2(s.double() - 127).repeat_interleave(32, -1) if sc.dtype == torch.uint8 else s.double()[..., None])
            else:
                val = rows.double()
            pair.append(val)
        out.append(pair)
    return out


def definition(q, kv, cu, lens, window, sinks, sm):
    """fp64 outputs [rows, Hq, D], sum p |v|, score error scale sum |q||k| sm
    (largest over the seen keys), max |q| sum |k| sm, seen keys, max |v|."""
    rows, Hq, D = q.shape
    q = q.double().cpu()
    o, pv, qk, qs = torch.zeros(rows, Hq, D, dtype=torch.float64), torch.zeros(rows, Hq, D, dtype=torch.float64), \
        torch.zeros(rows, Hq), torch.zeros(rows, Hq)
    keys, vmax = torch.zeros(rows), torch.zeros(rows, Hq)
    for b, (k, v) in enumerate(kv):
        n = cu[b + 1] - cu[b]
        G = Hq // k.shape[1]
        for i in range(n):
            p, r = lens[b] - n + i, cu[b] + i
            j = torch.arange(max(0, p + 1))
            if window:
                j = j[(j > p - window) | (j < sinks)]
            if len(j) == 0:
                continue
            kk, vv = k[j].repeat_interleave(G, 1), v[j].repeat_interleave(G, 1)      # [keys, Hq, D]
            s = torch.einsum("hd,khd->hk", q[r], kk) * sm
            w = torch.softmax(s, -1)
            o[r] = torch.einsum("hk,khd->hd", w, vv)
            pv[r] = torch.einsum("hk,khd->hd", w, vv.abs())
            qk[r] = (torch.einsum("hd,khd->hk", q[r].abs(), kk.abs()) * abs(sm)).amax(-1)
            qs[r] = q[r].abs().amax(-1) * kk.abs().sum(-1).amax(0) * abs(sm)
            keys[r], vmax[r] = len(j), vv.abs().amax((0, 2))
    return o, pv, qk, qs, keys, vmax


def check(out, cache, want, rows, kernel):
    o, pv, qk, qs, keys, vmax = (x[rows] for x in want)
    v16 = cache.v.dtype == torch.bfloat16
    d = cache.head_dim * 2.0 ** -23 * qk + 2.0 ** -19
    if kernel != "warp_mma":
        d = d + 2.0 ** -18 * qs
    tol = (2.0 ** (-8 if v16 else -11) + 4 * d)[..., None] * pv + (keys[:, None] * vmax * 2.0 ** -38)[..., None]
    got = out[rows].double().cpu()
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (o.abs() + tol)
    assert torch.isfinite(got).all()
    worst = ((got - o).abs() - tol).max().item()
    assert worst <= 0, f"past the tolerance by {worst:.3e}"


def run_case(dtype, D, Hq, Hkv, cached, new, page, seed, window=0, sinks=0, kernel="auto", splits=0, out_dtype=torch.float32,
             spread=0.0, pad=3):
    lens = [c + n for c, n in zip(cached, new)]
    cache = make_cache(dtype, D, Hkv, lens, page, seed, spread=spread)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn(cu[-1] + pad, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((cu[-1] + pad, Hq, D), 5.0, dtype=out_dtype, device="cuda")
    fk.fp8kv_chunk_attention(q, cache, _i32(cu), _i32(lens), window=window, sinks=sinks, num_splits=splits, out=out, kernel=kernel)
    assert fk.fp8kv_get_device_error() == 0
    want = definition(q, cache_values(cache, lens), cu, lens, window, sinks, 1 / math.sqrt(D))
    check(out, cache, want, slice(0, cu[-1]), kernel)
    assert bool((out[cu[-1]:] == 5.0).all()), "rows behind the last sequence changed"
    return out


DTYPES = ["k8v8", "k16v8", "k8v16", "k16v16", "mxk8v8"]
KERNELS = ["warp_mma", "tensor_cores"]


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", DTYPES)
def test_types(dtype, D, page):
    """Long chunks (64-row tiles) of odd lengths over prefixes that end inside
    tiles and pages, an idle sequence and a single token among them."""
    if dtype == "mxk8v8" and D == 64:
        pytest.skip("block-scaled keys are built for head dim 128")
    run_case(dtype, D, 6, 2, [0, 37, 130, 64], [67, 0, 41, 1], page, seed=1, kernel="warp_mma")


@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("dtype", ["k8v8", "k16v8", "k8v16", "k16v16"])
def test_types_tensor_cores(dtype, page):
    """The same on tcgen05, with 128-row tiles that are full, ragged, of one
    token, and longer than the rings."""
    run_case(dtype, 128, 6, 2, [0, 37, 130, 64, 700], [67, 0, 41, 1, 130], page, seed=1, kernel="tensor_cores")


@pytest.mark.parametrize("dtype", ["k8v8", "k16v16"])
@pytest.mark.parametrize("sm", [0.0, -0.11, 2.0])
def test_score_scale(dtype, sm):
    """A scale of zero (every seen key weighs the same), a negative and a large one."""
    lens, cu = [90, 200], [0, 50, 200]
    cache = make_cache(dtype, 128, 2, lens, 16, seed=21)
    q = torch.randn(200, 4, 128, device="cuda").to(torch.bfloat16)
    for kernel in KERNELS:
        out = fk.fp8kv_chunk_attention(q, cache, _i32(cu), _i32(lens), sm_scale=sm, out_dtype=torch.float32, kernel=kernel)
        assert fk.fp8kv_get_device_error() == 0
        o, pv, qk, qs, keys, vmax = definition(q, cache_values(cache, lens), cu, lens, 0, 0, sm)
        check(out, cache, (o, pv, qk, qs, keys, vmax), slice(0, 200), kernel)


@pytest.mark.parametrize("dtype,D", [("k8v8", 128), ("k8v8", 64), ("k16v16", 128), ("mxk8v8", 128), ("k8v16", 64)])
@pytest.mark.parametrize("new", [1, 2, 3, 6])
def test_few_rows(dtype, D, new):
    """Single and drafted tokens: the 8-, 16- and 32-row tiles, whose warps split
    the keys; one sequence holds the new tokens only."""
    run_case(dtype, D, 8, 2, [0, 15, 200, 63, 64], [new] * 5, 16, seed=2, kernel="warp_mma")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (3, 1), (7, 1), (10, 2), (16, 1), (11, 1)])
def test_groups(Hq, Hkv, kernel):
    """Group sizes that do and do not divide a tile's rows."""
    for new in ([5, 1, 40], [1, 1, 1]):
        run_case("k8v8", 128, Hq, Hkv, [70, 3, 0], new, 32, seed=3, kernel=kernel)


@pytest.mark.parametrize("dtype,D", [("k8v8", 128), ("k16v8", 64), ("k8v16", 128), ("k16v16", 64), ("mxk8v8", 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 1), (17, 40)])
def test_nine_to_sixteen_rows(dtype, D, window, sinks):
    """Tiles of two times eight query rows: 15 rows of 5 tokens x 3 heads, 11 and
    16 of one token, 14 of 2 x 7, with scales that differ widely."""
    for (Hq, Hkv), new in (((6, 2), [5, 4, 5, 5]), ((11, 1), [1] * 4), ((16, 1), [1, 0, 1, 2]), ((14, 2), [2] * 4)):
        run_case(dtype, D, Hq, Hkv, [0, 200, 63, 530], new, 16, seed=41, window=window, sinks=sinks, spread=6.0)
    run_case(dtype, D, 6, 2, [0, 200, 63, 530], [5, 4, 5, 5], 0, seed=42, window=window, sinks=sinks, splits=3,
             out_dtype=torch.bfloat16)


@pytest.mark.parametrize("dtype", ["k8v8", "k16v16"])
@pytest.mark.parametrize("Hq", [1, 2])
@pytest.mark.parametrize("what", ["nan", "inf", "scale"])
def test_few_rows_unseen_values(dtype, Hq, what):
    """Values that are not finite at a position that some queries of an 8- or
    16-row tile see and others do not; a huge value scale there."""
    lens, new, window = [203], [8], 5
    cache = make_cache(dtype, 128, 1, lens, 0, seed=43, poison=False)
    q = torch.randn(8, Hq, 128, device="cuda").to(torch.bfloat16)
    f = lambda: fk.fp8kv_chunk_attention(q, cache, _i32([0, 8]), _i32(lens), window=window, out_dtype=torch.float32)
    ref = f().clone()
    coded = dtype == "k8v8"
    if what == "scale":
        if not coded:
            pytest.skip("bf16 values have no scales")
        cache.v_scale[0, 0, 197] = float("inf")
        cache.v[0, 0, 197] = 0x38
    else:
        cache.v[0, 0, 197, 5] = 0xFF if coded else float(what)
    out = f()
    assert fk.fp8kv_get_device_error() == 0
    pos = torch.arange(195, 203)
    sees = (pos >= 197) & (pos < 197 + window)
    # the weights' two roundings (2^-11 or 2^-8 each) against other references
    assert torch.isfinite(out[~sees]).all() and (out[~sees] - ref[~sees]).abs().max() <= 2.0 ** -7 * 4.5
    assert not torch.isfinite(out[sees][..., 5]).any()
    if what != "scale":
        rest = [d for d in range(128) if d != 5]
        assert (out[sees][..., rest] - ref[sees][..., rest]).abs().max() <= 2.0 ** -7 * 4.5


@pytest.mark.parametrize("dtype", ["k8v8", "k16v8", "k8v16", "k16v16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 1), (64, 4), (100, 65), (2, 200)])
def test_many_rows_head_dim_64(dtype, window, sinks):
    """64-row tiles, full and ragged, of groups that do and do not divide them,
    with scales that differ widely and splits that are empty."""
    for Hq, Hkv, splits in ((4, 2, 0), (7, 1, 3), (16, 1, 0)):
        run_case(dtype, 64, Hq, Hkv, [0, 300, 129, 511], [150, 70, 1, 65], 16, seed=47, window=window, sinks=sinks, spread=6.0,
                 splits=splits)
    # the first queries come before the sequence's first token
    run_case(dtype, 64, 4, 1, [-20, 0], [90, 60], 0, seed=48, window=window, sinks=sinks, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("dtype", ["k8v8", "k16v16", "k8v16"])
@pytest.mark.parametrize("what", ["nan", "inf", "scale"])
def test_unseen_values_head_dim_64(dtype, what):
    """Values that are not finite where some queries of a 64-row tile see them and
    others do not."""
    lens, window = [200], 40
    cache = make_cache(dtype, 64, 1, lens, 0, seed=49, poison=False)
    q = torch.randn(120, 2, 64, device="cuda").to(torch.bfloat16)
    f = lambda: fk.fp8kv_chunk_attention(q, cache, _i32([0, 120]), _i32(lens), window=window, out_dtype=torch.float32)
    ref = f().clone()
    coded = dtype == "k8v8"
    for j in (100, 150):
        if what == "scale":
            if not coded:
                pytest.skip("bf16 values have no scales")
            cache.v_scale[0, 0, j] = float("inf")
            cache.v[0, 0, j] = 0x38
        else:
            cache.v[0, 0, j, 5] = 0xFF if coded else float(what)
    out = f()
    assert fk.fp8kv_get_device_error() == 0
    pos = torch.arange(80, 200)
    sees = torch.stack([(pos >= j) & (pos < j + window) for j in (100, 150)]).any(0)
    # the weights' two roundings (2^-11 or 2^-8 each) against other references
    assert torch.isfinite(out[~sees]).all() and (out[~sees] - ref[~sees]).abs().max() <= 2.0 ** -7 * 4.5
    assert not torch.isfinite(out[sees][..., 5]).any()
    if what != "scale":
        rest = [d for d in range(64) if d != 5]
        assert (out[sees][..., rest] - ref[sees][..., rest]).abs().max() <= 2.0 ** -7 * 4.5


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (63, 0), (64, 4), (65, 64), (100, 65), (130, 1000), (5000, 2), (2, 200)])
def test_windows(window, sinks, kernel):
    """Windows around the tile size and past the sequence, first tokens that
    end inside, at and past a tile and that meet the window."""
    run_case("k8v8", 128, 8, 2, [0, 300, 129, 511], [150, 70, 1, 65], 16, seed=4, window=window, sinks=sinks, kernel=kernel)
    run_case("k16v16", 64, 4, 4, [10, 300, 129, 0], [1, 1, 1, 1], 0, seed=5, window=window, sinks=sinks)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40])
def test_splits(splits, kernel):
    """More splits than a short sequence has tiles among them: empty splits."""
    out = run_case("k8v8", 128, 4, 1, [700, 0, 64], [30, 1, 2], 16, seed=6, splits=splits, kernel=kernel)
    one = run_case("k8v8", 128, 4, 1, [700, 0, 64], [30, 1, 2], 16, seed=6, splits=1, kernel=kernel)
    # the same tiles, joined in another order: fp32 re-association, and P
    # rounded against another reference (2 roundings of 2^-11)
    assert (out[:33] - one[:33]).abs().max() <= 2.0 ** -10 * 4.5


@pytest.mark.parametrize("dtype,D", [("k8v8", 64), ("k16v16", 128)])
@pytest.mark.parametrize("splits", [4, 9, 33, 70])
def test_joined_splits(dtype, D, splits):
    """Few rows of many splits (a CTA's warps share a row's splits, some of them
    empty), and many rows of as many (a warp a row)."""
    run_case(dtype, D, 4, 2, [2000, 0, 90], [1, 0, 3], 16, seed=44, splits=splits)
    run_case(dtype, D, 4, 1, [40, 900], [700, 30], 16, seed=45, splits=splits, out_dtype=torch.bfloat16)


def test_bf16_output_and_no_offsets():
    """cu_q None is one query per sequence; a bf16 output is the fp32 one rounded."""
    lens = [1, 77, 640, 0, 129]
    cache = make_cache("k8v8", 128, 2, lens, 16, seed=7)
    q = torch.randn(5, 8, 128, device="cuda").to(torch.bfloat16)
    f = fk.fp8kv_chunk_attention(q, cache, None, _i32(lens), out_dtype=torch.float32)
    h = fk.fp8kv_chunk_attention(q, cache, None, _i32(lens))
    c = fk.fp8kv_chunk_attention(q, cache, _i32(list(range(6))), _i32(lens), out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == 0
    assert torch.equal(f.to(torch.bfloat16), h) and torch.equal(f, c)
    assert bool((f[3] == 0).all())                 # a length of zero: a zero row
    ref = fk.fp8kv_decode_attention(q, cache, _i32(lens), out_dtype=torch.float32)
    # two roundings of the weights (bf16 there, f16 here) of values below 4.5
    assert (f - ref).abs().max() <= (2.0 ** -8 + 2.0 ** -11) * 4.5


@pytest.mark.parametrize("kernel", KERNELS)
def test_queries_before_the_first_token(kernel):
    """Fewer cached tokens than queries: the first queries see nothing."""
    lens, new = [3, 0, 70], [9, 4, 70]
    cache = make_cache("k8v8", 128, 1, lens, 16, seed=8)
    cu = [0, 9, 13, 83]
    q = torch.randn(83, 4, 128, device="cuda").to(torch.bfloat16)
    out = fk.fp8kv_chunk_attention(q, cache, _i32(cu), _i32(lens), out_dtype=torch.float32, kernel=kernel)
    assert fk.fp8kv_get_device_error() == 0
    assert bool((out[:6] == 0).all()) and bool((out[9:13] == 0).all())
    check(out, cache, definition(q, cache_values(cache, lens), cu, lens, 0, 0, 128 ** -0.5), slice(0, 83), kernel)


@pytest.mark.parametrize("kernel", KERNELS)
def test_v_scales_spread(kernel):
    """V rows scaled by 2^-9 .. 2^9, token by token."""
    run_case("k8v8", 128, 8, 2, [0, 500], [100, 33], 16, seed=9, spread=9.0, kernel=kernel)
    run_case("k8v8", 128, 8, 2, [900, 500], [1, 1], 16, seed=9, spread=9.0)


@pytest.mark.parametrize("dtype,kernel", [("k8v8", "warp_mma"), ("k16v16", "warp_mma"), ("k16v8", "warp_mma"),
                                          ("k8v8", "tensor_cores"), ("k16v16", "tensor_cores"), ("k8v16", "tensor_cores")])
@pytest.mark.parametrize("what", ["k_row", "v_nan", "v_inf", "v_huge"])
def test_unseen_poison(dtype, kernel, what):
    """Non-finite rows at some positions of the sequence itself: the queries
    that do not see them come out as if they were not there, those that do see
    a value that is not finite get one in that element (on the tensor-core
    kernel perhaps in the others of the row too)."""
    lens, new, window, sinks = [200], [120], 40, 3
    D, Hkv, Hq = 128, 1, 2
    bad = [100, 150, 199]
    clean = make_cache(dtype, D, Hkv, lens, 0, seed=10, poison=False)
    cu = [0, 120]
    q = torch.randn(120, Hq, D, device="cuda").to(torch.bfloat16)
    ref = fk.fp8kv_chunk_attention(q, clean, _i32(cu), _i32(lens), window=window, sinks=sinks, out_dtype=torch.float32, kernel=kernel)
    side = "k" if what == "k_row" else "v"
    t = getattr(clean, side)
    coded = t.dtype == torch.uint8
    for j in bad:
        if what == "k_row":
            t[0, 0, j] = 0x7F if coded else float("nan")
        elif what == "v_nan":
            t[0, 0, j, 5] = 0xFF if coded else float("nan")
        elif what == "v_huge":
            if coded:
                clean.v_scale[0, 0, j] = 2.0 ** 100
            t[0, 0, j] = 0x38 if coded else 2.0 ** 100
        elif coded:
            clean.v_scale[0, 0, j] = float("inf")
        else:
            t[0, 0, j, 5] = float("-inf")
    out = fk.fp8kv_chunk_attention(q, clean, _i32(cu), _i32(lens), window=window, sinks=sinks, out_dtype=torch.float32, kernel=kernel)
    assert fk.fp8kv_get_device_error() == 0
    pos = torch.arange(80, 200)
    sees = torch.stack([(pos >= j) & (pos < j + window) for j in bad]).any(0)
    assert torch.isfinite(out[~sees]).all()
    assert (out[~sees] - ref[~sees]).abs().max() <= 2.0 ** -7 * 4.5       # same weights, another rounding reference
    if what == "v_huge":
        assert (out[sees].abs() > 2.0 ** 60).all()
    else:
        assert not torch.isfinite(out[sees][..., 5]).any()
    if kernel == "warp_mma" and (what == "v_nan" or what == "v_inf" and not coded):
        rest = [d for d in range(D) if d != 5]
        assert torch.isfinite(out[sees][..., rest]).all()


def test_reported_lengths_offsets_and_pages():
    cache = make_cache("k8v8", 128, 1, [40, 40, 40], 16, seed=11)
    q = torch.randn(6, 2, 128, device="cuda").to(torch.bfloat16)
    good = fk.fp8kv_chunk_attention(q, cache, _i32([0, 2, 4, 6]), _i32([40, 40, 40]), out_dtype=torch.float32)
    for lens in ([40, 64 + 1, 40], [40, -1, 40]):       # capacity: 4 pages of 16
        out = fk.fp8kv_chunk_attention(q, cache, _i32([0, 2, 4, 6]), _i32(lens), out_dtype=torch.float32)
        assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:]) and bool((out[2:4] == 0).all())
    out = torch.full_like(good, 3.0)
    fk.fp8kv_chunk_attention(q, cache, _i32([0, 2, 9, 6]), _i32([40, 40, 40]), out=out, num_splits=1)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
    assert torch.equal(out[:2], good[:2]) and bool((out[2:] == 3.0).all())
    cache.page_table[1, 1] = cache.num_pages
    out = fk.fp8kv_chunk_attention(q, cache, _i32([0, 2, 4, 6]), _i32([40, 40, 40]), out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_BAD_PAGE
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])


def test_large_calls_repeat():
    """Calls of many CTAs, over and over: no wait runs out, and every run gives
    the same bits (nothing depends on the order in which warps arrive)."""
    rng = np.random.default_rng(31)
    new, cached = rng.integers(100, 400, 12).tolist(), rng.integers(500, 3000, 12).tolist()
    lens = [c + n for c, n in zip(cached, new)]
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    for dtype in ("k8v8", "k16v16", "k16v8"):
        cache = make_cache(dtype, 128, 4, lens, 16, seed=31, poison=False)
        q = torch.randn(cu[-1], 28, 128, device="cuda").to(torch.bfloat16)
        args = (q, cache, _i32(cu), _i32(lens))
        for window in (0, 200):
            ref = fk.fp8kv_chunk_attention(*args, window=window, sinks=5)
            for _ in range(20):
                assert torch.equal(fk.fp8kv_chunk_attention(*args, window=window, sinks=5), ref)
            other = fk.fp8kv_chunk_attention(*args, window=window, sinks=5, kernel="warp_mma")
            # two roundings of the weights on either side of values below 4.6, and bf16 outputs
            assert (ref.float() - other.float()).abs().max() <= 2 * 2.0 ** -8 * 4.6 + 2.0 ** -8 * 4.6
    assert fk.fp8kv_get_device_error() == 0


@pytest.mark.parametrize("dtype,D,new", [("k8v8", 128, [40, 3]), ("k8v8", 128, [1, 1]), ("k8v16", 64, [30, 1])])
def test_residual_keys(dtype, D, new):
    """A cache of keys less a fixed bias: the bias adds the same to every score of
    a query, so the outputs are those of the whole keys."""
    lens, Hkv = [100, 70], 2
    g = torch.Generator(device="cuda").manual_seed(40)
    bias = 5 * torch.randn(Hkv, D, generator=g, device="cuda")
    cache = fk.Fp8KVCache.contiguous(2, Hkv, D, 112, dtype, k_bias=bias)
    n = sum(lens)
    k = (torch.randn(n, Hkv, D, generator=g, device="cuda") + bias).to(torch.bfloat16)
    v = torch.randn(n, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    fk.fp8kv_append(cache, k, v, _i32([0] * 100 + [1] * 70), _i32(list(range(100)) + list(range(70))))
    cu = [0, new[0], sum(new)]
    q = torch.randn(cu[-1], 8, D, generator=g, device="cuda").to(torch.bfloat16)
    out = fk.fp8kv_chunk_attention(q, cache, _i32(cu), _i32(lens), out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == 0
    kv = [[x + bias.cpu().double(), y] for x, y in cache_values(cache, lens)]
    check(out, cache, definition(q, kv, cu, lens, 0, 0, D ** -0.5), slice(0, cu[-1]), "auto")


@pytest.mark.parametrize("dtype", ["k8v8", "k16v16"])
def test_smallest_caches(dtype):
    """A cache of 16 rows in all: fewer than a tile has keys.  One without room
    has no storage and is refused, as by the other calls."""
    for kernel in KERNELS:
        run_case(dtype, 128, 2, 1, [0], [11], 0, seed=17, kernel=kernel)
        cache = fk.Fp8KVCache.contiguous(2, 1, 128, 0, dtype)
        q = torch.randn(30, 2, 128, device="cuda").to(torch.bfloat16)
        with pytest.raises(fk.Fp8KVError):
            fk.fp8kv_chunk_attention(q, cache, _i32([0, 20, 30]), _i32([0, 0]), kernel=kernel)


def test_many_sequences():
    """The tile search over a large batch, many of them idle."""
    rng = np.random.default_rng(12)
    new = (rng.integers(0, 4, 1500) * (rng.random(1500) < 0.4)).tolist()
    cached = rng.integers(0, 40, 1500).tolist()
    run_case("k8v8", 64, 2, 1, cached, new, 16, seed=12)
    run_case("k8v8", 128, 2, 1, cached, new, 16, seed=12, kernel="tensor_cores")


@pytest.mark.parametrize("kernel", KERNELS)
def test_pages_behind_the_window_may_be_gone(kernel):
    """A windowed sequence whose old pages were given back: their table entries
    are out of range, and nothing reads them."""
    lens, cu = [900, 400], [0, 100, 101]
    cache = make_cache("k8v8", 128, 2, lens, 16, seed=22)
    q = torch.randn(101, 8, 128, device="cuda").to(torch.bfloat16)
    args = dict(window=50, sinks=4, out_dtype=torch.float32, kernel=kernel)
    ref = fk.fp8kv_chunk_attention(q, cache, _i32(cu), _i32(lens), **args)
    cache.page_table[0, 1:(900 - 100 - 50) // 16] = -5
    cache.page_table[1, 1:(400 - 50) // 16] = 1 << 30
    out = fk.fp8kv_chunk_attention(q, cache, _i32(cu), _i32(lens), **args)
    assert fk.fp8kv_get_device_error() == 0 and torch.equal(out, ref)


def test_offsets_past_32_bits():
    """Rows more than 2^32 bytes into the cache: pages at the end of a large pool."""
    D, Hkv, page, lens = 128, 8, 64, [100, 300]
    pages = (1 << 33) // (page * Hkv * D * 2) + 16        # 8 GiB of bf16 a side
    per = 5
    table = torch.arange(pages - 2 * per, pages, dtype=torch.int32).reshape(2, per)
    small = make_cache("k16v16", D, Hkv, lens, page, seed=13, poison=False)
    big = fk.Fp8KVCache.paged(table, pages, Hkv, D, page, "k16v16")
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            src, dst = int(small.page_table[b, i]), int(table[b, i])
            big.k[dst], big.v[dst] = small.k[src], small.v[src]
    q = torch.randn(31, 8, D, device="cuda").to(torch.bfloat16)
    for kernel in KERNELS:
        args = (_i32([0, 30, 31]), _i32(lens))
        assert torch.equal(fk.fp8kv_chunk_attention(q, big, *args, kernel=kernel), fk.fp8kv_chunk_attention(q, small, *args, kernel=kernel))
    assert fk.fp8kv_get_device_error() == 0


@pytest.mark.parametrize("splits", [1, 3, 9])
def test_calls_in_a_chain(splits):
    """Each call's queries are the last one's output and its workspace is shared:
    a call starts when the one before is done, eager and from a graph."""
    lens = [300, 17, 1200, 64]
    cache = make_cache("k8v8", 128, 2, lens, 16, seed=46)
    q = torch.randn(4, 8, 128, device="cuda").to(torch.bfloat16)
    a, b = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(fk.fp8kv_chunk_workspace_bytes(cache, 4, 8, num_splits=splits) + 16, dtype=torch.uint8, device="cuda")
    sl = _i32(lens)

    def chain(wait):
        x = q
        for i in range(12):
            x = fk.fp8kv_chunk_attention(x, cache, None, sl, num_splits=splits, out=(a, b)[i & 1], workspace=ws)
            if wait:
                torch.cuda.synchronize()
        return x

    want = chain(True).clone()
    assert torch.equal(chain(False), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain(False)
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and fk.fp8kv_get_device_error() == 0


def test_graphs_and_streams():
    """Two captured calls with a workspace each, replayed on two streams, with
    lengths that change between replays."""
    cache = make_cache("k8v8", 128, 2, [500] * 4, 16, seed=14, poison=False)
    q = torch.randn(4, 8, 128, device="cuda").to(torch.bfloat16)
    lens = [_i32([100] * 4), _i32([450] * 4)]
    need = fk.fp8kv_chunk_workspace_bytes(cache, 4, 8, num_splits=3)
    assert need == 4 * 8 * 3 * 130 * 4
    outs, graphs, works, side = [], [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(2):
        outs.append(torch.zeros(4, 8, 128, device="cuda"))
        works.append(torch.empty(need, dtype=torch.uint8, device="cuda"))
        graphs.append(torch.cuda.CUDAGraph())
        fk.fp8kv_chunk_attention(q, cache, None, lens[i], num_splits=3, out=outs[i], workspace=works[i])
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[i]):
            fk.fp8kv_chunk_attention(q, cache, None, lens[i], num_splits=3, out=outs[i], workspace=works[i])
    for new in (37, 499):
        for i in range(2):
            lens[i].fill_(new + i)
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(side[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], fk.fp8kv_chunk_attention(q, cache, None, lens[i], num_splits=3, out_dtype=torch.float32))
    assert fk.fp8kv_get_device_error() == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4)])
@pytest.mark.parametrize("dtype,page", [("k8v8", 16), ("k16v16", 0), ("mxk8v8", 32)])
def test_serving_steps(dtype, page, window, sinks):
    """Three steps as a server runs them: tables, rotation and append, chunk
    attention; a prompt next to decoding sequences, then single tokens.  The
    keys are the rotated ones of the whole history, kept beside in 64 bits."""
    D, Hq, Hkv, B = 128, 8, 2, 3
    cols = 12
    if page:
        cache = fk.Fp8KVCache.paged(torch.full((B, cols), -1, dtype=torch.int32), 40, Hkv, D, page, dtype)
        free, head = _i32(np.random.default_rng(1).permutation(40).tolist()), _i32([0])
    else:
        cache = fk.Fp8KVCache.contiguous(B, Hkv, D, 160, dtype)
        free = head = None
    cos, sin = fk.fp8kv_rope_tables(256, 64)
    lens = _i32([0] * B)
    g = torch.Generator(device="cuda").manual_seed(15)
    cached = [0] * B
    for new in ([90, 1, 0], [1, 30, 7], [1, 1, 1]):
        rows = sum(new) + 2
        t = fk.fp8kv_build_tables(cache, lens, _i32(new), rows, free, head)
        qkv = torch.randn(rows, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        q_rot = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device="cuda")
        fk.fp8kv_rope_append(cache, q, k, v, t["pos"], t["slots"], cos, sin, q_out=q_rot)
        out = fk.fp8kv_chunk_attention(q_rot, cache, t["cu_new"], t["seq_lens"], window=window, sinks=sinks, out_dtype=torch.float32)
        assert fk.fp8kv_get_device_error() == 0
        lens, head = t["seq_lens"], t["free_head"]
        cached = [c + n for c, n in zip(cached, new)]
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        assert lens.tolist() == cached and t["cu_new"].tolist() == cu
        check(out, cache, definition(q_rot, cache_values(cache, cached), cu, cached, window, sinks, D ** -0.5),
              slice(0, cu[-1]), "auto")
