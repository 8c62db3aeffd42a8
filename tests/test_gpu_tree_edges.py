"""Trees of drafted tokens at their edges: positions close to 2^31, rows in front
of the first tree, queries and scores that are not finite, residual keys, calls that
overlap, and a captured layer of a step with its projections."""
import math
import random

import pytest
import torch

import fp8_quantized_kv_gb300 as fk
from test_gpu_chunk import _i32, cache_values, check, make_cache
from test_gpu_tree import FORMS, ancestors, bits_of, cache_copy, make_step, random_tree, tree_definition

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_device_error():
    fk.fp8kv_get_device_error(clear=True)
    yield


@pytest.mark.parametrize("D,kernel,new", [(128, "warp_mma", 2), (128, "tensor_cores", 40), (64, "warp_mma", 70)])
def test_positions_up_to_31_bits(D, kernel, new):
    """A table row for 2^31 - 16 tokens, full, under a window, against the same tree
    behind 112 tokens: masks, positions, attention and the move of rows."""
    cols, window = (1 << 27) - 1, 15
    total = cols * 16
    small = make_cache("k8v8", D, 1, [112], 16, seed=65, poison=False)
    big = fk.Fp8KVCache.paged(torch.full((1, cols), -1, dtype=torch.int32), small.num_pages, 1, D, 16)
    for side in ("k", "v", "k_scale", "v_scale"):
        getattr(big, side).copy_(getattr(small, side))
    big.page_table[0, cols - 7:] = small.page_table[0, :7]
    q = torch.randn(new, 2, D, device="cuda").to(torch.bfloat16)
    parents, cu = _i32(random_tree(random.Random(3), new, 2)), _i32([0, new])
    outs = []
    for cache, n in ((small, 112), (big, total)):
        masks, pos = fk.fp8kv_tree_tables(parents, cu, _i32([n]), new)
        outs.append((masks, pos - n, fk.fp8kv_tree_attention(q, cache, cu, _i32([n]), masks, pos=pos, window=window, num_splits=1,
                                                             kernel=kernel, out_dtype=torch.float32)))
    assert fk.fp8kv_get_device_error() == 0 and all(torch.equal(a, b) for a, b in zip(*outs))
    tokens = torch.zeros(new, dtype=torch.int64, device="cuda")         # every node fits: the lowest children
    got = [fk.fp8kv_tree_accept([c], parents, tokens, tokens, cu, _i32([n]), 9) for c, n in ((small, 112), (big, total))]
    assert fk.fp8kv_get_device_error() == 0 and torch.equal(got[0]["path"], got[1]["path"])
    assert int(got[1]["lens"][0]) - total == int(got[0]["lens"][0]) - 112
    assert all(torch.equal(getattr(big, s), getattr(small, s)) for s in ("k", "v", "k_scale", "v_scale"))


@pytest.mark.parametrize("dtype,D,kernel", FORMS)
def test_rows_in_front_of_the_first_tree(dtype, D, kernel):
    cache, lens, cu, q, masks, seen, pos, _ = make_step(dtype, D, 4, 2, [90, 33], [20, 7], 16, seed=71, pad=0)
    front, gap = 5, [c + 5 for c in cu]
    pad = torch.randn(front, 4, D, device="cuda").to(torch.bfloat16)
    out = torch.full((front + cu[-1], 4, D), 2.0, device="cuda")
    fk.fp8kv_tree_attention(torch.cat([pad, q]), cache, _i32(gap), _i32(lens), torch.cat([bits_of([[0]] * front, 1), masks]), out=out,
                            kernel=kernel)
    assert fk.fp8kv_get_device_error() == 0 and bool((out[:front] == 2).all())
    want = tree_definition(q, cache_values(cache, lens), cu, lens, seen, pos, 0, 0, 1 / math.sqrt(D))
    check(out[front:], cache, want, slice(0, cu[-1]), kernel)
    masks2, pos2 = fk.fp8kv_tree_tables(_i32([9] * front + [-1] + [0] * 19 + [-1] + [0] * 6), _i32(gap), _i32(lens), 32)
    assert masks2[:front].tolist() == [[0]] * front and pos2.tolist() == [-1] * front + [90] + [91] * 19 + [33] + [34] * 6
    assert fk.fp8kv_get_device_error() == 0


@pytest.mark.parametrize("dtype,D,kernel", FORMS)
@pytest.mark.parametrize("splits", [1, 3])
def test_queries_that_are_not_finite(dtype, D, kernel, splits):
    """A NaN or infinite query makes its own rows NaN and no others."""
    cache, lens, cu, q, masks, seen, pos, _ = make_step(dtype, D, 2, 1, [200], [6], 16, seed=72, pad=0)
    want = tree_definition(q, cache_values(cache, lens), cu, lens, seen, pos, 0, 0, 1 / math.sqrt(D))
    for bad in (float("nan"), float("inf")):
        p = q.clone()
        p[2, :, 7] = bad
        out = fk.fp8kv_tree_attention(p, cache, _i32(cu), _i32(lens), masks, num_splits=splits, kernel=kernel, out_dtype=torch.float32)
        assert fk.fp8kv_get_device_error() == 0 and bool(torch.isnan(out[2]).all())
        check(out, cache, want, torch.tensor([r != 2 for r in range(6)]), kernel)


@pytest.mark.parametrize("kernel", ["warp_mma", "tensor_cores"])
@pytest.mark.parametrize("splits", [1, 2])
def test_scores_of_minus_infinity(kernel, splits):
    """Nodes whose seen keys all score -inf are NaN, those that see no key zero."""
    cache, lens, cu, q, masks, seen, pos, _ = make_step("k16v16", 128, 2, 1, [0], [5], 0, seed=73, pad=0)
    cache.k[0, :, :5, 0] = float("-inf")
    q[..., 0] = 1.0
    out = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, num_splits=splits, kernel=kernel, out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == 0 and bool(torch.isnan(out).all())
    out = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32([3]), masks, num_splits=splits, kernel=kernel, out_dtype=torch.float32)
    assert not bool(out[:2].any()) and bool(torch.isnan(out[2:]).all()) and fk.fp8kv_get_device_error() == 0


def test_residual_keys_move_and_attend():
    """Pre-bias residual keys: attention reads the residual codes (the bias cancels),
    acceptance moves them."""
    bias = torch.randn(2, 128, device="cuda") * 3
    cache = fk.Fp8KVCache.contiguous(1, 2, 128, 64, "k8v8", k_bias=bias)
    k, v = (torch.randn(40, 2, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    fk.fp8kv_append(cache, k, v, _i32([0] * 40), _i32(list(range(40))))
    parents = random_tree(random.Random(8), 10, 3)
    cu, lens, q = [0, 10], [40], torch.randn(10, 4, 128, device="cuda").to(torch.bfloat16)
    masks, pos = fk.fp8kv_tree_tables(_i32(parents), _i32(cu), _i32(lens), 10)
    out = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, out_dtype=torch.float32)
    seen = [ancestors(parents, i) for i in range(10)]
    want = tree_definition(q, cache_values(cache, lens), cu, lens, seen, pos.tolist(), 0, 0, 1 / math.sqrt(128))
    check(out, cache, want, slice(0, 10), "auto")
    before = cache_copy(cache)
    one = torch.ones(10, dtype=torch.int64, device="cuda")
    got = fk.fp8kv_tree_accept([cache], _i32(parents), one, one, _i32(cu), _i32(lens), 4)
    for j, i in enumerate(x for x in got["path"][0].tolist() if x >= 0):
        assert torch.equal(cache.k[0, :, 30 + j], before[0][0, :, 30 + i]) and torch.equal(cache.v_scale[0, :, 30 + j], before[3][0, :, 30 + i])
    assert fk.fp8kv_get_device_error() == 0


def test_calls_that_overlap():
    """Steps of two caches on two streams, each with its own workspace, again and again."""
    sets = []
    for i, (ctx, nodes) in enumerate((([3000, 200], [40, 9]), ([1500, 900], [3, 2]))):
        cache, lens, cu, q, masks, *_ = make_step("k8v8", 128, 8, 2, ctx, nodes, 16, seed=80 + i, pad=0)
        sets.append((q, cache, _i32(cu), _i32(lens), masks))
    want = [fk.fp8kv_tree_attention(*s, num_splits=4) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        got = [fk.fp8kv_tree_attention(*s, num_splits=4, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert fk.fp8kv_get_device_error() == 0


@pytest.mark.parametrize("nodes", [[5, 1, 20], [60, 33, 0]])
def test_captured_layer(nodes):
    """A layer of a verification step in one graph: product, masks, append, tree
    attention, quantisation, product, acceptance.  Replayed on new inputs it gives the
    bits of the same calls made one by one."""
    B, Hq, Hkv, D, C, n = 3, 8, 2, 128, 384, sum(nodes)
    g = torch.Generator(device="cuda").manual_seed(9)
    ctx = [50, 7, 130]
    lens = [c + x for c, x in zip(ctx, nodes)]
    cache = make_cache("k8v8", D, Hkv, lens, 16, seed=90, poison=False)
    base = cache_copy(cache)
    cu = _i32([0, nodes[0], nodes[0] + nodes[1], n])
    slots = torch.cat([cache.page_table[b].long()[t // 16] * 16 + t % 16 for b in range(B)
                       for t in [torch.arange(ctx[b], lens[b], device="cuda")]])
    w = [torch.randint(0, 120, s, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8) for s in (((Hq + 2 * Hkv) * D, C), (C, Hq * D))]
    ws = [torch.rand(x.shape[0] // 128, x.shape[1] // 128, generator=g, device="cuda") * 1e-3 for x in w]
    cos, sin = fk.fp8kv_rope_tables(256, D)
    x, parents, lens_t = torch.zeros(n, C, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda"), _i32(lens)
    tokens, choices = (torch.zeros(n, dtype=torch.int64, device="cuda") for _ in range(2))
    work = torch.empty(max(16, fk.fp8kv_tree_workspace_bytes(cache, n, Hq)), dtype=torch.uint8, device="cuda")

    def layer():
        codes, scales = fk.fp8kv_quantize(x.view(n, -1, 128))
        qkv = fk.fp8kv_block_matmul(codes.view(n, C), scales, w[0], ws[0])
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        masks, pos = fk.fp8kv_tree_tables(parents, cu, lens_t, 64)
        q = fk.fp8kv_rope_append(cache, q, k, v, pos, slots, cos, sin)
        o = fk.fp8kv_tree_attention(q, cache, cu, lens_t, masks, workspace=work)
        codes, scales = fk.fp8kv_quantize(o.view(n, Hq, D))
        y = fk.fp8kv_block_matmul(codes.view(n, Hq * D), scales, w[1], ws[1], out_dtype=torch.float32)
        return y, fk.fp8kv_tree_accept([cache], parents, tokens, choices, cu, lens_t, 8)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer()
    fk.fp8kv_get_device_error()                                         # (parents were all zero: node 0 under itself)
    r = random.Random(6)
    for _ in range(3):
        x.normal_(generator=g)
        parents.copy_(_i32([p for m in nodes for p in random_tree(r, m, 2)]))
        for t in (tokens, choices):
            t.random_(0, 2, generator=g)
        results = []
        for run in (lambda: (graph.replay(), captured)[1], layer):
            for t, o in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), base):
                t.copy_(o)
            y, kept = run()
            torch.cuda.synchronize()
            results.append([y.clone()] + [t.clone() for t in kept.values()] + cache_copy(cache))
        assert all(torch.equal(a, b) for a, b in zip(*results))
        assert torch.isfinite(results[0][0]).all() and fk.fp8kv_get_device_error() == 0


def many_trees(seed, batch, context, nodes):
    """Contexts of all lengths up to `context`, some empty, and trees of up to `nodes`, some without any."""
    r = random.Random(seed)
    ctx = [r.choice([0, 1, r.randint(1, context), context]) for _ in range(batch)]
    return ctx, [r.choice([0, 1, nodes, r.randint(1, nodes)]) for _ in range(batch)]


@pytest.mark.parametrize("dtype,D,kernel,batch,Hkv,nodes,splits", [
    ("k8v8", 128, "warp_mma", 40, 2, 5, 4), ("k16v16", 64, "warp_mma", 33, 1, 40, 8), ("k8v8", 128, "tensor_cores", 31, 2, 40, 4),
    ("k8v16", 128, "warp_mma", 300, 1, 3, 2), ("k8v8", 64, "auto", 1024, 1, 2, 1), ("k8v8", 64, "auto", 1025, 1, 2, 1), ("k8v8", 128, "auto", 256, 1, 4, 2),
    ("k8v8", 64, "auto", 257, 1, 2, 2), ("k16v16", 128, "warp_mma", 65, 2, 3, 3),
    ("k16v8", 128, "tensor_cores", 2, 4, 1024, 3)])
def test_long_sequences_first(dtype, D, kernel, batch, Hkv, nodes, splits):
    """More tiles than run at once, in the order of the sequences' lengths: every row is some tile's."""
    ctx, new = many_trees(batch, batch, 40 if batch > 100 else 200, nodes)
    if batch == 2:
        ctx, new = [700, 30], [600, 1024]
    cache, lens, cu, q, masks, seen, pos, _ = make_step(dtype, D, 2 * Hkv, Hkv, ctx, new, 16, seed=81, pad=4,
                                                        words=max(1, -(-max(new) // 32)))
    front = 3
    gap = [c + front for c in cu]
    q = torch.cat([q[-3:], q])
    masks = torch.cat([masks[-3:], masks])
    out = torch.full((gap[-1] + 4, 2 * Hkv, D), 6.0, device="cuda")
    fk.fp8kv_tree_attention(q, cache, _i32(gap), _i32(lens), masks, out=out, kernel=kernel, num_splits=splits)
    assert fk.fp8kv_get_device_error() == 0
    assert bool((out[:front] == 6).all()) and bool((out[gap[-1]:] == 6).all())
    want = tree_definition(q[front:], cache_values(cache, lens), cu, lens, seen, pos, 0, 0, 1 / math.sqrt(D))
    check(out[front:], cache, want, slice(0, cu[-1]), kernel)


def test_long_sequences_first_beside_bad_offsets():
    """Offsets that decrease leave the order as it comes; a row in front is right or as it was."""
    ctx, new = many_trees(5, 40, 200, 5)
    cache, lens, cu, q, masks, *_ = make_step("k8v8", 128, 4, 2, ctx, new, 16, seed=83)
    want = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, num_splits=4)
    bad = cu[:31] + [cu[30] - 1] + cu[32:]
    out = torch.full_like(want, 6.0)
    fk.fp8kv_tree_attention(q, cache, _i32(bad), _i32(lens), masks, num_splits=4, out=out)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
    assert bool(((out == want) | (out == 6)).all(-1).all(-1)[:cu[30] - 1].all()) and bool((out[cu[-1]:] == 6).all())


def test_node_0_with_a_bad_parent_is_accepted():
    cache = make_cache("k8v8", 128, 1, [40], 16, seed=85, poison=False)
    tokens = torch.ones(3, dtype=torch.int64, device="cuda")
    got = fk.fp8kv_tree_accept([cache], _i32([0, 0, 1]), tokens, tokens, _i32([0, 3]), _i32([40]), 4)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_BAD_TREE and got["path"].tolist() == [[0, 1, 2, -1]]


@pytest.mark.parametrize("dtype,D,nodes,batch", [("k8v8", 128, (30, 60), 24), ("k16v8", 128, (30, 60), 24), ("k16v16", 128, (2, 5), 60),
                                                 ("k8v8", 64, (30, 60), 24), ("mxk8v8", 128, (3, 9), 40)])
def test_large_calls_repeat_and_follow_lengths(dtype, D, nodes, batch):
    """More tiles than run at once: every run gives the same bits, on two streams at
    once too, and a captured call orders its tiles by the lengths of each replay."""
    r = random.Random(batch + D)
    ctx, new = [r.randint(100, 2500) for _ in range(batch)], [r.randint(*nodes) for _ in range(batch)]
    cache, lens, cu, q, masks, *_ = make_step(dtype, D, 16, 4, ctx, new, 16, seed=87, pad=0)
    lens_t, cu_t, outs = _i32(lens), _i32(cu), [torch.empty_like(q) for _ in range(3)]
    need = fk.fp8kv_tree_workspace_bytes(cache, q.shape[0], 16)
    spaces = [torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") for _ in range(3)]

    def call(i, stream=None):
        return fk.fp8kv_tree_attention(q, cache, cu_t, lens_t, masks, out=outs[i], workspace=spaces[i], stream=stream)

    want = call(0).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i, s in enumerate(streams):
            call(i, s)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(2)
    for shorter in ([n - min(c, 16 * (b % 5)) for b, (n, c) in enumerate(zip(lens, ctx))], [n if b % 2 else m + 7
                                                                                           for b, (n, m) in enumerate(zip(lens, new))]):
        lens_t.copy_(_i32(shorter))
        graph.replay()
        assert torch.equal(outs[2], call(0))
    assert fk.fp8kv_get_device_error() == 0


@pytest.mark.parametrize("down", [-100, -60, 90])
@pytest.mark.parametrize("D,nodes,kernel", [(128, 2, "warp_mma"), (128, 9, "warp_mma"), (128, 40, "tensor_cores"), (64, 60, "warp_mma")])
def test_value_scales_far_from_one(D, nodes, kernel, down):
    cache, lens, cu, q, masks, seen, pos, _ = make_step("k8v8", D, 4, 2, [300, 0, 41], [nodes, 1, nodes], 16, seed=89)
    cache.v_scale.mul_(2.0 ** down)
    cache.v_scale.view(-1)[::7] = 0
    out = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, kernel=kernel, out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == 0
    want = tree_definition(q, cache_values(cache, lens), cu, lens, seen, pos, 0, 0, 1 / math.sqrt(D))
    check(out, cache, want, slice(0, cu[-1]), kernel)
