"""Trees of drafted tokens: masks and positions (fp8kv_tree_tables), attention of
the nodes over the cache (fp8kv_tree_attention), acceptance with the move of
cache rows (fp8kv_tree_accept), and whole verification steps, against plain
walks of the trees and the definition in 64 bits.  The attention's tolerance is
derived in test_gpu_chunk (the same roundings)."""
import math
import random

import numpy as np
import pytest
import torch

import fp8_quantized_kv_gb300 as fk
from test_gpu_chunk import _i32, cache_values, check, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_device_error():
    fk.fp8kv_get_device_error(clear=True)
    yield


def random_tree(r, n, chain=0):
    """Parents of n nodes: a chain first, then anything above."""
    return [-1 if i == 0 else i - 1 if i < chain else r.randrange(i) for i in range(n)]


def ancestors(parents, i):
    """Node i and those above it."""
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out


def bits_of(rows, words):
    """Lists of node numbers as [rows, words] int32."""
    m = np.zeros((len(rows), words), np.uint32)
    for r, nodes in enumerate(rows):
        for i in nodes:
            m[r, i // 32] |= np.uint32(1 << (i % 32))
    return torch.from_numpy(m.view(np.int32)).cuda()


def tree_definition(q, kv, cu, lens, seen_nodes, pos, window, sinks, sm):
    """As test_gpu_chunk.definition: node i of sequence b sees its context (under a
    window a part of it), the nodes seen_nodes[row] and itself."""
    rows, Hq, D = q.shape
    q = q.double().cpu()
    o, pv = torch.zeros(rows, Hq, D, dtype=torch.float64), torch.zeros(rows, Hq, D, dtype=torch.float64)
    qk, qs, keys, vmax = torch.zeros(rows, Hq), torch.zeros(rows, Hq), torch.zeros(rows), torch.zeros(rows, Hq)
    for b, (k, v) in enumerate(kv):
        n = cu[b + 1] - cu[b]
        ctx = lens[b] - n
        G = Hq // k.shape[1]
        for i in range(n):
            r = cu[b] + i
            if ctx + i < 0:
                continue
            j = torch.arange(max(0, ctx))
            if window:
                p = min(max(pos[r], ctx), lens[b] - 1)
                j = j[(j > p - window) | (j < sinks)]
            nodes = sorted({x for x in seen_nodes[r] if x < n and ctx + x >= 0} | {i})
            j = torch.cat([j, torch.tensor([ctx + x for x in nodes], dtype=torch.long)])
            kk, vv = k[j].repeat_interleave(G, 1), v[j].repeat_interleave(G, 1)
            s = torch.einsum("hd,khd->hk", q[r], kk) * sm
            w = torch.softmax(s, -1)
            o[r] = torch.einsum("hk,khd->hd", w, vv)
            pv[r] = torch.einsum("hk,khd->hd", w, vv.abs())
            qk[r] = (torch.einsum("hd,khd->hk", q[r].abs(), kk.abs()) * abs(sm)).amax(-1)
            qs[r] = q[r].abs().amax(-1) * kk.abs().sum(-1).amax(0) * abs(sm)
            keys[r], vmax[r] = len(j), vv.abs().amax((0, 2))
    return o, pv, qk, qs, keys, vmax


def make_step(dtype, D, Hq, Hkv, ctx, nodes, page, seed, spread=0.0, pad=3, words=None, any_mask=False):
    lens = [c + n for c, n in zip(ctx, nodes)]
    cache = make_cache(dtype, D, Hkv, lens, page, seed, spread=spread)
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(int).tolist()
    r = random.Random(seed)
    seen, pos = [], []
    for c, n in zip(ctx, nodes):
        t = random_tree(r, n, r.randint(0, 4))
        for i in range(n):
            up = ancestors(t, i)
            pos.append(c + len(up) - 1)
            # any mask: nodes in front and behind, its own bit or not, bits past the tree
            seen.append([x for x in range(32 * (words or 1)) if r.random() < 0.3] if any_mask else up)
    words = words or max(1, -(-max(nodes) // 32))
    masks = bits_of(seen + [[0, 1]] * pad, words)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn(cu[-1] + pad, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    return cache, lens, cu, q, masks, seen, pos, _i32(pos + [-1] * pad)


def run_case(dtype, D, Hq, Hkv, ctx, nodes, page, seed, window=0, sinks=0, kernel="auto", splits=0, out_dtype=torch.float32,
             spread=0.0, pad=3, **kw):
    cache, lens, cu, q, masks, seen, pos, pos_t = make_step(dtype, D, Hq, Hkv, ctx, nodes, page, seed, spread, pad, **kw)
    out = torch.full((cu[-1] + pad, Hq, D), 5.0, dtype=out_dtype, device="cuda")
    fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, pos=pos_t if window else None, window=window, sinks=sinks,
                            num_splits=splits, out=out, kernel=kernel)
    assert fk.fp8kv_get_device_error() == 0
    want = tree_definition(q, cache_values(cache, lens), cu, lens, seen, pos, window, sinks, 1 / math.sqrt(D))
    check(out, cache, want, slice(0, cu[-1]), kernel)
    assert bool((out[cu[-1]:] == 5.0).all()), "rows behind the last tree changed"


# ----------------------------------------------------- masks and positions --
def want_tables(parents, cu, lens, rows, words):
    seen, pos = [[] for _ in range(rows)], [-1] * rows
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        if n > 32 * words or lens[b] < n:
            continue
        t = [p if -1 <= p < i else -1 for i, p in enumerate(parents[cu[b]:cu[b + 1]])]
        for i in range(n):
            seen[cu[b] + i] = ancestors(t, i)
            pos[cu[b] + i] = lens[b] - n + len(seen[cu[b] + i]) - 1
    return bits_of(seen, words), _i32(pos)


@pytest.mark.parametrize("nodes,words,chain,pad", [
    ([1], 1, 0, 0), ([0, 5, 0, 32, 1], 1, 3, 2), ([33, 64, 7], 2, 64, 0), ([200, 96, 1, 0, 160], 7, 9, 1100),
    ([1024, 1000], 32, 1024, 5), ([1024, 513], 32, 4, 0), ([3] * 700, 1, 2, 40)])
def test_tables(nodes, words, chain, pad):
    """Trees of nothing to 1,024 nodes, chains of all of them, more words than a tree needs, padding rows."""
    r = random.Random(len(nodes) + words)
    parents = [p for n in nodes for p in random_tree(r, n, chain)] + [77] * pad
    lens = [n + r.randrange(5000) for n in nodes]
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(int).tolist()
    masks, pos = fk.fp8kv_tree_tables(_i32(parents), _i32(cu), _i32(lens), 32 * words - 1)
    assert fk.fp8kv_get_device_error() == 0
    want = want_tables(parents, cu, lens, len(parents), words)
    assert torch.equal(masks, want[0]) and torch.equal(pos, want[1])


def test_tables_reports():
    """Parents that do not come before their node count as none; a tree with more
    nodes than bits or than its sequence has tokens gets nothing; offsets that
    decrease or pass the rows leave theirs."""
    lens, cu = [10, 20], [0, 4, 8]
    for bad in ([-1, 1, 0, 2], [-1, 0, -2, 1], [-1, 0, 1 << 30, 2], [-1, 0, 1, 3]):
        parents = [-1, 0, 0, 1] + bad
        masks, pos = fk.fp8kv_tree_tables(_i32(parents), _i32(cu), _i32(lens), 32)
        assert fk.fp8kv_get_device_error() == fk.DEVERR_BAD_TREE
        want = want_tables(parents, cu, lens, 8, 1)
        assert torch.equal(masks, want[0]) and torch.equal(pos, want[1])
    parents = random_tree(random.Random(1), 33) + random_tree(random.Random(2), 6)
    for lens in ([40, 6], [33, 5], [33, -4]):
        masks, pos = fk.fp8kv_tree_tables(_i32(parents), _i32([0, 33, 39]), _i32(lens), 32)
        assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
        want = want_tables(parents, [0, 33, 39], lens, 39, 1)
        assert torch.equal(masks, want[0]) and torch.equal(pos, want[1])
    for cu, kept in (([0, 6, 3], [0, 3]), ([0, 3, 12], [0, 3]), ([-2, 3, 6], [3, 6])):
        masks, pos = torch.full((8, 1), 9, dtype=torch.int32, device="cuda"), torch.full((8,), 9, dtype=torch.int32, device="cuda")
        fk.fp8kv_tree_tables(_i32([-1, 0, 1, -1, 0, 1, -1, 0]), _i32(cu), _i32([50, 50]), 32, masks=masks, pos=pos)
        assert fk.fp8kv_get_device_error() & fk.DEVERR_SEQ_TOO_LONG
        a, b = kept
        n = 6 if cu[1] == 6 else 3                                       # nodes of the tree that is fine
        assert masks[a:b, 0].tolist() == [1, 3, 7] and pos[a:b].tolist() == [50 - n, 51 - n, 52 - n]


def test_tables_overwrite_what_was_there():
    masks, pos = torch.full((40, 3), -1, dtype=torch.int32, device="cuda"), torch.full((40,), 5, dtype=torch.int32, device="cuda")
    fk.fp8kv_tree_tables(_i32([-1] + [0] * 36 + [4] * 3), _i32([0, 37]), _i32([100]), 96, masks=masks, pos=pos)
    want = want_tables([-1] + [0] * 36 + [-1] * 3, [0, 37], [100], 40, 3)
    assert fk.fp8kv_get_device_error() == 0 and torch.equal(masks, want[0]) and torch.equal(pos, want[1])


# ---------------------------------------------------------------- attention --
FORMS = [("k8v8", 128, "warp_mma"), ("k16v8", 128, "warp_mma"), ("k8v16", 64, "warp_mma"), ("k16v16", 64, "warp_mma"),
         ("mxk8v8", 128, "warp_mma"), ("k8v8", 64, "warp_mma"), ("k8v8", 128, "tensor_cores"), ("k16v8", 128, "tensor_cores"),
         ("k8v16", 128, "tensor_cores"), ("k16v16", 128, "tensor_cores")]


@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("dtype,D,kernel", FORMS)
def test_types(dtype, D, kernel, page):
    """Trees of none to 70 nodes behind contexts that end inside tiles and pages."""
    run_case(dtype, D, 6, 2, [0, 37, 130, 64, 700], [67, 0, 41, 1, 70], page, seed=1, kernel=kernel)


@pytest.mark.parametrize("dtype,D,kernel", FORMS)
@pytest.mark.parametrize("nodes", [1, 2, 3, 5])
def test_few_nodes(dtype, D, kernel, nodes):
    """Tiles of 8 and 16 rows; one sequence holds the nodes only."""
    run_case(dtype, D, 8, 2, [0, 15, 200, 63, 64], [nodes] * 5, 16, seed=2, kernel=kernel)


@pytest.mark.parametrize("dtype,D,kernel", FORMS)
@pytest.mark.parametrize("words", [1, 2, 3])
def test_any_mask(dtype, D, kernel, words):
    """Bits in any order: later nodes, one's own missing, nodes that are not there."""
    for nodes in ([33, 70, 3], [2, 1, 4]):
        if max(nodes) <= 32 * words:
            run_case(dtype, D, 4, 2, [70, 5, 129], nodes, 16, seed=5 + words, kernel=kernel, words=words, any_mask=True)


@pytest.mark.parametrize("kernel", ["warp_mma", "tensor_cores"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 1), (10, 2), (16, 1), (11, 1)])
def test_groups(Hq, Hkv, kernel):
    for nodes in ([5, 1, 40], [1, 1, 1]):
        run_case("k8v8", 128, Hq, Hkv, [70, 3, 0], nodes, 32, seed=3, kernel=kernel)


@pytest.mark.parametrize("dtype,D,kernel", FORMS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 1), (64, 0), (100, 70), (10000, 3)])
def test_windows(dtype, D, kernel, window, sinks):
    """Windows that end inside the context, at its end and before it."""
    for nodes in ([9, 40, 20], [2, 1, 3]):
        run_case(dtype, D, 4, 2, [300, 63, 0], nodes, 16, seed=7, window=window, sinks=sinks, kernel=kernel)


@pytest.mark.parametrize("dtype,D,kernel", FORMS)
@pytest.mark.parametrize("splits", [2, 7])
def test_splits(dtype, D, kernel, splits):
    run_case(dtype, D, 4, 1, [900, 100, 1], [30, 6, 64], 16, seed=8, splits=splits, kernel=kernel, spread=5.0)
    run_case(dtype, D, 4, 1, [900, 100, 1], [2, 1, 2], 0, seed=9, splits=splits, kernel=kernel, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("kernel", ["warp_mma", "tensor_cores"])
def test_widest(kernel):
    """A tree of 1,024 nodes, and one of 1,000 in the same call."""
    run_case("k8v8", 128, 2, 1, [77, 0], [1024, 1000], 16, seed=10, kernel=kernel, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("dtype,D,kernel", FORMS)
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_unseen_values(dtype, D, kernel, what):
    """A node whose key or value is not finite: those that do not see it are as if
    it were not there, those that do are not finite.  (A key that is infinite may
    score -inf, which weighs nothing: its rows are finite where it does.)"""
    for Hq, n in ((2, 3), (4, 40)):
        cache, lens, cu, q, masks, seen, pos, _ = make_step(dtype, D, Hq, 1, [130], [n], 16, seed=11, pad=0)
        kv = cache_values(cache, lens)
        want = tree_definition(q, kv, cu, lens, seen, pos, 0, 0, 1 / math.sqrt(D))
        bad = 1
        rows = torch.tensor([bad not in s for s in seen])
        page, off = int(cache.page_table[0, (130 + bad) // 16]), (130 + bad) % 16
        for side in ("k", "v"):
            t, sc = getattr(cache, side), getattr(cache, side + "_scale")
            minus = side == "k" and what == float("inf")
            kept = t[page, :, off].clone()
            t[page, :, off, 3] = 0x7F if t.dtype == torch.uint8 else what
            out = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, out_dtype=torch.float32, kernel=kernel)
            assert fk.fp8kv_get_device_error() == 0
            check(out, cache, want, rows, kernel)
            assert (minus and t.dtype != torch.uint8) or not bool(torch.isfinite(out[~rows.cuda()]).flatten(1).all(1).any())
            t[page, :, off] = kept
            if sc is not None and sc.dtype == torch.float32:
                kept = sc[page, :, off].clone()
                sc[page, :, off] = what
                out = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, out_dtype=torch.float32, kernel=kernel)
                check(out, cache, want, rows, kernel)
                assert minus or not bool(torch.isfinite(out[~rows.cuda()]).flatten(1).all(1).any())
                sc[page, :, off] = kept


@pytest.mark.parametrize("dtype,D,kernel", FORMS)
def test_nodes_that_are_not_in_the_cache(dtype, D, kernel):
    """Fewer tokens than nodes: the first nodes have no key and get zero rows; a
    tree with more nodes than bits, or of a sequence past the capacity, too."""
    cache = make_cache(dtype, D, 1, [50, 40, 60], 16, seed=12)
    lens, nodes = [5, 40, 60], [9, 33, 20]
    cu = [0, 9, 42, 62]
    seen = [list(range(i + 1)) for n in nodes for i in range(n)]
    q = torch.randn(62, 2, D, device="cuda").to(torch.bfloat16)
    out = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), bits_of([[x for x in s if x < 32] for s in seen], 1),
                                  out_dtype=torch.float32, kernel=kernel)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
    assert not bool(out[:4].any()) and not bool(out[9:42].any())
    want = tree_definition(q, cache_values(cache, [5, 40, 60]), cu, lens, seen, [0] * 62, 0, 0, 1 / math.sqrt(D))
    check(out, cache, want, torch.tensor([4 <= r < 9 or r >= 42 for r in range(62)]), kernel)
    out = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32([5, -1, cache.capacity + 1]), bits_of(seen, 2), kernel=kernel)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG and not bool(out[9:].any())


@pytest.mark.parametrize("kernel", ["warp_mma", "tensor_cores"])
@pytest.mark.parametrize("splits", [1, 4])
def test_bad_offsets_leave_their_rows(kernel, splits):
    cache, lens, cu, q, masks, *_ = make_step("k8v8", 128, 4, 1, [300, 300], [6, 6], 16, seed=13, pad=0)
    good = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, num_splits=splits, kernel=kernel)
    assert fk.fp8kv_get_device_error() == 0
    for cu in ([0, 6, 13], [0, 6, 2]):
        out = torch.full_like(good, 3.0)
        fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, num_splits=splits, kernel=kernel, out=out)
        assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
        assert bool((out[6:] == 3.0).all()) and bool(((out[:6] == good[:6]) | ((out[:6] == 3.0) if cu[2] < cu[1] else False)).all())


@pytest.mark.parametrize("kernel", ["warp_mma", "tensor_cores"])
def test_pages_behind_the_window_may_be_gone(kernel):
    """Pages that hold no first token and end before ctx - window + 1 are not looked at."""
    ctx, n, window, sinks = 500, 12, 70, 4
    for nodes in (n, 2):
        cache, lens, cu, q, masks, seen, pos, pos_t = make_step("k8v8", 128, 4, 1, [ctx], [nodes], 16, seed=14, pad=0)
        kv = cache_values(cache, lens)
        cache.page_table[0, 1:(ctx - window + 1) // 16] = 1 << 20
        out = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, pos=pos_t, window=window, sinks=sinks,
                                      out_dtype=torch.float32, kernel=kernel)
        assert fk.fp8kv_get_device_error() == 0
        check(out, cache, tree_definition(q, kv, cu, lens, seen, pos, window, sinks, 1 / math.sqrt(128)), slice(0, nodes), kernel)


def test_positions_outside_the_sequence_count_as_the_nearest():
    cache, lens, cu, q, masks, seen, pos, _ = make_step("k8v8", 128, 2, 1, [200], [10], 16, seed=15, pad=0)
    pos = [-(1 << 31), (1 << 31) - 1, 0, 199, 200, 209, 210, 205, -1, 1 << 30]
    out = fk.fp8kv_tree_attention(q, cache, _i32(cu), _i32(lens), masks, pos=_i32(pos), window=30, sinks=2, out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == 0
    check(out, cache, tree_definition(q, cache_values(cache, lens), cu, lens, seen, pos, 30, 2, 1 / math.sqrt(128)), slice(0, 10), "auto")


def test_chain_is_causal():
    """A tree that is one chain sees what causal chunk attention sees."""
    for dtype, D, n in (("k8v8", 128, 90), ("k16v16", 64, 90), ("k8v8", 128, 2)):
        cache = make_cache(dtype, D, 2, [300, n], 16, seed=16)
        cu, lens = _i32([0, n, 2 * n]), _i32([300, n])
        q = torch.randn(2 * n, 4, D, device="cuda").to(torch.bfloat16)
        masks, pos = fk.fp8kv_tree_tables(_i32(list(range(-1, n - 1)) * 2), cu, lens, n)
        assert pos.tolist() == list(range(300 - n, 300)) + list(range(n))
        a = fk.fp8kv_tree_attention(q, cache, cu, lens, masks, out_dtype=torch.float32)
        b = fk.fp8kv_chunk_attention(q, cache, cu, lens, out_dtype=torch.float32)
        # Each is the definition's row up to the rounding of its weights: u sum p |v| <= u max |v|,
        # u = 2^-11 beside e4m3 values and 2^-8 beside bf16 ones, relative to a reference that
        # depends on the share of keys (the two calls may split them differently).  Two rows
        # differ by twice that; fp32 sums add far less than the 1e-5 here.
        u = 2.0 ** (-8 if cache.v.dtype == torch.bfloat16 else -11)
        most = max(float(v.abs().max()) for _, v in cache_values(cache, [300, n]))
        assert fk.fp8kv_get_device_error() == 0 and (a - b).abs().max().item() <= 2 * u * most + 1e-5
        c = fk.fp8kv_tree_attention(q, cache, cu, lens, masks, out_dtype=torch.float32, num_splits=1)
        b = fk.fp8kv_chunk_attention(q, cache, cu, lens, out_dtype=torch.float32, num_splits=1)
        # one share each: the same scores and weights, only the order of rescalings can differ
        assert (c - b).abs().max().item() <= 1e-5


def test_graph_and_stream():
    """Captured and replayed with other trees in the same buffers; on a stream of its own."""
    cache, lens, cu, q, masks, seen, pos, _ = make_step("k8v8", 128, 8, 2, [900, 500], [40, 22], 16, seed=17, pad=0)
    parents = torch.zeros(62, dtype=torch.int32, device="cuda")
    cu_t, lens_t, out = _i32(cu), _i32(lens), torch.zeros(62, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, fk.fp8kv_tree_workspace_bytes(cache, 62, 8, num_splits=3)), dtype=torch.uint8, device="cuda")
    m, p = torch.empty(62, 2, dtype=torch.int32, device="cuda"), torch.empty(62, dtype=torch.int32, device="cuda")

    def step():
        fk.fp8kv_tree_tables(parents, cu_t, lens_t, 64, masks=m, pos=p)
        fk.fp8kv_tree_attention(q, cache, cu_t, lens_t, m, out=out, workspace=ws, num_splits=3)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_BAD_TREE             # (all zeros: node 0 under itself)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    r = random.Random(4)
    for _ in range(3):
        parents.copy_(_i32(random_tree(r, 40) + random_tree(r, 22)))
        graph.replay()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    again = fk.fp8kv_tree_attention(q, cache, cu_t, lens_t, m, num_splits=3, stream=other)
    other.synchronize()
    assert torch.equal(again, got) and fk.fp8kv_get_device_error() == 0


# --------------------------------------------------------------- acceptance --
def walk(parents, tokens, choices, most):
    path = [0] if parents else []
    while path and len(path) < most:
        hits = [i for i, p in enumerate(parents) if p == path[-1] and 0 <= p < i and tokens[i] == choices[p]]
        if not hits:
            break
        path.append(hits[0])
    return path


def cache_copy(cache):
    return [None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]


def check_accept(caches, before, parents, tokens, choices, cu, lens, most, got):
    paths = [walk(parents[a:b], tokens[a:b], choices[a:b], most) for a, b in zip(cu, cu[1:])]
    assert got["path"].tolist() == [p + [-1] * (most - len(p)) for p in paths]
    assert got["accepted"].tolist() == [len(p) for p in paths]
    assert got["next_tokens"].tolist() == [choices[a + p[-1]] if p else -1 for a, p in zip(cu, paths)]
    assert got["lens"].tolist() == [n - (b - a) + len(p) for n, a, b, p in zip(lens, cu, cu[1:], paths)]
    for cache, old in zip(caches, before):
        span = cache.page_size or cache.max_tokens
        for t, o in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), old):
            if t is None:
                continue
            want = o.clone()
            for b, p in enumerate(paths):
                ctx = lens[b] - (cu[b + 1] - cu[b])
                for k, i in enumerate(p):
                    at = [(int(cache.page_table[b, x // span]) if cache.page_size else b, x % span) for x in (ctx + i, ctx + k)]
                    want[at[1][0], :, at[1][1]] = o[at[0][0], :, at[0][1]]
            assert torch.equal(t.view(torch.uint8), want.view(torch.uint8))
    return paths


@pytest.mark.parametrize("page", [0, 16, 32])
@pytest.mark.parametrize("dtype,D", [("k8v8", 128), ("k16v8", 64), ("k8v16", 128), ("k16v16", 64), ("mxk8v8", 128)])
@pytest.mark.parametrize("nodes,most", [([1, 0, 9, 2], 4), ([64, 40, 30, 12], 30), ([200, 3, 0, 1], 200)])
def test_accept(dtype, D, page, nodes, most):
    """Paths of every kind: the whole chain, out of it, cut by max_path; several
    layers; rows that move over pages; ties between children."""
    r = random.Random(len(dtype) + most)
    ctx = [5, 0, 37, 16]
    lens = [c + n for c, n in zip(ctx, nodes)]
    caches = [make_cache(dtype, D, 3, lens, page, seed=20 + i, poison=False) for i in range(2)]
    before = [cache_copy(c) for c in caches]
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(int).tolist()
    parents = [p for n in nodes for p in random_tree(r, n, min(n, 5) if n < 100 else n)]
    tokens = [r.randrange(3) for _ in parents]                          # (siblings share tokens)
    choices = [r.randrange(3) for _ in parents]
    tokens[cu[0]:cu[1]] = choices[cu[0]:cu[1]] = [7 << 40] * nodes[0]   # every child fits; tokens past 32 bits
    i64 = dict(dtype=torch.int64, device="cuda")
    got = fk.fp8kv_tree_accept(caches, _i32(parents), torch.tensor(tokens, **i64), torch.tensor(choices, **i64), _i32(cu), _i32(lens), most)
    assert fk.fp8kv_get_device_error() == 0
    check_accept(caches, before, parents, tokens, choices, cu, lens, most, got)


def test_accept_many_layers_and_none():
    """More layers than one launch takes; no layer at all; a path along every second node."""
    n = 61
    parents = [-1, 0] + [i - 2 for i in range(2, n)]
    tokens = [i % 2 for i in range(n)]                                  # the even nodes are accepted
    choices, lens, cu = [0] * n, [n + 3], [0, n]
    parents[2] = 0
    caches = [make_cache("k8v8", 64, 1, lens, 16, seed=30 + i, poison=False) for i in range(63)]
    before = [cache_copy(c) for c in caches]
    i64 = dict(dtype=torch.int64, device="cuda")
    args = (_i32(parents), torch.tensor(tokens, **i64), torch.tensor(choices, **i64), _i32(cu), _i32(lens), 40)
    got = fk.fp8kv_tree_accept(caches, *args)
    assert fk.fp8kv_get_device_error() == 0
    paths = check_accept(caches, before, parents, tokens, choices, cu, lens, 40, got)
    assert paths[0] == list(range(0, n, 2))
    none = fk.fp8kv_tree_accept([], *args)
    assert all(torch.equal(none[k], got[k]) for k in got)


def test_accept_reports():
    """Trees that are refused accept nothing and move nothing, beside one that is fine."""
    i64 = dict(dtype=torch.int64, device="cuda")
    lens, cu = [40, 44], [0, 4, 8]
    cache = make_cache("k8v8", 128, 2, lens, 16, seed=31, poison=False)
    before = cache_copy(cache)

    def call(parents, cu, lens, tokens=(1,) * 8):
        for t, o in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
            t.copy_(o)
        return fk.fp8kv_tree_accept([cache], _i32(parents), torch.tensor(tokens, **i64), torch.ones(8, **i64), _i32(cu), _i32(lens), 8)

    got = call([-1, 0, 1, 3, -1, 0, -5, 6], cu, lens)                   # parents that do not come before their node
    assert fk.fp8kv_get_device_error() == fk.DEVERR_BAD_TREE
    assert got["accepted"].tolist() == [3, 2] and got["path"][1].tolist() == [0, 1] + [-1] * 6
    for bad_cu, bad_lens in (([0, 4, 2], lens), ([0, 4, 9], lens), (cu, [40, 3]), (cu, [40, -2])):
        got = call([-1, 0, 0, 2] * 2, bad_cu, bad_lens, (1, 2, 1, 1, 1, 2, 1, 1))
        assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
        assert got["accepted"].tolist() == [3, 0] and got["lens"].tolist() == [39, bad_lens[1]] and int(got["next_tokens"][1]) == -1
        check_accept([cache], [before], [-1, 0, 0, 2], [1, 2, 1, 1], [1] * 4, [0, 4], lens[:1], 8, {k: v[:1] for k, v in got.items()})
    got = call([-1, 0, 0, 2] * 2, cu, [40, cache.capacity + 1], (1, 2, 1, 1) * 2)         # walks, but moves nothing
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG and got["accepted"].tolist() == [3, 3]
    cache.page_table[1, 42 // 16] = -1
    got = call([-1, 0, 0, 2] * 2, cu, lens, (1, 2, 1, 1) * 2)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_BAD_PAGE and got["accepted"].tolist() == [3, 3]


# -------------------------------------------------------------- whole steps --
@pytest.mark.parametrize("dtype,page,window", [("k8v8", 16, 0), ("k16v8", 0, 0), ("mxk8v8", 32, 0), ("k8v8", 16, 50), ("k16v16", 64, 50)])
def test_verification_steps(dtype, page, window):
    """Prompts, then steps that draft trees, attend, accept and keep: after every
    step the kept cache is the one of a run that appended the accepted tokens alone,
    and the next step's attention is the definition's over it."""
    B, Hq, Hkv, D, cap = 3, 4, 2, 128, 192
    r, g = random.Random(page + window), torch.Generator(device="cuda").manual_seed(5)
    i64 = dict(dtype=torch.int64, device="cuda")

    def new_cache():
        if not page:
            return fk.Fp8KVCache.contiguous(B, Hkv, D, cap, dtype), None, None
        c = fk.Fp8KVCache.paged(torch.full((B, cap // page), -1, dtype=torch.int32), 3 * cap // page + 60, Hkv, D, page, dtype)
        return c, torch.randperm(c.num_pages, generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda(), _i32([0])

    cache, free, head = new_cache()
    plain, plain_free, plain_head = new_cache()
    cos, sin = fk.fp8kv_rope_tables(cap, D)

    def rows(n):
        return [torch.randn(n, h, D, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]

    def append(c, fr, hd, lens, new, q, k, v, pos=None):
        t = fk.fp8kv_build_tables(c, lens, _i32(new), sum(new), fr, hd)
        q = fk.fp8kv_rope_append(c, q, k, v, t["pos"] if pos is None else pos(t), t["slots"], cos, sin)
        return q, t

    lens = plain_lens = _i32([0, 0, 0])
    first = [40, 1, 17]
    qkv = rows(sum(first))
    _, t = append(cache, free, head, lens, first, *qkv)
    _, u = append(plain, plain_free, plain_head, plain_lens, first, *qkv)
    lens, head, plain_lens, plain_head = t["seq_lens"], t["free_head"], u["seq_lens"], u["free_head"]
    for step in range(4):
        nodes = [r.randint(1, 12), 0 if step == 1 else r.randint(1, 40), r.randint(3, 33)]
        parents = [p for n in nodes for p in random_tree(r, n, 3)]
        cu = np.concatenate([[0], np.cumsum(nodes)]).astype(int).tolist()
        ctx = lens.tolist()
        tables = {}

        def positions(t):
            tables["masks"], tables["pos"] = fk.fp8kv_tree_tables(_i32(parents), t["cu_new"], t["seq_lens"], 64)
            return tables["pos"]
        qkv = rows(cu[-1])
        q, t = append(cache, free, head, lens, nodes, *qkv, pos=positions)
        out = fk.fp8kv_tree_attention(q, cache, t["cu_new"], t["seq_lens"], tables["masks"], pos=tables["pos"], window=window, sinks=2,
                                      out_dtype=torch.float32)
        assert fk.fp8kv_get_device_error() == 0
        full = t["seq_lens"].tolist()
        seen = [ancestors(parents[a:b], i) for a, b in zip(cu, cu[1:]) for i in range(b - a)]
        want = tree_definition(q, cache_values(cache, full), cu, full, seen, tables["pos"].tolist(), window, 2, 1 / math.sqrt(D))
        check(out, cache, want, slice(0, cu[-1]), "auto")
        tokens, choices = [r.randrange(2) for _ in parents], [r.randrange(2) for _ in parents]
        got = fk.fp8kv_tree_accept([cache], _i32(parents), torch.tensor(tokens, **i64), torch.tensor(choices, **i64), t["cu_new"],
                                   t["seq_lens"], 9)
        paths = [walk(parents[a:b], tokens[a:b], choices[a:b], 9) for a, b in zip(cu, cu[1:])]
        assert got["path"].tolist() == [p + [-1] * (9 - len(p)) for p in paths]
        # the accepted tokens alone, at the same positions
        keep = [a + i for a, p in zip(cu, paths) for i in p]
        _, u = append(plain, plain_free, plain_head, plain_lens, [len(p) for p in paths], *[x[keep] for x in qkv])
        lens, plain_lens, plain_head = got["lens"], u["seq_lens"], u["free_head"]
        assert fk.fp8kv_get_device_error() == 0 and torch.equal(lens, plain_lens)
        for (k, v), (k2, v2) in zip(cache_values(cache, lens.tolist()), cache_values(plain, lens.tolist())):
            assert torch.equal(k, k2) and torch.equal(v, v2)
        if page:      # pages behind the new lengths go back to the free list
            back = [int(cache.page_table[b, i]) for b in range(B) for i in range(-(-int(lens[b]) // page), -(-full[b] // page))]
            rest = free[int(t["free_head"]):].tolist()
            free, head = _i32(back + rest), _i32([0])
        assert ctx == [f - n for f, n in zip(full, nodes)]
