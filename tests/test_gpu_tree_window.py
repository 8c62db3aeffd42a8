"""Trees deeper than a model's sliding window: the masks of fp8kv_tree_tables under a
window against a plain walk, and attention with them against causal chunk attention
under the same window."""
import random

import numpy as np
import pytest
import torch

import fp8_quantized_kv_gb300 as fk
from test_gpu_chunk import _i32, cache_values, make_cache
from test_gpu_tree import FORMS, ancestors, bits_of, random_tree, run_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_device_error():
    fk.fp8kv_get_device_error(clear=True)
    yield


@pytest.mark.parametrize("nodes,words,chain,pad", [([1], 1, 0, 0), ([0, 5, 0, 32, 1], 1, 9, 2), ([33, 64, 7], 2, 64, 0),
                                                   ([1024, 513], 32, 1024, 5), ([3] * 700, 1, 2, 40)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 0), (7, 3), (40, 200), (2000, 0), ((1 << 31) - 1, (1 << 31) - 1)])
def test_tables(nodes, words, chain, pad, window, sinks):
    """An ancestor at position a is seen from position p if a > p - window or a < sinks;
    contexts of nothing, so that nodes themselves are first tokens, and longer ones."""
    r = random.Random(len(nodes) + window % 97)
    trees = [random_tree(r, n, chain) for n in nodes]
    ctx = [r.choice([0, 1, 190, 5000]) for _ in nodes]
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(int).tolist()
    seen, at = [], []
    for c, t in zip(ctx, trees):
        depth = []
        for p in t:
            depth.append(depth[p] + 1 if p >= 0 else 0)
        for i in range(len(t)):
            at.append(c + depth[i])
            seen.append([a for a in ancestors(t, i) if c + depth[a] > at[-1] - window or c + depth[a] < sinks])
    parents, lens = [p for t in trees for p in t] + [77] * pad, [c + n for c, n in zip(ctx, nodes)]
    masks, pos = fk.fp8kv_tree_tables(_i32(parents), _i32(cu), _i32(lens), 32 * words, window=window, sinks=sinks)
    assert fk.fp8kv_get_device_error() == 0
    assert torch.equal(masks, bits_of(seen + [[]] * pad, words)) and pos.tolist() == at + [-1] * pad
    if window > max(nodes):
        plain, _ = fk.fp8kv_tree_tables(_i32(parents), _i32(cu), _i32(lens), 32 * words)
        assert torch.equal(masks, plain)


@pytest.mark.parametrize("kernel", ["warp_mma", "tensor_cores"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (20, 0), (70, 5), (100, 260)])
def test_chain_under_a_window(kernel, window, sinks):
    """A tree that is one chain, deeper than the window, sees what causal chunk attention
    sees under that window: each row is the definition's up to the rounding of its weights
    (2^-11 of max |v| beside e4m3 values, relative to a reference that may differ between
    the calls; fp32 sums add far less than 1e-5)."""
    n = 90
    cache = make_cache("k8v8", 128, 2, [300, n], 16, seed=16)
    cu, lens = _i32([0, n, 2 * n]), _i32([300, n])
    q = torch.randn(2 * n, 4, 128, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(torch.bfloat16)
    masks, pos = fk.fp8kv_tree_tables(_i32(list(range(-1, n - 1)) * 2), cu, lens, n, window=window, sinks=sinks)
    most = max(float(v.abs().max()) for _, v in cache_values(cache, [300, n]))
    for splits in (1, 3):
        kw = dict(window=window, sinks=sinks, num_splits=splits, out_dtype=torch.float32, kernel=kernel)
        a = fk.fp8kv_tree_attention(q, cache, cu, lens, masks, pos=pos, **kw)
        b = fk.fp8kv_chunk_attention(q, cache, cu, lens, **kw)
        assert fk.fp8kv_get_device_error() == 0 and (a - b).abs().max().item() <= 2 * 2.0 ** -11 * most + 1e-5


@pytest.mark.parametrize("dtype,D,kernel", FORMS)
@pytest.mark.parametrize("splits", [0, 5])
def test_wide_tree_under_a_small_window(dtype, D, kernel, splits):
    """A window far smaller than the tree: its nodes are most of the keys, and the shares
    divide them."""
    run_case(dtype, D, 4, 2, [200, 50], [300, 9], 16, seed=21, window=32, sinks=3, kernel=kernel, splits=splits)
