"""Page tables and slot maps (fp8kv_build_tables), rotary tables
(fp8kv_rope_tables) and the rotating append (fp8kv_rope_append) on the GPU
against plain implementations in whole numbers and 64 bits.

Tolerances.  Tables and slots are whole numbers: equal.  A rotary table entry
is the fp32 sine or cosine of an angle in [-pi/4, pi/4] that carries the
rounding of a 32-bit phase (2^-33 of a turn), of its conversion and scaling to
fp32 (2 x 2^-24 pi/4) and sine's own error (under 2 ulp of at most 1, 2^-23),
times the amplitude with one more rounding: under 2^-22 times the amplitude.
A rotated element a cos - b sin carries three fp32 roundings (3 x 2^-24 of
|a| + |b|) and, for queries and bf16 keys, one bf16 rounding (2^-8 of the
value).  Codes: the same fp32 operations in numpy give the same bits."""
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


# ------------------------------------------------------------------ tables --
def _plain_tables(cached, new, page, free, head, table, rows, num_pages):
    """The definition, sequence by sequence."""
    table = [list(r) for r in table]
    seq_idx, pos, slots, cu, lens = [], [], [], [0], []
    for b, (c, n) in enumerate(zip(cached, new)):
        first, last = -(-c // page), -(-(c + n) // page)
        for i in range(first, last):
            table[b][i] = free[head]
            head += 1
        for t in range(c, c + n):
            seq_idx.append(b)
            pos.append(t)
            slots.append(table[b][t // page] * page + t % page)
        cu.append(cu[-1] + n)
        lens.append(c + n)
    pad = rows - len(pos)
    return table, cu, lens, seq_idx + [-1] * pad, pos + [-1] * pad, slots + [-1] * pad, head


def _paged_state(rng, cached, new, page, extra_pages=7, kv_heads=1, dtype="k8v8", head_dim=64):
    need = [-(-(c + n) // page) for c, n in zip(cached, new)]
    have = [-(-c // page) for c in cached]
    cols, pages = max([1] + need) + 1, sum(need) + extra_pages
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((len(cached), cols), -1, np.int32)
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = perm[at:at + h]
        at += h
    cache = fk.Fp8KVCache.paged(torch.from_numpy(table.copy()), pages, kv_heads, head_dim, page, dtype)
    return cache, table, perm[at:]


LENGTHS = {
    "one": ([0], [1]),
    "one_full_page": ([16], [1]),
    "idle_and_empty": ([0, 5, 64, 0, 31], [0, 0, 3, 40, 1]),
    "page_edges": ([15, 16, 17, 31, 32, 33], [1, 1, 1, 33, 32, 31]),
    "none_new": ([3, 70], [0, 0]),
}


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("lengths", sorted(LENGTHS) + ["random_700"])
def test_tables_paged(page, lengths):
    rng = np.random.default_rng(5)
    if lengths == "random_700":      # several scan rounds, many row blocks, padding behind
        cached, new = rng.integers(0, 200, 700).tolist(), rng.integers(0, 50, 700).tolist()
    else:
        cached, new = LENGTHS[lengths]
    rows, head = sum(new) + 19, 2
    cache, table, free = _paged_state(rng, cached, new, page)
    want = _plain_tables(cached, new, page, free.tolist(), head, table.tolist(), rows, cache.num_pages)
    got = fk.fp8kv_build_tables(cache, _i32(cached), _i32(new), rows, torch.from_numpy(free).cuda(), _i32([head]))
    assert fk.fp8kv_get_device_error() == 0
    assert cache.page_table.tolist() == want[0]
    for name, w in zip(("cu_new", "seq_lens", "seq_idx", "pos", "slots"), want[1:6]):
        assert got[name].tolist() == w, name
    assert got["free_head"].tolist() == [want[6]]


def test_tables_contiguous():
    cached, new = [0, 7, 100], [4, 0, 28]
    cache = fk.Fp8KVCache.contiguous(3, 1, 64, 128)
    got = fk.fp8kv_build_tables(cache, _i32(cached), _i32(new), 40)
    assert fk.fp8kv_get_device_error() == 0
    assert got["cu_new"].tolist() == [0, 4, 4, 32] and got["seq_lens"].tolist() == [4, 7, 128]
    assert got["slots"].tolist() == [0, 1, 2, 3] + [2 * 128 + t for t in range(100, 128)] + [-1] * 8
    assert got["free_head"] is None


def test_tables_large_batch():
    """16384 sequences of one new token each: the largest batch."""
    B, page = 16384, 16
    rng = np.random.default_rng(9)
    cached = rng.integers(0, 40, B)
    cache, table, free = _paged_state(rng, cached.tolist(), [1] * B, page)
    got = fk.fp8kv_build_tables(cache, _i32(cached.tolist()), _i32([1] * B), B, torch.from_numpy(free).cuda(), _i32([0]))
    assert fk.fp8kv_get_device_error() == 0
    fresh = cached % page == 0
    base = np.cumsum(fresh) - fresh
    page_of = np.where(fresh, free[np.minimum(base, len(free) - 1)], table[np.arange(B), cached // page])
    assert np.array_equal(got["slots"].cpu().numpy(), page_of.astype(np.int64) * page + cached % page)
    assert got["free_head"].tolist() == [int(fresh.sum())]


def test_tables_refused_sequences():
    """Sequences that cannot be placed keep their rows (slot and position -1),
    change nothing in the table and raise their bits; the others are placed."""
    page = 16
    rng = np.random.default_rng(1)
    cache, table, free = _paged_state(rng, [8, 4, 20], [4, 30, 2], page)
    # sequence 1 is longer than its table row can hold, sequence 2 has a negative length
    got = fk.fp8kv_build_tables(cache, _i32([8, 4, 20]), _i32([4, 1000, -3]), 1004, torch.from_numpy(free).cuda(), _i32([0]))
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
    assert got["cu_new"].tolist() == [0, 4, 1004, 1004] and got["seq_lens"].tolist() == [12, 4, 20]
    assert got["slots"].tolist()[:4] == [int(table[0, 0]) * page + t for t in range(8, 12)]
    assert set(got["slots"].tolist()[4:]) == {-1} and set(got["pos"].tolist()[4:]) == {-1}
    assert cache.page_table.tolist() == table.tolist() and got["free_head"].tolist() == [0]


def test_tables_out_of_pages():
    page = 16
    rng = np.random.default_rng(2)
    cached, new = [0, 0, 5, 0], [20, 40, 3, 1]       # 2, 3, 0 and 1 fresh pages
    cache, table, free = _paged_state(rng, cached, new, page)
    got = fk.fp8kv_build_tables(cache, _i32(cached), _i32(new), 64, torch.from_numpy(free[:4].copy()).cuda(), _i32([0]))
    assert fk.fp8kv_get_device_error() == fk.DEVERR_NO_PAGES
    assert got["free_head"].tolist() == [2]           # sequence 1 and, needing pages too, sequence 3 got none
    assert got["seq_lens"].tolist() == [20, 0, 8, 0]
    s = got["slots"].tolist()
    assert min(s[:20]) >= 0 and set(s[20:60]) == {-1} and min(s[60:63]) >= 0 and s[63] == -1


def test_tables_far_more_pages_than_free():
    """Requests for 2^23 pages with three free: nothing is placed, and the
    pages that do not exist are not walked."""
    table = torch.full((8, 1 << 20), -7, dtype=torch.int32)
    cache = fk.Fp8KVCache.paged(table, 4, 1, 64, 16)
    got = fk.fp8kv_build_tables(cache, _i32([0] * 8), _i32([16 << 20] * 8), 8, _i32([1, 2, 3]), _i32([0]))
    assert fk.fp8kv_get_device_error() == fk.DEVERR_NO_PAGES | fk.DEVERR_SEQ_TOO_LONG
    assert got["seq_lens"].tolist() == [0] * 8 and got["free_head"].tolist() == [0] and got["slots"].tolist() == [-1] * 8
    assert bool((cache.page_table == -7).all())


def test_tables_bad_ids_and_short_rows():
    page = 16
    cache = fk.Fp8KVCache.paged(torch.tensor([[99, -1], [0, -1]], dtype=torch.int32), 4, 1, 64, page)
    free = _i32([1, 77])
    got = fk.fp8kv_build_tables(cache, _i32([3, 16]), _i32([1, 1]), 2, free, _i32([1]))
    assert fk.fp8kv_get_device_error() == fk.DEVERR_BAD_PAGE
    assert got["slots"].tolist() == [-1, -1] and cache.page_table.tolist() == [[99, -1], [0, -1]]
    got = fk.fp8kv_build_tables(cache, _i32([16, 0]), _i32([3, 0]), 2, free, _i32([0]))
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG       # three new rows, room for two
    assert got["slots"].tolist() == [16, 17]
    got = fk.fp8kv_build_tables(cache, _i32([0, 0]), _i32([1, 0]), 1, free, _i32([5]))
    assert fk.fp8kv_get_device_error() == fk.DEVERR_NO_PAGES           # a head outside the list


def test_tables_graph_steps():
    """Three decode steps from one captured graph: the lengths and the head of
    the free list are fed back on the device."""
    page, B = 16, 5
    rng = np.random.default_rng(3)
    cached = [14, 15, 16, 31, 0]
    cache, table, free = _paged_state(rng, cached, [3] * B, page)
    lens, head, ones, fr = _i32(cached), _i32([0]), _i32([1] * B), torch.from_numpy(free).cuda()
    out = fk.fp8kv_build_tables(cache, lens, ones, B, fr, head)
    cache.page_table.copy_(torch.from_numpy(table))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fk.fp8kv_build_tables(cache, lens, ones, B, fr, head, out["cu_new"], out["seq_lens"], out["seq_idx"], out["pos"],
                              out["slots"], out["free_head"])
        lens.copy_(out["seq_lens"])
        head.copy_(out["free_head"])
    h, t = 0, table.tolist()
    for step in range(3):
        g.replay()
        t, _, _, _, pos, slots, h = _plain_tables([c + step for c in cached], [1] * B, page, free.tolist(), h, t, B, 0)
        assert out["slots"].tolist() == slots and out["pos"].tolist() == pos and head.tolist() == [h]
        assert cache.page_table.tolist() == t
    assert fk.fp8kv_get_device_error() == 0


# ----------------------------------------------------------- rotary tables --
@pytest.mark.parametrize("rot", [2, 6, 64, 128, 256])
@pytest.mark.parametrize("kw", [{}, {"factor": 4.0}, {"factor": 8.0, "original_positions": 4096, "base": 500000.0},
                                {"factor": 3.0, "original_positions": 512, "ramp": (0.5, 32.0), "amplitude": 1.25},
                                {"base": 0.3}])
def test_rope_tables(rot, kw):
    n = 5000
    cos, sin = fk.fp8kv_rope_tables(n, rot, **kw)
    base, factor, orig = kw.get("base", 10000.0), kw.get("factor", 1.0), kw.get("original_positions", 0)
    lo, hi = kw.get("ramp", (1.0, 4.0))
    w = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if orig:
        g = np.clip((orig * w / (2 * math.pi) - lo) / (hi - lo), 0, 1)
        w = w * (g + (1 - g) / factor)
    else:
        w = w / factor
    a = np.arange(n)[:, None] * w
    amp = kw.get("amplitude", 1.0)
    tol = amp * 2.0 ** -22
    assert np.abs(cos.cpu().numpy() - amp * np.cos(a)).max() <= tol
    assert np.abs(sin.cpu().numpy() - amp * np.sin(a)).max() <= tol


def test_rope_tables_far_positions():
    """Two million positions: the last rows against exact turns (whole-number
    arithmetic on a 120-bit frequency)."""
    n, rot = 2_000_001, 4
    cos, sin = fk.fp8kv_rope_tables(n, rot, base=10.0)
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    for i in range(2):
        w = (Decimal(1) / Decimal(10) ** (Decimal(2 * i) / Decimal(rot))) / (2 * pi)
        for t in (0, 1, 999_999, 1_999_999, 2_000_000):
            x = Decimal(t) * w
            angle = float((x - x.to_integral_value()) * 2 * pi)
            assert abs(cos[t, i].item() - math.cos(angle)) <= 2.0 ** -22
            assert abs(sin[t, i].item() - math.sin(angle)) <= 2.0 ** -22


@pytest.mark.parametrize("rot,kw", [(64, {"base": 500000.0, "factor": 8.0}), (128, {"base": 1e6}), (256, {"base": 1e8, "factor": 40.0}),
                                    (6, {"base": 1e7})])
def test_rope_tables_small_angles(rot, kw):
    """Sines keep their leading digits: a sine is off by its own roundings, relative
    to it.  The angle is a 64-bit phase converted to fp32 in two parts (each part
    and each product rounded, the constants too, and the sum: 6 roundings of 2^-24
    at most), sine's polynomial adds 2^-27 and its last sum 2^-24: 8 x 2^-24 =
    2^-21 in all.  Beside it the frequency's own error, t 2^-53 of a turn."""
    n = 4096
    cos, sin = fk.fp8kv_rope_tables(n, rot, **kw)
    base, factor = kw["base"], kw.get("factor", 1.0)
    w = np.array([base ** (-2.0 * i / rot) / factor for i in range(rot // 2)])
    t = np.arange(n)[:, None]
    want = np.sin(t * w)
    # (numpy's own product t w and sine: 2^-52 of the angle)
    tol = 2.0 ** -21 * np.abs(want) + t * (2 * math.pi * 2.0 ** -53 + 2.0 ** -52 * w)
    assert np.all(np.abs(sin.cpu().numpy() - want) <= tol)
    want = np.cos(t * w)
    tol = 2.0 ** -21 * np.abs(want) + t * (2 * math.pi * 2.0 ** -53 + 2.0 ** -52 * w)
    assert np.all(np.abs(cos.cpu().numpy() - want) <= tol)


# ------------------------------------------------------------- rope append --
def _f32(t):
    return t.float().cpu().numpy()


def _rotate(x, c, s, rot, layout):
    """fp32, each product and each sum rounded once."""
    y = x.copy()
    i = np.arange(rot // 2)
    a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    c, s = c[:, None], s[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _e4m3(x, scale):
    """Codes of x / scale through torch's own e4m3 conversion on the CPU."""
    q = np.divide(x, scale[..., None], out=np.zeros_like(x), where=scale[..., None] > 0)
    return torch.from_numpy(np.clip(q, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _setup(dtype, D, page, n, Hq, Hkv, seed, fused=True, batch=3):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = rng.multinomial(n, [1 / batch] * batch)
    if page:
        per = -(-int(lens.max()) // page) + 1
        table = torch.from_numpy(rng.permutation(batch * per).astype(np.int32).reshape(batch, per))
        cache = fk.Fp8KVCache.paged(table, batch * per, Hkv, D, page, dtype)
    else:
        cache = fk.Fp8KVCache.contiguous(batch, Hkv, D, -(-(int(lens.max()) + 1) // 16) * 16, dtype)
    seq = np.repeat(np.arange(batch), lens)
    pos = np.concatenate([np.arange(x) for x in lens]).astype(np.int32)
    if page:
        slots = table.numpy()[seq, pos // page].astype(np.int64) * page + pos % page
    else:
        slots = seq.astype(np.int64) * cache.max_tokens + pos
    qkv = torch.randn(n, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = qkv[:, :Hq * D].unflatten(1, (Hq, D)), qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)), \
        qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return cache, q, k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda()


def _stored(cache, side, slots):
    """Rows of one side (and its scales) at the slots: [n, Hkv, ...]."""
    t, sc = getattr(cache, side), getattr(cache, side + "_scale")
    span = cache.page_size or cache.max_tokens
    pick = lambda x: x[slots // span, :, slots % span].cpu()      # noqa: E731
    return pick(t), None if sc is None else pick(sc)


def _check_rows(cache, side, slots, x):
    """x [n, Hkv, D] fp32 is what the slots hold, quantised from fp32."""
    got, sc = _stored(cache, side, slots)
    if got.dtype == torch.bfloat16:
        assert torch.equal(got, torch.from_numpy(x).to(torch.bfloat16))
    elif sc.dtype == torch.uint8:
        blocks = x.reshape(x.shape[:-1] + (4, 32))
        m, e = np.frexp(np.abs(blocks).max(-1))
        E = np.where(m == 0, -127, np.clip(np.where(m <= 0.875, e - 9, e - 8), -127, 127))
        assert np.array_equal(sc.numpy(), E + 127)
        want = torch.from_numpy(np.ldexp(blocks, -E[..., None]).reshape(x.shape).astype(np.float32))
        assert torch.equal(got.view(torch.float8_e4m3fn).float(), want.to(torch.float8_e4m3fn).float())
    else:
        scale = (np.abs(x).max(-1) / np.float32(448)).astype(np.float32)
        assert np.array_equal(sc.numpy(), scale)
        want = torch.from_numpy(_e4m3(x, scale)).view(torch.float8_e4m3fn).float()
        assert torch.equal(got.view(torch.float8_e4m3fn).float(), want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,D,rots", [("k8v8", 128, (8, 40, 64, 128)), ("mxk8v8", 128, (48, 96, 128)), ("k16v8", 64, (16, 64)),
                                          ("k8v16", 64, (24, 64)), ("k16v16", 128, (32, 128))])
@pytest.mark.parametrize("page", [0, 16])
def test_rope_append(layout, dtype, D, rots, page):
    for i, rot in enumerate(rots):
        Hq, Hkv = [(4, 1), (6, 3), (7, 7), (16, 2)][i % 4]
        cache, q, k, v, pos, slots = _setup(dtype, D, page, 61, Hq, Hkv, seed=10 * i + rot, fused=i % 2 == 0)
        cos, sin = fk.fp8kv_rope_tables(64, rot)
        out = fk.fp8kv_rope_append(cache, q, k, v, pos, slots, cos, sin, layout)
        assert fk.fp8kv_get_device_error() == 0
        at = pos.cpu().numpy()
        c, s = cos.cpu().numpy()[at], sin.cpu().numpy()[at]
        want = _rotate(_f32(q), c, s, rot, layout)
        assert torch.equal(out.cpu(), torch.from_numpy(want).to(torch.bfloat16))
        # and against 64 bits: three fp32 roundings and one to bf16
        x = _f32(q).astype(np.float64)
        exact = _rotate(x, c.astype(np.float64), s.astype(np.float64), rot, layout)
        assert np.all(np.abs(_f32(out) - exact) <= 2.0 ** -8 * np.abs(exact) + 6 * 2.0 ** -24 * np.abs(x).max(-1, keepdims=True))
        _check_rows(cache, "k", slots, _rotate(_f32(k), c, s, rot, layout))
        _check_rows(cache, "v", slots, _f32(v))


def test_rope_append_k_bias():
    """Residual keys: the bias, constant or turning, is subtracted from the
    rotated key; codes as fp8kv_append stores them for the same residual."""
    D, Hkv = 128, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    bias = torch.randn(Hkv, D, generator=g, device="cuda") * 20
    cos, sin = fk.fp8kv_rope_tables(64, D)
    for turning in (False, True):
        cache, q, k, v, pos, slots = _setup("k8v8", D, 0, 40, 4, Hkv, seed=8)
        kw = {"rope_cos": cos, "rope_sin": sin} if turning else {}
        cache = fk.Fp8KVCache.contiguous(3, Hkv, D, cache.max_tokens, "k8v8", k_bias=bias, **kw)
        fk.fp8kv_rope_append(cache, q, k, v, pos, slots, cos, sin)
        at = pos.cpu().numpy()
        c, s = cos.cpu().numpy()[at], sin.cpu().numpy()[at]
        x, b = _rotate(_f32(k), c, s, D, "half"), bias.cpu().numpy()
        if turning:
            c6, s6, lo, hi = c[:, None].astype(np.float64), s[:, None], b[:, :D // 2], b[:, D // 2:]
            # fma(b_d, cos, -(b sin)) with the product with sin rounded to fp32 first
            t0 = (lo * c6 - (hi * s6).astype(np.float64)).astype(np.float32)
            t1 = (hi * c6 + (lo * s6).astype(np.float64)).astype(np.float32)
            b = np.concatenate([t0, t1], -1)
        _check_rows(cache, "k", slots, (x - b).astype(np.float32))
    assert fk.fp8kv_get_device_error() == 0


def test_rope_append_turning_bias_has_its_own_table():
    """A position past the cache's own rotary table is reported, however long
    the call's table is."""
    D = 64
    cos, sin = fk.fp8kv_rope_tables(32, D)
    long_cos, long_sin = fk.fp8kv_rope_tables(4096, D)
    cache = fk.Fp8KVCache.contiguous(1, 1, D, 32, "k8v8", k_bias=torch.zeros(1, D, device="cuda"), rope_cos=cos, rope_sin=sin)
    q = torch.randn(2, 1, D, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 9.0)
    fk.fp8kv_rope_append(cache, q, q, q, _i32([3, 4000]), torch.tensor([3, 4], device="cuda"), long_cos, long_sin, q_out=out)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG
    assert bool((out[1] == 9.0).all()) and not bool((out[0] == 9.0).any())


def test_rope_append_padding_and_bad_rows():
    """Rows with a negative slot are left alone, rows without a table entry or
    with a slot past the cache are skipped and reported."""
    cache, q, k, v, pos, slots = _setup("k8v8", 128, 16, 12, 4, 2, seed=4)
    cos, sin = fk.fp8kv_rope_tables(64, 64)
    ref = fk.fp8kv_rope_append(cache, q, k, v, pos, slots, cos, sin)
    k_ref, s_ref = _stored(cache, "k", slots)
    cache.k.fill_(7)
    cache.k_scale.fill_(-1.0)
    slots2, pos2 = slots.clone(), pos.clone()
    slots2[3] = -1
    slots2[5] = cache.num_pages * 16
    pos2[7] = 64
    out = torch.full_like(ref, 9.0)
    fk.fp8kv_rope_append(cache, q, k, v, pos2, slots2, cos, sin, q_out=out)
    assert fk.fp8kv_get_device_error() == fk.DEVERR_SEQ_TOO_LONG | fk.DEVERR_BAD_PAGE
    ok = torch.tensor([i not in (3, 5, 7) for i in range(12)])
    assert torch.equal(out.cpu()[ok], ref.cpu()[ok]) and bool((out.cpu()[~ok] == 9.0).all())
    got, sc = _stored(cache, "k", slots)
    assert torch.equal(got[ok], k_ref[ok]) and torch.equal(sc[ok], s_ref[ok])
    assert bool((got[~ok] == 7).all()) and bool((sc[~ok] == -1).all())


def test_rope_append_in_place_and_zero_rows():
    cache, q, k, v, pos, slots = _setup("k8v8", 64, 0, 33, 5, 5, seed=6, fused=False)
    k[4] = 0
    v[5, 2] = 0
    cos, sin = fk.fp8kv_rope_tables(64, 48)
    ref = fk.fp8kv_rope_append(cache, q, k, v, pos, slots, cos, sin, "interleaved")
    _check_rows(cache, "v", slots, _f32(v))
    assert _stored(cache, "k", slots)[1][4].abs().max() == 0
    same = fk.fp8kv_rope_append(cache, q, k, v, pos, slots, cos, sin, "interleaved", q_out=q)
    assert same.data_ptr() == q.data_ptr() and torch.equal(same, ref)
    empty = fk.fp8kv_rope_append(cache, q[:0], k[:0], v[:0], pos[:0], slots[:0], cos, sin)
    assert empty.shape == (0, 5, 64)


def test_step_calls_on_another_stream():
    """Tables and append enqueued on a side stream behind a copy that fills
    their inputs: the calls wait for it, as they are on the same stream."""
    cache, q, k, v, pos, slots = _setup("k8v8", 128, 16, 64, 8, 2, seed=12)
    cos, sin = fk.fp8kv_rope_tables(64, 128)
    ref = fk.fp8kv_rope_append(cache, q, k, v, pos, slots, cos, sin)
    q2, pin = torch.zeros_like(q.contiguous()), q.contiguous().cpu().pin_memory()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q2.copy_(pin, non_blocking=True)
    out = fk.fp8kv_rope_append(cache, q2, k, v, pos, slots, cos, sin, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
