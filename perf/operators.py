"""Measured cases of the serving-step operators around the quantised cache.

One serving step over a ragged batch runs, in this order: the page tables and
slot maps of the step (`tables`), the rotary tables kept for the model's life
(`rope_tables`), the rotation of queries and keys with the quantising write
into the cache (`rope_append`), and the attention of the new tokens over the
cache, over all of it (`chunk`) or over a sliding window and a few first
tokens (`window`).  Each operator has a plain form in elementary torch
operations and the framework's own call; `own` says which one `run` takes.
"""
import math
import random

import torch

own = False

DEV = "cuda"
K_CODES = ("k8v8", "k8v16", "mxk8v8")
V_CODES = ("k8v8", "k16v8", "mxk8v8")


# ------------------------------------------------------------------- cases --
def _tables(name, batch, page, ctx, new, pad, lens_seed):
    return {"name": name, "op": "tables", "batch": batch, "page_size": page, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "new_lo": new[0], "new_hi": new[1], "pad": pad, "lens_seed": lens_seed}


def _rope_tables(name, positions, rot, base, factor, original, amplitude):
    return {"name": name, "op": "rope_tables", "positions": positions, "rot_dim": rot, "base": base, "factor": factor,
            "original": original, "amplitude": amplitude}


def _rope_append(name, dtype, heads, dim, page, rot, layout, batch, ctx, new, pad, lens_seed):
    return {"name": name, "op": "rope_append", "dtype": dtype, "q_heads": heads[0], "kv_heads": heads[1], "head_dim": dim,
            "page_size": page, "rot_dim": rot, "layout": layout, "batch": batch, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "new_lo": new[0], "new_hi": new[1], "pad": pad, "lens_seed": lens_seed}


def _attention(name, op, dtype, heads, dim, page, batch, ctx, new, window, sinks, pad, lens_seed):
    return {"name": name, "op": op, "dtype": dtype, "q_heads": heads[0], "kv_heads": heads[1], "head_dim": dim,
            "page_size": page, "batch": batch, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0], "new_hi": new[1],
            "window": window, "sinks": sinks, "pad": pad, "lens_seed": lens_seed}


def listed():
    return [
        # the tables of one decode step of the paged serving batch: every sequence gets one token
        _tables("tables_decode", 64, 16, (1024, 16384), (1, 1), 0, 3),
        # admission of many prompts at once, some requests idle this step, rows padded to a captured size
        _tables("tables_prompts", 300, 64, (0, 2000), (0, 800), 777, 5),
        # a model's rotary tables, made once at load: plain frequencies
        _rope_tables("rope_tables_16k", 16384, 128, 10000.0, 1.0, 0, 1.0),
        # the same for a context stretched eightfold, long wavelengths slowed, short ones kept
        _rope_tables("rope_tables_long", 131072, 64, 500000.0, 8.0, 16384, 1.0),
        # one decode step of the paged serving batch: 64 new rows
        _rope_append("rope_append_decode", "k8v8", (32, 8), 128, 16, 128, "half", 64, (1024, 16384), (1, 1), 0, 3),
        # block-scaled keys, part of the head rotated, an odd number of rows with padding behind them
        _rope_append("rope_append_mx", "mxk8v8", (16, 2), 128, 32, 96, "half", 5, (0, 900), (100, 300), 13, 7),
        # a prompt's rows, interleaved pairs on half of the head, keys kept in bf16
        _rope_append("rope_append_prompt", "k16v8", (28, 4), 128, 0, 64, "interleaved", 4, (0, 100), (1900, 2048), 0, 11),
        # a few drafted tokens for two short sequences, bf16 cache: latency alone
        _attention("chunk_small", "chunk", "k16v16", (4, 1), 64, 0, 2, (77, 128), (3, 9), 0, 0, 0, 13),
        # chunked prefill next to decoding sequences in one ragged batch
        _attention("chunk_mixed", "chunk", "k8v8", (32, 8), 128, 16, 16, (512, 8192), (1, 256), 0, 0, 5, 17),
        # long prompts behind cached prefixes
        _attention("chunk_prompt", "chunk", "k8v8", (28, 4), 128, 16, 2, (2048, 6144), (1500, 2048), 0, 0, 0, 19),
        # a decode step that sees a window and four first tokens of long contexts
        _attention("window_decode", "window", "k8v8", (32, 8), 128, 16, 64, (1024, 16384), (1, 1), 1024, 4, 0, 3),
        # prompts under a short window, bf16 cache
        _attention("window_prompt", "window", "k16v16", (16, 2), 128, 0, 4, (0, 4096), (1000, 2048), 512, 16, 0, 23),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope_tables", "rope_append", "rope_append", "chunk", "chunk", "window", "window"])
    seed = rng.randrange(1 << 20)
    page = rng.choice([0, 16, 32, 64])
    if op == "tables":
        hi = _log_int(rng, 1, 800)
        return _unnamed(_tables("", _log_int(rng, 1, 300), page or 16, (0, _log_int(rng, 16, 8000)), (rng.choice([0, 1]), hi),
                                rng.choice([0, 0, _log_int(rng, 1, 1000)]), seed))
    if op == "rope_tables":
        positions = _log_int(rng, 100, 131072)
        long = rng.random() < 0.5
        return _unnamed(_rope_tables("", positions, rng.choice([16, 32, 64, 96, 128] if positions < 60000 else [16, 32, 64]),
                                     rng.choice([10000.0, 500000.0]), rng.choice([2.0, 4.0, 8.0]) if long else 1.0,
                                     rng.choice([0, 4096, 8192]) if long else 0, rng.choice([1.0, 1.1])))
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["k8v8", "k8v8", "k16v8", "k8v16", "k16v16"] + (["mxk8v8"] if dim == 128 else []))
    group, kv = rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 2, 4, 8])
    while group * kv > 32:
        kv //= 2
    heads = (group * kv, kv)
    if op == "rope_append":
        batch = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, max(1, 6000 // batch))
        return _unnamed(_rope_append("", dtype, heads, dim, page, rng.choice([32, 48, dim // 2, dim]), rng.choice(["half", "interleaved"]),
                                     batch, (0, _log_int(rng, 16, 8192)), (max(1, new // 2), new), rng.choice([0, 0, 3]), seed))
    decode = rng.random() < 0.4
    batch = _log_int(rng, 1, 64) if decode else _log_int(rng, 1, 16)
    ctx = _log_int(rng, 16, 8192)
    new = rng.choice([1, 1, 4]) if decode else _log_int(rng, 2, min(2048, 8192 // batch))
    # the padded score matrix of the plain form, and the arithmetic, stay below the largest listed case's
    while batch * heads[0] * new * (ctx + new) > 3.5e8:
        new, ctx = max(1, new * 2 // 3), max(16, ctx * 2 // 3)
    window, sinks = (_log_int(rng, 1, 2048), rng.choice([0, 1, 4, 30])) if op == "window" else (0, 0)
    return _unnamed(_attention("", op, dtype, heads, dim, page, batch, (ctx // 4, ctx), (1 if decode else max(1, new // 3), new),
                               window, sinks, rng.choice([0, 0, 7]), seed))


def _unnamed(case):
    case.pop("name")
    return case


def _lengths(case):
    """Tokens already cached and new tokens of every sequence (part of the case: no seed changes them)."""
    r = random.Random(case["lens_seed"])
    return ([r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])],
            [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])])


# ------------------------------------------------------------------ inputs --
def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed(seed * 16 + salt)


def _e4m3_rows(x):
    scale = x.abs().amax(-1) / 448
    q = x / torch.where(scale > 0, scale, 1.0)[..., None]
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _mx_exponent(amax):
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8).clamp(-127, 127), -127)


def _mx_rows(x):
    b = x.unflatten(-1, (-1, 32))
    e = _mx_exponent(b.abs().amax(-1))
    codes = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    return codes, (e + 127).to(torch.uint8)


def _pool(case, totals, seed, fill):
    """Cache tensors for sequences of `totals` tokens: a pool of pages in random order, or one stretch per sequence."""
    B, H, D, P = case["batch"], case["kv_heads"], case["head_dim"], case["page_size"]
    s = {"page_size": P, "kv_heads": H, "head_dim": D, "dtype": case["dtype"], "batch": B}
    if P:
        per = [-(-t // P) for t in totals]
        cols, pages = max(1, max(per)), sum(per) + 2
        perm = torch.randperm(pages, generator=_gen(seed, 1), device=DEV, dtype=torch.int64)
        have = torch.tensor(per, device=DEV)
        col = torch.arange(cols, device=DEV)
        at = (have.cumsum(0) - have)[:, None] + col
        s["page_table"] = torch.where(col < have[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32)
        s["num_pages"], s["max_tokens"], lead = pages, 0, (pages, H, P)
    else:
        s["page_table"], s["num_pages"] = None, 0
        s["max_tokens"] = max(16, -(-max(totals) // 16) * 16)
        lead = (B, H, s["max_tokens"])
    for side, coded, salt in (("k", case["dtype"] in K_CODES, 2), ("v", case["dtype"] in V_CODES, 3)):
        mx = side == "k" and case["dtype"] == "mxk8v8"
        if not fill:
            s[side] = torch.zeros(lead + (D,), dtype=torch.uint8 if coded else torch.bfloat16, device=DEV)
            s[side + "_scale"] = (torch.zeros(lead + (4,), dtype=torch.uint8, device=DEV) if mx else
                                  torch.zeros(lead, dtype=torch.float32, device=DEV) if coded else None)
            continue
        x = torch.randn(lead + (D,), generator=_gen(seed, salt), device=DEV)
        if side == "k":
            x[..., 5::16] *= 4.0          # a few channels of the keys are much larger than the others
        if mx:
            s["k"], s["k_scale"] = _mx_rows(x.to(torch.bfloat16).float())
        elif coded:
            s[side], s[side + "_scale"] = _e4m3_rows(x.to(torch.bfloat16).float())
        else:
            s[side], s[side + "_scale"] = x.to(torch.bfloat16), None
    return s


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cos_sin(positions, rot, base):
    inv = base ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * inv
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def prepare(case, seed):
    op = case["op"]
    if op == "rope_tables":
        # the seed moves the base of the frequencies: other tables
        half = case["rot_dim"] // 2
        return {"case": case, "base": case["base"] * (1 + (seed % 97) / 100),
                "cos": torch.empty(case["positions"], half, device=DEV), "sin": torch.empty(case["positions"], half, device=DEV)}
    cached, new = _lengths(case)
    totals = [a + b for a, b in zip(cached, new)]
    s = {"case": case, "rows": sum(new) + case["pad"], "n": sum(new), "new_max": max(new), "cached": _i32(cached),
         "new": _i32(new), "seq_lens": _i32(totals)}
    cu = torch.zeros(case["batch"] + 1, dtype=torch.int32, device=DEV)
    cu[1:] = s["new"].cumsum(0)
    s["cu"] = cu
    if op == "tables":
        P = case["page_size"]
        cols, pages = -(-max(totals) // P) + 1, sum(-(-t // P) for t in totals) + 5
        perm = torch.randperm(pages, generator=_gen(seed, 1), device=DEV, dtype=torch.int64).to(torch.int32)
        have = (s["cached"] + P - 1) // P
        used = sum(-(-t // P) for t in cached)
        col = torch.arange(cols, device=DEV, dtype=torch.int32)
        at = (have.cumsum(0) - have)[:, None] + col
        s["page_table"] = torch.where(col < have[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32)
        s["free"], s["head"] = perm[used:].contiguous(), torch.zeros(1, dtype=torch.int32, device=DEV)
        s |= {"num_pages": pages, "page_size": P, "kv_heads": 1, "head_dim": 64, "dtype": "k8v8", "batch": case["batch"], "max_tokens": 0}
        for side in ("k", "v"):
            s[side] = torch.zeros(pages, 1, P, 64, dtype=torch.uint8, device=DEV)
            s[side + "_scale"] = torch.zeros(pages, 1, P, device=DEV)
        N, B = s["rows"], case["batch"]
        s["out"] = {"cu_new": torch.empty(B + 1, dtype=torch.int32, device=DEV), "seq_lens": torch.empty(B, dtype=torch.int32, device=DEV),
                    "seq_idx": torch.empty(N, dtype=torch.int32, device=DEV), "pos": torch.empty(N, dtype=torch.int32, device=DEV),
                    "slots": torch.empty(N, dtype=torch.int64, device=DEV), "free_head": torch.empty(1, dtype=torch.int32, device=DEV)}
        return s
    s |= _pool(case, totals, seed, fill=op != "rope_append")
    Hq, H, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    g = _gen(seed, 7)
    if op != "rope_append":
        s["q"] = torch.randn(s["rows"], Hq, D, generator=g, device=DEV).to(torch.bfloat16)
        s["out"] = torch.zeros(s["rows"], Hq, D, dtype=torch.bfloat16, device=DEV)
        s["max_len"] = max(totals)
        return s
    # queries, keys and values as one projection leaves them: side by side in a row
    qkv = torch.randn(s["rows"], (Hq + 2 * H) * D, generator=g, device=DEV).to(torch.bfloat16)
    s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    s["k_new"] = qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
    s["v_new"] = qkv[:, (Hq + H) * D:].unflatten(1, (H, D))
    seq = torch.repeat_interleave(torch.arange(case["batch"], device=DEV), s["new"].long())
    pos = s["cached"][seq] + torch.arange(s["n"], device=DEV) - s["cu"][seq]
    P = case["page_size"]
    slots = s["page_table"][seq, pos // P].long() * P + pos % P if P else seq * s["max_tokens"] + pos
    tail = torch.full((case["pad"],), -1, device=DEV, dtype=torch.int64)
    s["pos"], s["slots"] = torch.cat([pos, tail]).to(torch.int32), torch.cat([slots, tail])
    s["cos"], s["sin"] = _cos_sin(max(totals), case["rot_dim"], 10000.0)
    s["q_out"] = torch.zeros(s["rows"], Hq, D, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------- plain forms --
def _plain_tables(s):
    P, cols, out, N = s["page_size"], s["page_table"].shape[1], s["out"], s["rows"]
    cached, new = s["cached"].long(), s["new"].long()
    first, last = (cached + P - 1) // P, (cached + new + P - 1) // P
    base = s["head"].long() + (last - first).cumsum(0) - (last - first)
    col = torch.arange(cols, device=DEV)
    take = (base[:, None] + col - first[:, None]).clamp(0, s["free"].numel() - 1)
    fresh = (col >= first[:, None]) & (col < last[:, None])
    s["page_table"].copy_(torch.where(fresh, s["free"][take], s["page_table"]))
    out["cu_new"][:1] = 0
    out["cu_new"][1:] = new.cumsum(0)
    out["seq_lens"].copy_(cached + new)
    out["free_head"].copy_(s["head"] + (last - first).sum())
    row = torch.arange(N, device=DEV)
    real = row < out["cu_new"][-1]
    seq = torch.searchsorted(out["cu_new"].long(), row, right=True).clamp(max=s["batch"]) - 1
    pos = cached[seq] + row - out["cu_new"].long()[seq]
    page = s["page_table"][seq, (pos // P).clamp(0, cols - 1)].long()
    out["seq_idx"].copy_(torch.where(real, seq, -1))
    out["pos"].copy_(torch.where(real, pos, -1))
    out["slots"].copy_(torch.where(real, page * P + pos % P, -1))
    return {"page_table": s["page_table"], **out}


def _inv_freq(case, base, device):
    R = case["rot_dim"]
    inv = base ** (-torch.arange(0, R, 2, device=device, dtype=torch.float64) / R)
    if case["original"]:
        turns = case["original"] * inv / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return inv * (keep + (1 - keep) / case["factor"])
    return inv / case["factor"]


def _plain_rope_tables(s):
    c = s["case"]
    a = torch.arange(c["positions"], device=DEV, dtype=torch.float64)[:, None] * _inv_freq(c, s["base"], DEV)
    s["cos"].copy_(a.cos() * c["amplitude"])
    s["sin"].copy_(a.sin() * c["amplitude"])
    return {"cos": s["cos"], "sin": s["sin"]}


def _rotate(x, cos, sin, rot, layout):
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope_append(s):
    c, n, H, D = s["case"], s["n"], s["kv_heads"], s["head_dim"]
    pos, slots = s["pos"][:n].long(), s["slots"][:n]
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    s["q_out"][:n] = _rotate(s["q"][:n].float(), cos, sin, c["rot_dim"], c["layout"]).to(torch.bfloat16)
    span = s["page_size"] or s["max_tokens"]
    row = ((slots // span)[:, None] * H + torch.arange(H, device=DEV)) * span + (slots % span)[:, None]
    k, v = _rotate(s["k_new"][:n].float(), cos, sin, c["rot_dim"], c["layout"]), s["v_new"][:n].float()
    if c["dtype"] == "mxk8v8":
        codes, scale = _mx_rows(k)
        s["k"].view(-1, D)[row], s["k_scale"].view(-1, 4)[row] = codes, scale
    elif c["dtype"] in K_CODES:
        codes, scale = _e4m3_rows(k)
        s["k"].view(-1, D)[row], s["k_scale"].view(-1)[row] = codes, scale
    else:
        s["k"].view(-1, D)[row] = k.to(torch.bfloat16)
    if c["dtype"] in V_CODES:
        codes, scale = _e4m3_rows(v)
        s["v"].view(-1, D)[row], s["v_scale"].view(-1)[row] = codes, scale
    else:
        s["v"].view(-1, D)[row] = v.to(torch.bfloat16)
    return _cache_values(s)


def _cache_values(s):
    out = {"q": s["q_out"]}
    for side in ("k", "v"):
        t, scale = s[side], s[side + "_scale"]
        out[side] = t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t
        if scale is not None:
            out[side + "_scale"] = scale.view(torch.float8_e8m0fnu) if scale.dtype == torch.uint8 else scale
    return out


def _gather(s, side):
    """The sequences' rows of one side of the cache as [batch, kv_heads, max_len, head_dim] fp32."""
    x, scale = s[side], s[side + "_scale"]
    x = (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x)
    if s["page_size"]:
        pages = s["page_table"].clamp(min=0).long()
        x = x.view(torch.uint8)[pages].view(x.dtype).float().transpose(1, 2).flatten(2, 3)
        scale = None if scale is None else scale[pages].transpose(1, 2).flatten(2, 3)
    else:
        x = x.float()
    if scale is not None and scale.dtype == torch.uint8:
        x = (x.unflatten(-1, (4, 32)) * torch.exp2(scale.float() - 127)[..., None]).flatten(-2)
    elif scale is not None:
        x = x * scale[..., None]
    return x[:, :, :s["max_len"]]


def _plain_attention(s):
    c, n, m = s["case"], s["n"], s["new_max"]
    B, H, D, Hq = s["batch"], s["kv_heads"], s["head_dim"], c["q_heads"]
    G, T = Hq // H, s["max_len"]
    # queries padded to the longest chunk: [batch, kv_heads, group * chunk, head_dim]
    i = torch.arange(m, device=DEV)
    row = (s["cu"][:-1, None] + i).clamp(max=s["rows"] - 1).long()
    q = s["q"].float()[row].unflatten(2, (H, G)).permute(0, 2, 3, 1, 4).reshape(B, H, G * m, D)
    scores = torch.matmul(q, _gather(s, "k").transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, H, G, m, T)
    pos = (s["seq_lens"] - s["new"])[:, None] + i
    key = torch.arange(T, device=DEV)
    seen = (key <= pos[..., None]) & (i[:, None] < s["new"][:, None, None])
    if c["window"]:
        seen &= (key > pos[..., None] - c["window"]) | (key < c["sinks"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, G * m, T), _gather(s, "v")).view(B, H, G, m, D) / torch.where(total > 0, total, 1.0)
    # back to ragged rows; rows behind the last sequence stay as they were
    seq = torch.searchsorted(s["cu"], torch.arange(n, device=DEV, dtype=torch.int32), right=True) - 1
    at = torch.arange(n, device=DEV) - s["cu"][seq]
    s["out"][:n] = o[seq, :, :, at].flatten(1, 2).to(torch.bfloat16)
    return s["out"]


# --------------------------------------------------------------------- run --
def _cache(s):
    """The cache handle that a program keeps for the life of its cache."""
    if "handle" not in s:
        import fp8_quantized_kv_gb300 as fk
        s["handle"] = fk.Fp8KVCache(
            dtype=s["dtype"], layout=fk.LAYOUT_PAGED if s["page_size"] else fk.LAYOUT_CONTIGUOUS, batch=s["batch"],
            kv_heads=s["kv_heads"], head_dim=s["head_dim"], k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"],
            max_tokens=s["max_tokens"], page_size=s["page_size"], num_pages=s["num_pages"], page_table=s["page_table"])
    return s["handle"]


def _own(s):
    import fp8_quantized_kv_gb300 as fk
    c = s["case"]
    if c["op"] == "rope_tables":
        fk.fp8kv_rope_tables(c["positions"], c["rot_dim"], base=s["base"], factor=c["factor"], original_positions=c["original"],
                             ramp=(1.0, 4.0), amplitude=c["amplitude"], cos=s["cos"], sin=s["sin"])
        return {"cos": s["cos"], "sin": s["sin"]}
    cache = _cache(s)
    if c["op"] == "tables":
        o = s["out"]
        fk.fp8kv_build_tables(cache, s["cached"], s["new"], s["rows"], free_pages=s["free"], free_head=s["head"],
                              cu_new=o["cu_new"], seq_lens=o["seq_lens"], seq_idx=o["seq_idx"], pos=o["pos"], slots=o["slots"],
                              free_head_out=o["free_head"])
        return {"page_table": s["page_table"], **o}
    if c["op"] == "rope_append":
        fk.fp8kv_rope_append(cache, s["q"], s["k_new"], s["v_new"], s["pos"], s["slots"], s["cos"], s["sin"], layout=c["layout"],
                             q_out=s["q_out"])
        return _cache_values(s)
    if "workspace" not in s:
        need = fk.fp8kv_chunk_workspace_bytes(cache, s["rows"], c["q_heads"], window=c["window"], sinks=c["sinks"])
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    return fk.fp8kv_chunk_attention(s["q"], cache, s["cu"], s["seq_lens"], window=c["window"], sinks=c["sinks"], out=s["out"],
                                    workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "tables":
        return _plain_tables(state)
    if op == "rope_tables":
        return _plain_rope_tables(state)
    if op == "rope_append":
        return _plain_rope_append(state)
    return _plain_attention(state)


# -------------------------------------------------------------------- work --
def _row_bytes(dtype, side, D):
    if (side == "k" and dtype in K_CODES) or (side == "v" and dtype in V_CODES):
        return D + 4
    return 2 * D


def work(case):
    op = case["op"]
    if op == "rope_tables":
        # both tables written once; an angle is a product and a reduction, then a sine and a cosine
        n = case["positions"] * case["rot_dim"] / 2
        return {"bytes": 8 * n, "flops": 4 * n}
    cached, new = _lengths(case)
    n, B = sum(new), case["batch"]
    if op == "tables":
        P, rows = case["page_size"], n + case["pad"]
        fresh = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(cached, new))
        # lengths in; prefix sums, new pages and the three row maps out; one page id a row at most is read back
        return {"bytes": 4 * (2 * B + 2 * B + 1) + 8 * fresh + 16 * rows + 4 * B, "flops": 4 * rows}
    D, Hq, H, dt = case["head_dim"], case["q_heads"], case["kv_heads"], case["dtype"]
    if op == "rope_append":
        per = 4 * Hq * D + 4 * H * D + H * (_row_bytes(dt, "k", D) + _row_bytes(dt, "v", D)) + 12
        touched = len({p for a, b in zip(cached, new) for p in range(a, a + b)}) if n < 100000 else n
        return {"bytes": n * per + touched * case["rot_dim"] * 4, "flops": n * (3 * (Hq + H) * case["rot_dim"] + 4 * H * D)}
    W, S = case["window"], case["sinks"]
    keys = pairs = 0
    for a, b in zip(cached, new):
        # cache rows that any query of the chunk sees, and the (query, key) pairs of the chunk
        if W:
            low = max(0, a - W + 1)
            keys += (a + b - low + min(S, low)) if b else 0
            pairs += sum(min(p + 1, W + min(S, max(0, p + 1 - W))) for p in range(a, a + b))
        else:
            keys += (a + b) if b else 0
            pairs += b * a + b * (b + 1) // 2
    return {"bytes": keys * H * (_row_bytes(dt, "k", D) + _row_bytes(dt, "v", D)) + 4 * n * Hq * D, "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------------- exact --
def _e4m3_nearest(x):
    """Nearest e4m3 value of fp64 numbers up to 448 in size, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (x / step).round().mul(step).clamp(-448, 448)


def _exact_rotate(x, angle_cos, angle_sin, rot, layout):
    y = x.clone()
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c, t = angle_cos[:, None, i], angle_sin[:, None, i]
        y[..., a] = x[..., a] * c - x[..., b] * t
        y[..., b] = x[..., a] * t + x[..., b] * c
    return y


def _exact_values(s):
    """Code values times scales of the filled cache, one [tokens, kv_heads, head_dim] fp64 pair a sequence."""
    P = s["page_size"]
    for b in range(s["batch"]):
        t = torch.arange(int(s["seq_lens"][b]), device=DEV)
        if P:
            lead, off = s["page_table"][b].long()[t // P], t % P
        else:
            lead, off = torch.full_like(t, b), t
        pair = []
        for side in ("k", "v"):
            x, scale = s[side], s[side + "_scale"]
            if x.dtype == torch.uint8:
                u = x[lead, :, off].to(torch.int64)
                man, ex = (u & 7).double(), (u >> 3) & 15
                mag = torch.where(ex > 0, (8 + man) * torch.exp2(ex.double() - 10), man * 2.0 ** -9)
                val = torch.where(u >= 128, -mag, mag)
                sc = scale[lead, :, off].double()
                val = val * (torch.exp2(sc - 127).repeat_interleave(32, -1) if scale.dtype == torch.uint8 else sc[..., None])
            else:
                val = x[lead, :, off].double()
            pair.append(val)
        yield b, pair[0], pair[1]


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None
    s = prepare(case, seed)
    if op == "rope_tables":
        R, t = case["rot_dim"], torch.arange(case["positions"], device=DEV, dtype=torch.float64)
        cos, sin = torch.empty_like(s["cos"], dtype=torch.float64), torch.empty_like(s["sin"], dtype=torch.float64)
        for i in range(R // 2):
            w = s["base"] ** (-2.0 * i / R)
            if case["original"]:
                g = min(1.0, max(0.0, (case["original"] * w / (2 * math.pi) - 1.0) / 3.0))
                w = g * w + (1.0 - g) * w / case["factor"]
            else:
                w = w / case["factor"]
            cos[:, i], sin[:, i] = torch.cos(t * w) * case["amplitude"], torch.sin(t * w) * case["amplitude"]
        return {"cos": cos, "sin": sin}
    n, H, D = s["n"], s["kv_heads"], s["head_dim"]
    if op == "rope_append":
        at = s["pos"][:n].long()
        cos, sin = s["cos"][at].double(), s["sin"][at].double()
        out = {"q": torch.zeros(s["rows"], case["q_heads"], D, dtype=torch.float64, device=DEV)}
        out["q"][:n] = _exact_rotate(s["q"][:n].double(), cos, sin, case["rot_dim"], case["layout"])
        span, slots = s["page_size"] or s["max_tokens"], s["slots"][:n]
        lead, off = slots // span, slots % span
        for side, rows in (("k", _exact_rotate(s["k_new"][:n].double(), cos, sin, case["rot_dim"], case["layout"])),
                           ("v", s["v_new"][:n].double())):
            full = torch.zeros(s[side].shape, dtype=torch.float64, device=DEV)
            if s[side].dtype == torch.uint8 and s[side + "_scale"].dtype == torch.uint8:
                block = rows.unflatten(-1, (4, 32))
                need = block.abs().amax(-1)
                ex = torch.ceil(torch.log2(need / 448)).clamp(-127, 127)
                full[lead, :, off] = _e4m3_nearest(block / torch.exp2(ex)[..., None]).flatten(-2)
                out["k_scale"] = torch.full(s["k_scale"].shape, 2.0 ** -127, dtype=torch.float64, device=DEV)
                out["k_scale"][lead, :, off] = torch.exp2(ex)
            elif s[side].dtype == torch.uint8:
                amax = rows.abs().amax(-1)
                full[lead, :, off] = _e4m3_nearest(rows / torch.where(amax > 0, amax / 448, 1.0)[..., None])
                out[side + "_scale"] = torch.zeros(s[side + "_scale"].shape, dtype=torch.float64, device=DEV)
                out[side + "_scale"][lead, :, off] = amax / 448
            else:
                full[lead, :, off] = rows
            out[side] = full
        return out
    out = torch.zeros(s["rows"], case["q_heads"], D, dtype=torch.float64, device=DEV)
    G, W, S = case["q_heads"] // H, case["window"], case["sinks"]
    for b, k, v in _exact_values(s):
        r0, r1, T = int(s["cu"][b]), int(s["cu"][b + 1]), k.shape[0]
        p = torch.arange(T - (r1 - r0), T, device=DEV)[:, None]
        j = torch.arange(T, device=DEV)[None]
        hidden = j > p
        if W:
            hidden |= (j <= p - W) & (j >= S)
        for h in range(case["q_heads"]):
            z = (s["q"][r0:r1, h].double() @ k[:, h // G].T) / math.sqrt(D)
            z[hidden] = -math.inf
            out[r0:r1, h] = torch.softmax(z, -1) @ v[:, h // G]
    return out
