"""Measured cases of tree verification around the quantised cache and of the
8-bit projections on either side of its attention.

A step that verifies a tree of drafted tokens runs, in this order: the node
masks and rotary positions of the step's trees (`tables`), the projection of
the rows to queries, keys and values in 8 bits (`matmul`), the attention of
every node over the cached tokens and its own ancestors (`attention`), and,
once the model has chosen a token at every node, the walk along the accepted
nodes with the move of their cache rows to the places behind the context
(`accept`).  Each operator has a plain form in elementary torch operations and
the framework's own call; `own` says which one `run` takes.
"""
import math
import random

import torch

own = False

DEV = "cuda"
K_CODES = ("k8v8", "k8v16", "mxk8v8")
V_CODES = ("k8v8", "k16v8", "mxk8v8")


# ------------------------------------------------------------------- cases --
def _tables(name, batch, nodes, depth, max_nodes, ctx, pad, lens_seed):
    return {"name": name, "op": "tables", "batch": batch, "nodes_lo": nodes[0], "nodes_hi": nodes[1], "depth": depth,
            "max_nodes": max_nodes, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "pad": pad, "lens_seed": lens_seed}


def _attention(name, dtype, heads, dim, page, batch, ctx, nodes, depth, window, sinks, pad, lens_seed):
    return {"name": name, "op": "attention", "dtype": dtype, "q_heads": heads[0], "kv_heads": heads[1], "head_dim": dim,
            "page_size": page, "batch": batch, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "nodes_lo": nodes[0], "nodes_hi": nodes[1],
            "depth": depth, "max_nodes": nodes[1], "window": window, "sinks": sinks, "pad": pad, "lens_seed": lens_seed}


def _accept(name, dtype, kv_heads, dim, page, layers, batch, ctx, nodes, depth, lens_seed):
    return {"name": name, "op": "accept", "dtype": dtype, "kv_heads": kv_heads, "head_dim": dim, "page_size": page,
            "layers": layers, "batch": batch, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "nodes_lo": nodes[0], "nodes_hi": nodes[1],
            "depth": depth, "max_nodes": nodes[1], "lens_seed": lens_seed}


def _matmul(name, m, n, k, bias, out):
    return {"name": name, "op": "matmul", "m": m, "n": n, "k": k, "bias": bias, "out": out}


def listed():
    return [
        # the masks of one verification step of a serving batch: trees of up to 64 drafted tokens
        _tables("tables_trees", 64, (24, 64), 8, 64, (1024, 16384), 0, 3),
        # many wide trees, chains among them, rows padded to a captured size
        _tables("tables_wide", 300, (1, 256), 40, 256, (0, 2000), 777, 5),
        # small trees for two short sequences, bf16 cache: latency alone
        _attention("tree_small", "k16v16", (4, 1), 64, 0, 2, (77, 128), (3, 9), 4, 0, 0, 0, 13),
        # the paged serving batch, a few drafted tokens each: the cache is read once and nothing takes as long
        _attention("tree_decode", "k8v8", (32, 8), 128, 16, 64, (1024, 16384), (2, 4), 3, 0, 0, 0, 3),
        # wide trees of few sequences: the two products bound it
        _attention("tree_wide", "k8v8", (28, 4), 128, 16, 16, (2048, 8192), (33, 64), 8, 0, 0, 7, 19),
        # trees under a sliding window with first tokens, keys in bf16
        _attention("tree_window", "k16v8", (16, 2), 128, 32, 32, (500, 8192), (5, 31), 6, 1024, 4, 0, 23),
        # what a step keeps of its trees: one layer, contiguous cache
        _accept("accept_one", "k16v16", 2, 64, 0, 1, 16, (77, 128), (3, 9), 4, 13),
        # the same over twelve layers of a model, the serving batch
        _accept("accept_layers", "k8v8", 8, 128, 16, 12, 64, (20, 90), (24, 64), 8, 3),
        # one token's query, key and value projection (16 / 2 heads of 128): latency and the weights' bytes
        _matmul("matmul_token", 1, 2560, 2048, False, "bf16"),
        # one decode step of the serving batch (32 / 8 heads): the weights' bytes
        _matmul("matmul_decode", 64, 6144, 4096, False, "bf16"),
        # the rows of sixteen trees (28 / 4 heads, with the projection's bias)
        _matmul("matmul_trees", 997, 4608, 3584, True, "bf16"),
        # a prompt batch's rows (32 / 8 heads): arithmetic
        _matmul("matmul_prompt", 7940, 6144, 4096, False, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _unnamed(case):
    case.pop("name")
    return case


def draw(rng):
    op = rng.choice(["tables", "attention", "attention", "attention", "accept", "matmul", "matmul", "matmul"])
    seed = rng.randrange(1 << 20)
    page = rng.choice([0, 16, 32, 64])
    if op == "tables":
        hi = _log_int(rng, 1, 256)
        return _unnamed(_tables("", _log_int(rng, 1, 300), (max(1, hi // 4), hi), rng.choice([2, 6, 12, 40]), hi + rng.choice([0, 0, 9]),
                                (0, _log_int(rng, 16, 16000)), rng.choice([0, 0, _log_int(rng, 1, 700)]), seed))
    if op == "matmul":
        n = rng.choice([_log_int(rng, 1, 700), 8 * _log_int(rng, 8, 768), 8 * _log_int(rng, 64, 768)])
        k = rng.choice([16 * _log_int(rng, 1, 256), 128 * _log_int(rng, 2, 32)])
        return _unnamed(_matmul("", _log_int(rng, 1, 7900), n, k, rng.random() < 0.3, rng.choice(["bf16", "bf16", "f32"])))
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["k8v8", "k8v8", "k16v8", "k8v16", "k16v16"] + (["mxk8v8"] if dim == 128 else []))
    group, kv = rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 2, 4, 8])
    while group * kv > 32:
        kv //= 2
    hi = _log_int(rng, 1, 64)
    nodes, depth = (max(1, hi // 3), hi), rng.choice([2, 4, 8])
    if op == "accept":
        batch = _log_int(rng, 1, 64)
        return _unnamed(_accept("", dtype, kv, dim, page, _log_int(rng, 1, max(1, min(12, 700 // batch))), batch,
                                (0, _log_int(rng, 4, 90)), nodes, depth, seed))
    batch, ctx = _log_int(rng, 1, 64), _log_int(rng, 16, 16384)
    # the padded score matrix of the plain form, and the arithmetic, stay below the largest listed case's
    while batch * group * kv * hi * (ctx + hi) > 2.2e8:
        hi, ctx = max(1, hi * 2 // 3), max(16, ctx * 2 // 3)
    window, sinks = (_log_int(rng, 1, 2048), rng.choice([0, 1, 4, 30])) if rng.random() < 0.3 else (0, 0)
    return _unnamed(_attention("", dtype, (group * kv, kv), dim, page, batch, (ctx // 4, ctx), (max(1, hi // 3), hi), depth,
                               window, sinks, rng.choice([0, 0, 7]), seed))


def _plan(case):
    """Context lengths, trees (parents within the tree, -1 for the first node) and the accepted nodes of every
    sequence: part of the case, no seed changes them.  A tree starts with its likeliest chain; the other nodes
    hang anywhere above the largest depth.  The accepted path follows the chain and may leave it."""
    r = random.Random(case["lens_seed"])
    ctx, trees, paths = [], [], []
    for _ in range(case["batch"]):
        n = r.randint(case["nodes_lo"], case["nodes_hi"])
        chain = min(n, case["depth"])
        parents, depth, open_ = [], [], []
        for i in range(n):
            p = i - 1 if i < chain else open_[min(r.randrange(len(open_)), r.randrange(len(open_)))] if open_ else 0
            parents.append(p)
            depth.append(depth[p] + 1 if p >= 0 else 0)
            if depth[i] < case["depth"] - 1:
                open_.append(i)
        path, children = [0], {}
        for i, p in enumerate(parents):
            children.setdefault(p, []).append(i)
        while path[-1] in children and r.random() < 0.8:
            path.append(r.choice(children[path[-1]]))
        ctx.append(r.randint(case["ctx_lo"], case["ctx_hi"]))
        trees.append(parents)
        paths.append(path[:case["depth"]])
    return ctx, trees, paths


# ------------------------------------------------------------------ inputs --
def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed(seed * 16 + salt)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _e4m3_rows(x):
    scale = x.abs().amax(-1) / 448
    q = x / torch.where(scale > 0, scale, 1.0)[..., None]
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _mx_rows(x):
    b = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0, torch.where(m <= 0.875, e - 9, e - 8).clamp(-127, 127), -127)
    codes = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    return codes, (e + 127).to(torch.uint8)


def _blocks(x, rows):
    """Codes of a matrix and the scales of its blocks of `rows` x 128 (1 or 128 rows; the last ones may be short)."""
    R, K = x.shape
    pr, pk = -R % rows, -K % 128
    b = torch.nn.functional.pad(x, (0, pk, 0, pr)).unflatten(0, (-1, rows)).unflatten(2, (-1, 128))
    scale = b.abs().amax((1, 3)) / 448
    codes = (b / torch.where(scale > 0, scale, 1.0)[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).flatten(2, 3).flatten(0, 1)[:R, :K].contiguous(), scale.contiguous()


def _page_tables(case, totals, seed):
    """Table, pages and capacity of a cache for sequences of `totals` tokens (page size 0: contiguous)."""
    P = case["page_size"]
    if not P:
        return None, 0, max(16, -(-max(totals) // 16) * 16)
    per = [-(-t // P) for t in totals]
    cols, pages = max(1, max(per)), sum(per) + 2
    perm = torch.randperm(pages, generator=_gen(seed, 1), device=DEV, dtype=torch.int64)
    have = torch.tensor(per, device=DEV)
    col = torch.arange(cols, device=DEV)
    at = (have.cumsum(0) - have)[:, None] + col
    return torch.where(col < have[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32), pages, 0


def _cache(case, plan, seed, salt):
    table, pages, room = plan
    H, D, P = case["kv_heads"], case["head_dim"], case["page_size"]
    lead = (pages, H, P) if P else (case["batch"], H, room)
    c = {"page_size": P, "dtype": case["dtype"], "page_table": table, "num_pages": pages, "max_tokens": room}
    for side, coded, more in (("k", case["dtype"] in K_CODES, 0), ("v", case["dtype"] in V_CODES, 1)):
        x = torch.randn(lead + (D,), generator=_gen(seed, salt + more), device=DEV)
        if side == "k":
            x[..., 5::16] *= 4.0          # a few channels of the keys are much larger than the others
        x = x.to(torch.bfloat16)
        if side == "k" and case["dtype"] == "mxk8v8":
            c["k"], c["k_scale"] = _mx_rows(x.float())
        elif coded:
            c[side], c[side + "_scale"] = _e4m3_rows(x.float())
        else:
            c[side], c[side + "_scale"] = x, None
    return c


def _pack(ancestors, words):
    """Rows of node bits (Python integers) as [rows, words] int32."""
    flat = [(a >> (32 * w)) & 0xFFFFFFFF for a in ancestors for w in range(words)]
    return torch.tensor(flat, dtype=torch.int64, device=DEV).to(torch.int32).view(-1, words)


def prepare(case, seed):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        a = torch.randn(m, k, generator=_gen(seed, 1), device=DEV)
        a[:, 5::64] *= 8.0                # activations have a few large channels
        b = torch.randn(n, k, generator=_gen(seed, 2), device=DEV) / math.sqrt(k)
        s = {"case": case, "bias": torch.randn(n, generator=_gen(seed, 3), device=DEV) if case["bias"] else None,
             "out": torch.empty(m, n, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device=DEV)}
        s["a"], s["a_scale"] = _blocks(a.to(torch.bfloat16).float(), 1)
        s["b"], s["b_scale"] = _blocks(b.to(torch.bfloat16).float(), 128)
        return s
    ctx, trees, paths = _plan(case)
    n = [len(t) for t in trees]
    totals = [a + b for a, b in zip(ctx, n)]
    rows = sum(n) + case.get("pad", 0)
    words = -(-case["max_nodes"] // 32)
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    s = {"case": case, "rows": rows, "n": cu[-1], "widest": max(n), "words": words, "cu": _i32(cu), "seq_lens": _i32(totals),
         "trees": trees, "paths": paths, "max_len": max(totals)}
    pad = [-1] * (rows - cu[-1])
    parents = [p for t in trees for p in t] + pad
    if case["op"] == "tables":
        # the seed moves the contexts' lengths
        s["seq_lens"] += seed % 4093
        # and hangs some nodes under their parent's parent: other trees of the same sizes, none deeper
        r = random.Random(seed)
        for b, t in enumerate(trees):
            for i in range(min(len(t), case["depth"]), len(t)):
                if r.random() < 0.5:
                    parents[cu[b] + i] = max(0, t[t[i]])
        s["parents"] = _i32(parents)
        s["out"] = {"masks": torch.empty(rows, words, dtype=torch.int32, device=DEV), "pos": torch.empty(rows, dtype=torch.int32, device=DEV)}
        return s
    s["parents"] = _i32(parents)
    plan = _page_tables(case, totals, seed)
    if case["op"] == "accept":
        g = _gen(seed, 2)
        tokens = torch.randperm(1 << 17, generator=g, device=DEV)[:rows]
        choices = torch.randint(1 << 17, 1 << 18, (rows,), generator=g, device=DEV)       # nobody's token
        at = [cu[b] + i for b, p in enumerate(paths) for i in p[:-1]]
        to = [cu[b] + i for b, p in enumerate(paths) for i in p[1:]]
        if at:
            choices[torch.tensor(at, device=DEV)] = tokens[torch.tensor(to, device=DEV)]
        s["tokens"], s["choices"] = tokens, choices
        s["layers"] = [_cache(case, plan, seed, 16 * (1 + i)) for i in range(case["layers"])]
        B = case["batch"]
        s["out"] = {"path": torch.empty(B, case["depth"], dtype=torch.int32, device=DEV), "accepted": torch.empty(B, dtype=torch.int32, device=DEV),
                    "next_tokens": torch.empty(B, dtype=torch.int64, device=DEV), "lens": torch.empty(B, dtype=torch.int32, device=DEV)}
        return s
    s["cache"] = _cache(case, plan, seed, 2)
    ancestors, depths = [], []
    for t in trees:
        first = len(ancestors)
        for i, p in enumerate(t):
            ancestors.append((ancestors[first + p] if p >= 0 else 0) | 1 << i)
            depths.append(depths[first + p] + 1 if p >= 0 else 0)
    s["masks"] = _pack(ancestors + [0] * len(pad), words)
    s["pos"] = _i32([c + d for c, d in zip((ctx[b] for b, t in enumerate(trees) for _ in t), depths)] + pad)
    s["q"] = torch.randn(rows, case["q_heads"], case["head_dim"], generator=_gen(seed, 7), device=DEV).to(torch.bfloat16)
    s["out"] = torch.zeros(rows, case["q_heads"], case["head_dim"], dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------- plain forms --
def _rows_of(s):
    """Sequence and node of every row of the trees (padding apart)."""
    row = torch.arange(s["n"], device=DEV)
    seq = torch.searchsorted(s["cu"].long(), row, right=True) - 1
    return row, seq, row - s["cu"].long()[seq]


def _plain_tables(s):
    row, seq, node = _rows_of(s)
    start, ctx = s["cu"].long()[seq], (s["seq_lens"] - (s["cu"][1:] - s["cu"][:-1])).long()[seq]
    bits = torch.zeros(s["rows"], s["words"] * 32, dtype=torch.bool, device=DEV)
    depth = torch.full_like(row, -1)
    at = node.clone()
    for _ in range(s["case"]["depth"] + 1):       # up the trees, all rows at once
        live = at >= 0
        bits[row, torch.where(live, at, node)] = True
        depth += live
        at = torch.where(live, s["parents"].long()[start + at.clamp(min=0)], -1)
    weight = torch.ones((), dtype=torch.int64, device=DEV) << torch.arange(32, device=DEV)
    s["out"]["masks"].copy_((bits.view(-1, s["words"], 32) * weight).sum(-1))
    s["out"]["pos"].fill_(-1)
    s["out"]["pos"][:s["n"]] = ctx + depth
    return s["out"]


def _values(c, side):
    t = c[side]
    return t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t


def _gather(s, side):
    """The sequences' rows of one side of the cache as [batch, kv_heads, max_len, head_dim] fp32."""
    c = s["cache"]
    x, scale = _values(c, side), c[side + "_scale"]
    if c["page_size"]:
        pages = c["page_table"].clamp(min=0).long()
        x = (x.view(torch.uint8)[pages].view(x.dtype) if x.dtype == torch.float8_e4m3fn else x[pages]).float().transpose(1, 2).flatten(2, 3)
        scale = None if scale is None else scale[pages].transpose(1, 2).flatten(2, 3)
    else:
        x = x.float()
    if scale is not None and scale.dtype == torch.uint8:
        x = (x.unflatten(-1, (4, 32)) * torch.exp2(scale.float() - 127)[..., None]).flatten(-2)
    elif scale is not None:
        x = x * scale[..., None]
    return x[:, :, :s["max_len"]]


def _plain_attention(s):
    c, m, T = s["case"], s["widest"], s["max_len"]
    B, H, D, Hq = c["batch"], c["kv_heads"], c["head_dim"], c["q_heads"]
    G = Hq // H
    # queries padded to the widest tree: [batch, kv_heads, group * nodes, head_dim]
    i = torch.arange(m, device=DEV)
    have = s["cu"][1:] - s["cu"][:-1]
    row = (s["cu"][:-1, None] + i).clamp(max=s["rows"] - 1).long()
    q = s["q"].float()[row].unflatten(2, (H, G)).permute(0, 2, 3, 1, 4).reshape(B, H, G * m, D)
    scores = torch.matmul(q, _gather(s, "k").transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, H, G, m, T)
    # a node sees the context (under a window: its end and its first tokens) and the nodes of its mask
    ctx = (s["seq_lens"] - have)[:, None]
    key = torch.arange(T, device=DEV)
    node = key - ctx                                                     # [batch, keys]
    word = s["masks"][row].gather(2, (node.clamp(0, m - 1) >> 5)[:, None].expand(B, m, T))
    seen = ((word >> (node.clamp(min=0) & 31)[:, None]) & 1).bool() & (node >= 0)[:, None] & (node < have[:, None])[:, None]
    cached = (node < 0)[:, None].expand(B, m, T)
    if c["window"]:
        cached = cached & ((key > s["pos"][row][..., None] - c["window"]) | (key < c["sinks"]))
    seen = (seen | cached) & (i[:, None] < have[:, None, None])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, G * m, T), _gather(s, "v")).view(B, H, G, m, D) / torch.where(total > 0, total, 1.0)
    # back to ragged rows; rows behind the last sequence stay as they were
    _, seq, at = _rows_of(s)
    s["out"][:s["n"]] = o[seq, :, :, at].flatten(1, 2).to(torch.bfloat16)
    return s["out"]


def _slots(c, seq, pos):
    """Pool page (or sequence) and place of each position."""
    P = c["page_size"]
    return (c["page_table"][seq, pos // P].long(), pos % P) if P else (seq, pos)


def _plain_accept(s):
    out, B, m, steps = s["out"], s["case"]["batch"], s["widest"], s["case"]["depth"]
    start, have = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(m, device=DEV)
    row = (start[:, None] + i).clamp(max=s["rows"] - 1)
    real = i < have[:, None]
    parent, token = torch.where(real, s["parents"].long()[row], -2), s["tokens"][row]
    at, alive = torch.zeros(B, dtype=torch.int64, device=DEV), have > 0
    path = torch.full((B, steps), -1, dtype=torch.int64, device=DEV)
    path[:, 0] = torch.where(alive, 0, -1)
    for k in range(1, steps):
        hit = (parent == at[:, None]) & (token == s["choices"][start + at][:, None])
        alive = alive & hit.any(1)
        at = torch.where(alive, hit.int().argmax(1), at)
        path[:, k] = torch.where(alive, at, -1)
    taken = (path >= 0).sum(1)
    ctx = s["seq_lens"].long() - have
    out["path"].copy_(path)
    out["accepted"].copy_(taken)
    out["next_tokens"].copy_(s["choices"][start + at])
    out["lens"].copy_(ctx + taken)
    # rows of the accepted nodes to the places behind the context; the others stay where they are
    k = torch.arange(steps, device=DEV)
    seq = torch.arange(B, device=DEV)[:, None].expand(B, steps)
    keep = path >= 0
    to = torch.where(keep, ctx[:, None] + k, ctx[:, None].clamp(max=s["max_len"] - 1))
    frm = torch.where(keep, ctx[:, None] + path, to)
    result = dict(out)
    for i, c in enumerate(s["layers"]):
        a, b = _slots(c, seq, frm), _slots(c, seq, to)
        for name in ("k", "v", "k_scale", "v_scale"):
            if c[name] is not None:
                c[name][b[0], :, b[1]] = c[name][a[0], :, a[1]].clone()
        result |= _layer_values(c, i)
    return result


def _layer_values(c, i):
    out = {f"k{i}": _values(c, "k"), f"v{i}": _values(c, "v")}
    for name in ("k_scale", "v_scale"):
        if c[name] is not None:
            out[f"{name}{i}"] = c[name].view(torch.float8_e8m0fnu) if c[name].dtype == torch.uint8 else c[name]
    return out


def _dequantised(codes, scale, rows):
    R, K = codes.shape
    wide = scale.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :K]
    return codes.view(torch.float8_e4m3fn).float() * wide


def _plain_matmul(s):
    y = torch.matmul(_dequantised(s["a"], s["a_scale"], 1), _dequantised(s["b"], s["b_scale"], 128).T)
    if s["bias"] is not None:
        y = y + s["bias"]
    s["out"].copy_(y)
    return s["out"]


# --------------------------------------------------------------------- run --
def _handle(c, case):
    """The cache handle that a program keeps for the life of its cache."""
    if "handle" not in c:
        import fp8_quantized_kv_gb300 as fk
        c["handle"] = fk.Fp8KVCache(
            dtype=c["dtype"], layout=fk.LAYOUT_PAGED if c["page_size"] else fk.LAYOUT_CONTIGUOUS, batch=case["batch"],
            kv_heads=case["kv_heads"], head_dim=case["head_dim"], k=c["k"], v=c["v"], k_scale=c["k_scale"], v_scale=c["v_scale"],
            max_tokens=c["max_tokens"], page_size=c["page_size"], num_pages=c["num_pages"], page_table=c["page_table"])
    return c["handle"]


def _own(s):
    import fp8_quantized_kv_gb300 as fk
    c = s["case"]
    if c["op"] == "matmul":
        return fk.fp8kv_block_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], bias=s["bias"], out=s["out"])
    if c["op"] == "tables":
        fk.fp8kv_tree_tables(s["parents"], s["cu"], s["seq_lens"], c["max_nodes"], masks=s["out"]["masks"], pos=s["out"]["pos"])
        return s["out"]
    if c["op"] == "accept":
        o = s["out"]
        if "handles" not in s:
            s["handles"] = [_handle(x, c) for x in s["layers"]]
        fk.fp8kv_tree_accept(s["handles"], s["parents"], s["tokens"], s["choices"], s["cu"], s["seq_lens"], c["depth"],
                             path=o["path"], accepted=o["accepted"], next_tokens=o["next_tokens"], new_lens=o["lens"])
        result = dict(o)
        for i, x in enumerate(s["layers"]):
            result |= _layer_values(x, i)
        return result
    cache = _handle(s["cache"], c)
    if "workspace" not in s:
        need = fk.fp8kv_tree_workspace_bytes(cache, s["rows"], c["q_heads"], window=c["window"], sinks=c["sinks"])
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    return fk.fp8kv_tree_attention(s["q"], cache, s["cu"], s["seq_lens"], s["masks"], pos=s["pos"], window=c["window"],
                                   sinks=c["sinks"], out=s["out"], workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "attention": _plain_attention, "accept": _plain_accept, "matmul": _plain_matmul}[state["case"]["op"]](state)


# -------------------------------------------------------------------- work --
def _row_bytes(case, side):
    D = case["head_dim"]
    return D + 4 if case["dtype"] in (K_CODES if side == "k" else V_CODES) else 2 * D


def work(case):
    op = case["op"]
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // 128)
        return {"bytes": m * k + n * k + 4 * kb * (m + -(-n // 128)) + (4 if case["out"] == "f32" else 2) * m * n + (4 * n if case["bias"] else 0),
                "flops": 2.0 * m * n * k}
    ctx, trees, paths = _plan(case)
    n, B = sum(len(t) for t in trees), case["batch"]
    if op == "tables":
        rows, words = n + case["pad"], -(-case["max_nodes"] // 32)
        return {"bytes": 4 * n + 8 * B + 4 * rows * (words + 1), "flops": float(rows * words)}
    row = case["kv_heads"] * (_row_bytes(case, "k") + _row_bytes(case, "v"))
    if op == "accept":
        moved = sum(1 for p in paths for k, i in enumerate(p) if k != i)
        return {"bytes": 20 * n + 8 * B + B * (16 + 4 * case["depth"]) + 2 * moved * row * case["layers"], "flops": float(n)}
    W, S, Hq, D = case["window"], case["sinks"], case["q_heads"], case["head_dim"]
    keys = pairs = 0
    for c, t in zip(ctx, trees):
        low = max(0, c - W + 1) if W else 0
        keys += c - low + min(S, low) + len(t)
        depth = []
        for p in t:
            depth.append(depth[p] + 1 if p >= 0 else 0)
            first = max(0, c + depth[-1] - W + 1) if W else 0
            pairs += max(0, c - first) + min(S, min(first, c)) + depth[-1] + 1
    return {"bytes": keys * row + 4 * n * Hq * D + 4 * n * -(-case["max_nodes"] // 32), "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------------- exact --
def _code_values(codes):
    """fp64 values of e4m3 codes, from their bits."""
    u = codes.to(torch.int64)
    man, ex = (u & 7).double(), (u >> 3) & 15
    mag = torch.where(ex > 0, (8 + man) * torch.exp2(ex.double() - 10), man * 2.0 ** -9)
    return torch.where(u >= 128, -mag, mag)


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "accept":
        # row by row along the accepted paths, on the values that the rows stand for
        out = dict.fromkeys(s["out"])
        for i, c in enumerate(s["layers"]):
            for name in _layer_values(c, i):
                x = c[name[:-len(str(i))]]
                out[name] = x.double() if x.dtype != torch.uint8 else torch.exp2(x.double() - 127) if "scale" in name else _code_values(x)
        P = case["page_size"]
        for b, path in enumerate(s["paths"]):
            first = int(s["seq_lens"][b]) - len(s["trees"][b])
            for k, node in enumerate(path):
                (p0, r0), (p1, r1) = (((int(c["page_table"][b, t // P]), t % P) if P else (b, t)) for t in (first + node, first + k))
                for x in out.values():
                    if x is not None:
                        x[p1, :, r1] = x[p0, :, r0]
        return out
    if case["op"] == "matmul":
        # block by block: sums of code products, each scaled once
        y = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
        a, b = _code_values(s["a"]), _code_values(s["b"])
        block = torch.arange(case["n"], device=DEV) // 128
        for j in range(s["a_scale"].shape[1]):
            cut = slice(128 * j, min(128 * j + 128, case["k"]))
            y += (a[:, cut] @ b[:, cut].T) * s["a_scale"][:, j, None].double() * s["b_scale"][block, j].double()
        return y if s["bias"] is None else y + s["bias"].double()
    c, D, W, S = s["cache"], case["head_dim"], case["window"], case["sinks"]
    out = torch.zeros(s["rows"], case["q_heads"], D, dtype=torch.float64, device=DEV)
    G, r0 = case["q_heads"] // case["kv_heads"], 0
    for b, tree in enumerate(s["trees"]):
        T, n = int(s["seq_lens"][b]), len(tree)
        t = torch.arange(T, device=DEV)
        lead, off = _slots(c, torch.full_like(t, b), t)
        pair = []
        for side in ("k", "v"):
            x, scale = c[side][lead, :, off], c[side + "_scale"]
            if x.dtype != torch.uint8:
                pair.append(x.double())
                continue
            sc = scale[lead, :, off].double()
            pair.append(_code_values(x) * (torch.exp2(sc - 127).repeat_interleave(32, -1) if scale.dtype == torch.uint8 else sc[..., None]))
        hidden = torch.ones(n, T, dtype=torch.bool)
        for i in range(n):
            at, up = i, []
            while at >= 0:
                up.append(at)
                at = tree[at]
            low = max(0, T - n + len(up) - 1 - W + 1) if W else 0
            hidden[i, min(low, T - n):T - n] = False
            hidden[i, :min(S if W else 0, T - n)] = False
            hidden[i, [T - n + j for j in up]] = False
        hidden = hidden.to(DEV)
        for h in range(case["q_heads"]):
            z = (s["q"][r0:r0 + n, h].double() @ pair[0][:, h // G].T) / math.sqrt(D)
            z[hidden] = -math.inf
            out[r0:r0 + n, h] = torch.softmax(z, -1) @ pair[1][:, h // G]
        r0 += n
    return out
