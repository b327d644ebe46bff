"""What is measured of the operators for a decode batch of many requests.

What the requests of a batch share is read and computed once for all of them,
what each has of its own beside it: the linear shards on 4-bit weights with
the low-rank adapters of the tokens' requests, attention over a shared prefix
and every sequence's own tokens in a paged cache, and the store into that
cache.  Sizes are those of this library's decode workloads (1, 2, 4 and 8
ranks, hidden sizes 4096 and 8192 in heads of 128 with 8 of them in the
cache, 1 to 128 sequences) and of prompts run through the same layers.

`own` is False for the plain forms (elementary torch operations in binary32)
and True for the library's kernels.
"""
import random

import torch

own = False

E4M3_EMAX, E4M3_MAX = 8, 448.0
E2M1_EMAX, E2M1_MAX = 2, 6.0
BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
#: most work of a drawn attention: what the largest listed one has, roughly
ATTEND_MOST = 128 * 64 * 128 * 32768
#: most tokens x heads x dim of a drawn attention's own cache
CACHE_MOST = 8 * 32768 * 8 * 128


def up(n, m):
    return (n + m - 1) // m * m


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode token of a request with an adapter, a layer split over 8 ranks: nothing but latency
        {"name": "adapters_n8_1x4096x512_r16", "op": "adapters", "ranks": 8, "split": "rows", "m": 1, "n": 4096,
         "k": 512, "x": "bf16", "y": "bf16", "adapters": 32, "rank": 16, "index": "each"},
        # a decode batch of 16 requests, every one with an adapter of its own
        {"name": "adapters_n4_16x8192x2048_r16", "op": "adapters", "ranks": 4, "split": "rows", "m": 16, "n": 8192,
         "k": 2048, "x": "mx8", "y": "bf16", "adapters": 64, "rank": 16, "index": "each"},
        # ragged: tokens of 7 adapters and of none in any order, outputs split over the ranks, no size a multiple of a tile
        {"name": "adapters_n2_777x4000x2080_r24", "op": "adapters", "ranks": 2, "split": "columns", "m": 777, "n": 4000,
         "k": 2080, "x": "mx4", "y": "f32", "adapters": 7, "rank": 24, "index": "mixed"},
        # prompts of 8 requests one after the other: the matrix cores' rate
        {"name": "adapters_4096x8192x8192_r64", "op": "adapters", "ranks": 1, "split": "rows", "m": 4096, "n": 8192,
         "k": 8192, "x": "mx8", "y": "bf16", "adapters": 8, "rank": 64, "index": "requests"},
        # a decode step's keys and values into an 8-bit cache
        {"name": "append_16x1_row8", "op": "append", "sequences": 16, "queries": 1, "kv_heads": 8, "dim": 128,
         "page": 16, "own": 1000, "type": "bf16", "cache": "row8"},
        # chunks of 8 prompts into a cache of their own type
        {"name": "append_8x512_bf16", "op": "append", "sequences": 8, "queries": 512, "kv_heads": 8, "dim": 128,
         "page": 64, "own": 2048, "type": "bf16", "cache": "same"},
        # one request behind a system prompt
        {"name": "attend_1_prefix1000_own500", "op": "attend", "sequences": 1, "queries": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "prefix": 1000, "own": 500, "type": "bf16", "cache": "same"},
        # a decode batch behind a long one
        {"name": "attend_16_prefix8192_own1024", "op": "attend", "sequences": 16, "queries": 1, "heads": 64,
         "kv_heads": 8, "dim": 128, "page": 64, "prefix": 8192, "own": 1024, "type": "bf16", "cache": "same"},
        # two tokens at a time (one of them guessed), heads of 96, an odd prefix that ends inside a page
        {"name": "attend_37x2_prefix4999_d96", "op": "attend", "sequences": 37, "queries": 2, "heads": 40,
         "kv_heads": 8, "dim": 96, "page": 32, "prefix": 4999, "own": 777, "type": "f16", "cache": "same"},
        # few requests whose own text is long: the stream of the cache
        {"name": "attend_8_prefix512_own32768", "op": "attend", "sequences": 8, "queries": 1, "heads": 64,
         "kv_heads": 8, "dim": 128, "page": 64, "prefix": 512, "own": 32768, "type": "bf16", "cache": "same"},
        # many requests over one long document, 8-bit cache: the matrix cores' rate
        {"name": "attend_128_prefix32768_row8", "op": "attend", "sequences": 128, "queries": 1, "heads": 64,
         "kv_heads": 8, "dim": 128, "page": 64, "prefix": 32768, "own": 2048, "type": "bf16", "cache": "row8"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "attend", "attend", "append"])
    if op == "adapters":
        ranks = rng.choice([1, 2, 4, 8])
        m = _log(rng, 1, 4096 // ranks)
        n, k = _log(rng, 256, 8192), _log(rng, 256, 8192 // ranks)
        if rng.random() < 0.5:
            n, k = up(n, 16), up(k, 32)
        return {"op": op, "ranks": ranks, "split": rng.choice(["rows", "columns"]), "m": m, "n": n, "k": k,
                "x": rng.choice(["bf16", "mx8", "mx4", "row8"]), "y": rng.choice(["bf16", "f32"]),
                "adapters": _log(rng, 1, 16), "rank": _log(rng, 4, 64), "index": rng.choice(["each", "mixed", "requests"])}
    kv = rng.choice([1, 2, 4, 8])
    dim, page = rng.choice([64, 80, 96, 128, 128, 192, 256]), rng.choice([16, 32, 64, 128])
    t, cache = rng.choice(["bf16", "bf16", "f16"]), rng.choice(["same", "row8"])
    if op == "append":
        sequences, queries = _log(rng, 1, 128), _log(rng, 1, 32)
        return {"op": op, "sequences": sequences, "queries": queries, "kv_heads": kv, "dim": dim, "page": page,
                "own": queries + _log(rng, 1, 1024), "type": t, "cache": cache}
    sequences, queries = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 5, 8])
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    rows = sequences * queries * heads * dim
    prefix = rng.choice([0, 1, 1, 1, 1]) * min(_log(rng, 16, 32768), ATTEND_MOST // (2 * rows))
    most = min(ATTEND_MOST // (2 * rows), CACHE_MOST // (sequences * kv * dim), 32768)
    return {"op": op, "sequences": sequences, "queries": queries, "heads": heads, "kv_heads": kv, "dim": dim,
            "page": page, "prefix": prefix, "own": queries + min(_log(rng, 1, 32768), most), "type": t, "cache": cache}


def _lengths(case):
    """Tokens of each sequence: the first has all of them, the others from a quarter on; in a batch
    of more than four, one has none yet."""
    rng = random.Random(131 * case["own"] + case["sequences"])
    n = [max(case["queries"], case["own"] - int(0.75 * case["own"] * rng.random())) for _ in range(case["sequences"])]
    n[0] = case["own"]
    if len(n) > 4:
        n[len(n) // 2] = 0
    return n


# ----------------------------------------------------- formats, plain form --

def _pow2(e):
    """2**e in binary32 for whole e in [-149, 127]."""
    return torch.ldexp(torch.ones((), device=e.device, dtype=torch.float64), e).float()


def _mx(v, emax):
    """Block values times 2**-e and the biased exponents, of finite rows."""
    rows, cols = v.shape
    b = torch.nn.functional.pad(v, (0, up(cols, BLOCK) - cols)).view(rows, -1, BLOCK)
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 1 - emax).clamp(-127, 127)
    e = torch.where(amax == 0, -127, e)
    return b * _pow2(-e).unsqueeze(-1), (e + 127).to(torch.uint8)


def _e2m1(q):
    """Nearest 4-bit value (ties to the even mantissa), as binary32."""
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=E2M1_MAX), q)


def _to_mx8(v):
    q, s = _mx(v, E4M3_EMAX)
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(v.shape[0], -1), s


def _to_mx4(v):
    q, s = _mx(v, E2M1_EMAX)
    return _e2m1(q).view(v.shape[0], -1), s


def _to_row8(v):
    """8-bit codes of rows (the last dimension) and a scale for each."""
    s = (v.abs().amax(-1) / E4M3_MAX).clamp(min=2.0 ** -126)
    return (v * (1 / s).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def _pack4(q):
    """4-bit values (binary32) -> codes, two in a byte, the even column low."""
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack4(codes):
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return lut[c.int()]


def _values(codes, scales, fmt):
    """What codes and scales stand for, in binary32."""
    if fmt == "row8":
        return codes.float() * scales.unsqueeze(-1)
    q = _unpack4(codes) if fmt == "mx4" else codes.float()
    s = _pow2(scales.int() - 127)
    return (q.unflatten(-1, (-1, BLOCK)) * s.unsqueeze(-1)).flatten(-2)


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _pad_scales(s):
    """Scale rows of a multiple of 4 bytes."""
    return torch.nn.functional.pad(s, (0, up(s.shape[1], 4) - s.shape[1]))


def _index(case, g):
    """The adapter of every token, -1 for none."""
    m, count = case["m"], case["adapters"]
    if case["index"] == "each":          # a batch of single tokens
        return (torch.randperm(up(m, count), generator=g, device="cuda")[:m] % count).int()
    if case["index"] == "mixed":         # any order, some without
        return torch.randint(-1, count, (m,), generator=g, device="cuda", dtype=torch.int32)
    return (torch.arange(m, device="cuda") * count // m).int()


def _prepare_adapters(case, g, s):
    ranks, m, n, k, columns = case["ranks"], case["m"], case["n"], case["k"], case["split"] == "columns"
    count, rank = case["adapters"], case["rank"]
    inputs = k if columns else ranks * k
    w4, ws = _to_mx4(_normal(g, ranks * n, k) * inputs ** -0.5)
    s["w"], s["w_scales"] = _pack4(w4).view(ranks, n, -1), _pad_scales(ws).view(ranks, n, -1)
    del w4
    xr = 1 if columns else ranks         # the ranks share the tokens, or each has a slice of them
    x = _normal(g, xr * m, k) * torch.empty((xr * m, 1), device="cuda").uniform_(0.5, 2, generator=g)
    if case["x"] == "bf16":
        s["x"], s["x_scales"] = torch.zeros((xr, m, up(k, 8)), dtype=torch.bfloat16, device="cuda"), None
        s["x"][..., :k] = x.view(xr, m, k)
    elif case["x"] == "row8":
        c, sc = _to_row8(x)
        s["x"] = torch.zeros((xr, m, up(k, 16)), dtype=torch.float8_e4m3fn, device="cuda")
        s["x"].view(torch.uint8)[..., :k] = c.view(torch.uint8).view(xr, m, k)
        s["x_scales"] = sc.view(xr, m)
    else:
        c, sc = _to_mx8(x) if case["x"] == "mx8" else _to_mx4(x)
        s["x"] = (c if case["x"] == "mx8" else _pack4(c)).view(xr, m, -1)
        s["x_scales"] = _pad_scales(sc).view(xr, m, -1)
    ar, br = (1, ranks) if columns else (ranks, 1)
    s["a"] = torch.zeros((ar, count, rank, up(k, 8)), dtype=torch.bfloat16, device="cuda")
    s["a"][..., :k] = _normal(g, ar, count, rank, k) * inputs ** -0.5
    s["b"] = torch.zeros((br, count, n, up(rank, 8)), dtype=torch.bfloat16, device="cuda")
    s["b"][..., :rank] = _normal(g, br, count, n, rank) * (0.5 * rank ** -0.5)
    s["index"] = _index(case, g)
    s["scale"] = torch.empty(count, device="cuda").uniform_(0.25, 1, generator=g)
    s["y"] = torch.empty((ranks, m, n), dtype=TYPES[case["y"]], device="cuda")
    if own:
        from collective_synchronization_amd import abi
        x, xs, w, ws, a, b, y = s["x"], s["x_scales"], s["w"], s["w_scales"], s["a"], s["b"], s["y"]
        s["linear"] = abi.linear_params(
            ranks, m, n, k, case["x"], x, x.stride(1), 0 if columns else x.stride(0),
            xs, 0 if xs is None or case["x"] == "row8" else xs.stride(1), 0 if xs is None or columns else xs.stride(0),
            w, w.stride(1), w.stride(0), ws, ws.stride(1), ws.stride(0), case["y"], y, y.stride(1), y.stride(0))
        s["adapters"] = abi.adapter_params(
            count, rank, s["index"], s["scale"], a, a.stride(2), a.stride(1), 0 if columns else a.stride(0),
            b, b.stride(2), b.stride(1), b.stride(0) if columns else 0)
        s["work"] = torch.empty(abi.ar_adapter_work_bytes(s["linear"], s["adapters"]), dtype=torch.uint8, device="cuda")


def _prepare_cache(case, g, s):
    """The paged cache, its tables in an order of no meaning, and the sequences' tokens."""
    n, kv, dim, page = case["sequences"], case["kv_heads"], case["dim"], case["page"]
    prefix = case.get("prefix", 0)
    lengths = _lengths(case)
    width = max(1, up(case["own"], page) // page)
    used = [up(x, page) // page for x in lengths]
    shared = up(prefix, page) // page
    pages = shared + sum(used) + 1
    order = torch.randperm(pages, generator=g, device="cuda").int()
    s["prefix_pages"] = order[:shared].contiguous()
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    at = shared
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    s["pages"] = table
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for name in ("k", "v"):
        shape = (pages, page, kv, dim)
        if case["op"] == "append":       # free pages
            rows = torch.zeros(shape, dtype=TYPES[case["type"]], device="cuda")
        else:
            rows = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16).to(TYPES[case["type"]])
        if case["cache"] == "row8":
            c = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
            sc = torch.empty(shape[:3], device="cuda")
            for i in range(0, pages, 4096):
                c[i:i + 4096], sc[i:i + 4096] = _to_row8(rows[i:i + 4096].float())
            s[name + "_cache"], s[name + "_scales"] = c, sc
        else:
            s[name + "_cache"], s[name + "_scales"] = rows, None
    if own:
        from collective_synchronization_amd import abi
        k, ks = s["k_cache"], s["k_scales"]
        strides = (0, 0, 0) if ks is None else ks.stride()
        s["cache"] = abi.cache_params(case["type"] if ks is None else "row8", pages, page, kv, dim, k, s["v_cache"],
                                      k.stride(0), k.stride(1), k.stride(2), ks, s["v_scales"], *strides)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "adapters":
        _prepare_adapters(case, g, s)
        return s
    _prepare_cache(case, g, s)
    t, tokens, dim = TYPES[case["type"]], case["sequences"] * case["queries"], case["dim"]
    if op == "append":
        s["k"] = _normal(g, tokens, case["kv_heads"], dim).to(t)
        s["v"] = _normal(g, tokens, case["kv_heads"], dim).to(t)
        return s
    # some heads look at few tokens, some at all
    sharp = torch.empty((1, case["heads"], 1), device="cuda").uniform_(0.5, 3, generator=g)
    s["q"] = (_normal(g, tokens, case["heads"], dim) * sharp).to(t)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((tokens, case["heads"]), device="cuda")
    if own:
        from collective_synchronization_amd import abi
        q, out = s["q"], s["out"]
        s["attention"] = abi.attention_params(
            s["cache"], case["sequences"], case["queries"], case["heads"], dim ** -0.5, case["type"],
            q, q.stride(0), q.stride(1), out, out.stride(0), out.stride(1), s["lse"], s["lse"].stride(0),
            case["prefix"], s["prefix_pages"], s["lengths"], s["pages"], s["pages"].stride(0), s["pages"].shape[1])
        s["work"] = torch.empty(abi.ar_prefix_attention_work_bytes(s["attention"]), dtype=torch.uint8, device="cuda")
    return s


# -------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if op == "adapters":
        return _run_adapters_own(s) if own else _run_adapters_plain(s)
    if op == "append":
        return _run_append_own(s) if own else _run_append_plain(s)
    return _run_attend_own(s) if own else _run_attend_plain(s)


def _run_adapters_own(s):
    from collective_synchronization_amd import abi
    abi.ar_mx4_linear_adapters(s["linear"], s["adapters"], s["work"])
    return {"y": s["y"]}


def _run_adapters_plain(s):
    case = s["case"]
    ranks, m, k, rank, count = case["ranks"], case["m"], case["k"], case["rank"], case["adapters"]
    x = s["x"]
    if case["x"] == "bf16":
        x = x.float()
    else:
        x = _values(x, s["x_scales"] if case["x"] == "row8" else s["x_scales"][..., :up(k, BLOCK) // BLOCK], case["x"])
    x = x[..., :k].contiguous()
    w = _values(s["w"], s["w_scales"][..., :up(k, BLOCK) // BLOCK], "mx4")[..., :k]
    y = torch.matmul(x, w.transpose(1, 2).contiguous())
    index = s["index"].long()
    none = (index < 0) | (index >= count)
    if m <= 64:                          # every token's own adapter
        at = index.clamp(0, count - 1)
        a = s["a"][:, at, :, :k].float()                             # [a ranks, m, rank, k]
        t = torch.matmul(a, x.unsqueeze(-1)).squeeze(-1)             # [x ranks, m, rank]
        t = torch.where(none.unsqueeze(-1), 0.0, t * s["scale"][at].unsqueeze(-1))
        y += torch.matmul(s["b"][:, at, :, :rank].float(), t.unsqueeze(-1)).squeeze(-1)
    else:                                # one adapter after the other
        for i in range(count):
            a, b = s["a"][:, i, :, :k].float(), s["b"][:, i, :, :rank].float()
            t = torch.matmul(x, a.transpose(1, 2).contiguous()) * s["scale"][i]
            t = torch.where((index == i).unsqueeze(-1), t, 0.0)
            y += torch.matmul(t, b.transpose(1, 2).contiguous())
    return {"y": y.to(TYPES[case["y"]])}


def _cache_out(s):
    out = {"k": s["k_cache"], "v": s["v_cache"]}
    if s["k_scales"] is not None:
        out |= {"k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    return out


def _run_append_own(s):
    from collective_synchronization_amd import abi
    case, k, v = s["case"], s["k"], s["v"]
    abi.ar_cache_append(s["cache"], case["sequences"], case["queries"], case["type"], k, k.stride(0), k.stride(1),
                        v, v.stride(0), v.stride(1), s["lengths"], s["pages"], s["pages"].stride(0),
                        s["pages"].shape[1])
    return _cache_out(s)


def _run_append_plain(s):
    case = s["case"]
    n, page = case["queries"], case["page"]
    at = (s["lengths"].long().unsqueeze(1) - n + torch.arange(n, device=s["k"].device)).flatten()
    seq = torch.arange(case["sequences"], device=s["k"].device).repeat_interleave(n)
    keep = at >= 0
    at, seq = at[keep], seq[keep]
    where = s["pages"][seq, at // page].long(), at % page
    for name in ("k", "v"):
        rows, cache, scales = s[name][keep], s[name + "_cache"], s[name + "_scales"]
        if scales is None:
            cache[where] = rows
        else:
            c, sc = _to_row8(rows.float())
            cache.view(torch.uint8)[where] = c.view(torch.uint8)
            scales[where] = sc
    return _cache_out(s)


def _run_attend_own(s):
    from collective_synchronization_amd import abi
    abi.ar_prefix_attention(s["attention"], s["work"])
    return {"out": s["out"], "lse": s["lse"]}


def _gather(s, name, pages):
    """Pages' rows in binary32: [..., tokens, kv_heads, dim]."""
    rows = s[name + "_cache"]
    if s[name + "_scales"] is None:
        return rows[pages].float().flatten(-4, -3)
    return (rows.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
            * s[name + "_scales"][pages].unsqueeze(-1)).flatten(-4, -3)


def _run_attend_plain(s):
    case = s["case"]
    b, n, heads, kv, dim, prefix = (case[x] for x in ("sequences", "queries", "heads", "kv_heads", "dim", "prefix"))
    group = heads // kv
    q = s["q"].float().view(b, n, kv, group, dim).permute(2, 0, 1, 3, 4).contiguous()      # [kv, b, n, group, dim]
    # every sequence's own tokens, masked behind its length and behind each query
    pages = s["pages"].long().clamp(min=0)
    k, v = (_gather(s, x, pages).permute(2, 0, 1, 3).contiguous() for x in ("k", "v"))     # [kv, b, tokens, dim]
    so = torch.matmul(q.flatten(2, 3), k.transpose(2, 3).contiguous()) * dim ** -0.5
    limit = s["lengths"].unsqueeze(1) - n + 1 + torch.arange(n, device=q.device)           # [b, n]
    seen = torch.arange(k.shape[2], device=q.device) < limit.unsqueeze(-1)
    so = so.view(kv, b, n, group, -1).masked_fill(~seen[:, :, None, :], float("-inf"))
    m = so.amax(-1)
    if prefix:
        # the shared ones, all sequences' queries at once
        at = s["prefix_pages"].long()
        pk, pv = (_gather(s, x, at)[:prefix].transpose(0, 1).contiguous() for x in ("k", "v"))
        sp = torch.matmul(q.flatten(1, 3), pk.transpose(1, 2).contiguous()) * dim ** -0.5
        sp = sp.view(kv, b, n, group, prefix)
        m = torch.maximum(m, sp.amax(-1))
    safe = torch.where(m == float("-inf"), 0.0, m).unsqueeze(-1)
    po = torch.exp(so - safe)
    l, o = po.sum(-1), torch.matmul(po.flatten(2, 3), v).view(kv, b, n, group, dim)
    if prefix:
        pp = torch.exp(sp - safe)
        l += pp.sum(-1)
        o += torch.matmul(pp.flatten(1, 3), pv).view(kv, b, n, group, dim)
    o /= torch.where(l > 0, l, 1.0).unsqueeze(-1)
    lse = m + torch.log(l)
    return {"out": o.permute(1, 2, 0, 3, 4).reshape(b * n, heads, dim).to(s["q"].dtype),
            "lse": lse.permute(1, 2, 0, 3).reshape(b * n, heads)}


# ------------------------------------------------------- work and 64 bits --

def _row_bytes(cols, fmt):
    """Bytes of one row of a format, its scales among them."""
    if fmt in TYPES:
        return cols * TYPES[fmt].itemsize
    if fmt == "row8":
        return cols + 4
    return (cols if fmt == "mx8" else cols / 2) + up(cols, BLOCK) / BLOCK


def _adapters_used(case):
    if case["index"] == "each":
        return min(case["m"], case["adapters"])
    return min(case["adapters"], case["m"])


def work(case):
    if case["op"] == "adapters":
        ranks, m, n, k, rank = (case[x] for x in ("ranks", "m", "n", "k", "rank"))
        ar, br = (1, ranks) if case["split"] == "columns" else (ranks, 1)
        used = _adapters_used(case)
        b = ranks * (n * _row_bytes(k, "mx4") + m * n * TYPES[case["y"]].itemsize)
        b += ar * (m * _row_bytes(k, case["x"]) + used * rank * k * 2) + br * used * n * rank * 2
        tokens = m * case["adapters"] / (case["adapters"] + 1) if case["index"] == "mixed" else m
        return {"bytes": b, "flops": 2.0 * ranks * m * n * k + 2.0 * tokens * rank * (ar * k + ranks * n)}
    lengths, n = _lengths(case), case["queries"]
    kv, dim, size = case["kv_heads"], case["dim"], TYPES[case["type"]].itemsize
    row = dim * size if case["cache"] == "same" else dim + 4
    if case["op"] == "append":
        return {"bytes": 2 * kv * sum(min(x, n) for x in lengths) * (dim * size + row), "flops": 0}
    rows = case["sequences"] * n * case["heads"]
    keys = sum(max(x - n + 1 + i, 0) for x in lengths for i in range(n)) * case["heads"] + rows * case["prefix"]
    return {"bytes": 2 * kv * (case["prefix"] + sum(lengths)) * row + rows * (2 * dim * size + 4),
            "flops": 4.0 * keys * dim}


def _grid(values, v):
    """The nearest of the ascending `values` to each |v|, ties to the even place, with v's sign."""
    t = torch.tensor(values, dtype=torch.float64, device=v.device)
    mid = (t[1:] + t[:-1]) / 2
    a = v.abs().contiguous()
    lo, hi = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)  # they differ at a tie alone
    return torch.copysign(t[torch.where(lo % 2 == 0, lo, hi)], v)


def _exact_adapters(case, s):
    k, rank = case["k"], case["rank"]
    four = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")

    def blocks(scales):
        return torch.pow(2.0, scales.double() - 127).repeat_interleave(32, -1)[..., :k]

    def nibbles(codes):
        c = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.int64, device="cuda")
        c[..., ::2], c[..., 1::2] = codes % 16, codes // 16
        return (four[c % 8] * (1 - 2 * (c // 8)))[..., :k]

    if case["x"] == "mx4":
        x = nibbles(s["x"]) * blocks(s["x_scales"])
    else:
        x = s["x"][..., :k].double()
        if case["x"] == "row8":
            x = x * s["x_scales"].double()[..., None]
        elif case["x"] == "mx8":
            x = x * blocks(s["x_scales"])
    out = []
    for r in range(case["ranks"]):
        xr, a, b = (s_[r % s_.shape[0]] for s_ in (x, s["a"], s["b"]))
        y = xr @ (nibbles(s["w"][r]) * blocks(s["w_scales"][r])).t().contiguous()
        for i in set(s["index"].tolist()) - {-1}:
            at = (s["index"] == i).nonzero().flatten()
            t = xr[at] @ a[i, :, :k].double().t().contiguous() * s["scale"][i].double()
            y[at] += t @ b[i, :, :rank].double().t().contiguous()
        out.append(y)
    return {"y": torch.stack(out)}


def _exact_append(case, s):
    n, page = case["queries"], case["page"]
    out = {x: y.double().clone() for x, y in _cache_out(s).items()}
    values = [m / 512 for m in range(8)] + [2.0 ** (e - 7) * (1 + m / 8) for e in range(1, 16) for m in range(8)][:-1]
    for i, length in enumerate(_lengths(case)):
        first = max(0, n - length)       # a sequence of fewer tokens takes none that come before its first
        at = torch.arange(length - n + first, length, device="cuda")
        where = s["pages"][i].long()[at // page], at % page
        for name in ("k", "v"):
            rows = s[name][i * n + first:(i + 1) * n].double()
            if case["cache"] == "row8":
                sc = (rows.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
                out[name + "_scales"][where] = sc
                rows = _grid(values, rows / sc[..., None])
            out[name][where] = rows
    return out


def _exact_attend(case, s):
    n, heads, kv, dim, page = (case[x] for x in ("queries", "heads", "kv_heads", "dim", "page"))
    group = heads // kv
    out = torch.zeros((case["sequences"] * n, heads, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((case["sequences"] * n, heads), float("-inf"), dtype=torch.float64, device="cuda")

    def rows(name, table, count):
        t = table[:up(count, page) // page].long()
        v = s[name + "_cache"].view(torch.uint8)[t].view(s[name + "_cache"].dtype).double()
        if s[name + "_scales"] is not None:
            v = v * s[name + "_scales"][t].double()[..., None]
        return v.flatten(0, 1)[:count]

    shared = [rows(x, s["prefix_pages"], case["prefix"]) for x in ("k", "v")]
    for i, length in enumerate(_lengths(case)):
        mine = [rows(x, s["pages"][i], length) for x in ("k", "v")]
        for j in range(n):
            seen = max(0, length - n + 1 + j)
            for h in range(kv):
                k, v = (torch.cat((a[:, h], b[:seen, h])) for a, b in zip(shared, mine))
                if not len(k):
                    continue
                at = i * n + j, slice(h * group, (h + 1) * group)
                score = s["q"][at].double() @ k.t().contiguous() / dim ** 0.5
                lse[at] = torch.logsumexp(score, -1)
                out[at] = torch.exp(score - lse[at][:, None]) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"adapters": _exact_adapters, "append": _exact_append, "attend": _exact_attend}[case["op"]](case, s)
