"""Performance cases of the operators that a decoding step needs beside the MoE layer.

Four operators over one paged key-value cache: the attention of one new token per sequence, the append of
new keys and values (and reading them back), the page operations (fork with copy-on-write, compaction), and
the selection of a beam search. ``run`` computes one pass: with ``own`` false in plain torch operations, with
``own`` true through the package's entry points. ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF16, F32, D64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
INF = math.inf


# --------------------------------------------------------------------------- cases
def _attn(name, B, L, heads, kv_heads, D, page, precision="bf16", ragged=False, window=0):
    return dict(name=name, op="attn", B=B, L=L, heads=heads, kv_heads=kv_heads, D=D, page=page, precision=precision,
                ragged=ragged, window=window)


def _append(name, kind, n, L, kv_heads, D, page, precision):
    return dict(name=name, op="append", kind=kind, n=n, L=L, kv_heads=kv_heads, D=D, page=page, precision=precision)


def _pages(name, kind, groups, beams, L, layers, kv_heads, D, page, precision):
    return dict(name=name, op="pages", kind=kind, groups=groups, beams=beams, L=L, layers=layers, kv_heads=kv_heads,
                D=D, page=page, precision=precision)


def _beam(name, N, W, V, K, dtype, done=False, first=False):
    return dict(name=name, op="beam", N=N, W=W, V=V, K=K, dtype=dtype, done=done, first=first)


def listed():
    return [
        # the first tokens after a short prompt, one sequence: nothing but latency
        _attn("attention 1 x 100", 1, 100, 32, 8, 128, 16),
        # one very long sequence: the cache's length is all there is to split
        _attn("attention 1 x 131072", 1, 131072, 32, 8, 128, 16),
        # a serving batch whose sequences are anywhere between their first token and 8192
        _attn("attention 64 ragged", 64, 8192, 32, 8, 128, 16, ragged=True),
        # the 8-bit cache of a full batch, the largest there is
        _attn("attention 32 x 16384 mxfp8", 32, 16384, 32, 8, 128, 32, precision="mxfp8"),
        # seven query heads to a key head, narrow heads, a sliding window, lengths and pages that end anywhere
        _attn("attention 5 ragged, window 1000", 5, 20011, 56, 8, 64, 24, ragged=True, window=1000),
        # the append of one decoding step
        _append("append 64 tokens", "step", 64, 512, 8, 128, 16, "bf16"),
        # prompts written to the 8-bit cache and read back for their own attention
        _append("append 8192 tokens mxfp8", "prompt", 8192, 1021, 8, 128, 32, "mxfp8"),
        # one beam search's step: 4 beams, one layer
        _pages("fork 4 beams", "fork", 1, 4, 300, 1, 8, 128, 16, "bf16"),
        # a batch of beam searches over four layers: tables, page counts and the copied last pages
        _pages("fork 32 x 8 beams, 4 layers", "fork", 32, 8, 2048, 4, 8, 128, 16, "bf16"),
        # a fragmented pool made dense again
        _pages("compact 2 layers", "compact", 16, 4, 4096, 2, 8, 128, 16, "bf16"),
        # one beam search over a small vocabulary
        _beam("beams 1 x 4 x 32000", 1, 4, 32000, 8, "fp32"),
        # a batch of beam searches over a large one
        _beam("beams 32 x 8 x 131072 bf16", 32, 8, 131072, 16, "bf16", done=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "pages", "beam", "beam"])
    kv_heads, page = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    precision = rng.choice(["bf16", "bf16", "mxfp8"])
    D = rng.choice([64, 128, 128, 256, 96] + ([80] if precision == "bf16" else []))
    if op == "attn":
        B = _log(rng, 1, 256)
        L = _log(rng, 1, 131072)
        L = max(1, min(L, 131072 * 8 * 128 // (B * kv_heads * D)))
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        return dict(op="attn", B=B, L=L, heads=kv_heads * group, kv_heads=kv_heads, D=D, page=page, precision=precision,
                    ragged=rng.random() < 0.6, window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))
    if op == "append":
        kind = rng.choice(["step", "prompt"])
        n = _log(rng, 1, 256) if kind == "step" else _log(rng, 1, 8192)
        return dict(op="append", kind=kind, n=n, L=_log(rng, 1, 512 if kind == "step" else 4096), kv_heads=kv_heads, D=D,
                    page=page, precision=precision)
    if op == "pages":
        groups, beams = _log(rng, 1, 32), rng.choice([1, 2, 4, 5, 8])
        L, layers = _log(rng, 1, 4096), rng.choice([1, 2, 4])
        L = max(1, min(L, 2 ** 28 // (groups * beams * layers * kv_heads * D)))
        return dict(op="pages", kind=rng.choice(["fork", "compact"]), groups=groups, beams=beams, L=L, layers=layers,
                    kv_heads=kv_heads, D=D, page=max(page, 8), precision=precision)
    N, W = _log(rng, 1, 32), _log(rng, 1, 16)
    V = min(_log(rng, 64, 200000), 32 * 8 * 131072 // (N * W))
    return dict(op="beam", N=N, W=W, V=V, K=rng.choice([W, 2 * W]), dtype=rng.choice(["bf16", "fp32"]),
                done=rng.random() < 0.4, first=rng.random() < 0.2)


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(shape, std, g, dtype):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):                 # bounds the 32-bit temporary
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV).mul_(std))
    return out


def _mxfp8(v):
    """fp32 or fp64 [..., C] -> (codes, scale bytes): per 32 elements the power of two
    floor(log2(amax)) - 8, elements rounded to nearest even and saturated to +-448."""
    b = v.unflatten(-1, (v.shape[-1] // 32, 32))
    amax = b.abs().amax(-1)
    byte = (torch.frexp(amax).exponent - 1 - 8 + 127).clamp(0, 254)
    byte = torch.where(amax == 0, torch.full_like(byte, 127), byte)
    scaled = b * torch.exp2((127 - byte).to(v.dtype)).unsqueeze(-1)
    codes = scaled.clamp(-448, 448).to(F32).to(torch.float8_e4m3fn).flatten(-2)
    return codes.view(torch.uint8), byte.to(torch.uint8)


def _mxfp8_value(codes, byte, dtype):
    v = codes.view(torch.float8_e4m3fn).to(F32).to(dtype).unflatten(-1, (codes.shape[-1] // 32, 32))
    return (v * torch.exp2(byte.to(dtype) - 127).unsqueeze(-1)).flatten(-2)


def _pool(c, pages, std, g):
    """(values or codes, scale bytes) [pages, kv_heads, page, D] of one side of the cache."""
    shape = (pages, c["kv_heads"], c["page"], c["D"])
    if c["precision"] == "bf16":
        return _normal(shape, std, g, BF16), None
    codes = torch.empty(shape, dtype=torch.uint8, device=DEV)
    byte = torch.empty(shape[:-1] + (c["D"] // 32,), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, pages, step):
        codes[i:i + step], byte[i:i + step] = _mxfp8(_normal((min(step, pages - i),) + shape[1:], std, g, F32))
    return codes, byte


def _lengths(c):
    """The sequences' lengths, by the case alone: so many tokens are there to read or to hold."""
    L = c["L"]
    r = random.Random(L * 7919 + c.get("B", 0) + c.get("n", 0) + c.get("groups", 0))
    if c["op"] == "attn":
        if not c["ragged"]:
            return [L] * c["B"]
        drawn = [min(L, int(math.exp(r.random() * math.log(L + 1)))) for _ in range(c["B"])]
        return [0 if r.random() < 0.03 else n for n in drawn]  # a slot without a sequence
    if c["op"] == "append":
        if c["kind"] == "step":
            return [r.randint(0, L) for _ in range(c["n"])]
        S = (c["n"] + L - 1) // L                              # whole prompts of L tokens, the last one shorter
        return [L] * (S - 1) + [c["n"] - (S - 1) * L]
    drawn = [max(1, int(L / math.exp(r.random() * math.log(L) * 0.5))) for _ in range(c["groups"])]
    return [n for n in drawn for _ in range(c["beams"])]       # a group's beams are of one length


def _rows(lengths, page, width, spare, g):
    """Pages for the sequences' lengths in random order: (table [rows, width], pages of the pool)."""
    held = (lengths + page - 1) // page
    mine = torch.arange(width, device=DEV)[None] < held[:, None]
    n = int(held.sum())
    pages = n + spare
    table = torch.full(mine.shape, -1, dtype=I32, device=DEV)
    table[mine] = torch.randperm(pages, generator=g, device=DEV)[:n].to(I32)
    return table, pages


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "beam":
        N, W, V = c["N"], c["W"], c["V"]
        s = dict(case=c, logits=_normal((N, W, V), 2.5, g, BF16 if c["dtype"] == "bf16" else F32), done=None,
                 scores=-10 * torch.rand((N, W), generator=g, device=DEV))
        if c["first"]:                                         # a search's first step: one beam lives
            s["scores"][:, 0] = 0.0
            s["scores"][:, 1:] = -INF
        if c["done"]:
            s["done"] = torch.rand((N, W), generator=g, device=DEV) < 0.2
        return s
    page, L, D = c["page"], c["L"], c["D"]
    width = (L + page) // page                                 # room for a token past the longest
    lengths = torch.tensor(_lengths(c), dtype=I32, device=DEV)
    if c["op"] == "attn":
        B = c["B"]
        table, pages = _rows(lengths, page, width, 7, g)
        k, ks = _pool(c, pages, 1.0, g)
        v, vs = _pool(c, pages, 1.0, g)
        return dict(case=c, q=_normal((B, c["heads"], D), 1.5, g, BF16), k=k, k_scales=ks, v=v, v_scales=vs, table=table,
                    lengths=lengths)
    if c["op"] == "append":
        n = c["n"]
        if c["kind"] == "step":                                # one token to each sequence, some slots empty
            table, pages = _rows(lengths + 1, page, width, 3, g)
            rows, positions = None, lengths.clone()
            positions[torch.rand(n, generator=g, device=DEV) < 0.05] = -1
        else:
            at = torch.arange(n, device=DEV, dtype=I32)
            rows, positions = at // L, at % L
            table, pages = _rows(lengths, page, width, 3, g)
        qkv = _normal((n, 3 * c["kv_heads"], D), 1.0, g, BF16)  # keys and values are slices of one projection
        k, ks = _pool(c, pages, 1.0, g)
        v, vs = _pool(c, pages, 1.0, g)
        return dict(case=c, qkv=qkv, k=k, k_scales=ks, v=v, v_scales=vs, table=table, rows=rows, positions=positions)
    S = c["groups"] * c["beams"]
    table, pages = _rows(lengths, page, width, 0, g)
    if c["kind"] == "fork":
        # the beams' first half of pages is the one prefix that they share
        shared = (lengths // 2 // page)[:, None] > torch.arange(width, device=DEV)[None]
        first = table.view(c["groups"], c["beams"], width)[:, :1].expand(-1, c["beams"], -1).reshape(S, width)
        table = torch.where(shared, first, table)
        parents = torch.randint(0, c["beams"], (c["groups"], c["beams"]), generator=g, device=DEV, dtype=I32)
        parents += torch.arange(c["groups"], device=DEV, dtype=I32)[:, None] * c["beams"]
        parents = parents.view(-1)
        parents[torch.rand(S, generator=g, device=DEV) < 0.02] = -1             # a beam that ends
        pages += S
    else:
        # every third sequence or so has left
        gone = torch.rand(S, generator=g, device=DEV) < 0.35
        table[gone] = -1
        parents = None
    layers = [dict(zip(("k", "k_scales", "v", "v_scales"), _pool(c, pages, 1.0, g) + _pool(c, pages, 1.0, g)))
              for _ in range(c["layers"])]
    return dict(case=c, table=table, lengths=lengths, parents=parents, pages=pages, layers=layers)


# --------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    return {"attn": _plain_attn, "append": _plain_append, "pages": _plain_pages, "beam": _plain_beam}[c["op"]](c, state)


def _cache(c, s):
    from dropless_moe_expert_router_gb300 import api
    return api.PagedCache(c["precision"], s["k"].shape[0], c["kv_heads"], c["page"], c["D"], s["k"], s["k_scales"], s["v"],
                          s["v_scales"])


def _run_own(c, s):
    from dropless_moe_expert_router_gb300 import api
    if c["op"] == "beam":
        if "workspace" not in s:                               # what a server keeps
            s["workspace"] = api.moe_beam_select_workspace(s["logits"], c["K"])
        o = api.moe_beam_select(s["logits"], s["scores"], c["K"], done=s["done"], pad=1, workspace=s["workspace"])
        return dict(scores=o.scores, parents=o.parents, tokens=o.tokens)
    if c["op"] == "attn":
        if "cache" not in s:
            s["cache"] = _cache(c, s)
            s["workspace"] = api.moe_paged_attention_workspace(s["cache"], c["B"], c["heads"])
        out, lse = api.moe_paged_attention(s["q"], s["cache"], s["table"], s["lengths"], window=c["window"],
                                           workspace=s["workspace"])
        return dict(out=out, lse=lse)
    if c["op"] == "append":
        if "cache" not in s:
            s["cache"] = _cache(c, s)
        h = c["kv_heads"]
        api.moe_cache_append(s["qkv"][:, h:2 * h], s["qkv"][:, 2 * h:], s["cache"], s["table"], s["positions"],
                             rows=s["rows"])
        if c["precision"] == "bf16":
            return dict(k=s["k"], v=s["v"])
        k, v = api.moe_cache_gather(s["cache"], s["table"], s["positions"], rows=s["rows"])
        return dict(k=k, v=v)
    if "caches" not in s:
        s["caches"] = [_cache(c, layer) for layer in s["layers"]]
        s["workspace"] = api.moe_cache_pages_workspace(s["pages"], s["table"].shape[0], DEV)
    if c["kind"] == "fork":
        o = api.moe_cache_fork(s["table"], s["lengths"], s["parents"], s["pages"], c["page"], room=1,
                               workspace=s["workspace"])
        out = dict(table=o.table, lengths=o.lengths, src=o.src, dst=o.dst, used=o.used)
    else:
        o = api.moe_cache_compact(s["table"], s["pages"], workspace=s["workspace"])
        out = dict(table=o.table, src=o.src, dst=o.dst, used=o.used)
    api.moe_cache_copy_pages(s["caches"], o.src, o.dst)
    return dict(out, layers=_layers_out(c, s))


def _layers_out(c, s):
    """The pools; what is held in 8 bits as the values of the layers' codes and their scales' exponents."""
    if c["precision"] == "bf16":
        return [(p["k"], p["v"]) for p in s["layers"]]
    fp8 = torch.float8_e4m3fn
    return [(p["k"].view(fp8), p["k_scales"], p["v"].view(fp8), p["v_scales"]) for p in s["layers"]]


def _side(c, s, name, page, offset):
    """Rows of one side of the cache in 32 bits: [..., kv_heads, D] at the pages and offsets."""
    v = s[name][page, :, offset]
    if c["precision"] == "bf16":
        return v.to(F32)
    return _mxfp8_value(v, s[name + "_scales"][page, :, offset], F32)


def _plain_attn(c, s):
    B, D, page, kv = c["B"], c["D"], c["page"], c["kv_heads"]
    group = c["heads"] // kv
    at = torch.arange(c["L"], device=DEV)
    pages = s["table"].long()[:, at // page].clamp(min=0)
    offset = (at % page)[None].expand(B, -1)
    k = _side(c, s, "k", pages, offset).transpose(1, 2)                       # [B, kv, L, D]
    v = _side(c, s, "v", pages, offset).transpose(1, 2)
    q = s["q"].to(F32).view(B, kv, group, D)
    scores = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(D)
    seen = at[None] < s["lengths"][:, None]
    if c["window"]:
        seen = seen & (at[None] >= s["lengths"][:, None] - c["window"])
    scores = scores.masked_fill(~seen[:, None, None], -INF)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -INF, torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.masked_fill(~seen[:, None, :, None], 0.0)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).squeeze(-1)
    return dict(out=out.view(B, c["heads"], D).to(BF16), lse=lse.view(B, c["heads"]))


def _places(c, s):
    """(page, offset) of every token's position, and which of them there are."""
    pos = s["positions"].long()
    ok = pos >= 0
    row = s["rows"].long() if s["rows"] is not None else torch.arange(c["n"], device=DEV)
    at = pos.clamp(min=0)
    return s["table"].long()[row, at // c["page"]], at % c["page"], ok


def _plain_append(c, s):
    h = c["kv_heads"]
    page, offset, ok = _places(c, s)
    new = dict(k=s["qkv"][:, h:2 * h], v=s["qkv"][:, 2 * h:])
    if c["precision"] == "bf16":
        for name, t in new.items():
            s[name][page[ok], :, offset[ok]] = t[ok]
        return dict(k=s["k"], v=s["v"])
    out = {}
    for name, t in new.items():
        codes, byte = _mxfp8(t.to(F32))
        s[name][page[ok], :, offset[ok]] = codes[ok]
        s[name + "_scales"][page[ok], :, offset[ok]] = byte[ok]
        got = _side(c, s, name, page.clamp(min=0), offset)
        out[name] = got.masked_fill(~ok[:, None, None], 0.0).to(BF16)
    return out


def _plain_pages(c, s):
    table, P, page = s["table"].long(), s["pages"], c["page"]
    S, M = table.shape
    col = torch.arange(M, device=DEV)[None]
    if c["kind"] == "fork":
        par = s["parents"].long()
        live = par >= 0
        length = torch.where(live, s["lengths"].long()[par.clamp(min=0)], 0)
        held = (length + page - 1) // page
        mine = col < held[:, None]
        t = torch.where(mine, table[par.clamp(min=0)], -1)
        # who keeps a page: the row with the most of it, then the first
        key = (length[:, None] - col * page).clamp(0, page) * S + (S - 1 - torch.arange(S, device=DEV)[:, None])
        best = torch.full((P,), -1, dtype=torch.int64, device=DEV).scatter_reduce_(0, t[mine], key[mine], "amax")
        last = (held - 1).clamp(min=0)[:, None]
        last_page = t.gather(1, last).squeeze(1)
        copy = (length % page != 0) & (best[last_page.clamp(min=0)] != key.gather(1, last).squeeze(1))
        fresh = live & (length % page == 0) & (held < M)
        need = copy.long() + fresh.long()
        free = best < 0
        rank = torch.cumsum(free.long(), 0) - 1
        order = torch.empty(P + 1, dtype=torch.int64, device=DEV)
        order[torch.where(free, rank, P)] = torch.arange(P, device=DEV)
        got = order[(torch.cumsum(need, 0) - need).clamp(max=P - 1)]          # the next free page to each that needs one
        where = torch.where(copy, held - 1, held).clamp(max=M - 1)[:, None]
        t.scatter_(1, where, torch.where(need > 0, got, t.gather(1, where).squeeze(1))[:, None])
        src, dst = torch.where(copy, last_page, -1), torch.where(copy, got, -1)
        used = (P - free.sum() + need.sum()).reshape(1)
        out = dict(table=t.to(I32), lengths=length.to(I32), src=src.to(I32), dst=dst.to(I32), used=used.to(I32))
    else:
        live = torch.zeros(P + 1, dtype=torch.bool, device=DEV)
        live[torch.where(table >= 0, table, P)] = True
        live = live[:P]
        used = live.sum()
        at = torch.arange(P, device=DEV)
        moved, hole = live & (at >= used), ~live & (at < used)
        n = P // 2                                                             # moves there can be at most
        src = torch.full((n + 1,), -1, dtype=torch.int64, device=DEV)
        dst = src.clone()
        src[torch.where(moved, torch.cumsum(moved.long(), 0) - 1, n)] = torch.where(moved, at, -1)
        dst[torch.where(hole, torch.cumsum(hole.long(), 0) - 1, n)] = torch.where(hole, at, -1)
        src, dst = src[:n], dst[:n]
        to = torch.cat([at, at.new_full((1,), -1)])
        to[torch.where(src >= 0, src, P)] = torch.where(src >= 0, dst, -1)
        out = dict(table=to[torch.where(table >= 0, table, P)].to(I32), src=src.to(I32), dst=dst.to(I32),
                   used=used.reshape(1).to(I32))
    ok = src >= 0
    src, dst = src[ok], dst[ok]
    for layer in s["layers"]:
        for t in layer.values():
            if t is not None:
                t[dst] = t[src]
    return dict(out, layers=_layers_out(c, s))


def _plain_beam(c, s):
    N, W, V, K = c["N"], c["W"], c["V"], c["K"]
    # (in 64 bits: candidates of different beams come close to one another)
    x, score = s["logits"].to(D64), s["scores"].to(D64).unsqueeze(-1)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))).add_(score)
    x.masked_fill_(score == -INF, -INF)
    if s["done"] is not None:                                  # a beam that is done goes on with the padding token alone
        pad = torch.where(torch.arange(V, device=DEV) == 1, score, torch.full_like(score, -INF))
        x = torch.where(s["done"].unsqueeze(-1), pad, x)
    v, at = torch.sort(x.view(N, W * V), dim=1, descending=True, stable=True)
    v, at = v[:, :K], at[:, :K]
    rows = at // V + torch.arange(N, device=DEV)[:, None] * W
    return dict(scores=v.to(F32), parents=rows.to(I32), tokens=(at % V).to(I32))


# --------------------------------------------------------------------------- floors
def work(case):
    c = case
    if c["op"] == "beam":
        n = c["N"] * c["W"] * c["V"]
        return {"bytes": n * (2 if c["dtype"] == "bf16" else 4) + c["N"] * (4 * c["W"] + 12 * c["K"]), "flops": 4 * n}
    side = c["kv_heads"] * c["D"] * (2 if c["precision"] == "bf16" else 1 + 1 / 32)    # bytes of a token's keys
    if c["op"] == "attn":
        n = sum(min(x, c["window"]) if c["window"] else x for x in _lengths(c))
        return {"bytes": 2 * n * side + c["B"] * c["heads"] * (4 * c["D"] + 4) + 4 * n / c["page"],
                "flops": 4 * n * c["heads"] * c["D"]}
    if c["op"] == "append":
        bf16 = c["kv_heads"] * c["D"] * 2
        back = side + bf16 if c["precision"] == "mxfp8" else 0
        return {"bytes": 2 * c["n"] * (bf16 + side + back) + 12 * c["n"], "flops": 4 * c["n"] * c["kv_heads"] * c["D"]}
    S, W = c["groups"] * c["beams"], c["beams"]
    width = (c["L"] + c["page"]) // c["page"]
    lengths = _lengths(c)
    if c["kind"] == "fork":
        # beams of a group less the parents that are chosen at all, where the last page is not full
        copies = sum(n % c["page"] != 0 for n in lengths) / W * (W - W * (1 - (1 - 1 / W) ** W))
    else:
        copies = sum((n + c["page"] - 1) // c["page"] for n in lengths) * 0.65 * 0.35
    return {"bytes": copies * 4 * c["layers"] * side * c["page"] + 8 * S * width + 12 * S, "flops": S * width}


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "beam":
        if c["N"] * c["W"] * c["V"] > 5e7:
            return None
        scores = torch.empty((c["N"], c["K"]), dtype=D64, device=DEV)
        for n in range(c["N"]):
            c_n = torch.log_softmax(s["logits"][n].to(D64), -1) + s["scores"][n].to(D64)[:, None]
            if s["done"] is not None:
                for w in s["done"][n].nonzero()[:, 0].tolist():
                    c_n[w] = -INF
                    c_n[w, 1] = s["scores"][n, w].to(D64)
            scores[n] = torch.topk(c_n.flatten(), c["K"]).values
        return dict(scores=scores, parents=None, tokens=None)
    fp8 = c["precision"] == "mxfp8"
    if c["op"] == "attn":
        B, D, group = c["B"], c["D"], c["heads"] // c["kv_heads"]
        out = torch.zeros((B, c["heads"], D), dtype=D64, device=DEV)
        lse = torch.full((B, c["heads"]), -INF, dtype=D64, device=DEV)
        for b, n in enumerate(s["lengths"].tolist()):
            first = max(0, n - c["window"]) if c["window"] else 0
            if n == first:
                continue
            pages = s["table"][b, first // c["page"]:(n - 1) // c["page"] + 1].long()

            def whole(name):
                t = s[name][pages]
                t = _mxfp8_value(t, s[name + "_scales"][pages], D64) if fp8 else t.to(D64)
                t = t.permute(1, 0, 2, 3).reshape(c["kv_heads"], -1, D)
                skip = first % c["page"]
                return t[:, skip:skip + n - first].repeat_interleave(group, 0)

            z = torch.einsum("hd,hnd->hn", s["q"][b].to(D64), whole("k")) * D ** -0.5
            lse[b] = torch.logsumexp(z, -1)
            out[b] = torch.einsum("hn,hnd->hd", torch.softmax(z, -1), whole("v"))
        return dict(out=out, lse=lse)
    if c["op"] == "append":
        new = dict(k=s["qkv"][:, c["kv_heads"]:2 * c["kv_heads"]], v=s["qkv"][:, 2 * c["kv_heads"]:])
        pos = s["positions"].tolist()
        if fp8:
            there = torch.tensor([p >= 0 for p in pos], device=DEV)[:, None, None]
            return {name: _mxfp8_value(*_mxfp8(t.to(D64)), D64) * there for name, t in new.items()}
        table = s["table"].tolist()
        rows = s["rows"].tolist() if s["rows"] is not None else range(c["n"])
        to = [(i, table[r][p // c["page"]], p % c["page"]) for i, (r, p) in enumerate(zip(rows, pos)) if p >= 0]
        i, pg, off = (torch.tensor(t, dtype=torch.int64, device=DEV) for t in zip(*to)) if to else [torch.empty(0, dtype=torch.int64, device=DEV)] * 3
        out = {}
        for name, t in new.items():
            whole = s[name].to(D64).transpose(1, 2).contiguous()
            whole[pg, off] = t[i].to(D64)
            out[name] = whole.transpose(1, 2)
        return out
    return None                                                # whole numbers and copies: nothing is computed
