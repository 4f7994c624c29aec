"""The paged cache's rows and pages (append, gather, copies, fork, compact) against plain Python. Everything
here is exact: rows are copied or quantised by the layer's MXFP8 rule, the rest is whole numbers."""
import random

import pytest
import torch

from dropless_moe_expert_router_gb300 import api
from dropless_moe_expert_router_gb300.api import MoeError

pytestmark = pytest.mark.gpu
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dropless_moe_expert_router_gb300 import build
    build.build()


def _i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _rows(n, heads, dim, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn((n, heads, dim), generator=g, device="cuda") * std).to(BF) for _ in range(2)]


def _quant(t):
    """The rows' MXFP8 codes and scales by the plain rule in 32 bits."""
    b = t.float().unflatten(-1, (t.shape[-1] // 32, 32))
    amax = b.abs().amax(-1)
    byte = (torch.frexp(amax).exponent - 1 - 8 + 127).clamp(0, 254)
    byte = torch.where(amax == 0, torch.full_like(byte, 127), byte)
    codes = (b * torch.exp2((127 - byte).float()).unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(-2)
    return codes.view(U8), byte.to(U8)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("heads,dim,page", [(1, 32, 1), (2, 64, 16), (3, 96, 5), (8, 128, 16), (1, 256, 33)])
@pytest.mark.parametrize("n", [1, 7, 300])
def test_append_and_gather(n, heads, dim, page, precision):
    r = random.Random(n * 31 + page)
    S, M = 9, (400 + page - 1) // page
    pages = S * M + 2
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(n))[:S * M].view(S, M).to(I32).cuda()
    places = r.sample([(s, p) for s in range(S) for p in range(400)], n)
    rows, pos = [p[0] for p in places], [p[1] for p in places]
    for i in range(0, n, 5):                                          # padding
        if i % 2:
            pos[i] = -1 - i
        elif n > 1:
            rows[i] = -1
    k, v = _rows(n, heads, dim, seed=n)
    if n > 5:
        k[3] = 0                                                      # a block of zeros
    cache = api.cache_buffers(pages, heads, page, dim, "cuda", precision)
    old = {}
    for name in ("k", "v", "k_scales", "v_scales"):
        t = getattr(cache, name)
        if t is not None:
            t.view(U8).random_(0, 100)
            old[name] = t.clone()
    api.moe_cache_append(k, v, cache, table, _i32(pos), rows=_i32(rows))
    want = {name: t.clone() for name, t in old.items()}
    ok = [i for i in range(n) if pos[i] >= 0 and rows[i] >= 0]
    for name, t in (("k", k), ("v", v)):
        codes, byte = _quant(t) if precision == "mxfp8" else (t, None)
        for i in ok:
            p, o = int(table[rows[i], pos[i] // page]), pos[i] % page
            want[name][p, :, o] = codes[i]
            if byte is not None:
                want[name + "_scales"][p, :, o] = byte[i]
    for name, t in want.items():
        assert torch.equal(getattr(cache, name).view(U8), t.view(U8)), name      # the other positions as they were
    gk, gv = api.moe_cache_gather(cache, table, _i32(pos), rows=_i32(rows))
    for name, got, t in (("k", gk, k), ("v", gv, v)):
        if precision == "mxfp8":
            codes, byte = _quant(t)
            t = (codes.view(torch.float8_e4m3fn).float().unflatten(-1, (dim // 32, 32)) *
                 torch.exp2(byte.float() - 127).unsqueeze(-1)).flatten(-2).to(BF)
        t = t.clone()
        t[[i for i in range(n) if i not in ok]] = 0
        assert torch.equal(got, t), name
    assert api.moe_get_device_errors() == 0


def test_quantised_rows_are_those_of_the_permute():
    k, v = _rows(64, 2, 64, seed=3, std=0.01)
    k[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -0.0, 1e30], device="cuda")
    cache = api.cache_buffers(4, 2, 16, 64, "cuda", "mxfp8")
    table = _i32([[3, 1, 0, 2]])
    api.moe_cache_append(k, v, cache, table, torch.arange(64, dtype=I32, device="cuda"),
                         rows=torch.zeros(64, dtype=I32, device="cuda"))
    p = api.moe_permute(k.view(128, 64), torch.zeros((128, 1), dtype=I32, device="cuda"), 1, fuse_mxfp8=True)
    order = table[0].long()
    assert torch.equal(cache.k[order].permute(0, 2, 1, 3).reshape(128, 64), p.x_perm)
    assert torch.equal(cache.k_scales[order].permute(0, 2, 1, 3).reshape(128, 2), p.x_perm_scales)


def test_append_of_a_projection_s_slices_and_of_one_token_each():
    qkv = _rows(6, 12, 64, seed=1)[0]
    cache = api.cache_buffers(20, 2, 4, 64, "cuda")
    cache.k.zero_(), cache.v.zero_()
    table = torch.arange(20, dtype=I32, device="cuda").view(10, 2)     # more sequences than tokens: the rest untouched
    pos = _i32([0, 7, 3, -1, 4, 2])
    api.moe_cache_append(qkv[:, 8:10], qkv[:, 10:], cache, table, pos)
    k, v = api.moe_cache_gather(cache, table, pos)
    ok = [0, 1, 2, 4, 5]
    assert torch.equal(k[ok], qkv[ok, 8:10]) and torch.equal(v[ok], qkv[ok, 10:]) and not k[3].any()
    assert int((cache.k != 0).any(-1).sum()) == 10
    one = qkv[:1, 3:5]                                                 # a single token, any stride
    api.moe_cache_append(one, one, cache, table, _i32([5]), rows=_i32([9]))
    assert torch.equal(api.moe_cache_gather(cache, table, _i32([5]), rows=_i32([9]))[0], one)
    assert api.moe_get_device_errors() == 0


def test_bad_positions_are_skipped_and_told():
    k, v = _rows(3, 2, 64, seed=1)
    cache = api.cache_buffers(6, 2, 4, 64, "cuda")
    cache.k.zero_(), cache.v.zero_()
    for table, pos, rows, bad in (([[0, 1], [2, 9]], [8, 1, 1], [0, 0, 1], 0), ([[0, 1], [2, 9]], [0, 1, 4], [0, 0, 1], 2),
                                  ([[0, -1], [2, 3]], [4, 1, 1], [0, 0, 1], 0), ([[0, 1], [2, 3]], [1, 1, 2], [2, 0, 1], 0)):
        api.moe_cache_append(k, v, cache, _i32(table), _i32(pos), rows=_i32(rows))
        assert api.moe_get_device_errors() == api.MOE_DEVERR_BAD_ID
        got, _ = api.moe_cache_gather(cache, _i32(table), _i32(pos), rows=_i32(rows))
        assert api.moe_get_device_errors() == api.MOE_DEVERR_BAD_ID
        assert all(torch.equal(got[i], k[i]) if i != bad else not got[i].any() for i in range(3))
    assert not cache.k[4:].any()


# ------------------------------------------------------------------ fork
def _fork_plain(table, lengths, parents, pages, page, rooms):
    S, M = len(table), len(table[0])
    S2 = len(parents)
    new, lens = [], []
    for p in parents:
        n = max(0, min(lengths[p], M * page)) if 0 <= p < S else 0
        held = (n + page - 1) // page
        new.append([table[p][j] if j < held and 0 <= table[p][j] < pages else -1 for j in range(M)])
        lens.append(n)
    keeper = {}
    for i in range(S2):
        for j in range(M):
            t = new[i][j]
            if t >= 0:
                fill = min(page, lens[i] - j * page)
                if t not in keeper or fill > keeper[t][0]:
                    keeper[t] = (fill, i, j)
    free = [p for p in range(pages) if p not in keeper]
    wanted, short = 0, False
    src, dst = [-1] * S2, [-1] * S2
    named = len(keeper)
    for i, p in enumerate(parents):
        room = max(0, rooms[i])
        if not 0 <= p < S or room == 0:
            continue
        n = lens[i]
        held, end = (n + page - 1) // page, min(M, (n + room + page - 1) // page)

        def take():
            nonlocal wanted, short
            wanted += 1
            if wanted > len(free):
                short = True
                return -1
            return free[wanted - 1]
        if n % page:
            t = new[i][held - 1]
            if t >= 0 and keeper[t] != (n - (held - 1) * page, i, held - 1):
                to = take()
                src[i], dst[i] = (t, to) if to >= 0 else (-1, -1)
                new[i][held - 1] = to
        for j in range(held, end):
            new[i][j] = take()
    return new, lens, src, dst, named + wanted, short


def _state(r, S, M, page, pages, share=0.5):
    """Rows with pages of their own behind a prefix that they may share with an earlier row."""
    order = list(range(pages))
    r.shuffle(order)
    table, lengths = [], []
    for s in range(S):
        n = r.randint(0, M * page)
        row = [-1] * M
        held = (n + page - 1) // page
        common = 0
        if s and r.random() < share:
            o = r.randrange(s)
            common = r.randint(0, min(held, (lengths[o] + page - 1) // page))
            row[:common] = table[o][:common]
        for j in range(common, held):
            if not order:
                held, n = j, j * page
                break
            row[j] = order.pop()
        table.append(row)
        lengths.append(n)
    return table, lengths


def _check_fork(table, lengths, parents, pages, page, room, workspace=None):
    M = len(table[0])
    rooms = room if isinstance(room, list) else [room] * len(parents)
    want = _fork_plain(table, lengths, parents, pages, page, rooms)
    got = api.moe_cache_fork(_i32(table).view(len(table), M), _i32(lengths), _i32(parents), pages, page,
                             room=_i32(room) if isinstance(room, list) else room, workspace=workspace)
    assert got.table.tolist() == want[0]
    assert got.lengths.tolist() == want[1]
    assert got.src.tolist() == want[2] and got.dst.tolist() == want[3]
    assert got.used.item() == want[4]
    assert (api.moe_get_device_errors() == api.MOE_DEVERR_NO_PAGE) == want[5]
    return got


@pytest.mark.parametrize("S,M,page,pages", [(1, 1, 1, 3), (4, 5, 4, 40), (8, 9, 16, 100), (33, 7, 3, 400), (64, 130, 2, 9000),
                                            (300, 40, 8, 13_000), (5, 3, 16, 70_001), (300, 100, 2, 31_000), (2, 20_000, 1, 30_000)])
@pytest.mark.parametrize("room", [0, 1, 5])
def test_fork(S, M, page, pages, room):
    for seed in range(4):
        r = random.Random(seed * 1000 + S)
        table, lengths = _state(r, S, M, page, pages)
        S2 = r.choice([S, 2 * S, max(1, S // 2)])
        parents = [r.randint(-1, S - 1) for _ in range(S2)]
        ws = api.moe_cache_pages_workspace(pages, S2, "cuda").fill_(255 * (seed % 2))
        _check_fork(table, lengths, parents, pages, page, room, ws)
        _check_fork(table, lengths, list(range(S)), pages, page, [r.randint(-1, 2 * page) for _ in range(S)])


def test_fork_runs_short_of_pages():
    table, lengths = [[0, 1, -1], [2, -1, -1]], [5, 4]
    got = _check_fork(table, lengths, [0, 0, 1, 1], 4, 4, 1)         # wants a copy and two more pages: one is free
    assert got.used.item() == 6
    _check_fork(table, lengths, [0, 1], 3, 4, [1, 1])
    _check_fork([[0, 1, 2]], [12], [0], 4, 4, 5)                      # no column left: nothing is wanted
    assert api.moe_get_device_errors() == 0


def test_fork_of_each_from_itself_and_of_none():
    table, lengths = _i32([[4, -1], [2, 0]]), _i32([3, 8])
    got = api.moe_cache_fork(table, lengths, None, 6, 4)
    assert got.table.tolist() == [[4, -1], [2, 0]] and got.src.tolist() == [-1, -1] and got.used.item() == 3
    got = api.moe_cache_fork(table, lengths, _i32([-1, -1, -1]), 6, 4)
    assert got.table.tolist() == [[-1, -1]] * 3 and got.lengths.tolist() == [0] * 3 and got.used.item() == 0
    got = api.moe_cache_fork(table[:0], lengths[:0], None, 6, 4)
    assert got.table.shape == (0, 2) and got.used.item() == 0
    assert api.moe_get_device_errors() == 0


def test_fork_tells_bad_ids():
    for table, lengths, parents in (([[4, 1]], [5], [1]), ([[4, 1]], [5], [-2]), ([[9, 1]], [5], [0]), ([[-1, 1]], [5], [0]),
                                    ([[4, 1]], [9], [0])):
        want = _fork_plain(table, lengths, parents, 6, 4, [1])
        got = api.moe_cache_fork(_i32(table), _i32(lengths), _i32(parents), 6, 4)
        assert got.table.tolist() == want[0] and got.used.item() == want[4]
        assert api.moe_get_device_errors() == api.MOE_DEVERR_BAD_ID


# ------------------------------------------------------------------ compact
def _compact_plain(table, pages):
    live = sorted({t for row in table for t in row if 0 <= t < pages})
    n = len(live)
    movers = [p for p in live if p >= n]
    named = set(live)
    holes = [p for p in range(n) if p not in named]
    to = dict(zip(movers, holes))
    pad = [-1] * (pages // 2 - len(movers))
    return [[to.get(t, t) if 0 <= t < pages else -1 for t in row] for row in table], movers + pad, holes + pad, n


@pytest.mark.parametrize("S,M,pages", [(1, 1, 1), (1, 1, 2), (4, 5, 40), (9, 9, 81), (33, 7, 400), (64, 130, 9000), (300, 40, 60_000),
                                       (5, 3, 70_001), (300, 100, 29_000), (2, 20_000, 30_000)])
def test_compact(S, M, pages):
    for seed in range(5):
        r = random.Random(seed * 77 + S)
        fill = r.choice([0.0, 0.1, 0.5, 0.9, 1.0])
        order = list(range(pages))
        r.shuffle(order)
        if seed == 3:
            order = sorted(order)                                     # nothing below to move to
        table = [[order.pop() if order and r.random() < fill else -1 for _ in range(M)] for _ in range(S)]
        if S > 2:
            table[1] = list(table[0])                                 # shared pages
        want = _compact_plain(table, pages)
        t = _i32(table).view(S, M)
        got = api.moe_cache_compact(t, pages, workspace=api.moe_cache_pages_workspace(pages, 0, "cuda").fill_(255))
        assert got.table.tolist() == want[0] and got.src.tolist() == want[1] and got.dst.tolist() == want[2]
        assert got.used.item() == want[3]
        api.moe_cache_compact(t, pages, out=got._replace(table=t))    # in place
        assert t.tolist() == want[0]
    assert api.moe_get_device_errors() == 0
    api.moe_cache_compact(_i32([[pages]]), pages)
    assert api.moe_get_device_errors() == api.MOE_DEVERR_BAD_ID


# ------------------------------------------------------------------ copies
@pytest.mark.parametrize("heads,page,dim,precision", [(1, 1, 32, "mxfp8"), (2, 16, 64, "bf16"), (3, 5, 32, "mxfp8"), (8, 64, 128, "mxfp8"),
                                                      (8, 64, 128, "bf16"), (1, 1, 16, "bf16")])
@pytest.mark.parametrize("n", [1, 40, 5000])
def test_copy_pages(heads, page, dim, precision, n):
    pages = 2 * n + 5
    caches = []
    for _ in range(3):
        c = api.cache_buffers(pages, heads, page, dim, "cuda", precision) if n * heads * page * dim < 2 ** 26 else None
        if c is None:
            pytest.skip("the small pools cover the lists' lengths")
        for t in c[5:]:
            if t is not None:
                t.view(U8).random_(0, 256)
        caches.append(c)
    want = [[None if t is None else t.clone() for t in c[5:]] for c in caches]
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(n))
    src, dst = order[:n].clone(), order[n:2 * n].clone()
    skip = torch.rand(n, generator=torch.Generator().manual_seed(1)) < 0.4
    skip[0] = False
    src[skip], dst[skip & (torch.arange(n) % 2 == 0)] = -1, -1
    src[:n // 3] = src[0]                                             # one source, many destinations
    ok = (src >= 0) & (dst >= 0)
    for w in want:
        for t in w:
            if t is not None:
                t[dst[ok].cuda()] = t[src[ok].cuda()]
    api.moe_cache_copy_pages(caches, src.to(I32).cuda(), dst.to(I32).cuda())
    for c, w in zip(caches, want):
        for t, x in zip(c[5:], w):
            assert x is None or torch.equal(t.view(U8), x.view(U8))
    assert api.moe_get_device_errors() == 0


def test_copy_pages_of_many_layers_and_bad_ids():
    caches = [api.cache_buffers(4, 1, 2, 32, "cuda", "mxfp8" if i % 3 else "bf16") for i in range(150)]
    for c in caches:
        for t in c[5:]:
            if t is not None:
                t.view(U8).random_(0, 256)
    before = [c.k.view(U8).clone() for c in caches]                   # (any bits: NaN among them)
    api.moe_cache_copy_pages(caches, _i32([3, 9, -5, 1]), _i32([0, 1, 2, 4]))
    assert api.moe_get_device_errors() == api.MOE_DEVERR_BAD_ID
    for c, b in zip(caches, before):
        now = c.k.view(U8)
        assert torch.equal(now[0], b[3]) and torch.equal(now[1:], b[1:])
        assert c.v_scales is None or torch.equal(c.v_scales[0], c.v_scales[3])
    api.moe_cache_copy_pages([], _i32([0]), _i32([1]))
    api.moe_cache_copy_pages(caches, _i32([]), _i32([]))


def test_pages_calls_in_a_graph_and_on_a_stream():
    r = random.Random(4)
    table, lengths = _state(r, 12, 20, 4, 500)
    parents = [r.randint(-1, 11) for _ in range(12)]
    t, l, p = _i32(table), _i32(lengths), _i32(parents)
    cache = api.cache_buffers(500, 2, 4, 32, "cuda")
    cache.k.normal_(), cache.v.normal_()
    ref = api.moe_cache_fork(t, l, p, 500, 4)
    ws = api.moe_cache_pages_workspace(500, 12, "cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.moe_cache_fork(t, l, p, 500, 4, workspace=ws, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    out = api.CacheFork(*[torch.empty_like(x) for x in ref])
    packed = api.moe_cache_compact(t, 500)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_cache_fork(t, l, p, 500, 4, workspace=ws, out=out)
        api.moe_cache_copy_pages(cache, out.src, out.dst)
        api.moe_cache_compact(out.table, 500, workspace=ws, out=packed)
    p2 = [r.randint(-1, 11) for _ in range(12)]
    p.copy_(torch.tensor(p2))
    graph.replay()
    torch.cuda.synchronize()
    want = _fork_plain(table, lengths, p2, 500, 4, [1] * 12)
    assert out.table.tolist() == want[0] and out.src.tolist() == want[2]
    for a, b in zip(want[2], want[3]):
        assert a < 0 or torch.equal(cache.k[a], cache.k[b])
    assert packed.table.tolist() == _compact_plain(want[0], 500)[0]


def test_refusals():
    t, l = _i32([[0, 1]]), _i32([3])
    cache = api.cache_buffers(4, 2, 4, 32, "cuda", "mxfp8")
    k, v = _rows(1, 2, 32, seed=1)
    with pytest.raises(ValueError):
        api.moe_cache_append(k.float(), v, cache, t, l)
    with pytest.raises(ValueError):
        api.moe_cache_append(k, v[:, :1], cache, t, l)
    with pytest.raises(ValueError):
        api.moe_cache_append(k, v, cache, t[0], l)
    with pytest.raises(ValueError):
        api.moe_cache_append(k, v, cache._replace(k_scales=None), t, l)
    with pytest.raises(ValueError):
        api.moe_cache_append(k, v, cache, t, l.long())
    with pytest.raises(MoeError):                                     # more tokens than sequences, and no rows
        api.moe_cache_append(k.expand(2, 2, 32).contiguous(), v.expand(2, 2, 32).contiguous(), cache, t, _i32([0, 1]))
    with pytest.raises(ValueError):
        api.moe_cache_gather(cache, t, l, k=torch.empty((1, 2, 32), device="cuda"))
    with pytest.raises(ValueError):
        api.moe_cache_fork(t, l, _i32([0]).long(), 4, 4)
    with pytest.raises(MoeError):
        api.moe_cache_fork(t, l, _i32([0]), 4, 0)
    with pytest.raises(MoeError):
        api.moe_cache_fork(t, l, _i32([0]), 4, 4, workspace=torch.empty(16, dtype=U8, device="cuda"))
    with pytest.raises(ValueError):
        f = api.moe_cache_fork(t, l, None, 4, 4)
        api.moe_cache_fork(t, l, None, 4, 4, out=f._replace(table=t))
    with pytest.raises(ValueError):
        api.moe_cache_fork(t, l, None, 4, 4, out=f._replace(lengths=l))
    for big in ((1 << 32) + 4, 4), (4, (1 << 32) + 4):
        with pytest.raises(ValueError):
            api.moe_cache_fork(t, l, None, *big)
    with pytest.raises(ValueError):
        api.moe_cache_compact(t, (1 << 32) + 4)
    for room in (-1, 1 << 31):
        with pytest.raises(ValueError):
            api.moe_cache_fork(t, l, None, 4, 4, room=room)
    with pytest.raises(ValueError):
        api.moe_cache_copy_pages(cache, _i32([0]), _i32([0, 1]))
    with pytest.raises(ValueError):
        api.moe_cache_copy_pages([cache, api.cache_buffers(5, 2, 4, 32, "cuda")], _i32([0]), _i32([1]))
    with pytest.raises(ValueError):
        api.moe_cache_copy_pages(cache, torch.tensor([0], dtype=I32), torch.tensor([1], dtype=I32))


def test_fork_of_sequences_near_two_to_the_31():
    """2046 * 1049601 = 2^31 - 2 positions a row: lengths whose sum with a page passes 31 bits."""
    page, M = 2046, 1_049_601
    table = torch.arange(M, dtype=I32, device="cuda")[None]
    for n, room in ((page * M - 1, 1), (page * M, 1), (page * M, 0), (page * M - page, 7)):
        got = api.moe_cache_fork(table, _i32([n]), _i32([0, 0]), M + 2, page, room=room)
        want = table.expand(2, M).clone()
        src, dst, used = [-1, -1], [-1, -1], M
        if n % page:                                                  # the second row's copy of the page that both would write
            src[1], dst[1], want[1, -1], used = M - 1, M, M, M + 1
        elif n < page * M:                                            # a page behind for each (M - 1 is free, too)
            want[:, -1], used = torch.tensor([M - 1, M], dtype=I32, device="cuda"), M + 1
        assert torch.equal(got.table, want) and got.lengths.tolist() == [n, n]
        assert got.src.tolist() == src and got.dst.tolist() == dst and got.used.item() == used
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("n,heads,dim,page", [(777, 8, 128, 16), (20_003, 1, 32, 7), (2501, 3, 96, 5), (90, 24, 256, 33), (513, 8, 128, 1)])
def test_append_and_gather_of_many_tokens(n, heads, dim, page, precision):
    """Sizes at which a thread has four tokens, the last ones fewer; slices of one projection; padding; other rows as they were."""
    M = (n + page - 1) // page
    g = torch.Generator(device="cuda").manual_seed(n)
    table = torch.randperm(M + 3, generator=g, device="cuda")[:M].to(I32)[None].contiguous()
    pos = torch.randperm(n, generator=g, device="cuda").to(I32)
    pos[::7] = -1
    rows = torch.where(torch.arange(n, device="cuda") % 11 == 3, -1, 0).to(I32)
    qkv = torch.randn((n, 3 * heads, dim), generator=g, device="cuda").to(BF)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    cache = api.cache_buffers(M + 3, heads, page, dim, "cuda", precision)
    want = {}
    for name in ("k", "v", "k_scales", "v_scales"):
        t = getattr(cache, name)
        if t is not None:
            t.view(U8).random_(0, 100)
            want[name] = t.clone()
    api.moe_cache_append(k, v, cache, table, pos, rows=rows)
    ok = (pos >= 0) & (rows >= 0)
    p, o = table[0, (pos[ok] // page).long()].long(), (pos[ok] % page).long()
    back = {}
    for name, t in (("k", k), ("v", v)):
        codes, byte = _quant(t) if precision == "mxfp8" else (t, None)
        want[name][p, :, o] = codes[ok]
        if byte is not None:
            want[name + "_scales"][p, :, o] = byte[ok]
            codes = (codes.view(torch.float8_e4m3fn).float().unflatten(-1, (dim // 32, 32)) *
                     torch.exp2(byte.float() - 127).unsqueeze(-1)).flatten(-2).to(BF)
        back[name] = codes.masked_fill(~ok[:, None, None], 0)
    for name, t in want.items():
        assert torch.equal(getattr(cache, name).view(U8), t.view(U8)), name
    gk, gv = api.moe_cache_gather(cache, table, pos, rows=rows)
    assert torch.equal(gk, back["k"]) and torch.equal(gv, back["v"])
    assert api.moe_get_device_errors() == 0
