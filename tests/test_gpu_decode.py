"""A beam search over decoder blocks (norm, attention over the paged cache, norm, MoE layer) with its cache, step by
step, against a plain 64-bit implementation that keeps every beam's whole history.

Every expert is chosen (K = E), so no near tie of the router can part the two. Bars: the stream passes eight
bf16 roundings a block (norm, projections, attention, expert values, output, sums), each of 2^-8 at most of values of the
stream's size and independent; two blocks: 4 * 2^-8 = 1.6e-2 of the largest value, twice that allowed. An MXFP8 key or value errs
by 2^-3 of itself at most: a block's largest element, scaled into [256, 512), saturates at 448, (512 - 448) / 512 = 2^-3
(the others round by half a step, 2^-4). That is the bar of what the cache holds, with the stream's own, and of what
comes out of attention over it, an average of such values with weights from such keys."""
import pytest
import torch

from dropless_moe_expert_router_gb300 import api
from dropless_moe_expert_router_gb300.block import Attention, MoEBlock
from dropless_moe_expert_router_gb300.cache import SequenceCache

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
H, F, E, Q, KV, D, V, LAYERS = 256, 256, 4, 4, 2, 64, 61, 2
BAR = {"bf16": 2 ** -5, "mxfp8": 2 ** -3 + 2 ** -5}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dropless_moe_expert_router_gb300 import build
    build.build()


def _params(seed):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, std, dtype=BF):
        return (torch.randn(shape, generator=g) * std).to(dtype)
    return dict(embed=n(V, H, std=1.0), layers=[dict(
        w1=n(E, H, F, std=0.06), w3=n(E, H, F, std=0.06), w2=n(E, F, H, std=0.06), router=n(E, H, std=0.1, dtype=F32),
        norm=1 + n(H, std=0.1, dtype=F32), bias=n(H, std=0.1, dtype=F32), qkv=n((Q + 2 * KV) * D, H, std=0.08),
        out=n(H, Q * D, std=0.06), anorm=1 + n(H, std=0.1, dtype=F32)) for _ in range(LAYERS)])


def _blocks(p, slots, window):
    blocks = []
    for i, q in enumerate(p["layers"]):
        c = {k: v.cuda() for k, v in q.items()}
        att = Attention(c["qkv"], c["out"], c["anorm"], q_heads=Q, kv_heads=KV, window=window)
        blocks.append(MoEBlock(c["w1"], c["w3"], c["w2"], c["router"], c["norm"], c["bias"], T=slots, K=E, renorm=True,
                               attention=att, index=i))
    return blocks


def _norm(s, w, b=None):
    var, mean = torch.var_mean(s, -1, unbiased=False, keepdim=True)
    y = (s - mean) * (var + 1e-5).rsqrt() * w.double()
    return y if b is None else y + b.double()


def _plain(p, tokens, window):
    """Logits of the last token of a history, and each layer's keys and values [n, KV, D], in 64 bits."""
    x, kv = p["embed"].double()[tokens], []
    n = len(tokens)
    mask = torch.ones((n, n), dtype=torch.bool).tril()
    if window:
        mask &= ~torch.ones((n, n), dtype=torch.bool).tril(-window)
    for q in p["layers"]:
        hn = _norm(x, q["anorm"])
        a = (hn @ q["qkv"].double().t()).view(n, Q + 2 * KV, D)
        k, v = a[:, Q:Q + KV], a[:, Q + KV:]
        kv.append((k, v))
        s = torch.einsum("ihd,jhd->hij", a[:, :Q], k.repeat_interleave(Q // KV, 1)) * D ** -0.5
        w = torch.softmax(s.masked_fill(~mask, -float("inf")), -1)
        x = x + torch.einsum("hij,jhd->ihd", w, v.repeat_interleave(Q // KV, 1)).reshape(n, -1) @ q["out"].double().t()
        hn = _norm(x, q["norm"], q["bias"])
        r = torch.softmax(hn @ q["router"].double().t(), 1)
        for e in range(E):
            up, gate = hn @ q["w1"][e].double(), hn @ q["w3"][e].double()
            x = x + r[:, e:e + 1] * ((up * torch.sigmoid(up) * gate) @ q["w2"][e].double())
    return x[-1] @ p["embed"].double().t(), kv


def _step(p, blocks, cache, embed, tokens, parents):
    cache.advance(parents)
    x, delta = embed[tokens.view(-1).long()], None
    for b in blocks:
        x, delta = b.step(x, delta, cache)
    cache.grow()
    return torch.mm((x.float() + delta.float()), embed.float().t())


@pytest.mark.parametrize("precision,window,page", [("bf16", 0, 4), ("bf16", 5, 3), ("mxfp8", 0, 4)])
def test_beam_search(precision, window, page):
    N, W, steps = 2, 3, 11
    p = _params(1)
    blocks = _blocks(p, N * W, window)
    embed = p["embed"].cuda()
    cache = SequenceCache(LAYERS, N * W, pages=60, heads=KV, page_size=page, dim=D, max_length=steps + 2, precision=precision)
    tokens = torch.tensor([[3], [9]], dtype=I32).expand(N, W).cuda()
    parents = torch.arange(N * W, dtype=I32, device="cuda")
    scores = torch.tensor([[0.0] + [-float("inf")] * (W - 1)] * N, device="cuda")
    history = [[3 if i < W else 9] for i in range(N * W)]
    total = [0.0] * (N * W)
    for step in range(steps):
        logits = _step(p, blocks, cache, embed, tokens, parents)
        ref = [_plain(p, h, window) for h in history]
        want = torch.stack([r[0] for r in ref])
        assert (logits.double().cpu() - want).abs().max() <= BAR[precision] * want.abs().max(), step
        assert cache.lengths.tolist() == [step + 1] * (N * W)
        # every beam's whole cache is its own history's
        n = step + 1
        rows = torch.arange(N * W, dtype=I32, device="cuda").repeat_interleave(n)
        pos = torch.arange(n, dtype=I32, device="cuda").repeat(N * W)
        for layer in range(LAYERS):
            k, v = api.moe_cache_gather(cache.layers[layer], cache.table, pos, rows=rows)
            for got, which in ((k, 0), (v, 1)):
                w = torch.stack([r[1][layer][which] for r in ref])
                err = (got.double().cpu().view_as(w) - w).abs().max()
                assert err <= BAR[precision] * w.abs().max(), (step, layer)
        # (a beam that is dead in the first step's scores has the same history as its first one)
        sel = cache.select(logits.view(N, W, V), scores)
        tokens, scores, parents = sel.tokens, sel.scores, sel.parents.view(-1)
        par, tok = parents.tolist(), tokens.view(-1).tolist()
        logp = torch.log_softmax(want, 1)
        total = [total[a] + logp[a, t].item() for a, t in zip(par, tok)]
        assert (scores.view(-1).double().cpu() - torch.tensor(total)).abs().max() <= (step + 1) * 2 * BAR[precision] * want.abs().max()
        assert all(i // W == a // W for i, a in enumerate(par))
        history = [history[a] + [t] for a, t in zip(par, tok)]
        if step % 4 == 3:
            before = cache.used.item()
            cache.compact()
            live = {t for row in cache.table.tolist() for t in row if t >= 0}
            assert live == set(range(len(live))) and cache.used.item() == len(live) <= before
        # no page is written by two beams: pages are shared only behind what they have in common
        assert api.moe_get_device_errors() == 0
    cache.advance(torch.full((N * W,), -1, dtype=I32, device="cuda"))
    assert cache.used.item() == 0 and not cache.lengths.any()


def test_a_step_in_a_graph():
    """One captured step (cache, blocks, selection), replayed, makes the search that eager steps make."""
    N, W, steps = 1, 4, 9
    p = _params(2)
    blocks = _blocks(p, N * W, 0)
    embed = p["embed"].cuda()

    def fresh():
        cache = SequenceCache(LAYERS, N * W, pages=40, heads=KV, page_size=4, dim=D, max_length=steps + 1)
        return (cache, torch.full((N, W), 7, dtype=I32, device="cuda"), torch.arange(W, dtype=I32, device="cuda"),
                torch.tensor([[0.0, -float("inf"), -float("inf"), -float("inf")]], device="cuda"))

    def step(cache, tokens, parents, scores):
        logits = _step(p, blocks, cache, embed, tokens, parents)
        sel = cache.select(logits.view(N, W, V), scores)
        tokens.copy_(sel.tokens), scores.copy_(sel.scores), parents.copy_(sel.parents.view(-1))
        return logits
    eager, state = [], fresh()
    for _ in range(steps):
        eager.append((step(*state).clone(), state[1].clone(), state[2].clone(), state[3].clone()))
    state = fresh()
    torch.cuda.synchronize()
    warm = fresh()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(*warm)
    torch.cuda.current_stream().wait_stream(s)
    state[0].attend(0, torch.zeros((N * W, Q, D), dtype=BF, device="cuda"))     # (its workspaces)
    state[0].select(torch.zeros((N, W, V), device="cuda"), state[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = step(*state)
    for want in eager:
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((logits,) + state[1:], want):
            assert torch.equal(a, b)
    assert api.moe_get_device_errors() == 0


def test_prompts_and_slots_that_come_and_go():
    """Prompts written at once, a slot that ends and one that begins, others that go on."""
    cache = SequenceCache(1, 4, pages=30, heads=1, page_size=4, dim=32, max_length=20)
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(n):
        return torch.randn((n, 1, 32), generator=g, device="cuda").to(BF)
    lens = [5, 0, 8, 3]
    room = torch.tensor(lens, dtype=I32, device="cuda")
    cache.advance(torch.tensor([0, -1, 2, 3], dtype=I32, device="cuda"), room=room)
    rows = torch.tensor([i for i, n in enumerate(lens) for _ in range(n)], dtype=I32, device="cuda")
    pos = torch.tensor([j for n in lens for j in range(n)], dtype=I32, device="cuda")
    k, v = rand(16), rand(16)
    cache.write(0, k, v, rows, pos)
    cache.grow(room)
    assert cache.lengths.tolist() == lens
    got = cache.read(0, rows, pos)
    assert torch.equal(got[0], k) and torch.equal(got[1], v)
    full = [[k[0:5], v[0:5]], None, [k[5:13], v[5:13]], [k[13:16], v[13:16]]]
    for parents, src in (([0, 2, 2, -1], [0, 2, 2, None]), ([0, 1, 2, 3], [0, 1, 2, 3]), (None, [0, 1, 2, 3]),
                         ([-1, 1, 1, 1], [None, 1, 1, 1])):
        cache.advance(None if parents is None else torch.tensor(parents, dtype=I32, device="cuda"))
        nk, nv = rand(4), rand(4)
        cache.append(0, nk, nv)
        q = rand(4).expand(4, 2, 32).contiguous()
        out = cache.attend(0, q)
        cache.grow()
        empty = torch.empty((0, 1, 32), dtype=BF, device="cuda")
        old, full = full, []
        for i, a in enumerate(src):
            if a is None:
                full.append(None)
                assert not out[i].any() and cache.lengths[i] == 0
                continue
            ok, ov = old[a] if old[a] is not None else (empty, empty)
            full.append([torch.cat([ok, nk[i:i + 1]]), torch.cat([ov, nv[i:i + 1]])])
            kk, vv = full[i][0][:, 0].double(), full[i][1][:, 0].double()
            w = torch.softmax(q[i].double() @ kk.t() * 32 ** -0.5, -1)
            # the weights' and the output's roundings, 2^-8 each
            assert bool(((out[i].double() - w @ vv).abs() <= 2 ** -7 * (w @ vv.abs()) + 2 ** -12).all())
            assert cache.lengths[i] == len(kk)
    assert api.moe_get_device_errors() == 0


def test_refusals():
    p = _params(3)
    with pytest.raises(ValueError):
        SequenceCache(0, 1, pages=4, heads=1, page_size=4, dim=32, max_length=8)
    cache = SequenceCache(1, 2, pages=4, heads=KV, page_size=4, dim=D, max_length=8)
    blocks = _blocks(p, 2, 0)
    x = torch.zeros((2, H), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        blocks[0].step(x)                                     # no cache
    with pytest.raises(ValueError):
        blocks[0].forward(x)
    q = p["layers"][0]
    c = {k: v.cuda() for k, v in q.items()}
    plain = MoEBlock(c["w1"], c["w3"], c["w2"], c["router"], c["norm"], T=2, K=E)
    with pytest.raises(ValueError):
        plain.step(x, None, cache)
    with pytest.raises(ValueError):
        MoEBlock(c["w1"], c["w3"], c["w2"], c["router"], c["norm"], T=2, K=E, attention=blocks[0].attention, training=True)
    with pytest.raises(ValueError):
        Attention(c["qkv"], c["out"], c["anorm"], q_heads=3, kv_heads=KV)
    with pytest.raises(ValueError):
        cache.select(torch.zeros((1, 3, V), device="cuda"), torch.zeros((1, 3), device="cuda"))
    with pytest.raises(ValueError):
        cache.append(0, x.view(2, 4, 64), x.view(2, 4, 64))


def test_a_step_that_finds_too_few_pages():
    """Nothing that was stored is lost, nothing is written, and the step is made once there is room."""
    cache = SequenceCache(2, 3, pages=5, heads=1, page_size=4, dim=32, max_length=16)
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(n):
        return torch.randn((n, 1, 32), generator=g, device="cuda").to(BF)

    def parents(*p):
        return torch.tensor(p, dtype=I32, device="cuda")
    room = parents(6, 3, 0)
    cache.advance(parents(0, 1, -1), room=room)
    rows, pos = parents(*[0] * 6 + [1] * 3), parents(*range(6), *range(3))
    data = [(rand(9), rand(9)) for _ in range(2)]
    for layer, (k, v) in enumerate(data):
        cache.write(layer, k, v, rows, pos)
    cache.grow(room)

    def stored():
        return all(torch.equal(a, b) for layer in range(2) for a, b in zip(cache.read(layer, rows, pos), data[layer]))
    assert stored() and cache.lengths.tolist() == [6, 3, 0] and api.moe_get_device_errors() == 0
    table, pools = cache.table.clone(), [t.clone() for c in cache.layers for t in (c.k, c.v)]
    # slots 0 and 2 go on from slot 0, slot 1 is given up: of its last page there is to be a copy, and 20 positions more
    cache.advance(parents(0, -1, 0), room=20)
    assert api.moe_get_device_errors() == api.MOE_DEVERR_NO_PAGE and cache.used.item() > cache.pages
    assert torch.equal(cache.table, table) and cache.lengths.tolist() == [6, 3, 0] and cache.positions.tolist() == [-1] * 3
    cache.append(0, rand(3), rand(3))                         # a step that does not know yet
    assert not cache.attend(0, rand(3)).any()
    cache.grow()
    assert cache.lengths.tolist() == [6, 3, 0] and stored()
    assert all(torch.equal(a, b) for a, b in zip(pools, (t for c in cache.layers for t in (c.k, c.v))))
    assert api.moe_get_device_errors() == 0
    cache.advance(parents(0, -1, 0))                          # one position more each: the copy's page is there
    assert cache.active.tolist() == [True, False, True] and cache.positions.tolist() == [6, -1, 6]
    new = rand(3)
    for layer in range(2):
        cache.append(layer, new, new)
    cache.grow()
    assert cache.lengths.tolist() == [7, 0, 7] and api.moe_get_device_errors() == 0
    for slot in (0, 2):
        for layer in range(2):
            k, v = cache.read(layer, parents(*[slot] * 7), parents(*range(7)))
            assert torch.equal(k, torch.cat([data[layer][0][:6], new[slot:slot + 1]]))
            assert torch.equal(v, torch.cat([data[layer][1][:6], new[slot:slot + 1]]))


def test_steps_of_every_slot_that_find_too_few_pages():
    """Slots that go on from themselves find no page for a step or more, and all go on where they were when one is free."""
    cache = SequenceCache(1, 3, pages=3, heads=1, page_size=2, dim=32, max_length=8)

    def parents(*p):
        return torch.tensor(p, dtype=I32, device="cuda")
    cache.advance(parents(0, 1, 2))
    kv = torch.randn((3, 1, 32), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)
    for n in (1, 2):
        cache.append(0, kv, kv)
        cache.grow()
        if n == 1:
            cache.advance()
    for _ in range(3):                                        # three pages more are wanted, none is free
        cache.advance()
        assert api.moe_get_device_errors() == api.MOE_DEVERR_NO_PAGE
        cache.append(0, kv, kv)
        cache.grow()
        assert cache.lengths.tolist() == [2, 2, 2] and cache.active.all() and cache.used.item() == 6
    cache.advance(parents(0, -1, -1))
    cache.append(0, kv, kv)
    cache.grow()
    assert cache.lengths.tolist() == [3, 0, 0] and cache.active.tolist() == [True, False, False]
    k, v = cache.read(0, parents(0, 0, 0), parents(0, 1, 2))
    assert torch.equal(k, kv[:1].expand(3, 1, 32)) and torch.equal(v, k)
    assert api.moe_get_device_errors() == 0
