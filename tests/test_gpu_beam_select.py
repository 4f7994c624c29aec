"""Selection of a beam search's step against a plain 64-bit implementation, through the C ABI.

Bars. The sum under a beam's logarithm is of at most 2^11 terms a thread in fp32, each off by 2^-22 of itself
(exp), and in a few levels above that; so lse errs by 2^-12 at most. What is compared is ids: they have to be the
reference's wherever its candidates are further apart than that, and everywhere in one beam, whose candidates
all have the same error, and where nothing is rounded (equal beams, finished beams, -inf)."""
from fractions import Fraction

import pytest
import torch

from dropless_moe_expert_router_gb300 import api
from dropless_moe_expert_router_gb300.api import MoeError

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
INF = float("inf")
BAR = 2.0 ** -12


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dropless_moe_expert_router_gb300 import build
    build.build()


def _plain(logits, scores, K, done=None, pad=0):
    x, s = logits.double().cpu(), scores.double().cpu()
    N, W, V = x.shape
    lse = torch.logsumexp(x, -1)
    alive = torch.isfinite(lse) & torch.isfinite(s)
    # (the maximum first: a row of the type's lowest values has a logarithm that 64 bits would lose beside them)
    top = torch.where(torch.isfinite(lse), x.amax(-1), torch.zeros_like(lse))[..., None]
    c = s[..., None] + ((x - top) - torch.log(torch.exp(x - top).sum(-1, keepdim=True)))
    c = torch.where(alive[..., None], c, torch.full_like(c, -INF))
    if done is not None:
        only = torch.full((V,), -INF, dtype=torch.float64)
        only[pad] = 0.0
        fin = torch.where(torch.isfinite(s), s, torch.full_like(s, -INF))[..., None] + only
        c = torch.where(done.cpu()[..., None], fin, c)
    v, at = torch.sort(c.view(N, -1), dim=1, descending=True, stable=True)
    return c.view(N, -1), v[:, :K], at[:, :K]


def _check(logits, scores, K, done=None, pad=0, exact=False, **kw):
    N, W, V = logits.shape
    o = api.moe_beam_select(logits, scores, K, done=done, pad=pad, **kw)
    c, v, at = _plain(logits, scores, K, done, pad)
    assert o.scores.dtype == F32 and o.parents.dtype == I32 and o.tokens.dtype == I32
    rows, tok = o.parents.cpu().long(), o.tokens.cpu().long()
    base = torch.arange(N)[:, None] * W
    assert bool(((rows >= base) & (rows < base + W) & (tok >= 0) & (tok < V)).all())
    got = (rows - base) * V + tok
    val = torch.gather(c, 1, got)
    # no candidate twice, their own values in order, and as good as the reference's
    assert all(len(set(r)) == K for r in got.tolist())
    fin = torch.isfinite(v)
    assert torch.equal(fin, torch.isfinite(val)) and torch.equal(fin, torch.isfinite(o.scores.cpu()))
    err = BAR + 2.0 ** -23 * v[fin].abs()
    assert bool(((val - v)[fin].abs() <= 2 * err).all())
    assert bool(((o.scores.cpu().double() - val)[fin].abs() <= err).all())
    assert torch.equal(got[~fin], at[~fin])                          # -inf: the lowest indices
    if exact or W == 1:
        assert torch.equal(got, at)
    else:
        # where the reference's neighbours are further apart than the bar, the ids are its own
        gap = torch.full((N, K + 1), INF, dtype=torch.float64)
        gap[:, 1:K] = v[:, :-1] - v[:, 1:]
        nxt = torch.sort(c, 1, descending=True).values
        if c.shape[1] > K:
            gap[:, K] = v[:, -1] - nxt[:, K]
        sure = torch.minimum(gap[:, :-1], gap[:, 1:]) > 2 * BAR
        assert torch.equal(got[sure & fin], at[sure & fin])
    assert api.moe_get_device_errors() == 0
    return o


def _inputs(N, W, V, dtype, seed, std=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.randn((N, W, V), generator=g, device="cuda") * std).to(dtype),
            -8 * torch.rand((N, W), generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,W,V,K", [(1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 15), (1, 4, 32000, 8), (5, 5, 1001, 10), (3, 2, 4096, 64),
                                     (2, 8, 50021, 16), (1, 1, 200_003, 32), (40, 4, 513, 4), (1, 64, 257, 64), (2, 16, 8192, 1),
                                     (1, 3, 31, 64), (300, 1, 100, 3), (2, 7, 33333, 33)])
def test_selection(N, W, V, K, dtype):
    logits, scores = _inputs(N, W, V, dtype, seed=V + K)
    _check(logits, scores, K)
    done = torch.rand((N, W), generator=torch.Generator().manual_seed(V)) < 0.4
    _check(logits, scores, K, done=done.cuda(), pad=V // 2)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_first_step_and_dead_beams(dtype):
    logits, scores = _inputs(3, 4, 2000, dtype, seed=1)
    scores[:, 1:] = -INF
    _check(logits, scores, 8)
    scores[1] = -INF                                                  # no beam lives: -inf, lowest indices
    _check(logits, scores, 8)
    done = torch.ones((3, 4), dtype=torch.bool, device="cuda")
    _check(logits, scores, 8, done=done, pad=1999)                    # fewer candidates than K
    scores[0, 2], scores[2, 1] = float("nan"), INF
    _check(logits, scores, 8)
    _check(logits, scores, 8, done=done, pad=3)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_masked_and_bad_logits(dtype):
    """Forbidden tokens (-inf, the type's lowest), rows that forbid everything, NaN and +inf rows."""
    logits, scores = _inputs(4, 3, 777, dtype, seed=2)
    logits[0, :, 5:] = -INF                                           # 15 candidates are left
    logits[1, 1] = -INF
    logits[2, 0] = torch.finfo(dtype).min
    logits[2, 1, 100:] = torch.finfo(dtype).min
    logits[3, 0, 50], logits[3, 1, 51] = float("nan"), INF
    _check(logits, scores, 12)
    _check(logits, scores, 20)


def test_ties_go_to_the_lowest_beam_then_token():
    for dtype in (F32, BF):
        logits = torch.zeros((2, 4, 3000), device="cuda", dtype=dtype)
        scores = torch.zeros((2, 4), device="cuda")
        o = _check(logits, scores, 40, exact=True)
        assert o.tokens[0].tolist() == list(range(40)) and o.parents[1].tolist() == [4] * 40
        one, _ = _inputs(1, 1, 3000, BF, seed=3, std=1.0)             # a few hundred values: many ties
        logits = one.to(dtype).expand(2, 4, 3000).contiguous()
        _check(logits, scores, 64, exact=True)
        logits = torch.full((1, 2, 70_000), -3.0, device="cuda", dtype=dtype)
        logits[0, :, 69_990:] = 2.0
        o = _check(logits, scores[:1, :2].contiguous(), 30, exact=True)
        assert o.tokens[0].tolist() == list(range(69_990, 70_000)) * 2 + list(range(10))


def test_ascending_and_descending_rows():
    """The best at the end, where every element beats those before it, and at the start."""
    for flip in (False, True):
        row = torch.linspace(-5, 5, 60_000, device="cuda")
        logits = (row.flip(0) if flip else row).expand(1, 2, 60_000).contiguous()
        _check(logits, torch.tensor([[0.0, -0.5]], device="cuda"), 64)


@pytest.mark.parametrize("dtype,V", [(F32, 32_768), (F32, 30_001), (BF, 70_003)])
@pytest.mark.parametrize("kind", ["random", "ascending", "equal", "few values"])
def test_many_rows_a_block(dtype, V, kind):
    """More units than blocks, so that a block has several of a row and several rows: the threshold that is kept from
    unit to unit, and more ties and larger logits than the buffer holds."""
    N, K = 700, 40
    g = torch.Generator(device="cuda").manual_seed(V)
    if kind == "random":
        x = torch.randn((N, V), generator=g, device="cuda") * 2.5
    elif kind == "ascending":
        x = torch.linspace(-9, 9, V, device="cuda").expand(N, V) + torch.arange(N, device="cuda")[:, None] * 0.001
    elif kind == "equal":
        x = torch.zeros((N, V), device="cuda")
    else:
        x = torch.randint(0, 5, (N, V), generator=g, device="cuda").float()
    logits = x.to(dtype)[:, None].contiguous()
    del x
    scores = torch.linspace(-3, 0, N, device="cuda")[:, None].contiguous()
    o = api.moe_beam_select(logits, scores, K)
    assert torch.equal(o.parents, torch.arange(N, dtype=I32, device="cuda")[:, None].expand(N, K))
    rows = logits[:, 0].float()
    want, at = torch.sort(rows, dim=1, descending=True, stable=True)
    assert torch.equal(o.tokens.long(), at[:, :K])
    lse = torch.logsumexp(rows.double(), 1, keepdim=True)
    ref = scores.double() + want[:, :K].double() - lse
    assert bool(((o.scores.double() - ref).abs() <= BAR + 2.0 ** -23 * ref.abs()).all())
    assert api.moe_get_device_errors() == 0


def test_repeats_on_any_workspace_stream_and_graph():
    logits, scores = _inputs(3, 6, 40_000, F32, seed=9)
    ref = _check(logits, scores, 12)
    ws = api.moe_beam_select_workspace(logits, 12)
    s = torch.cuda.Stream()
    for fill in (0, 255):
        ws.fill_(fill)
        s.wait_stream(torch.cuda.current_stream())
        got = api.moe_beam_select(logits, scores, 12, workspace=ws, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    out = api.BeamSelected(*[torch.empty_like(t) for t in ref])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_beam_select(logits, scores, 12, workspace=ws, out=out)
    ws.fill_(255)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    logits.copy_(logits.flip(2))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.tokens, 39_999 - ref.tokens)


def test_refusals():
    logits, scores = _inputs(2, 3, 50, F32, seed=1)
    with pytest.raises(ValueError):
        api.moe_beam_select(logits.half(), scores, 4)
    with pytest.raises(ValueError):
        api.moe_beam_select(logits.transpose(1, 2), scores, 4)
    with pytest.raises(ValueError):
        api.moe_beam_select(logits, scores[:1], 4)
    with pytest.raises(ValueError):
        api.moe_beam_select(logits, scores.double(), 4)
    with pytest.raises(ValueError):
        api.moe_beam_select(logits, scores, 4, done=torch.zeros((2, 3), device="cuda"))
    with pytest.raises(ValueError):
        api.moe_beam_select(logits.cpu(), scores, 4)
    for K in (0, 65, 151):
        with pytest.raises(MoeError):
            api.moe_beam_select(logits, scores, K)
    done = torch.zeros((2, 3), dtype=torch.bool, device="cuda")
    for big in (dict(K=4, pad=1 << 32), dict(K=1 << 32)):        # (not what is left of them in 32 bits)
        with pytest.raises(ValueError):
            api.moe_beam_select(logits, scores, done=done, **big)
    for pad in (-1, 50):
        with pytest.raises(MoeError):
            api.moe_beam_select(logits, scores, 4, done=done, pad=pad)
    with pytest.raises(MoeError):
        api.moe_beam_select(logits, scores, 4, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert api.moe_beam_select(logits[:0], scores[:0], 4).tokens.shape == (0, 4)


def _ordered(logits, scores, K):
    """The K best of every search by the definition, as (beam, token) and their scores in 64 bits, compared without rounding
    (a score of -1e32 swallows a logit in 64 bits). A candidate that fp32 rounds to -inf counts as -inf."""
    out = []
    for x, s in zip(logits.double().cpu(), scores.double().cpu()):
        lp = x - torch.logsumexp(x, -1)[:, None]
        c = (s[:, None] + lp).float()
        keys = [(-Fraction(s[w].item()) - Fraction(lp[w, t].item()) if c[w, t] > -INF else INF, w, t)
                for w in range(x.shape[0]) for t in range(x.shape[1])]
        out.append([(w, t, -float(v)) for v, w, t in sorted(keys)[:K]])
    return out


@pytest.mark.parametrize("dtype", [F32, BF])
def test_sums_below_the_lowest_number(dtype):
    """Forbidden tokens of the type's lowest value in beams whose score is the lowest number or near it, and a row of both ends
    of the range: what fp32 cannot hold is -inf, last and in the indices' order. A score is rounded once, 2^-24 of itself, and lse
    errs by BAR."""
    logits, _ = _inputs(4, 3, 61, dtype, seed=12)
    low, lowest = torch.finfo(dtype).min, torch.finfo(F32).min
    scores = torch.tensor([[-1.0, lowest, -1e32], [lowest, -1e32, lowest], [lowest, lowest, lowest], [0.0, -2.0, lowest]], device="cuda")
    logits[0, :, 5:] = low                                            # fewer tokens than K are allowed
    logits[1, :, 3:] = low
    logits[2, :, :58] = low
    logits[3, 0] = 0.0
    logits[3, 0, 7], logits[3, 0, [9, 20]] = 3e38, -3e38
    for K in (1, 10, 40, 64):
        o = api.moe_beam_select(logits, scores, K)
        rows, tokens, got = o.parents.tolist(), o.tokens.tolist(), o.scores.tolist()
        for n, want in enumerate(_ordered(logits, scores, K)):
            assert [(r - 3 * n, t) for r, t in zip(rows[n], tokens[n])] == [(w, t) for w, t, _ in want], (n, K)
            for g, (_, _, v) in zip(got[n], want):
                assert g == v if v == -INF else abs(g - v) <= BAR + 2.0 ** -23 * abs(v), (n, K, g, v)
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("dtype,N,W,V", [(BF, 32, 8, 131_072), (F32, 32, 8, 65_536), (BF, 32, 8, 50_257), (F32, 32, 8, 30_001),
                                         (BF, 3, 5, 40_003), (F32, 700, 2, 9_001), (BF, 1, 64, 1_001)])
def test_equal_beams_of_many_units(dtype, N, W, V):
    """Beams with the same logits and scores are taken in their order wherever the blocks' stretches cut their rows and
    wherever the rows begin against 16 bytes: their values are the same bits."""
    K = 2 * W if W <= 32 else W
    g = torch.Generator(device="cuda").manual_seed(V)
    one = (torch.randn((N, 1, V), generator=g, device="cuda") * 2.5).to(dtype)
    scores = (-8 * torch.rand((N, 1), generator=g, device="cuda")).expand(N, W).contiguous()
    o = api.moe_beam_select(one.expand(N, W, V).contiguous(), scores, K)
    for n in range(N):
        at = torch.sort(one[n].float().expand(W, V).reshape(-1), descending=True, stable=True).indices[:K]
        assert torch.equal(o.parents[n].long(), n * W + at // V) and torch.equal(o.tokens[n].long(), at % V), n
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("dtype,V", [(BF, 131_072), (F32, 20_000), (BF, 50_257), (F32, 33_333), (BF, 333)])
def test_a_search_does_not_depend_on_its_place(dtype, V):
    """The same search at every place of a batch, and alone, gives the same bits."""
    logits, scores = _inputs(1, 5, V, dtype, seed=V)
    alone = api.moe_beam_select(logits, scores, 16)
    N = 31
    o = api.moe_beam_select(logits.expand(N, 5, V).contiguous(), scores.expand(N, 5).contiguous(), 16)
    base = 5 * torch.arange(N, dtype=I32, device="cuda")[:, None]
    assert torch.equal(o.scores, alone.scores.expand(N, 16)) and torch.equal(o.tokens, alone.tokens.expand(N, 16))
    assert torch.equal(o.parents - base, alone.parents.expand(N, 16))
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("N,W,V,dtype", [(260, 1, (1 << 24) - 1, BF), (2, 3, (1 << 24) - 1, F32), (1, 2, (1 << 24) - 8, BF)])
def test_the_largest_vocabulary(N, W, V, dtype):
    """Rows of the most logits, off 16 bytes and on them; 260 of them lie past 2^32 logits."""
    K = 24
    logits = torch.empty((N, W, V), dtype=dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(N))
    scores = -8 * torch.rand((N, W), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    if W > 1:
        scores[:, 1:] = -1e4                                          # far behind: the first beam's tokens in their order
    logits[-1, 0, [5, V - 1, V // 2]] = 20.0                          # ties, the row's last logit among them
    o = api.moe_beam_select(logits, scores, K)
    for n in sorted({0, 1, N // 2, N - 1} & set(range(N))):
        x = logits[n, 0].float()
        want, at = torch.sort(x, descending=True, stable=True)
        assert torch.equal(o.tokens[n].long(), at[:K]) and bool((o.parents[n] == n * W).all()), n
        ref = scores[n, 0].double() + want[:K].double() - torch.logsumexp(x.double(), 0)
        assert bool(((o.scores[n].double() - ref).abs() <= BAR + 2.0 ** -23 * ref.abs()).all()), n
    assert o.tokens[-1, :3].tolist() == [5, V // 2, V - 1]
    assert api.moe_get_device_errors() == 0
