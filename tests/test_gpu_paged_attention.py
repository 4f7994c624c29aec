"""Attention of one new token over a paged cache against a plain 64-bit implementation, through the C ABI.

Bars. u = 2^-24. A score is a sum of dim products in fp32 and a product with the scale, so it errs by at most
e = (dim + 4) u scale sum |q k|; a weight exp(s - m) then errs by 2 e of itself (both s and m), by its rounding to
16 bits (at most half a step of bf16, 2^-8) and by 2^-12 for exp, the rescalings and the sums (a thread adds
fewer than 2^11 terms in a row). With A = sum w |v| the output errs by (2^-8 + 2 e + 2^-12) A and its own
rounding, 2^-8 of itself; lse by e + 2^-12 and its rounding."""
import math

import pytest
import torch

from dropless_moe_expert_router_gb300 import api
from dropless_moe_expert_router_gb300.api import MoeError

pytestmark = pytest.mark.gpu
BF, F32, I32, D64 = torch.bfloat16, torch.float32, torch.int32, torch.float64
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dropless_moe_expert_router_gb300 import build
    build.build()


def _randn(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _cache(lengths, heads, dim, page, precision="bf16", seed=0, spare=3, fill=float("nan"), extra_cols=1, std=1.0):
    """A cache whose unused positions and pages hold `fill`, its table, and the dense K, V in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lengths)
    held = [(n + page - 1) // page for n in lengths]
    pages = sum(held) + spare
    M = max(held + [0]) + extra_cols
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((B, M), -1, dtype=I32)
    for b, h in enumerate(held):
        for j in range(h):
            table[b, j] = order.pop()
    cache = api.cache_buffers(pages, heads, page, dim, "cuda", precision)
    for t in (cache.k, cache.v):
        t.fill_(fill) if precision == "bf16" else t.fill_(0x7f)              # (0x7f: an E4M3 NaN)
    for t in (cache.k_scales, cache.v_scales):
        if t is not None:
            t.fill_(255)
    table = table.cuda()
    total = sum(lengths)
    rows = torch.cat([torch.full((n,), b, dtype=I32) for b, n in enumerate(lengths)] or [torch.empty(0, dtype=I32)]).cuda()
    pos = torch.cat([torch.arange(n, dtype=I32) for n in lengths] or [torch.empty(0, dtype=I32)]).cuda()
    k, v = _randn((total, heads, dim), g, std).to(BF), _randn((total, heads, dim), g, std).to(BF)
    api.moe_cache_append(k, v, cache, table, pos, rows=rows)
    if precision == "mxfp8":
        k, v = api.moe_cache_gather(cache, table, pos, rows=rows)
    at, dense = 0, []
    for n in lengths:
        dense.append((k[at:at + n].double(), v[at:at + n].double()))
        at += n
    return cache, table, dense


def _check(q, cache, table, lengths, dense, out, lse, scale=None, window=0):
    dim = q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    group = q.shape[1] // cache.heads
    for b, n in enumerate(lengths):
        first = max(0, n - window) if window else 0
        if n == 0:
            assert not out[b].any() and bool((lse[b] == -float("inf")).all())
            continue
        k, v = (t[first:n].repeat_interleave(group, 1) for t in dense[b])
        x = q[b].double()
        s = torch.einsum("hd,jhd->hj", x, k) * scale
        e = (dim + 4) * 2.0 ** -24 * abs(scale) * torch.einsum("hd,jhd->hj", x.abs(), k.abs()).amax(1)
        ref_lse = torch.logsumexp(s, 1)
        assert bool(((lse[b].double() - ref_lse).abs() <= e + 2.0 ** -12 + 2.0 ** -23 * ref_lse.abs()).all())
        w = torch.softmax(s, 1)
        ref = torch.einsum("hj,jhd->hd", w, v)
        A = torch.einsum("hj,jhd->hd", w, v.abs())
        bar = (2.0 ** -8 + 2 * e[:, None] + 2.0 ** -12) * A + 2.0 ** -8 * ref.abs() + 1e-38
        assert out.dtype == BF and bool(((out[b].double() - ref).abs() <= bar).all()), b


def _run(lengths, q_heads, heads, dim, page, precision="bf16", window=0, scale=None, seed=0, std=1.0):
    cache, table, dense = _cache(lengths, heads, dim, page, precision, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = _randn((len(lengths), q_heads, dim), g, std).to(BF)
    lens = torch.tensor(lengths, dtype=I32, device="cuda")
    out, lse = api.moe_paged_attention(q, cache, table, lens, window=window, scale=scale)
    _check(q, cache, table, lengths, dense, out, lse, scale, window)
    assert api.moe_get_device_errors() == 0
    return q, cache, table, lens, dense, out, lse


LENGTHS = [[1], [0], [2, 0, 17], [100], [128, 129, 127], [1, 0, 0, 5, 1000, 16, 15], [3001, 64], [0, 0]]


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("lengths", LENGTHS, ids=[str(i) for i in range(len(LENGTHS))])
@pytest.mark.parametrize("q_heads,heads", [(8, 2), (1, 1), (7, 1)])
def test_lengths(lengths, q_heads, heads, precision):
    _run(lengths, q_heads, heads, 128, 16, precision)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 128, 160, 192, 256])
@pytest.mark.parametrize("q_heads,heads", [(3, 3), (6, 2), (18, 2)])
def test_widths(dim, q_heads, heads, precision):
    if precision == "mxfp8" and dim % 32:
        pytest.skip("MXFP8 rows are whole 32-element blocks")
    _run([333, 1, 40, 77], q_heads, heads, dim, 16, precision)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("page", [1, 3, 8, 24, 32, 128, 513])
def test_pages_that_end_anywhere(page, precision):
    _run([700, 33, 1, 0, page, page + 1], 8, 2, 64, page, precision)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("q_heads", [2, 5, 8, 9, 12, 16, 17, 24, 32, 33, 64, 100, 128])
def test_heads_of_a_group(q_heads, precision):
    _run([257, 0, 90], q_heads, 1, 128, 16, precision)
    _run([257, 90], q_heads * 3, 3, 64, 16, precision)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 1000, 100000, (1 << 32) + 5])
def test_window(window, precision):
    _run([700, 33, 1, 0, 100, 101], 8, 2, 128, 16, precision, window=window)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_long_and_many(precision):
    _run([70_000], 8, 1, 128, 16, precision)
    _run([20_000, 1, 20_001, 5000], 4, 4, 128, 32, precision)
    _run([(37 * i) % 500 for i in range(300)], 16, 2, 64, 16, precision)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_large_scores_and_scales(precision):
    """Weights that leave one position, scores far from zero in both directions, a negative scale."""
    _run([500, 31], 8, 2, 128, 16, precision, std=8.0)
    _run([500, 31], 8, 2, 128, 16, precision, scale=-0.3)
    _run([500, 31], 8, 2, 128, 16, precision, scale=0.0)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("factor", [2.0 ** -60, 2.0 ** -20, 2.0 ** 20, 2.0 ** 60, 2.0 ** 110])
def test_values_of_any_size(precision, factor):
    """Values by a power of two larger or smaller give outputs by it larger or smaller, bit for bit; one token's
    values 2^20 times the others' leave those where its weight is small."""
    lengths = [300, 45]
    q, cache, table, lens, dense, out, lse = _run(lengths, 8, 2, 128, 16, precision)
    rows = torch.cat([torch.full((n,), b, dtype=I32) for b, n in enumerate(lengths)]).cuda()
    pos = torch.cat([torch.arange(n, dtype=I32) for n in lengths]).cuda()
    k, v = api.moe_cache_gather(cache, table, pos, rows=rows)
    api.moe_cache_append(k, (v.float() * factor).to(BF), cache, table, pos, rows=rows)
    out2, lse2 = api.moe_paged_attention(q, cache, table, lens)
    assert torch.equal(lse2, lse) and torch.equal(out2.float(), out.float() * factor)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_an_unattended_outlier_among_the_values(precision):
    """A token with values 2^20 times the others' and a weight below 2^-60 changes nothing that can be seen."""
    lengths = [400]
    cache, table, dense = _cache(lengths, 1, 64, 16, precision)
    pos = torch.arange(400, dtype=I32, device="cuda")
    rows = torch.zeros(400, dtype=I32, device="cuda")
    k, v = api.moe_cache_gather(cache, table, pos, rows=rows)
    q = torch.ones((1, 4, 64), device="cuda", dtype=BF)
    for at in (0, 5, 130, 399):
        k2, v2 = k.clone(), v.clone()
        k2[at] = -8.0                                       # its score is -64 at scale 1 / 8
        v2[at] *= 2.0 ** 20
        api.moe_cache_append(k2, v2, cache, table, pos, rows=rows)
        out, lse = api.moe_paged_attention(q, cache, table, torch.tensor([400], dtype=I32, device="cuda"))
        k3, v3 = api.moe_cache_gather(cache, table, pos, rows=rows)
        _check(q, cache, table, lengths, [(k3.double(), v3.double())], out, lse)


@pytest.mark.parametrize("factor", [2.0 ** -40, 1.0, 2.0 ** 40])
def test_values_of_zeros_beside_small_and_large_ones(factor):
    """Rows of zeros, whose MXFP8 scale is 1 whatever the others' is, and scales that differ from block to block."""
    lengths = [150, 33]
    cache, table, dense = _cache(lengths, 2, 96, 16, "mxfp8")
    rows = torch.cat([torch.full((n,), b, dtype=I32) for b, n in enumerate(lengths)]).cuda()
    pos = torch.cat([torch.arange(n, dtype=I32) for n in lengths]).cuda()
    k, v = api.moe_cache_gather(cache, table, pos, rows=rows)
    v = v * factor
    v[::3] = 0
    v[1::3, :, 32:64] *= 2.0 ** -9
    v[2::3, 1] *= 2.0 ** 5
    api.moe_cache_append(k, v, cache, table, pos, rows=rows)
    k, v = api.moe_cache_gather(cache, table, pos, rows=rows)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = _randn((2, 6, 96), g).to(BF)
    out, lse = api.moe_paged_attention(q, cache, table, torch.tensor(lengths, dtype=I32, device="cuda"))
    dense = [(k[:150].double(), v[:150].double()), (k[150:].double(), v[150:].double())]
    _check(q, cache, table, lengths, dense, out, lse)


def test_a_nan_in_8_bits():
    lengths = [70]
    cache, table, dense = _cache(lengths, 1, 64, 16, "mxfp8")
    q = torch.ones((1, 2, 64), device="cuda", dtype=BF)
    lens = torch.tensor(lengths, dtype=I32, device="cuda")
    page, off = int(table[0, 2]), 7                           # position 39
    for codes, scales in ((cache.v, cache.v_scales), (cache.k, cache.k_scales)):
        for t, at, bad in ((codes, 40, 0x7f), (codes, 40, 0xff), (scales, 1, 255)):
            keep = t[page, 0, off, at].clone()
            t[page, 0, off, at] = bad
            out, lse = api.moe_paged_attention(q, cache, table, lens)
            if codes is cache.v:                              # its own elements: a code's one, a scale's 32
                hit = torch.zeros(64, dtype=torch.bool, device="cuda")
                hit[40 if at == 40 else slice(32, 64)] = True
                assert torch.isnan(out[0][:, hit]).all() and torch.isfinite(out[0][:, ~hit]).all() and torch.isfinite(lse).all()
            else:
                assert torch.isnan(out).all() and torch.isnan(lse).all()
            out, lse = api.moe_paged_attention(q, cache, table, lens, window=30)
            assert torch.isfinite(out).all() and torch.isfinite(lse).all()
            t[page, 0, off, at] = keep


def test_strided_queries_and_given_outputs():
    lengths = [90, 300, 0, 12]
    cache, table, dense = _cache(lengths, 2, 64, 16)
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = _randn((4, 12, 64), g).to(BF)
    q = qkv[:, 2:8]
    lens = torch.tensor(lengths, dtype=I32, device="cuda")
    ref, ref_lse = api.moe_paged_attention(q.contiguous(), cache, table, lens)
    out, lse = torch.full((4, 6, 64), 7.0, dtype=BF, device="cuda"), torch.full((4, 6), 7.0, device="cuda")
    api.moe_paged_attention(q, cache, table, lens, out=out, lse=lse)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    _check(q, cache, table, lengths, dense, out, lse)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_repeats_bit_for_bit_on_any_workspace_stream_and_graph(precision):
    lengths = [5000, 0, 333, 1, 70]
    q, cache, table, lens, dense, out, lse = _run(lengths, 8, 2, 128, 16, precision)
    ws = api.moe_paged_attention_workspace(cache, 5, 8)
    s = torch.cuda.Stream()
    for fill in (0, 255):
        ws.fill_(fill)
        s.wait_stream(torch.cuda.current_stream())
        o2, l2 = api.moe_paged_attention(q, cache, table, lens, workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    o3, l3 = torch.empty_like(out), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_paged_attention(q, cache, table, lens, workspace=ws, out=o3, lse=l3)
    ws.fill_(255)
    graph.replay()
    # lengths that a replay finds changed
    fewer = [4999, 3, 0, 1, 69]
    torch.cuda.synchronize()
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    lens.copy_(torch.tensor([4999, 0, 0, 1, 69], dtype=I32))
    graph.replay()
    torch.cuda.synchronize()
    _check(q, cache, table, [4999, 0, 0, 1, 69], [(k[:n], v[:n]) for (k, v), n in zip(dense, fewer)], o3, l3)


def test_two_calls_at_once_with_their_own_workspaces():
    a = _run([3000, 40], 8, 2, 128, 16, seed=3)
    b = _run([900, 4000], 8, 2, 128, 16, seed=4)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = []
        for st, (q, cache, table, lens, _, _, _) in zip(s, (a, b)):
            st.wait_stream(torch.cuda.current_stream())
            got.append(api.moe_paged_attention(q, cache, table, lens, stream=st))
        torch.cuda.synchronize()
        for (o, l), r in zip(got, (a, b)):
            assert torch.equal(o, r[5]) and torch.equal(l, r[6])


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_bad_pages_and_lengths_are_left_out_and_told(precision):
    lengths = [200, 64]
    cache, table, dense = _cache(lengths, 2, 64, 16, precision, extra_cols=0)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = _randn((2, 8, 64), g).to(BF)
    lens = torch.tensor(lengths, dtype=I32, device="cuda")
    for bad in (-1, cache.pages, 1 << 30, -7):
        t = table.clone()
        t[0, 3] = bad
        out, lse = api.moe_paged_attention(q, cache, t, lens)
        keep = [j for j in range(200) if not 48 <= j < 64]
        _check(q, cache, t, [184, 64], [tuple(x[keep] for x in dense[0]), dense[1]], out, lse)
        assert api.moe_get_device_errors() == api.MOE_DEVERR_BAD_ID
    # every page of a sequence gone: nothing to attend to
    t = table.clone()
    t[1] = -1
    out, lse = api.moe_paged_attention(q, cache, t, lens)
    _check(q, cache, t, [200, 0], dense, out, lse)
    assert api.moe_get_device_errors() == api.MOE_DEVERR_BAD_ID
    # longer than the table, and negative
    long = torch.tensor([13 * 16 + 1, -5], dtype=I32, device="cuda")
    assert table.shape[1] == 13
    out, lse = api.moe_paged_attention(q, cache, table, long)
    assert not out[1].any() and api.moe_get_device_errors() == api.MOE_DEVERR_BAD_ID


def test_nan_and_inf_where_they_are_attended():
    """What is attended to reaches the output: a NaN key every element, a NaN value its own; masked ones nothing."""
    lengths = [100]
    cache, table, dense = _cache(lengths, 1, 64, 16)
    q = torch.ones((1, 4, 64), device="cuda", dtype=BF)
    lens = torch.tensor(lengths, dtype=I32, device="cuda")
    page, off = int(table[0, 3]), 5                           # position 53
    keep = cache.v[page, 0, off, 7].clone()
    cache.v[page, 0, off, 7] = float("nan")
    out, lse = api.moe_paged_attention(q, cache, table, lens)
    assert torch.isnan(out[0, :, 7]).all() and torch.isfinite(out[0, :, :7]).all() and torch.isfinite(lse).all()
    out, lse = api.moe_paged_attention(q, cache, table, lens, window=100 - 54)
    assert torch.isfinite(out).all()
    cache.v[page, 0, off, 7] = keep
    cache.k[page, 0, off, 9] = float("nan")
    out, lse = api.moe_paged_attention(q, cache, table, lens)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_offsets_past_32_bits(precision):
    """Pages that lie past 2^32 elements of a pool."""
    heads, page, dim = 8, 64, 128
    pages = (1 << 32) // (heads * page * dim) + 40
    cache = api.cache_buffers(pages, heads, page, dim, "cuda", precision)
    n = 500
    table = torch.arange(pages - 8, pages, dtype=I32, device="cuda").flip(0)[None].contiguous()
    pos, rows = torch.arange(n, dtype=I32, device="cuda"), torch.zeros(n, dtype=I32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = _randn((n, heads, dim), g).to(BF), _randn((n, heads, dim), g).to(BF)
    api.moe_cache_append(k, v, cache, table, pos, rows=rows)
    k2, v2 = api.moe_cache_gather(cache, table, pos, rows=rows)
    if precision == "bf16":
        assert torch.equal(k2, k) and torch.equal(v2, v)
    q = _randn((1, 16, dim), g).to(BF)
    out, lse = api.moe_paged_attention(q, cache, table, torch.tensor([n], dtype=I32, device="cuda"))
    _check(q, cache, table, [n], [(k2.double(), v2.double())], out, lse)
    # a page moved across the border
    api.moe_cache_copy_pages(cache, table[0, :1].clone(), torch.tensor([2], dtype=I32, device="cuda"))
    table[0, 0] = 2
    o2, l2 = api.moe_paged_attention(q, cache, table, torch.tensor([n], dtype=I32, device="cuda"))
    assert torch.equal(o2, out) and torch.equal(l2, lse) and api.moe_get_device_errors() == 0


def test_refusals():
    cache, table, dense = _cache([20, 30], 2, 64, 16)
    q = torch.zeros((2, 8, 64), device="cuda", dtype=BF)
    lens = torch.tensor([20, 30], dtype=I32, device="cuda")
    call = api.moe_paged_attention
    with pytest.raises(ValueError):
        call(q.float(), cache, table, lens)
    with pytest.raises(ValueError):
        call(q[:, :7], cache, table, lens)                    # 7 heads over 2
    with pytest.raises(ValueError):
        call(q[..., :32], cache, table, lens)
    with pytest.raises(ValueError):
        call(q.transpose(0, 1).contiguous().transpose(0, 1), cache, table, lens)
    with pytest.raises(ValueError):
        call(q, cache, table[:1], lens)
    with pytest.raises(ValueError):
        call(q, cache, table.long(), lens)
    with pytest.raises(ValueError):
        call(q, cache, table, lens.long())
    with pytest.raises(ValueError):
        call(q, cache, table, lens[:1])
    with pytest.raises(ValueError):
        call(q.cpu(), cache, table, lens)
    with pytest.raises(ValueError):
        call(q, cache, table, lens, out=torch.empty((2, 8, 64), device="cuda"))
    with pytest.raises(MoeError):
        call(q, cache, table, lens, window=-1)
    with pytest.raises(MoeError):
        call(q, cache, table, lens, scale=float("nan"))
    with pytest.raises(MoeError):
        call(q, cache, table, lens, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        call(q, cache._replace(page_size=8), table, lens)
    with pytest.raises(MoeError):                             # tokens that do not start on 16 bytes
        wide = torch.zeros((2, 8 * 64 + 4), device="cuda", dtype=BF)
        call(wide[:, :512].unflatten(1, (8, 64)), cache, table, lens)
    assert api.moe_paged_attention(q[:0], cache, table[:0], lens[:0])[0].shape == (0, 8, 64)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_a_length_near_two_to_the_31(precision):
    """2^31 - 2 positions, every one of the 1049601 pages of 2046 positions the same: the attention over one page, and lse by
    ln 1049601 larger. With a block on each of 152 SMs or more, a lane adds to its sums at most 2^31 / (152 * 4 * 16) < 2^18 times in
    a row (sixteen positions of a warp's at a time). So the sum of weights errs by 2^18 * 2^-24 = 2^-6 at most, which is the bar
    of lse, and the numerators by 2^-5 (the matrix unit may cut where it adds, 2^-23). The values are between 1 and 2; two more
    roundings of 2^-8."""
    page, M = 2046, 1_049_601
    cache, table, dense = _cache([page], 1, 32, page, precision, spare=0)
    v = torch.rand((page, 1, 32), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") + 1
    k = dense[0][0].to(BF)
    pos, rows = torch.arange(page, dtype=I32, device="cuda"), torch.zeros(page, dtype=I32, device="cuda")
    api.moe_cache_append(k, v.to(BF), cache, table, pos, rows=rows)
    k, v = api.moe_cache_gather(cache, table, pos, rows=rows)
    q = _randn((1, 2, 32), torch.Generator(device="cuda").manual_seed(3)).to(BF)
    many = torch.zeros((1, M), dtype=I32, device="cuda")
    n = torch.tensor([page * M], dtype=I32, device="cuda")
    out, lse = api.moe_paged_attention(q, cache, many, n)
    s = q[0].double() @ k[:, 0].double().t() * 32 ** -0.5
    ref = torch.softmax(s, 1) @ v[:, 0].double()
    assert bool(((lse[0].double() - torch.logsumexp(s, 1) - math.log(M)).abs() <= 2.0 ** -6 + 2.0 ** -12).all())
    assert bool(((out[0].double() - ref).abs() <= (2.0 ** -5 + 2.0 ** -6 + 2.0 ** -7) * ref).all())
    # the last positions of it: one page less its first position
    out, lse = api.moe_paged_attention(q, cache, many, n, window=page - 1)
    ref = torch.softmax(s[:, 1:], 1) @ v[1:, 0].double()
    assert bool(((out[0].double() - ref).abs() <= (2.0 ** -7 + 2.0 ** -11) * ref).all())
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("dim,q_heads,heads", [(64, 4, 2), (128, 8, 1), (256, 2, 1), (96, 20, 1)])
def test_values_of_the_smallest_scale(dim, q_heads, heads):
    """Values whose scale bytes are 0 (2^-127), alone and beside the next ones. Their codes are 1 and above, so that each is a
    bf16 number."""
    lengths = [37, 300, 1]
    cache, table, _ = _cache(lengths, heads, dim, 16, "mxfp8")
    g = torch.Generator(device="cuda").manual_seed(dim)
    cache.v.copy_(torch.randint(0x38, 0x7f, cache.v.shape, generator=g, device="cuda"))
    q = _randn((3, q_heads, dim), g).to(BF)
    rows = torch.cat([torch.full((n,), b, dtype=I32) for b, n in enumerate(lengths)]).cuda()
    pos = torch.cat([torch.arange(n, dtype=I32) for n in lengths]).cuda()
    for most in (1, 2, 4):
        cache.v_scales.copy_(torch.randint(0, most, cache.v_scales.shape, generator=g, device="cuda"))
        k, v = api.moe_cache_gather(cache, table, pos, rows=rows)
        out, lse = api.moe_paged_attention(q, cache, table, torch.tensor(lengths, dtype=I32, device="cuda"))
        dense = [(k[rows == b].double(), v[rows == b].double()) for b in range(3)]
        assert min(d[1].min() for d in dense) >= 2.0 ** -127
        _check(q, cache, table, lengths, dense, out, lse)
        # (the bar of _check has 1e-38 for what fp32 cannot hold; these outputs are all well above)
        assert out.float().min() >= 2.0 ** -127


@pytest.mark.parametrize("dim,offset", [(32, 1), (64, 2), (96, 3), (160, 1), (192, 2), (224, 3)])
def test_scales_that_begin_off_a_word(dim, offset):
    """Pools of scales that begin and end inside words whose other bytes are NaN's, every page of them in use: outputs are those of
    pools of their own, bit for bit."""
    lengths = [15, 9, 1]
    cache, table, dense = _cache(lengths, 3, dim, 5, "mxfp8", spare=0)
    q = _randn((3, 6, dim), torch.Generator(device="cuda").manual_seed(dim)).to(BF)
    lens = torch.tensor(lengths, dtype=I32, device="cuda")
    out, lse = api.moe_paged_attention(q, cache, table, lens)
    _check(q, cache, table, lengths, dense, out, lse)
    moved = []
    for t in (cache.k_scales, cache.v_scales):
        buf = torch.full((t.numel() + 16,), 255, dtype=torch.uint8, device="cuda")
        moved.append(buf[offset:offset + t.numel()].view(t.shape).copy_(t))
    o2, l2 = api.moe_paged_attention(q, cache._replace(k_scales=moved[0], v_scales=moved[1]), table, lens)
    assert torch.equal(o2, out) and torch.equal(l2, lse) and api.moe_get_device_errors() == 0


@pytest.mark.parametrize("precision,apart", [("bf16", False), ("mxfp8", False), ("mxfp8", True)])
@pytest.mark.parametrize("dim,q_heads", [(64, 1), (128, 12), (256, 3), (128, 20)])
def test_weights_keep_their_bits(dim, q_heads, precision, apart):
    """Positions whose weights are all the same, and one whose value takes away what they sum to: a rounding of the weights is
    all that is left of the output. Bars: those of _check, with the weight's rounding 2^-16 (two bf16) in the place of 2^-8, or 2^-11
    (fp16). apart: scales of the values further apart than fp16 weights take, which are 16 bits then, too."""
    lengths = [40, 130, 7, 300, 64, 33, 90, 18, 250, 500] * 2
    cache, table, _ = _cache(lengths, 1, dim, 16, precision)
    rows = torch.cat([torch.full((n,), b, dtype=I32) for b, n in enumerate(lengths)]).cuda()
    pos = torch.cat([torch.arange(n, dtype=I32) for n in lengths]).cuda()
    first = pos == 0
    c = 0.02 + 0.011 * rows.float()                           # scores of 0 and -c sqrt(dim): weights 1 and exp(-c sqrt(dim))
    k = torch.where(first, torch.zeros_like(c), -c)[:, None, None].expand(-1, 1, dim).to(BF).contiguous()
    w = torch.exp(k[:, 0, 0].double() * dim ** 0.5)
    n = torch.tensor(lengths, device="cuda")[rows.long()].double()
    v = torch.where(first, -(n - 1) * torch.exp(-c.to(BF).double() * dim ** 0.5), torch.ones_like(w))
    v = v[:, None, None].expand(-1, 1, dim).to(BF).contiguous()
    if apart:
        v[pos % 5 == 3] *= 2.0 ** -20
    api.moe_cache_append(k, v, cache, table, pos, rows=rows)
    k, v = api.moe_cache_gather(cache, table, pos, rows=rows)
    q = torch.ones((len(lengths), q_heads, dim), dtype=BF, device="cuda")
    out, lse = api.moe_paged_attention(q, cache, table, torch.tensor(lengths, dtype=I32, device="cuda"))
    at = 0
    for b, n in enumerate(lengths):
        kb, vb = k[at:at + n, 0].double(), v[at:at + n, 0].double()
        at += n
        s = q[b].double() @ kb.t() * dim ** -0.5
        e = (dim + 4) * 2.0 ** -24 * s.abs().amax()
        p = torch.softmax(s, 1)
        ref, A = p @ vb, p @ vb.abs()
        bar = ((2.0 ** -11 if precision == "mxfp8" and not apart else 2.0 ** -16) + 2 * e + 2.0 ** -12) * A + 2.0 ** -8 * ref.abs()
        assert bool(((out[b].double() - ref).abs() <= bar).all()), b
    assert api.moe_get_device_errors() == 0


def test_infinite_values_stay_infinite():
    lengths = [100, 300]
    cache, table, dense = _cache(lengths, 1, 64, 16)
    q = torch.ones((2, 4, 64), device="cuda", dtype=BF)
    lens = torch.tensor(lengths, dtype=I32, device="cuda")
    for at in (0, 7, 53, 99):
        page, off = int(table[0, at // 16]), at % 16
        cache.v[page, 0, off, 7], cache.v[page, 0, off, 8] = INF, -INF
        out, _ = api.moe_paged_attention(q, cache, table, lens)
        assert bool((out[0, :, 7] == INF).all() and (out[0, :, 8] == -INF).all()) and torch.isfinite(out[1]).all()
        cache.v[page, 0, off, 7:9] = 0
    one = _cache([1], 1, 64, 16)                              # (a weight of one: its second part would be 0)
    one[0].v[one[1][0, 0], 0, 0, 7] = INF
    out, _ = api.moe_paged_attention(q[:1], one[0], one[1], torch.ones(1, dtype=I32, device="cuda"))
    assert bool((out[0, :, 7] == INF).all() and torch.isfinite(out[0, :, :7]).all())
