"""The whole layer for a few tokens against a plain 64-bit implementation, through the C ABI.

Bars. ids: equal. probs: 1e-6 absolute (the router's bar). y, with A = sum over the routes of
p sum |h||W2| (the sum of the magnitudes that y is summed from):
  2^-8 |y|       the one rounding of y to bf16 (half a unit of the last of 8 significant bits);
  2^-12 A        bf16 h: where an fp32 sum falls on the other side of a rounding boundary, h
                 differs by one step, at most 2^-7 of itself; fewer than one in 32 do;
  2^-10 A        MXFP8 h: a step is at most 2^-3 of the value, fewer than one in 128 differ.
"""
import numpy as np
import pytest
import torch

from dropless_moe_expert_router_gb300 import api
from dropless_moe_expert_router_gb300.api import MoeError

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dropless_moe_expert_router_gb300 import build
    build.build()
    api.moe_get_device_errors(clear=True)


def _mxfp8(v):
    """Row-wise 1x32 MXFP8 of a float64 array, as values."""
    b = v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32))
    amax = np.abs(b).max(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))) - 8, 0.0)
    e = np.clip(e, -127, 127)
    scaled = np.clip(b / 2.0 ** e, -448, 448)
    q = torch.from_numpy(scaled.astype(np.float32)).to(torch.float8_e4m3fn).to(torch.float32).numpy()
    return (q.astype(np.float64) * 2.0 ** e).reshape(v.shape)


def _decoded(codes, scales):
    v = codes.cpu().view(torch.float8_e4m3fn).to(torch.float64).numpy()
    s = 2.0 ** (scales.cpu().to(torch.float64).numpy() - 127)
    return (v.reshape(v.shape[:-1] + (-1, 32)) * s[..., None]).reshape(v.shape)


def _weights(E, H, F, precision, seed, std=0.05):
    g = torch.Generator().manual_seed(seed)
    w1, w3 = ((torch.randn((E, H, F), generator=g) * std).to(torch.bfloat16) for _ in range(2))
    w2 = (torch.randn((E, F, H), generator=g) * std).to(torch.bfloat16)
    return (w1, w3, w2), api.moe_prepare_weights(w1.cuda(), w3.cuda(), w2.cuda(), precision)


def _reference(x, ids, probs, packed, largest=False):
    """(y, A) in 64 bits from bf16 x, integer ids, probs and the packed weights; largest: A is the largest of
    the magnitudes that y is summed from, not their sum."""
    fp8 = packed.precision == "mxfp8"
    T, K = ids.shape
    E, H, F = packed.E, packed.H, packed.F
    X = x.double().cpu().numpy()
    if fp8:
        X = _mxfp8(X)
    first = np.arange(F) // 128 * 256 + np.arange(F) % 128
    y, A = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        at = [(t, k) for t in range(T) for k in range(K) if ids[t, k] == e]
        if not at:
            continue
        if fp8:
            w13 = _decoded(packed.w13[e], packed.w13_scales[e])
            w2 = _decoded(packed.w2[e], packed.w2_scales[e])
        else:
            w13, w2 = packed.w13[e].double().cpu().numpy(), packed.w2[e].double().cpu().numpy()
        a, b = X[[t for t, _ in at]] @ w13[first].T, X[[t for t, _ in at]] @ w13[first + 128].T
        h = a / (1 + np.exp(-a)) * b
        h = _mxfp8(h) if fp8 else torch.from_numpy(h).to(torch.bfloat16).double().numpy()
        d = h @ w2.T
        m = np.stack([(np.abs(r) * np.abs(w2)).max(1) for r in h]) if largest else np.abs(h) @ np.abs(w2.T)
        for i, (t, k) in enumerate(at):
            y[t] += float(probs[t, k]) * d[i]
            A[t] = np.maximum(A[t], float(probs[t, k]) * m[i]) if largest else A[t] + float(probs[t, k]) * m[i]
    return y, A


def _check(y, x, ids, probs, packed):
    ref, A = _reference(x, ids.cpu().numpy(), probs.cpu().numpy(), packed)
    got = y.double().cpu().numpy()
    bar = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 if packed.precision == "mxfp8" else 2.0 ** -12) * A
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= bar).all(), float((np.abs(got - ref) / np.maximum(bar, 1e-30)).max())


def _inputs(T, H, E, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, H), generator=g).to(torch.bfloat16).cuda(), torch.randn((T, E), generator=g).cuda()


CASES = [
    (1, 256, 8, 2, 512, "bf16", False, torch.int32),
    (3, 128, 1, 1, 128, "bf16", True, torch.int32),        # one expert
    (7, 384, 5, 5, 128, "bf16", False, torch.int16),       # K = E
    (16, 256, 4, 2, 640, "bf16", True, torch.int32),
    (17, 640, 3, 1, 256, "bf16", False, torch.int32),
    (64, 256, 33, 3, 384, "bf16", True, torch.int32),
    (64, 128, 64, 64, 128, "bf16", False, torch.int16),    # T * K = 4096
    (5, 256, 2304, 36, 128, "bf16", False, torch.int16),
    (33, 128, 700, 20, 128, "bf16", True, torch.int32),
    (2, 1152, 2, 1, 2176, "bf16", False, torch.int32),
    (1, 512, 4, 2, 512, "mxfp8", False, torch.int32),
    (9, 512, 40, 8, 1024, "mxfp8", True, torch.int32),
    (64, 1024, 8, 2, 512, "mxfp8", True, torch.int16),
    (31, 512, 300, 7, 512, "mxfp8", False, torch.int32),
]


@pytest.mark.parametrize("T,H,E,K,F,precision,renorm,idt", CASES)
def test_few_tokens_matches_plain(T, H, E, K, F, precision, renorm, idt):
    x, lg = _inputs(T, H, E, seed=T * 31 + E)
    _, packed = _weights(E, H, F, precision, seed=E + F)
    y, ids, probs = api.moe_layer_few_tokens(x, lg, packed, K, renorm=renorm, id_dtype=idt)
    want_ids, want_p = api.moe_route_topk(lg, K, renorm=renorm, id_dtype=idt)
    assert ids.dtype == idt and torch.equal(ids, want_ids)
    assert (probs - want_p).abs().max().item() <= 1e-6
    _check(y, x, ids, probs, packed)
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("T,H,E,K,F,precision", [
    (1, 4096, 2, 1, 128, "bf16"),          # two tiles, each by dozens of blocks
    (64, 2048, 3, 2, 512, "bf16"),         # few tiles, many tokens
    (40, 7168, 1, 1, 128, "bf16"),
    (5, 4096, 3, 2, 512, "mxfp8"),
    (64, 7168, 2, 2, 512, "mxfp8"),
    (17, 1024, 21, 4, 2048, "mxfp8"),      # more tiles than blocks, shared ones among them
    (6, 1536, 30, 6, 1280, "bf16"),
])
def test_few_tokens_shared_tiles(T, H, E, K, F, precision):
    """Sizes whose tiles are shared between the GPU's blocks and joined from partial sums. With F as
    small as 128 a single step of h weighs more than the bars' share of all terms: they are joined
    by two steps (2^-7 each, MXFP8 2^-3) of the largest term."""
    x, lg = _inputs(T, H, E, seed=T + H)
    _, packed = _weights(E, H, F, precision, seed=E + F, std=0.02)
    y, ids, probs = api.moe_layer_few_tokens(x, lg, packed, K)
    ref, A = _reference(x, ids.cpu().numpy(), probs.cpu().numpy(), packed)
    _, M = _reference(x, ids.cpu().numpy(), probs.cpu().numpy(), packed, largest=True)
    fp8 = precision == "mxfp8"
    bar = 2.0 ** -8 * np.abs(ref) + 2.0 ** (-10 if fp8 else -12) * A + 2.0 ** (-2 if fp8 else -6) * M
    assert (np.abs(y.double().cpu().numpy() - ref) <= bar).all()
    assert torch.equal(y, api.moe_layer_few_tokens(x, lg, packed, K)[0])
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("E,K", [(200, 17), (256, 128), (257, 100), (1024, 9), (2304, 36), (8192, 40)])
def test_few_tokens_router_ties(E, K):
    """Equal logits, a few values only, both zeros and infinities: ties go to the lower index."""
    T = 8
    lg = torch.zeros((T, E))
    g = torch.Generator().manual_seed(E)
    lg[1] = torch.randint(0, 3, (E,), generator=g).float()
    lg[2, ::2] = -0.0
    lg[3] = torch.randint(0, 2, (E,), generator=g).float() * -1e30
    lg[4] = float("-inf")
    lg[4, E // 2:] = torch.arange(E - E // 2).float() % 5
    lg[5] = torch.arange(E).float()
    lg[6] = -torch.arange(E).float()
    lg[7] = (torch.arange(E) % 7).float() * 1e-40                   # subnormal
    _, packed = _weights(1, 128, 128, "bf16", seed=1)
    w = packed._replace(E=E, w13=packed.w13.expand(E, -1, -1).contiguous(), w2=packed.w2.expand(E, -1, -1).contiguous())
    x, _ = _inputs(T, 128, 1, seed=3)
    y, ids, _ = api.moe_layer_few_tokens(x, lg.cuda(), w, K)
    want = torch.sort(lg.double(), dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(ids.cpu().long(), want)
    assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("idt", [torch.int16, torch.int32])
def test_few_tokens_given_routes(precision, idt):
    """Routes of the caller's: invalid ones, a token with none (zeros), an expert named twice by
    one token (both weights count), one expert taken by every token."""
    T, H, E, K, F = 19, 512, 11, 4, 512
    x, _ = _inputs(T, H, E, seed=5)
    _, packed = _weights(E, H, F, precision, seed=6)
    g = torch.Generator().manual_seed(7)
    ids = torch.randint(0, E, (T, K), generator=g).to(idt)
    ids[:, 0] = 3
    ids[0] = -1
    ids[1, 1:] = -1
    ids[2] = 9
    ids[T - 1] = torch.tensor([-1, 4, -1, 4]).to(idt)
    probs = torch.rand((T, K), generator=g)
    probs[4] = 0.0
    ids, probs = ids.cuda(), probs.cuda()
    keep_i, keep_p = ids.clone(), probs.clone()
    y, i2, p2 = api.moe_layer_few_tokens(x, None, packed, K, ids=ids, probs=probs)
    assert i2 is ids and p2 is probs and torch.equal(ids, keep_i) and torch.equal(probs, keep_p)
    _check(y, x, ids, probs, packed)
    assert not y[0].any() and not y[4].any()
    assert api.moe_get_device_errors() == 0
    ids[5, 2] = E                                                    # outside [-1, E): invalid, and flagged
    ids[6, 1] = -2
    y, _, _ = api.moe_layer_few_tokens(x, None, packed, K, ids=ids, probs=probs)
    _check(y, x, ids, probs, packed)
    assert api.moe_get_device_errors() == api.MOE_DEVERR_BAD_ID


def test_few_tokens_no_valid_route_at_all():
    x, _ = _inputs(6, 256, 8, seed=1)
    _, packed = _weights(8, 256, 128, "bf16", seed=2)
    ids = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    y, _, _ = api.moe_layer_few_tokens(x, None, packed, 2, ids=ids, probs=torch.ones((6, 2), device="cuda"),
                                       y=torch.full((6, 256), 7.0, dtype=torch.bfloat16, device="cuda"))
    assert not y.any()


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_few_tokens_skewed_to_one_expert(precision):
    x, lg = _inputs(64, 512, 16, seed=8)
    lg[:, 7] += 100.0
    _, packed = _weights(16, 512, 512, precision, seed=9)
    y, ids, probs = api.moe_layer_few_tokens(x, lg, packed, 1)
    assert (ids == 7).all()
    _check(y, x, ids, probs, packed)


def test_few_tokens_bad_values_stay_in_their_token():
    """A NaN and an infinity in two tokens, NaN weights in an expert nobody chose: the other
    tokens' results are those without them."""
    T, H, E, K, F = 20, 256, 6, 2, 256
    x, lg = _inputs(T, H, E, seed=11)
    lg[:, 5] = -100.0
    _, packed = _weights(E, H, F, "bf16", seed=12)
    y0, _, _ = api.moe_layer_few_tokens(x, lg, packed, K)
    packed.w13[5] = float("nan")
    packed.w2[5] = float("nan")
    x2 = x.clone()
    x2[3, 17] = float("nan")
    x2[8, 200] = float("inf")
    y1, _, _ = api.moe_layer_few_tokens(x2, lg, packed, K)
    clean = [t for t in range(T) if t not in (3, 8)]
    assert torch.equal(y0[clean], y1[clean])
    assert not torch.isfinite(y1[3].float()).all() and not torch.isfinite(y1[8].float()).all()


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_few_tokens_repeats_bit_for_bit(precision):
    """The same call on a workspace of any contents, another stream and a graph's replay."""
    x, lg = _inputs(13, 1024, 24, seed=21)
    _, packed = _weights(24, 1024, 1024, precision, seed=22)
    ws = api.moe_layer_few_tokens_workspace(packed, 13, 3)
    first = api.moe_layer_few_tokens(x, lg, packed, 3, workspace=ws)[0].clone()
    for fill in (0, 255, 1):
        ws.fill_(fill)
        assert torch.equal(api.moe_layer_few_tokens(x, lg, packed, 3, workspace=ws)[0], first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = api.moe_layer_few_tokens(x, lg, packed, 3, workspace=ws, stream=s)[0]
    s.synchronize()
    assert torch.equal(y, first)
    y = torch.empty_like(first)
    ids, probs = torch.empty((13, 3), dtype=torch.int32, device="cuda"), torch.empty((13, 3), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_layer_few_tokens(x, lg, packed, 3, ids=ids, probs=probs, y=y, workspace=ws)
    for seed in (31, 32):
        x2, lg2 = _inputs(13, 1024, 24, seed=seed)
        x.copy_(x2)
        lg.copy_(lg2)
        graph.replay()
        got = y.clone()
        assert torch.equal(got, api.moe_layer_few_tokens(x2, lg2, packed, 3)[0])


def test_few_tokens_zero_tokens_and_refusals():
    _, packed = _weights(4, 256, 128, "bf16", seed=2)
    y, ids, probs = api.moe_layer_few_tokens(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"),
                                             torch.empty((0, 4), device="cuda"), packed, 2)
    assert y.shape == (0, 256) and ids.shape == (0, 2) and probs.shape == (0, 2)
    x, lg = _inputs(3, 256, 4, seed=1)
    with pytest.raises(MoeError):
        api.moe_layer_few_tokens(x, lg, packed, 5)                                    # K > E
    with pytest.raises(MoeError):
        api.moe_layer_few_tokens(*_inputs(65, 256, 4, seed=1), packed, 2)             # T > 64
    with pytest.raises(MoeError):
        api.moe_layer_few_tokens(x, lg, packed, 2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        api.moe_layer_few_tokens(x, lg[:, :3].contiguous(), packed, 2)
    with pytest.raises(ValueError):
        api.moe_layer_few_tokens(x.t(), lg, packed, 2)
    with pytest.raises(ValueError):
        api.moe_layer_few_tokens(x.float(), lg, packed, 2)
    with pytest.raises(ValueError):
        api.moe_layer_few_tokens(x, None, packed, 2)
    with pytest.raises(ValueError):
        api.moe_layer_few_tokens(x.cpu(), lg, packed, 2)
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("T,H,E,K,F,precision", [
    (64, 256, 40, 4, 1024, "bf16"), (33, 512, 16, 2, 2048, "bf16"), (17, 128, 64, 4, 1024, "bf16"),
    (64, 512, 16, 4, 2048, "mxfp8"), (9, 128, 128, 16, 512, "bf16"), (50, 384, 100, 3, 640, "bf16")])
def test_few_tokens_joined_in_two_steps(T, H, E, K, F, precision):
    """Few output tiles and many tokens: a tile's many blocks are joined in groups first. The tokens'
    results do not depend on when the blocks arrive."""
    x, lg = _inputs(T, H, E, seed=2 * T + H)
    _, packed = _weights(E, H, F, precision, seed=E + 3 * F)
    y, ids, probs = api.moe_layer_few_tokens(x, lg, packed, K)
    _check(y, x, ids, probs, packed)
    for _ in range(5):
        assert torch.equal(y, api.moe_layer_few_tokens(x, lg, packed, K)[0])
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("T,E,K", [(64, 2304, 36), (40, 1024, 100), (64, 8192, 16)])
def test_few_tokens_renormalised_probs_repeat_bit_for_bit(T, E, K):
    """Above 256 experts the chosen logits are listed in the order in which the threads find them; the sum
    over them is not in that order."""
    _, packed = _weights(1, 128, 128, "bf16", seed=1)
    w = packed._replace(E=E, w13=packed.w13.expand(E, -1, -1).contiguous(), w2=packed.w2.expand(E, -1, -1).contiguous())
    x, lg = _inputs(T, 128, E, seed=E + K)
    ws = api.moe_layer_few_tokens_workspace(w, T, K)
    y, ids, probs = api.moe_layer_few_tokens(x, lg, w, K, renorm=True, workspace=ws)
    chosen = torch.gather(lg.double(), 1, ids.long())
    assert (probs.double() - torch.softmax(chosen, 1)).abs().max().item() <= 1e-6
    for _ in range(200):
        y2, ids2, probs2 = api.moe_layer_few_tokens(x, lg, w, K, renorm=True, workspace=ws)
        assert torch.equal(ids, ids2) and torch.equal(probs, probs2) and torch.equal(y, y2)


@pytest.mark.parametrize("T,K,E,precision", [(64, 64, 8192, "bf16"), (32, 128, 8192, "bf16"), (63, 65, 4097, "bf16"),
                                             (64, 64, 2304, "mxfp8"), (32, 128, 2304, "mxfp8"), (64, 32, 8192, "mxfp8")])
def test_few_tokens_largest_plans(T, K, E, precision):
    """As many routes and experts as are taken. Expert e's W3 and W2 are one expert's times powers of two,
    by which h and its products scale exactly, so a token's output is that expert's output times
    sum p 2^(a(e) + b(e)). A step of h is the same for all of a token's experts: the bars join it from the
    largest term of the sum as in the test of shared tiles."""
    fp8 = precision == "mxfp8"
    H = F = 512 if fp8 else 128
    _, one = _weights(1, H, F, precision, seed=K)
    e = torch.arange(E, device="cuda")
    a, b = e % 3 - 1, e % 5 - 2
    linear = torch.arange(2 * F, device="cuda") // 128 % 2 == 1
    by = torch.where(linear[None], a[:, None], 0)
    w13, w2 = one.w13.expand(E, -1, -1).contiguous(), one.w2.expand(E, -1, -1).contiguous()
    s13 = s2 = None
    if fp8:
        s13 = (one.w13_scales.int() + by[..., None]).to(torch.uint8)
        s2 = (one.w2_scales.int() + b[:, None, None]).to(torch.uint8)
    else:
        w13.mul_(torch.exp2(by.float()).to(torch.bfloat16)[..., None])
        w2.mul_(torch.exp2(b.float()).to(torch.bfloat16)[:, None, None])
    w = one._replace(E=E, w13=w13, w13_scales=s13, w2=w2, w2_scales=s2)
    x, lg = _inputs(T, H, E, seed=E + K)
    y, ids, probs = api.moe_layer_few_tokens(x, lg, w, K, renorm=True)
    assert torch.equal(ids.long(), torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :K])
    zeros, ones = np.zeros((T, 1), dtype=np.int64), np.ones((T, 1))
    d, A = _reference(x, zeros, ones, one)
    _, M = _reference(x, zeros, ones, one, largest=True)
    c = (probs.double() * torch.exp2((a + b).double())[ids.long()]).sum(1, keepdim=True).cpu().numpy()
    bar = c * (2.0 ** -8 * np.abs(d) + 2.0 ** (-10 if fp8 else -12) * A + 2.0 ** (-2 if fp8 else -6) * M)
    assert (np.abs(y.double().cpu().numpy() - c * d) <= bar).all()
    assert torch.equal(y, api.moe_layer_few_tokens(x, lg, w, K, renorm=True)[0])
    assert api.moe_get_device_errors() == 0
