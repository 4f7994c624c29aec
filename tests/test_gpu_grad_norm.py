"""Global gradient norm and clipping against a plain 64-bit implementation, through the C ABI.

Bars, u = 2^-24: a thread adds at most n squares in fp32, so the norm errs by less than (n / 2 + 8) u of
itself; n <= 2^11 holds for every size here (the rest is a tree): 2^-14. Outputs: the scale's
error, and half a unit of the last place (2^-8 of a bf16 value, u of an fp32 one)."""
import pytest
import torch

from dropless_moe_expert_router_gb300 import api
from dropless_moe_expert_router_gb300.api import MoeError

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NORM_BAR = 2.0 ** -14


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dropless_moe_expert_router_gb300 import build
    build.build()


def _grads(sizes, seed, std=0.05, off=0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = BF if i % 3 != 1 else F32
        buf = (torch.randn(n + off, generator=g) * std).to(dt).cuda()
        out.append(buf[off:])
    return out


def _norm(grads):
    return sum(t.double().square().sum() for t in grads).sqrt().item() if grads else 0.0


def _check_out(outs, grads, c):
    for o, t in zip(outs, grads):
        ref = t.double() * c
        half = 2.0 ** -8 if t.dtype == BF else 2.0 ** -24
        assert o.dtype == t.dtype
        assert bool(((o.double() - ref).abs() <= (1.01 * half + NORM_BAR) * ref.abs() + 1e-45).all())


LISTS = [[1], [7], [5, 0, 3], [16384], [16385, 1, 8191], [100003, 4096, 33, 0, 250001], [3_000_001, 2_000_000],
         [17] * 300, [1000 + 37 * i for i in range(120)]]


@pytest.mark.parametrize("off", [0, 1, 4])
@pytest.mark.parametrize("sizes", LISTS, ids=[str(i) for i in range(len(LISTS))])
def test_norm_and_clip(sizes, off):
    grads = _grads(sizes, seed=len(sizes) + off, off=off)
    ref = _norm(grads)
    got = api.moe_grad_norm(grads)
    assert abs(got.item() - ref) <= NORM_BAR * ref
    for factor in (0.25, 4.0):                                       # clipped, and left alone
        outs = [torch.full_like(t, 9.0) for t in grads]
        keep = [t.clone() for t in grads]
        norm = api.moe_grad_clip(grads, factor * ref, out=outs)
        assert abs(norm.item() - ref) <= NORM_BAR * ref
        assert all(torch.equal(a, b) for a, b in zip(grads, keep))
        _check_out(outs, grads, min(1.0, factor * ref / (ref + 1e-6)))
        if factor > 1:
            assert all(torch.equal(a, b) for a, b in zip(outs, grads))
    keep = [t.clone() for t in grads]
    norm = api.moe_grad_clip(grads, 0.5 * ref)                       # in place
    _check_out(grads, keep, 0.5 * ref / (ref + 1e-6))
    again = api.moe_grad_norm(grads)
    assert abs(again.item() - 0.5 * ref) <= 0.01 * ref


def test_zero_gradients_and_zero_norm():
    z = [torch.zeros(1000, dtype=BF, device="cuda"), torch.zeros(3, device="cuda")]
    assert api.moe_grad_clip(z, 1.0).item() == 0.0 and not z[0].any()
    g = _grads([50, 60], seed=1)
    api.moe_grad_clip(g, 0.0)
    assert not g[0].any() and not g[1].any()
    norm = torch.full((1,), 5.0, device="cuda")
    assert api.moe_grad_clip([], 1.0, norm=norm).item() == 0.0
    e = [torch.empty(0, dtype=BF, device="cuda")]
    assert api.moe_grad_norm(e).item() == 0.0


@pytest.mark.parametrize("bad,dt", [(float("nan"), BF), (float("nan"), F32), (float("inf"), BF), (1e30, F32)])
def test_bad_values_reach_the_norm_and_every_output(bad, dt):
    g = [torch.ones(5000, dtype=dt, device="cuda"), torch.ones(100, device="cuda")]
    g[0][4321] = bad
    outs = [torch.empty_like(t) for t in g]
    norm = api.moe_grad_clip(g, 1.0, out=outs).item()
    if bad != bad:
        assert norm != norm and all(torch.isnan(o.float()).all() for o in outs)
    else:                                                            # infinite norm: c = 0
        assert norm == float("inf")
        assert not outs[1].any() and not outs[0][:4321].any()
        if bad == float("inf"):
            assert torch.isnan(outs[0][4321].float())


def test_repeats_bit_for_bit_on_any_workspace_and_stream():
    g = _grads([700_001, 3, 90_000], seed=3)
    ref = api.moe_grad_norm(g)
    n = int(api._lib.load().moe_grad_norm_workspace_size(3))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(t) for t in g]
    s = torch.cuda.Stream()
    for fill in (0, 255):
        ws.fill_(fill)
        s.wait_stream(torch.cuda.current_stream())
        norm = api.moe_grad_clip(g, 1.0, out=outs, workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(norm, ref)
    want = [t.clone() for t in outs]
    norm = torch.empty(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_grad_clip(g, 1.0, out=outs, norm=norm, workspace=ws)
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, ref) and all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    g = _grads([100, 200], seed=1)
    with pytest.raises(MoeError):
        api.moe_grad_clip(g, -1.0)
    with pytest.raises(MoeError):
        api.moe_grad_clip(g, float("nan"))
    with pytest.raises(ValueError):
        api.moe_grad_clip(g, 1.0, out=g[:1])
    with pytest.raises(ValueError):
        api.moe_grad_clip(g, 1.0, out=[g[0], g[1].to(BF)])
    with pytest.raises(ValueError):
        api.moe_grad_norm([g[0].half()])
    with pytest.raises(ValueError):
        api.moe_grad_norm([g[0].cpu()])
    with pytest.raises(ValueError):
        api.moe_grad_norm([torch.ones((4, 6), device="cuda").t()])
    with pytest.raises(ValueError):
        api.moe_grad_norm([])
    with pytest.raises(MoeError):
        api.moe_grad_norm(g, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dt", [BF, F32])
def test_zero_gradients_and_no_room_at_all_stay_zero(dt):
    """max_norm = 0, eps = 0 and a norm of 0: nothing to clip, not 0 / 0."""
    z = [torch.zeros(3000, dtype=dt, device="cuda"), torch.zeros(5, device="cuda")]
    outs = [torch.full_like(t, 3.0) for t in z]
    assert api.moe_grad_clip(z, 0.0, eps=0.0, out=outs).item() == 0.0
    assert not any(o.any() for o in outs)
    assert api.moe_grad_clip(z, 0.0, eps=0.0).item() == 0.0
    assert not any(t.any() for t in z)


def test_an_infinite_bound_clips_nothing():
    """max_norm = inf only measures, also where the squares overflow fp32."""
    for value in (0.5, 1e25):
        g = [torch.full((2000,), value, device="cuda"), torch.full((70,), -1.0, dtype=BF, device="cuda")]
        keep = [t.clone() for t in g]
        outs = [torch.empty_like(t) for t in g]
        norm = api.moe_grad_clip(g, float("inf"), out=outs).item()
        assert norm == float("inf") if value > 1 else abs(norm - _norm(keep)) <= NORM_BAR * _norm(keep)
        assert all(torch.equal(a, b) for a, b in zip(outs, keep))
        api.moe_grad_clip(g, float("inf"))
        assert all(torch.equal(a, b) for a, b in zip(g, keep))
    g = [torch.tensor([1.0, float("nan")], device="cuda")]
    api.moe_grad_clip(g, float("inf"))
    assert torch.isnan(g[0]).all()                                       # a NaN still reaches every output
