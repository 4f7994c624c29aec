"""Calls on a given stream that runs late: what they allocate stays theirs until their kernels are done,
although the current stream allocates and fills blocks of the same sizes meanwhile, and although
the caller keeps some of the results only."""
import pytest
import torch

from dropless_moe_expert_router_gb300 import api
from dropless_moe_expert_router_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dropless_moe_expert_router_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def ballast():
    return torch.randn((8192, 8192), device="cuda").to(BF)


def _late(ballast, call, sizes):
    """call(stream) on a stream that is some milliseconds behind, the current stream filling fresh blocks of
    these sizes as soon as the call has returned."""
    want = call(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(12):
            torch.mm(ballast, ballast)
        behind = torch.cuda.Event()
        behind.record()
    got = call(s)
    late = not behind.query()
    fills = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert late                                   # (else the test shows nothing)
    assert all(bool((f == 255).all()) for f in fills)      # nothing of the call's went into them
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def _normal(shape, seed, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_few_tokens(ballast, score):
    T, E, H, F, K = 24, 16, 512, 512, 4
    w = [_normal((E, H, F), 1, 0.05), _normal((E, H, F), 2, 0.05), _normal((E, F, H), 3, 0.05)]
    x, lg = _normal((T, H), 4), _normal((T, E), 5, dtype=torch.float32)
    L = MoELayer(*w, T=T, K=K, score=score)
    sizes = [T * K * 4, T * H * 2]
    _late(ballast, lambda s: [L.forward_few(x, lg, stream=s)], sizes)
    n = api.moe_layer_few_tokens_workspace(L.weights, T, K).numel()
    _late(ballast, lambda s: [api.moe_layer_few_tokens(x, lg, L.weights, K, stream=s)[0]], sizes + [n])
    L = MoELayer(*w, T=T, K=K, score=score)
    _late(ballast, lambda s: [L.forward_few(x, lg, stream=s)], sizes + [n])


def test_layer_norm(ballast):
    T, H = 600, 1024
    x, dy = _normal((T, H), 1), _normal((T, H), 2)
    w = _normal((H,), 3)
    _late(ballast, lambda s: [api.moe_layer_norm(x, w, stream=s).y], [T * 4, T * H * 2])
    o = api.moe_layer_norm(x, w)
    n = api.moe_layer_norm_backward_workspace_size(T, H)
    _late(ballast, lambda s: api.moe_layer_norm_backward(dy, x, w, o.mean, o.rstd, stream=s), [n, T * H * 2, H * 2])


def test_gradient_clipping(ballast):
    g = [_normal((300_001,), 1), _normal((77_000,), 2, dtype=torch.float32)]
    outs = [torch.empty_like(t) for t in g]
    n = int(api._lib.load().moe_grad_norm_workspace_size(2))

    def clip(s):
        norm = api.moe_grad_clip(g, 1.0, out=outs, stream=s)
        if s is not None:
            return [norm] + outs
        return [norm] + [t.clone() for t in outs]
    _late(ballast, clip, [n, 4])
    _late(ballast, lambda s: [api.moe_grad_norm(g, stream=s)], [n, 4])


def test_permute(ballast):
    x = _normal((900, 256), 1)
    ids = torch.randint(0, 64, (900, 4), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    n = api.moe_permute_workspace_size(900, 4, 64)
    _late(ballast, lambda s: list(api.moe_permute(x, ids, 64, stream=s)[2:5]), [n])
