"""The pre-norm MoE block (norm, layer, few-token step, backward, clipping) against a plain
64-bit implementation with torch's own differentiation.

Bars, as the largest error over the largest value: 1e-2 for what passes one or two bf16 roundings
of 2^-8 (s, hn, delta'), 3e-2 for gradients, which pass four (dy_perm, dab, dx, dhn), each of them
a sum of many terms whose roundings are independent; 1e-3 for the norm of all of them."""
import pytest
import torch

from dropless_moe_expert_router_gb300 import api
from dropless_moe_expert_router_gb300.block import MoEBlock
from dropless_moe_expert_router_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dropless_moe_expert_router_gb300 import build
    build.build()


def _rel(a, b):
    return ((a.double().cpu() - b).abs().max() / b.abs().max()).item()


def _params(E, H, F, seed):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, std):
        return torch.randn(shape, generator=g) * std
    bf = torch.bfloat16
    return dict(w1=n(E, H, F, std=0.06).to(bf), w3=n(E, H, F, std=0.06).to(bf), w2=n(E, F, H, std=0.06).to(bf),
                router=n(E, H, std=0.1), norm_weight=1 + n(H, std=0.1), norm_bias=n(H, std=0.1))


def _block(p, T, K, **kw):
    c = {k: v.cuda() for k, v in p.items()}
    return MoEBlock(c["w1"], c["w3"], c["w2"], c["router"], c["norm_weight"], c["norm_bias"], T=T, K=K, **kw)


def _plain(q, x, delta, ids, K):
    """The block in 64 bits with the routes given -> (s, delta')."""
    s = x + delta
    var, mean = torch.var_mean(s, 1, unbiased=False)
    hn = (s - mean[:, None]) * (var[:, None] + 1e-5).rsqrt() * q["norm_weight"] + q["norm_bias"]
    p = torch.softmax(torch.gather(hn @ q["router"].t(), 1, ids), 1)
    out = torch.zeros_like(s)
    for e in range(q["w1"].shape[0]):
        w = (p * (ids == e)).sum(1, keepdim=True)
        a, b = hn @ q["w1"][e], hn @ q["w3"][e]
        out = out + w * ((a * torch.sigmoid(a) * b) @ q["w2"][e])
    return s, out


def test_training_step():
    T, H, E, K, F = 192, 256, 8, 2, 256
    p = _params(E, H, F, seed=1)
    blk = _block(p, T, K, renorm=True, training=True)
    g = torch.Generator().manual_seed(2)
    x, delta, ds, dd = ((torch.randn((T, H), generator=g) * k).to(torch.bfloat16) for k in (1.0, 0.5, 0.1, 0.1))
    s, out = blk.forward(x.cuda(), delta.cuda())
    ids = blk.layer.ids.cpu().long()
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    xs = x.double().requires_grad_()
    rs, ro = _plain(q, xs, delta.double(), ids, K)
    assert _rel(s, rs.detach()) <= 1e-2 and _rel(out, ro.detach()) <= 1e-2
    dx = blk.backward(ds.cuda(), dd.cuda())
    torch.autograd.backward([rs, ro], [ds.double(), dd.double()])
    assert _rel(dx, xs.grad) <= 3e-2
    for k, v in blk.gradients.items():
        assert v.dtype == p[k].dtype and v.shape == p[k].shape
        assert _rel(v, q[k].grad) <= 3e-2, k
    before = {k: v.clone() for k, v in blk.gradients.items()}
    ref = sum(v.double().square().sum() for v in before.values()).sqrt().item()
    norm = blk.clip_gradients(0.5 * ref).item()
    assert abs(norm - ref) <= 1e-3 * ref
    for k, v in blk.gradients.items():
        assert _rel(v, 0.5 * before[k].double().cpu()) <= 1e-2
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("kw", [dict(renorm=True), dict(precision="mxfp8"), dict(score="sigmoid", renorm=True)])
def test_step_agrees_with_forward(kw):
    """The few-token step against the batched forward on the same tokens, with and without an update
    to add; tokens one at a time give what they give together."""
    T, H, E, K, F = 24, 512, 16, 4, 512
    p = _params(E, H, F, seed=3)
    blk = _block(p, T, K, **kw)
    g = torch.Generator().manual_seed(4)
    x, delta = (torch.randn((T, H), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    for d in (None, delta):
        s, out = blk.forward(x, d)
        s2, out2 = blk.step(x, d)
        assert torch.equal(s, s2)
        assert _rel(out2, out.double().cpu()) <= 1e-2
        one = torch.cat([blk.step(x[i:i + 1], None if d is None else d[i:i + 1])[1] for i in range(T)])
        assert _rel(one, out2.double().cpu()) <= 1e-2
    assert api.moe_get_device_errors() == 0


def test_block_refusals():
    p = _params(4, 256, 128, seed=5)
    blk = _block(p, 8, 2)
    x = torch.zeros((8, 256), dtype=torch.bfloat16, device="cuda")
    blk.forward(x)
    with pytest.raises(ValueError):
        blk.backward(x, x)                                       # not a training layer
    with pytest.raises(ValueError):
        _block(dict(p, router=p["router"][:2]), 8, 2)
    with pytest.raises(api.MoeError):
        blk.step(torch.zeros((65, 256), dtype=torch.bfloat16, device="cuda"))


def test_workspaces_of_another_kind_are_refused():
    """A workspace on the host, of another type, or with gaps never reaches a kernel."""
    p = _params(4, 256, 128, seed=5)
    blk = _block(p, 8, 2)
    x = torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda")
    lg = torch.zeros((2, 4), device="cuda")
    w = torch.ones(256, device="cuda")
    o = api.moe_layer_norm(x, w)
    n = 1 << 22
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(n, device="cuda"),
               torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            api.moe_layer_few_tokens(x, lg, blk.layer.weights, 2, workspace=ws)
        with pytest.raises(ValueError):
            api.moe_layer_norm_backward(x, x, w, o.mean, o.rstd, workspace=ws)
        with pytest.raises(ValueError):
            api.moe_grad_norm([x], workspace=ws)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_two_training_steps(precision):
    """Forward, backward, an update of every parameter in place, and again: the second step and the
    few-token step compute with the updated weights. MXFP8 rounds each operand by up to 2^-4, and with it
    every product of the forward by that much of one of many independent terms: its bar is 8e-2."""
    T, H, E, K, F = 128, 512, 8, 2, 512
    p = _params(E, H, F, seed=21)
    blk = _block(p, T, K, renorm=True, training=True, precision=precision)
    mine = dict(w1=blk.layer._w[0], w3=blk.layer._w[1], w2=blk.layer._w[2], router=blk.router,
                norm_weight=blk.norm_weight, norm_bias=blk.norm_bias)
    g = torch.Generator().manual_seed(22)
    x, ds, dd = ((torch.randn((T, H), generator=g) * k).to(torch.bfloat16) for k in (1.0, 0.1, 0.1))
    bar, gbar = (1e-2, 3e-2) if precision == "bf16" else (8e-2, 2e-1)
    for step in range(2):
        _, out = blk.forward(x.cuda())
        ids = blk.layer.ids.cpu().long()
        q = {k: v.detach().cpu().double().requires_grad_() for k, v in mine.items()}
        xs = x.double().requires_grad_()
        rs, ro = _plain(q, xs, torch.zeros_like(xs), ids, K)
        assert _rel(out, ro.detach()) <= bar
        assert _rel(blk.step(x[:24].cuda())[1], ro.detach()[:24]) <= bar
        dx = blk.backward(ds.cuda(), dd.cuda())
        torch.autograd.backward([rs, ro], [ds.double(), dd.double()])
        assert _rel(dx, xs.grad) <= gbar
        for k, v in blk.gradients.items():
            assert _rel(v, q[k].grad) <= gbar, k
        before = {k: v.clone() for k, v in mine.items()}
        for k, v in blk.gradients.items():                       # a step that changes every weight by about itself
            scale = mine[k].float().abs().mean() / v.float().abs().mean().clamp_min(1e-30)
            mine[k].copy_((mine[k].float() - scale * v.float()).to(v.dtype))
        assert all(not torch.equal(before[k], v) for k, v in mine.items())
        blk.repack()
    assert api.moe_get_device_errors() == 0


@pytest.mark.parametrize("precision", ["bf16", "mxfp8", "nvfp4"])
def test_repack_gives_what_a_new_layer_gives(precision):
    """In the buffers that were there: a captured graph and layers that share them see the new weights."""
    p = _params(4, 512, 512, seed=31)
    w = [p[k].cuda() for k in ("w1", "w3", "w2")]
    L = MoELayer(*w, T=40, K=2, precision=precision)
    shared = MoELayer(*w, T=40, K=2, precision=precision, packed_weights=L.weights)
    g = torch.Generator().manual_seed(32)
    x, lg = torch.randn((40, 512), generator=g).to(torch.bfloat16).cuda(), torch.randn((40, 4), generator=g).cuda()
    L.forward(x, lg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward(x, lg)
    at = [t.data_ptr() for t in L.weights if torch.is_tensor(t)]
    for t, seed in zip(w, (33, 34, 35)):
        t.copy_((torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)) * 0.06).to(torch.bfloat16))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    L.repack(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    new = MoELayer(*w, T=40, K=2, precision=precision)
    for a, b in zip(L.weights, new.weights):
        assert torch.equal(a, b) if torch.is_tensor(a) else a == b
    assert at == [t.data_ptr() for t in L.weights if torch.is_tensor(t)]
    want = new.forward(x, lg).clone()
    graph.replay()
    assert torch.equal(L.y, want) and torch.equal(shared.forward(x, lg), want)


def test_repack_into_other_weights_is_refused():
    p = _params(4, 512, 512, seed=41)
    w = [p[k].cuda() for k in ("w1", "w3", "w2")]
    packed, bwd = api.moe_prepare_weights(*w), api.moe_prepare_weights_bwd(*w)
    small = [t[:2].contiguous() for t in w]
    for bad in (lambda: api.moe_prepare_weights(*w, "mxfp8", out=packed), lambda: api.moe_prepare_weights(*small, out=packed),
                lambda: api.moe_prepare_weights(*w, out=bwd), lambda: api.moe_prepare_weights_bwd(*w, out=packed),
                lambda: api.moe_prepare_weights_bwd(*small, out=bwd), lambda: api.moe_prepare_weights_nvfp4(*w, out=packed),
                lambda: api.moe_prepare_weights(*w, out=packed._replace(w2=packed.w2[:, :, 8:])),
                lambda: api.moe_prepare_weights(*w, out=packed._replace(w13=packed.w13.cpu())),
                lambda: api.moe_prepare_weights(*w, out=packed._replace(w13=None))):
        with pytest.raises(ValueError):
            bad()


def test_clip_before_backward_is_refused():
    p = _params(4, 256, 128, seed=5)
    blk = _block(p, 8, 2, training=True)
    with pytest.raises(ValueError):
        blk.clip_gradients(1.0)
    blk.forward(torch.zeros((8, 256), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        blk.clip_gradients(1.0)
