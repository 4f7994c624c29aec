"""Performance cases of the operators around the dropless MoE layer.

Four operators: the whole layer for a few tokens, the layer norm and its backward pass, and the
global gradient norm with clipping. ``run`` computes one pass: with ``own`` false in plain 32-bit
torch operations, with ``own`` true through the package's entry points. ``exact`` is the
definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "fp32": F32}
SIZES = {"bf16": 2, "fp32": 4}
LN_EPS = 1e-5
CLIP_EPS = 1e-6


# --------------------------------------------------------------------------- cases
def _few(name, T, H, E, K, F, precision="bf16", renorm=False, id_bits=32):
    return dict(name=name, op="few", T=T, H=H, E=E, K=K, F=F, precision=precision, renorm=renorm, id_bits=id_bits)


def _ln(name, op, T, H, dtype, wdtype, residual):
    return dict(name=name, op=op, T=T, H=H, dtype=dtype, wdtype=wdtype, residual=residual)


def listed():
    return [
        # serving one token of the smallest workload's layer: nothing but latency
        _few("few tiny, 1 token", 1, 256, 8, 2, 512),
        # a decode step of one sequence: the Mixtral-like layer, two experts of eight
        _few("few Mixtral-like, 1 token", 1, 4096, 8, 2, 14336, renorm=True),
        # a decode step of a small batch: every expert of the Mixtral-like layer is read
        _few("few Mixtral-like, 32 tokens", 32, 4096, 8, 2, 14336, renorm=True),
        # a decode step of the DeepSeek-V3-like MXFP8 slice
        _few("few DeepSeek-V3-like mxfp8, 8 tokens", 8, 7168, 32, 4, 2048, precision="mxfp8"),
        # an odd batch of the 2,304-expert layer: 36 small experts a token
        _few("few 2,304 experts, 5 tokens", 5, 512, 2304, 36, 512, id_bits=16),
        # the pre-norm of one decoded token, the residual added on the way
        _ln("norm 1 x 4096", "ln", 1, 4096, "bf16", "bf16", True),
        # the pre-norm of a training batch of the Mixtral-like layer
        _ln("norm 8192 x 4096", "ln", 8192, 4096, "bf16", "bf16", True),
        # its backward pass at the DeepSeek-V3-like width, the residual path's gradient added
        _ln("norm backward 8192 x 7168", "ln_bwd", 8192, 7168, "bf16", "fp32", True),
        # an odd width and row count in fp32: no alignment to rely on
        _ln("norm backward 777 x 1021 fp32", "ln_bwd", 777, 1021, "fp32", "fp32", False),
        # clipping after a step of the smallest workload: a few small tensors
        dict(name="clip tiny layer", op="clip", kind="layer", E=8, H=256, F=512, max_norm=1.0),
        # clipping after a step of the Mixtral-like layer: 2.8 GB of gradients
        dict(name="clip Mixtral-like layer", op="clip", kind="layer", E=8, H=4096, F=14336, max_norm=1.0),
        # many tensors of ragged sizes and both types, as a whole model's list has them
        dict(name="clip 40 ragged tensors", op="clip", kind="ragged", n=40, total=24_000_000, max_norm=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "ln", "ln_bwd", "clip"])
    if op == "few":
        precision = rng.choice(["bf16", "bf16", "mxfp8"])
        step_h, step_f = (512, 512) if precision == "mxfp8" else (256, 128)
        E = _log(rng, 1, 2304)
        K = min(E, _log(rng, 1, 36))
        # the experts' weights hold at most half of the largest listed case's values
        budget = 3 * 4096 * 14336 * 4 // E
        H = step_h * max(1, min(7168 // step_h, _log(rng, 1, 7168 // step_h)))
        H = min(H, max(step_h, budget // (3 * step_f) // step_h * step_h))
        F = step_f * max(1, min(14336 // step_f, budget // (3 * H * step_f), _log(rng, 1, 14336 // step_f)))
        T = min(_log(rng, 1, 64), max(1, 2304 // K))
        return dict(op="few", T=T, H=H, E=E, K=K, F=F, precision=precision, renorm=rng.random() < 0.5,
                    id_bits=rng.choice([16, 32]))
    if op in ("ln", "ln_bwd"):
        T, H = _log(rng, 1, 16384), _log(rng, 8, 8192)
        if rng.random() < 0.5:
            H = (H + 7) // 8 * 8
        T = min(T, max(1, 8192 * 4096 // H))
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, T=T, H=H, dtype=dtype, wdtype=rng.choice([dtype, "fp32"]), residual=rng.random() < 0.5)
    if rng.random() < 0.5:
        return dict(op="clip", kind="layer", E=_log(rng, 1, 32), H=256 * _log(rng, 1, 8), F=128 * _log(rng, 1, 32),
                    max_norm=rng.choice([0.1, 1.0, 1e6]))
    return dict(op="clip", kind="ragged", n=rng.randint(1, 60), total=_log(rng, 1000, 100_000_000),
                max_norm=rng.choice([0.1, 1.0, 1e6]))


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


def _mxfp8_weights(shape, std, g):
    codes = torch.empty(shape, dtype=torch.uint8, device=DEV)
    byte = torch.empty(shape[:-1] + (shape[-1] // 32,), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (shape[1] * shape[2]))
    for i in range(0, shape[0], step):
        c, b = _mxfp8(torch.randn((min(step, shape[0] - i),) + tuple(shape[1:]), generator=g, device=DEV) * std)
        codes[i:i + step], byte[i:i + step] = c, b
    return codes, byte


def _clip_shapes(c):
    """[(elements, dtype)] of the gradient list."""
    if c["kind"] == "layer":
        E, H, F = c["E"], c["H"], c["F"]
        # expert weights, the router's projection, and the norm's weight and bias
        return [(E * H * F, BF16)] * 3 + [(E * H, F32), (H, F32), (H, F32)]
    r = random.Random(c["n"] * 7919 + c["total"])
    cuts = [math.exp(r.uniform(0.0, 6.0)) for _ in range(c["n"])]
    return [(max(1, int(c["total"] * q / sum(cuts))), r.choice([BF16, BF16, F32])) for q in cuts]


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "few":
        T, H, E, F = c["T"], c["H"], c["E"], c["F"]
        s = dict(case=c, x=_normal((T, H), 1.0, g, BF16),      # normalised activations
                 logits=torch.randn((T, E), generator=g, device=DEV))
        # W1 and W3 packed per 128 columns of F, W2 transposed: what the layer keeps of its weights
        if c["precision"] == "mxfp8":
            s["w13"], s["w13_scales"] = _mxfp8_weights((E, 2 * F, H), 0.02, g)
            s["w2"], s["w2_scales"] = _mxfp8_weights((E, H, F), 0.02, g)
        else:
            s["w13"], s["w13_scales"] = _normal((E, 2 * F, H), 0.02, g, BF16), None
            s["w2"], s["w2_scales"] = _normal((E, H, F), 0.02, g, BF16), None
        return s
    if c["op"] in ("ln", "ln_bwd"):
        T, H, dt, wdt = c["T"], c["H"], DTYPES[c["dtype"]], DTYPES[c["wdtype"]]
        s = dict(case=c, x=_normal((T, H), 1.5, g, dt), residual=None,
                 weight=(1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(wdt),
                 bias=(0.1 * torch.randn(H, generator=g, device=DEV)).to(wdt))
        if c["residual"]:
            s["residual"] = _normal((T, H), 0.5, g, dt)
        if c["op"] == "ln_bwd":
            s["dy"] = _normal((T, H), 0.02, g, dt)
            x = s["x"].to(F32)
            s["mean"] = x.mean(-1)
            s["rstd"] = (x.var(-1, unbiased=False) + LN_EPS).rsqrt()
        return s
    shapes = _clip_shapes(c)
    grads = [_normal((n,), 0.02, g, dt) for n, dt in shapes]
    return dict(case=c, grads=grads, out=[torch.empty_like(t) for t in grads])


# --------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["op"] == "few":
        return _plain_few(c, state)
    if c["op"] == "ln":
        return _plain_ln(state)
    if c["op"] == "ln_bwd":
        return _plain_ln_bwd(state)
    return _plain_clip(c, state)


def _run_own(c, s):
    from dropless_moe_expert_router_gb300 import api
    if c["op"] == "few":
        if "weights" not in s:                                   # the handle and workspace a server keeps
            s["weights"] = api.PackedWeights(c["precision"], c["E"], c["H"], c["F"], s["w13"], s["w13_scales"], s["w2"],
                                             s["w2_scales"])
            s["workspace"] = api.moe_layer_few_tokens_workspace(s["weights"], c["T"], c["K"])
        y, ids, probs = api.moe_layer_few_tokens(s["x"], s["logits"], s["weights"], c["K"], renorm=c["renorm"],
                                                 id_dtype=torch.int16 if c["id_bits"] == 16 else torch.int32,
                                                 workspace=s["workspace"])
        return dict(y=y, ids=ids, probs=probs)
    if c["op"] == "ln":
        o = api.moe_layer_norm(s["x"], s["weight"], s["bias"], LN_EPS, residual=s["residual"])
        out = dict(y=o.y, mean=o.mean, rstd=o.rstd)
        if c["residual"]:
            out["sum"] = o.sum
        return out
    if c["op"] == "ln_bwd":
        dx, dw, db = api.moe_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], dx_add=s["residual"])
        return dict(dx=dx, dweight=dw, dbias=db)
    norm = api.moe_grad_clip(s["grads"], c["max_norm"], eps=CLIP_EPS, out=s["out"])
    return dict(norm=norm, grads=s["out"])


def _plain_few(c, s):
    T, H, E, K, F = c["T"], c["H"], c["E"], c["K"], c["F"]
    logits = s["logits"]
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :K]      # ties: the lower index
    chosen = torch.gather(logits, 1, ids)
    over = chosen if c["renorm"] else logits
    top = over.amax(1, keepdim=True)
    probs = torch.exp(chosen - top) / torch.exp(over - top).sum(1, keepdim=True)

    def weights(name, which):
        w = s[name][which] if which is not None else s[name]
        if c["precision"] == "mxfp8":
            byte = s[name + "_scales"]
            return _mxfp8_value(w, byte[which] if which is not None else byte, F32)
        return w.to(F32)

    def quantised(v):
        return _mxfp8_value(*_mxfp8(v), F32) if c["precision"] == "mxfp8" else v

    def hidden(ab):                                               # [..., 2F] packed per 128 -> h [..., F]
        a, b = ab.unflatten(-1, (F // 128, 2, 128)).unbind(-2)
        h = (a / (1 + torch.exp(-a)) * b).flatten(-2)
        return quantised(h) if c["precision"] == "mxfp8" else h.to(BF16).to(F32)

    x = quantised(s["x"].to(F32))
    if T * K <= E:
        # each route's own expert
        e = ids.reshape(-1)
        xr = x.unsqueeze(1).expand(T, K, H).reshape(T * K, H, 1)
        h = hidden(torch.bmm(weights("w13", e), xr).squeeze(-1))
        yr = torch.bmm(weights("w2", e), h.unsqueeze(-1)).squeeze(-1).view(T, K, H)
        y = (probs.unsqueeze(-1) * yr).sum(1)
    else:
        # every expert on every token, weighted with zero where it was not chosen
        h = hidden(torch.matmul(x, weights("w13", None).transpose(1, 2)))              # [E, T, F]
        p = torch.zeros((T, E), device=DEV).scatter_(1, ids, probs)
        y = (torch.matmul(h, weights("w2", None).transpose(1, 2)) * p.t().unsqueeze(-1)).sum(0)
    return dict(y=y.to(BF16), ids=ids.to(torch.int16 if c["id_bits"] == 16 else torch.int32), probs=probs)


def _plain_ln(s):
    x = s["x"]
    if s["residual"] is not None:
        x = (x.to(F32) + s["residual"].to(F32)).to(x.dtype)        # the stored stream is what is normalised
    v = x.to(F32)
    mean = v.sum(-1) / v.shape[-1]
    d = v - mean.unsqueeze(-1)
    rstd = 1 / torch.sqrt((d * d).sum(-1) / v.shape[-1] + LN_EPS)
    y = (d * rstd.unsqueeze(-1) * s["weight"].to(F32) + s["bias"].to(F32)).to(x.dtype)
    out = dict(y=y, mean=mean, rstd=rstd)
    if s["residual"] is not None:
        out["sum"] = x
    return out


def _plain_ln_bwd(s):
    dy, x, w = s["dy"].to(F32), s["x"].to(F32), s["weight"].to(F32)
    rstd = s["rstd"].unsqueeze(-1)
    xh = (x - s["mean"].unsqueeze(-1)) * rstd
    g = dy * w
    H = x.shape[-1]
    dx = rstd * (g - g.sum(-1, keepdim=True) / H - xh * ((g * xh).sum(-1, keepdim=True) / H))
    if s["residual"] is not None:
        dx = dx + s["residual"].to(F32)
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * xh).sum(0).to(s["weight"].dtype),
                dbias=dy.sum(0).to(s["weight"].dtype))


def _plain_clip(c, s):
    norm = torch.sqrt(sum(t.to(F32).square().sum() for t in s["grads"]))
    scale = torch.clamp(c["max_norm"] / (norm + CLIP_EPS), max=1.0)
    return dict(norm=norm.reshape(1), grads=[(t.to(F32) * scale).to(t.dtype) for t in s["grads"]])


# --------------------------------------------------------------------------- floors
def work(case):
    c = case
    if c["op"] == "few":
        T, H, E, K, F = c["T"], c["H"], c["E"], c["K"], c["F"]
        distinct = E * (1 - (1 - K / E) ** T)                      # experts chosen at least once
        per = 3 * H * F * (1 + 1 / 32 if c["precision"] == "mxfp8" else 2)
        small = T * H * 4 + T * E * 4 + T * K * (4 + c["id_bits"] // 8)
        return {"bytes": distinct * per + small, "flops": 6 * T * K * H * F}
    if c["op"] in ("ln", "ln_bwd"):
        n, size, H = c["T"] * c["H"], SIZES[c["dtype"]], c["H"]
        stats = 8 * c["T"]
        if c["op"] == "ln":
            return {"bytes": n * size * (4 if c["residual"] else 2) + stats + 2 * H * SIZES[c["wdtype"]], "flops": 8 * n}
        return {"bytes": n * size * (4 if c["residual"] else 3) + stats + 3 * H * SIZES[c["wdtype"]], "flops": 14 * n}
    shapes = _clip_shapes(c)
    return {"bytes": sum(2 * n * (2 if dt == BF16 else 4) for n, dt in shapes) + 4, "flops": sum(3 * n for n, _ in shapes)}


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    D = torch.float64
    if c["op"] == "few":
        T, H, E, K, F = c["T"], c["H"], c["E"], c["K"], c["F"]
        if T * K * H * F > 3e10:
            return None
        fp8 = c["precision"] == "mxfp8"
        lg = s["logits"].to(D).cpu()
        order = torch.arange(E)
        rows = [sorted(order.tolist(), key=lambda e: (-lg[t, e].item(), e))[:K] for t in range(T)]
        x = s["x"].to(D)
        if fp8:
            x = _mxfp8_value(*_mxfp8(x), D)
        y = torch.zeros((T, H), dtype=D, device=DEV)
        probs = torch.zeros((T, K), dtype=D)
        for t in range(T):
            over = lg[t, rows[t]] if c["renorm"] else lg[t]
            probs[t] = torch.exp(lg[t, rows[t]] - torch.logsumexp(over, 0))
        for e in sorted({e for r in rows for e in r}):
            at = [(t, r.index(e)) for t, r in enumerate(rows) if e in r]
            t_of = torch.tensor([t for t, _ in at], device=DEV)
            w13, w2 = s["w13"][e], s["w2"][e]
            w13 = _mxfp8_value(w13, s["w13_scales"][e], D) if fp8 else w13.to(D)
            w2 = _mxfp8_value(w2, s["w2_scales"][e], D) if fp8 else w2.to(D)
            first = torch.arange(F, device=DEV)
            first = first // 128 * 256 + first % 128                # rows of W1; W3's come 128 later
            a, b = x[t_of] @ w13[first].t(), x[t_of] @ w13[first + 128].t()
            h = a * torch.sigmoid(a) * b
            h = _mxfp8_value(*_mxfp8(h), D) if fp8 else h.to(BF16).to(D)
            p = torch.stack([probs[t, k] for t, k in at]).to(DEV)
            y.index_add_(0, t_of, p.unsqueeze(1) * (h @ w2.t()))
        return dict(y=y, ids=None, probs=probs)
    if c["op"] == "ln":
        x = s["x"].to(D)
        if c["residual"]:
            x = (x + s["residual"].to(D)).to(s["x"].dtype).to(D)
        var, mean = torch.var_mean(x, -1, unbiased=False)
        rstd = (var + LN_EPS).rsqrt()
        y = (x - mean[:, None]) * rstd[:, None] * s["weight"].to(D) + s["bias"].to(D)
        out = dict(y=y, mean=mean, rstd=rstd)
        if c["residual"]:
            out["sum"] = x
        return out
    if c["op"] == "ln_bwd":
        x, dy = s["x"].to(D), s["dy"].to(D)
        # from the statistics that the call is given
        xh = x.sub_(s["mean"].to(D)[:, None]).mul_(s["rstd"].to(D)[:, None])
        dw, db = torch.einsum("th,th->h", dy, xh), dy.sum(0)
        g = dy.mul_(s["weight"].to(D))
        m1, m2 = g.mean(-1, keepdim=True), torch.einsum("th,th->t", g, xh)[:, None] / c["H"]
        dx = (g - m1 - xh * m2) * s["rstd"].to(D)[:, None]
        if c["residual"]:
            dx += s["residual"].to(D)
        return dict(dx=dx, dweight=dw, dbias=db)
    total = torch.zeros((), dtype=D, device=DEV)
    for t in s["grads"]:
        for part in t.split(1 << 27):
            total += torch.linalg.vector_norm(part.to(D)) ** 2
    norm = total.sqrt()
    scale = min(1.0, c["max_norm"] / (norm.item() + CLIP_EPS))
    big = sum(t.numel() for t in s["grads"]) > 4e8
    return dict(norm=norm.reshape(1), grads=[None if big else t.to(D) * scale for t in s["grads"]])
