"""Layer norm forward and backward against a plain 64-bit implementation, through the C ABI.

Bars, with u = 2^-24 and G = (H / 32 + 64) u, the worst relative error of an fp32 sum of H terms
that 32 threads or more share: every statistic errs by G of the mean magnitude it is summed from,
every output by the statistics' error carried through its formula, 16 u of the largest term, and
(bf16) half a unit of the last of its 8 significant bits, 2^-8 of itself.
"""
import pytest
import torch

from dropless_moe_expert_router_gb300 import api
from dropless_moe_expert_router_gb300.api import MoeError

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dropless_moe_expert_router_gb300 import build
    build.build()


def _half(dt):
    return 2.0 ** -8 if dt == BF else U


def _inputs(T, H, dt, wdt, seed, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, H), generator=g) * 1.5 + mean).to(dt).cuda()
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(wdt).cuda()
    b = (0.2 * torch.randn(H, generator=g)).to(wdt).cuda()
    r = torch.randn((T, H), generator=g).to(dt).cuda()
    dy = torch.randn((T, H), generator=g).to(dt).cuda()
    return x, w, b, r, dy


def _within(got, ref, bar):
    d = (got.double() - ref).abs()
    assert bool((d <= bar).all()), float((d / bar.clamp_min(1e-300)).max())


def _forward_check(o, s, w, b, eps):
    S, H = s.double(), s.shape[1]
    G = (H / 32 + 64) * U
    mean = S.mean(1)
    var = (S - mean[:, None]).square().mean(1)
    rstd = (var + eps).rsqrt()
    mag = S.abs().mean(1)
    e_mean = G * mag + 1e-30
    _within(o.mean, mean, e_mean)
    # d(rstd)/rstd = d(var + eps) / (2 (var + eps)); (s - mean) errs by u |s| and the mean's error
    e_rstd = rstd * (0.5 * (G * var + e_mean ** 2 + 4 * U * S.abs().amax(1) * var.sqrt()) * rstd ** 2 + 8 * U)
    _within(o.rstd, rstd, e_rstd)
    W, B = w.double(), torch.zeros(H, device=s.device).double() if b is None else b.double()
    y = (S - mean[:, None]) * rstd[:, None] * W + B
    e = ((e_mean + 4 * U * S.abs().amax(1)) * rstd)[:, None] * W.abs() + ((y - B).abs() * (e_rstd / rstd)[:, None]) \
        + 16 * U * (y.abs() + B.abs())
    _within(o.y, y, e + _half(o.y.dtype) * y.abs() * 1.01 + 1e-38)


SHAPES = [(1, 1), (1, 8), (3, 7), (2, 33), (5, 1021), (1, 4096), (130, 256), (33, 4096), (9, 7168), (4, 8192),
          (3, 8200), (2, 16384), (2, 65536), (1000, 129), (2, 20001)]


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H, dt, wdt):
    x, w, b, r, _ = _inputs(T, H, dt, wdt, seed=T + H)
    eps = 1e-5
    o = api.moe_layer_norm(x, w, b, eps)
    assert o.sum is x
    _forward_check(o, x, w, b, eps)
    o = api.moe_layer_norm(x, w, None, eps, residual=r)
    s = (x.float() + r.float()).to(dt)
    assert torch.equal(o.sum, s)
    _forward_check(o, s, w, None, eps)


def _backward_reference(dy, s, w, mean, rstd, add):
    DY, S, W = dy.double(), s.double(), w.double()
    R = rstd.double()[:, None]
    xh = (S - mean.double()[:, None]) * R
    g = DY * W
    a, c = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = R * (g - a - xh * c)
    if add is not None:
        dx = dx + add.double()
    return dx, (DY * xh).sum(0), DY.sum(0), xh, g


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("T,H", SHAPES + [(2500, 64), (1700, 1000)])
def test_backward(T, H, dt, wdt):
    x, w, b, r, dy = _inputs(T, H, dt, wdt, seed=3 * T + H)
    o = api.moe_layer_norm(x, w, b)
    G, GT = (H / 32 + 64) * U, (T + 64) * U
    for add in (None, r):
        dx, dw, db = api.moe_layer_norm_backward(dy, x, w, o.mean, o.rstd, dx_add=add)
        rx, rw, rb, xh, g = _backward_reference(dy, x, w, o.mean, o.rstd, add)
        R = o.rstd.double()[:, None]
        exh = 4 * U * (x.double().abs() + o.mean.double().abs()[:, None]) * R
        sums = G * (g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) \
            + xh.abs() * (g.abs() * exh).mean(1, keepdim=True)
        terms = g.abs() + g.mean(1, keepdim=True).abs() + (xh.abs() + exh) * (g * xh).mean(1, keepdim=True).abs()
        e = R * (sums + 16 * U * terms + exh * (g * xh).mean(1, keepdim=True).abs())
        if add is not None:
            e = e + 2 * U * (add.double().abs() + rx.abs())
        _within(dx, rx, e + 1.01 * _half(dt) * rx.abs() + 1e-38)
        D = dy.double().abs()
        _within(dw, rw, GT * (D * xh.abs()).sum(0) + (D * exh).sum(0) + 1.01 * _half(wdt) * rw.abs() + 1e-38)
        _within(db, rb, GT * D.sum(0) + 1.01 * _half(wdt) * rb.abs() + 1e-38)


def test_backward_against_differences():
    """<dx, v>, <dw, v>, <db, v> against central differences of L = sum(dy y), y of the fp32 kernel.
    Step 2^-6 along unit-variance v: truncation 2^-12 / 6 of third derivatives of order 1 per value;
    rounding 16 u sum|dy y| / 2^-6; both well under 2^-9 of the sum of |terms|."""
    T, H = 6, 96
    x, w, b, _, dy = _inputs(T, H, F32, F32, seed=1)
    g = torch.Generator().manual_seed(2)
    o = api.moe_layer_norm(x, w, b)
    dx, dw, db = api.moe_layer_norm_backward(dy, x, w, o.mean, o.rstd)
    h = 2.0 ** -6

    def loss(x_, w_, b_):
        return (api.moe_layer_norm(x_, w_, b_).y.double() * dy.double()).sum().item()

    for d, at in ((dx, 0), (dw, 1), (db, 2)):
        v = torch.randn(d.shape, generator=g).cuda()
        up, down = [x, w, b], [x, w, b]
        up[at], down[at] = up[at] + h * v, down[at] - h * v
        diff = (loss(*up) - loss(*down)) / (2 * h)
        dot = (d.double() * v.double()).sum().item()
        assert abs(diff - dot) <= 2.0 ** -9 * (d.double().abs() * v.double().abs()).sum().item()


@pytest.mark.parametrize("dt", [BF, F32])
def test_in_place(dt):
    x, w, b, r, dy = _inputs(40, 520, dt, F32, seed=9)
    want = api.moe_layer_norm(x, w, b, residual=r)
    x2, r2 = x.clone(), r.clone()
    got = api.moe_layer_norm(x2, w, b, residual=r2, sum=r2, y=x2)
    assert torch.equal(got.y, want.y) and torch.equal(r2, want.sum) and got.y is x2
    x3 = x.clone()
    assert torch.equal(api.moe_layer_norm(x3, w, b, y=x3).y, api.moe_layer_norm(x, w, b).y)
    ref = api.moe_layer_norm_backward(dy, want.sum, w, want.mean, want.rstd, dx_add=r)
    for alias in ("dy", "add"):
        d2, a2 = dy.clone(), r.clone()
        got = api.moe_layer_norm_backward(d2, want.sum, w, want.mean, want.rstd, dx_add=a2, dx=d2 if alias == "dy" else a2)
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("off", [1, 3, 4])
def test_unaligned_bases(dt, off):
    """Contiguous tensors that start off a 16-byte boundary, at a width that is a multiple of 8."""
    T, H = 37, 512
    x, w, b, r, dy = _inputs(T, H, dt, dt, seed=off)

    def moved(t):
        buf = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
        v = buf[off:].view(t.shape)
        v.copy_(t)
        return v
    o = api.moe_layer_norm(moved(x), moved(w), moved(b), residual=moved(r), y=moved(x), sum=moved(x))
    s = (x.float() + r.float()).to(dt)
    assert torch.equal(o.sum, s)
    _forward_check(o, s, w, b, 1e-5)
    ref = api.moe_layer_norm_backward(dy, s, w, o.mean, o.rstd, dx_add=r)
    got = api.moe_layer_norm_backward(moved(dy), moved(s), moved(w), o.mean, o.rstd, dx_add=moved(r), dx=moved(x),
                                      dweight=moved(w), dbias=moved(b))
    rx, rw, rb, _, _ = _backward_reference(dy, s, w, o.mean, o.rstd, r)
    for a, c, e in zip(got, ref, (rx, rw, rb)):
        bar = (2 * _half(dt) + 1e-5) * e.abs() + 1e-4
        _within(a, e, bar)
        _within(c, e, bar)


def test_degenerate_rows_stay_apart():
    """Constant rows (variance 0), a NaN row and an infinite one beside ordinary rows."""
    x, w, b, _, dy = _inputs(8, 640, F32, F32, seed=4)
    clean = api.moe_layer_norm(x, w, b)
    x2 = x.clone()
    x2[1] = 3.0
    x2[2] = 0.0
    x2[4, 5] = float("nan")
    x2[6, 639] = float("inf")
    o = api.moe_layer_norm(x2, w, b)
    rows = [0, 3, 5, 7]
    assert torch.equal(o.y[rows], clean.y[rows]) and torch.equal(o.rstd[rows], clean.rstd[rows])
    for t, v in ((1, 3.0), (2, 0.0)):
        assert abs(o.mean[t].item() - v) <= 1e-6 and abs(o.rstd[t].item() - 1e-5 ** -0.5) <= 1e-2
        assert (o.y[t] - b).abs().max().item() <= 1e-3
    assert torch.isnan(o.y[4]).all() and torch.isnan(o.y[6]).any()
    dx, _, _ = api.moe_layer_norm_backward(dy, x2, w, o.mean, o.rstd)
    ref, _, _ = api.moe_layer_norm_backward(dy, x, w, clean.mean, clean.rstd)
    assert torch.equal(dx[rows], ref[rows])


def test_repeats_bit_for_bit_on_any_workspace_and_stream():
    x, w, b, r, dy = _inputs(3000, 1000, BF, F32, seed=6)
    o = api.moe_layer_norm(x, w, b)
    ref = api.moe_layer_norm_backward(dy, x, w, o.mean, o.rstd)
    ws = torch.empty(api.moe_layer_norm_backward_workspace_size(3000, 1000), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    for fill in (0, 255):
        ws.fill_(fill)
        s.wait_stream(torch.cuda.current_stream())
        got = api.moe_layer_norm_backward(dy, x, w, o.mean, o.rstd, workspace=ws, stream=s)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, ref))
    y, sm = torch.empty_like(x), torch.empty_like(x)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    mean, rstd = torch.empty(3000, device="cuda"), torch.empty(3000, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_layer_norm(x, w, b, residual=r, y=y, sum=sm, mean=mean, rstd=rstd)
        api.moe_layer_norm_backward(dy, sm, w, mean, rstd, dx=dx, dweight=dw, dbias=db, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    o = api.moe_layer_norm(x, w, b, residual=r)
    assert torch.equal(y, o.y)
    assert all(torch.equal(p, q) for p, q in
               zip((dx, dw, db), api.moe_layer_norm_backward(dy, o.sum, w, o.mean, o.rstd)))


def test_no_rows_and_refusals():
    x, w, b, r, dy = _inputs(4, 64, BF, F32, seed=1)
    z = torch.empty((0, 64), dtype=BF, device="cuda")
    o = api.moe_layer_norm(z, w, b, residual=z)
    assert o.y.shape == (0, 64)
    dx, dw, db = api.moe_layer_norm_backward(z, z, w, o.mean, o.rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    with pytest.raises(ValueError):
        api.moe_layer_norm(x.half(), w, b)
    with pytest.raises(ValueError):
        api.moe_layer_norm(x, w[:32].contiguous(), b)
    with pytest.raises(ValueError):
        api.moe_layer_norm(x, w, b.to(BF))
    with pytest.raises(ValueError):
        api.moe_layer_norm(x.t(), w, b)
    with pytest.raises(ValueError):
        api.moe_layer_norm(x, w, b, residual=r.float())
    with pytest.raises(MoeError):
        api.moe_layer_norm(x, w, b, eps=-1.0)
    with pytest.raises(MoeError):
        api.moe_layer_norm(torch.zeros((1, 65537), device="cuda"), torch.zeros(65537, device="cuda"))
    o = api.moe_layer_norm(x, w, b)
    with pytest.raises(ValueError):
        api.moe_layer_norm_backward(dy[:3].contiguous(), x, w, o.mean, o.rstd)
    with pytest.raises(ValueError):
        api.moe_layer_norm_backward(dy, x, w, o.mean[:2], o.rstd)
    with pytest.raises(MoeError):
        api.moe_layer_norm_backward(dy, x, w, o.mean, o.rstd, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))


def _backward_check(got, dy, s, w, mean, rstd, add):
    T, H = s.shape
    G, GT = (H / 32 + 64) * U, (T + 64) * U
    dx, dw, db = got
    rx, rw, rb, xh, g = _backward_reference(dy, s, w, mean, rstd, add)
    R = rstd.double()[:, None]
    exh = 4 * U * (s.double().abs() + mean.double().abs()[:, None]) * R
    sums = G * (g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) \
        + xh.abs() * (g.abs() * exh).mean(1, keepdim=True)
    terms = g.abs() + g.mean(1, keepdim=True).abs() + (xh.abs() + exh) * (g * xh).mean(1, keepdim=True).abs()
    e = R * (sums + 16 * U * terms + exh * (g * xh).mean(1, keepdim=True).abs())
    if add is not None:
        e = e + 2 * U * (add.double().abs() + rx.abs())
    _within(dx, rx, e + 1.01 * _half(s.dtype) * rx.abs() + 1e-38)
    D = dy.double().abs()
    _within(dw, rw, GT * (D * xh.abs()).sum(0) + (D * exh).sum(0) + 1.01 * _half(w.dtype) * rw.abs() + 1e-38)
    _within(db, rb, GT * D.sum(0) + 1.01 * _half(w.dtype) * rb.abs() + 1e-38)


class _Fenced:
    """Contiguous tensors `off` elements past a 16-byte boundary, NaN before and behind them."""

    def __init__(self, off):
        self.off, self.all = off, []

    def __call__(self, t):
        n, pre = t.numel(), 64 + self.off
        buf = torch.full((pre + n + 64,), float("nan"), dtype=t.dtype, device="cuda")
        v = buf[pre:pre + n].view(t.shape)
        v.copy_(t)
        self.all.append((buf, pre, n))
        return v

    def intact(self):
        return all(bool(torch.isnan(b[:p]).all()) and bool(torch.isnan(b[p + n:]).all()) for b, p, n in self.all)


@pytest.mark.parametrize("dt,wdt,off", [(BF, BF, 0), (BF, F32, 3), (BF, BF, 7), (F32, F32, 0), (F32, BF, 1)])
@pytest.mark.parametrize("T,H", [(1, 129), (2, 131), (7, 258), (8, 33), (9, 255), (40, 100), (3000, 33), (777, 1021), (23, 2047), (500, 4099),
                                 (5, 8185), (2, 8191), (3, 8193), (2, 16383), (6, 1024), (3000, 1024), (2100, 1021), (4200, 513),
                                 (8300, 257)])
def test_rows_off_the_boundary(T, H, dt, wdt, off):
    """Rows that start anywhere against 16 bytes: nothing beside a row or a tensor is used or written."""
    x, w, b, r, dy = _inputs(T, H, dt, wdt, seed=T + 5 * H)
    at = _Fenced(off)
    for res in (None, r):
        s = x if res is None else (x.float() + r.float()).to(dt)
        o = api.moe_layer_norm(at(x), w, b, residual=None if res is None else at(res), y=at(dy),
                               sum=None if res is None else at(dy))
        _forward_check(o, s, w, b, 1e-5)
        assert res is None or torch.equal(o.sum, s)
        got = api.moe_layer_norm_backward(at(dy), at(s), w, o.mean, o.rstd, dx_add=None if res is None else at(res), dx=at(x))
        _backward_check(got, dy, s, w, o.mean, o.rstd, res)
    assert at.intact()


@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_off_the_boundary_in_place(dt):
    x, w, b, r, dy = _inputs(400, 1021, dt, F32, seed=11)
    want = api.moe_layer_norm(x, w, b, residual=r)
    x2, r2 = x.clone(), r.clone()
    got = api.moe_layer_norm(x2, w, b, residual=r2, sum=r2, y=x2)
    assert torch.equal(got.y, want.y) and torch.equal(r2, want.sum)
    ref = api.moe_layer_norm_backward(dy, want.sum, w, want.mean, want.rstd, dx_add=r)
    for alias in ("dy", "add"):
        d2, a2 = dy.clone(), r.clone()
        got = api.moe_layer_norm_backward(d2, want.sum, w, want.mean, want.rstd, dx_add=a2, dx=d2 if alias == "dy" else a2)
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_non_finite_rows_off_the_boundary_stay_apart():
    """A NaN row and an infinite one, whose elements share 16-byte pieces with their neighbours'."""
    x, w, b, _, dy = _inputs(40, 1021, BF, F32, seed=4)
    clean = api.moe_layer_norm(x, w, b)
    x2 = x.clone()
    x2[4] = float("nan")
    x2[6] = float("inf")
    o = api.moe_layer_norm(x2, w, b)
    rows = [t for t in range(40) if t not in (4, 6)]
    assert torch.equal(o.y[rows], clean.y[rows]) and torch.equal(o.rstd[rows], clean.rstd[rows])
    assert torch.isnan(o.y[4]).all() and torch.isnan(o.y[6]).all()
    d2 = dy.clone()
    d2[9] = float("nan")
    dx, _, _ = api.moe_layer_norm_backward(d2, x2, w, o.mean, o.rstd)
    ref, _, _ = api.moe_layer_norm_backward(dy, x, w, clean.mean, clean.rstd)
    rows.remove(9)
    assert torch.equal(dx[rows], ref[rows]) and torch.isnan(dx[9]).all()


@pytest.mark.parametrize("dt,wdt", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,H", [(300, 8264), (33, 16392), (9, 40000), (70, 9001)])
def test_long_rows_by_the_dozen(T, H, dt, wdt):
    """Rows that do not fit the ring, enough of them for several partial sums a column."""
    x, w, b, r, dy = _inputs(T, H, dt, wdt, seed=T * 3 + H)
    s = (x.float() + r.float()).to(dt)
    o = api.moe_layer_norm(x, w, b, residual=r)
    assert torch.equal(o.sum, s)
    _forward_check(o, s, w, b, 1e-5)
    got = api.moe_layer_norm_backward(dy, s, w, o.mean, o.rstd, dx_add=r)
    _backward_check(got, dy, s, w, o.mean, o.rstd, r)
    d2 = dy.clone()
    again = api.moe_layer_norm_backward(d2, s, w, o.mean, o.rstd, dx_add=r, dx=d2)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,H", [(700, 3001), (40, 8000), (9, 2048), (3, 9001), (300, 100)])
def test_tensors_off_the_boundary_differently(T, H, dt):
    """Each tensor starts elsewhere against 16 bytes, so no piece of one is a piece of the others."""
    x, w, b, r, dy = _inputs(T, H, dt, F32, seed=T + 7 * H)
    s = (x.float() + r.float()).to(dt)
    a0, a1, a2 = _Fenced(0), _Fenced(1), _Fenced(2)
    o = api.moe_layer_norm(a0(x), w, b, residual=a1(r), y=a2(dy), sum=a1(dy))
    assert torch.equal(o.sum, s)
    _forward_check(o, s, w, b, 1e-5)
    got = api.moe_layer_norm_backward(a1(dy), a0(s), w, o.mean, o.rstd, dx_add=a2(r), dx=a1(x))
    _backward_check(got, dy, s, w, o.mean, o.rstd, r)
    assert a0.intact() and a1.intact() and a2.intact()


def _large_mean_check(dy, s, w, add, dx=None):
    """The backward of rows whose mean is many standard deviations, from statistics exact to fp32. The
    bars take xh to 4 u of itself, two roundings with room, whatever the mean: s - mean loses nothing."""
    S = s.double()
    mean64 = S.mean(1)
    mean = mean64.float()
    rstd = ((S - mean64[:, None]).square().mean(1) + 1e-5).rsqrt().float()
    got = api.moe_layer_norm_backward(dy, s, w, mean, rstd, dx_add=add, dx=dx)
    T, H = s.shape
    G, GT = (H / 32 + 64) * U, (T + 64) * U
    rx, rw, rb, xh, g = _backward_reference(dy, s, w, mean, rstd, add)
    R = rstd.double()[:, None]
    exh = 4 * U * xh.abs()
    c = (g * xh).mean(1, keepdim=True).abs()
    sums = G * (g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) \
        + xh.abs() * (g.abs() * exh).mean(1, keepdim=True)
    terms = g.abs() + g.mean(1, keepdim=True).abs() + xh.abs() * c
    e = R * (sums + 16 * U * terms + exh * c)
    if add is not None:
        e = e + 2 * U * (add.double().abs() + rx.abs())
    _within(got[0], rx, e + 1.01 * _half(s.dtype) * rx.abs() + 1e-38)
    D = dy.double().abs()
    _within(got[1], rw, GT * (D * xh.abs()).sum(0) + (D * exh).sum(0) + 1.01 * _half(w.dtype) * rw.abs() + 1e-38)
    _within(got[2], rb, GT * D.sum(0) + 1.01 * _half(w.dtype) * rb.abs() + 1e-38)


@pytest.mark.parametrize("ratio", [1e2, 1e3, 1e4])
@pytest.mark.parametrize("T,H", [(2500, 128), (40, 1024), (200, 4096), (9, 8192), (40, 1021), (1100, 1021), (40, 2001),
                                 (9, 8001), (20, 9001), (20, 12288)])
def test_backward_of_rows_with_a_large_mean(T, H, ratio):
    """Every kernel of the backward: rows in registers, through the ring (on and off the boundary), long ones."""
    x, w, _, r, dy = _inputs(T, H, F32, F32, seed=T + H, mean=1.5 * ratio)
    for add in (None, r):
        _large_mean_check(dy, x, w, add)


@pytest.mark.parametrize("dt,wdt,ratio", [(F32, BF, 1e3), (BF, BF, 1e2), (BF, F32, 1e2)])
@pytest.mark.parametrize("T,H", [(40, 2048), (33, 8184), (1500, 1021), (20, 8193)])
def test_backward_of_rows_with_a_large_mean_other_types(T, H, dt, wdt, ratio):
    x, w, _, r, dy = _inputs(T, H, dt, wdt, seed=T + H, mean=1.5 * ratio)
    _large_mean_check(dy, x, w, r)


def test_backward_of_rows_with_a_large_mean_elsewhere_against_16_bytes():
    x, w, _, r, dy = _inputs(40, 3001, F32, F32, seed=1, mean=1.5e3)
    _large_mean_check(dy, x, w, r, dx=_Fenced(1)(x))


@pytest.mark.parametrize("T,H", [(40, 1024), (9, 8192), (1100, 1021), (20, 12288)])
def test_backward_of_constant_rows(T, H):
    """s = mean in every place: xh is 0, so no weight gradient comes of it."""
    _, w, _, _, dy = _inputs(T, H, F32, F32, seed=3)
    s = torch.full((T, H), 1000.1, device="cuda")
    mean, rstd = s[:, 0].contiguous(), torch.full((T,), 1e-5 ** -0.5, device="cuda")
    _, dw, db = api.moe_layer_norm_backward(dy, s, w, mean, rstd)
    assert not dw.any() and db.any()
