"""Refusals of the few-token layer, the layer norm and the gradient norm that need no GPU: bad
shapes, types, pointers and workspaces return a status before any CUDA call
(1 invalid argument, 2 unsupported, 3 workspace, 5 alignment)."""
import ctypes as C

import pytest

P = C.c_void_p(4096)             # stands for a buffer: never dereferenced on these paths
ODD = C.c_void_p(4097)
BF16, MXFP8, F32 = 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from dropless_moe_expert_router_gb300 import _lib, build
    build.build()
    return _lib.load()


def _few(lib, T=4, H=512, K=2, E=8, F=512, dtype=BF16, x=P, logits=P, w13=P, s13=P, w2=P, s2=P, ids=P, idt=1, probs=P,
         y=P, flags=0, ws=P, nbytes=1 << 40):
    return lib.moe_layer_few_tokens(x, T, H, logits, K, E, F, w13, s13, w2, s2, dtype, ids, idt, probs, y, flags, ws,
                                    nbytes, None)


def test_few_tokens(lib):
    assert _few(lib, T=-1) == 1 and _few(lib, K=0) == 1 and _few(lib, K=9) == 1 and _few(lib, E=0) == 1
    assert _few(lib, idt=2) == 1 and _few(lib, flags=2) == 1 and _few(lib, dtype=F32) == 1
    assert _few(lib, T=65) == 2 and _few(lib, H=192) == 2 and _few(lib, F=192) == 2
    assert _few(lib, H=256, dtype=MXFP8) == 2 and _few(lib, F=768, dtype=MXFP8) == 2
    assert _few(lib, K=129, E=200) == 2 and _few(lib, T=64, K=65, E=200) == 2 and _few(lib, E=8193) == 2
    assert _few(lib, T=0, x=None, y=None, ws=None) == 0
    for name in ("x", "w13", "w2", "ids", "probs", "y"):
        assert _few(lib, **{name: None}) == 1
    assert _few(lib, dtype=MXFP8, s13=None) == 1 and _few(lib, dtype=MXFP8, s2=None) == 1
    assert _few(lib, ws=None) == 3 and _few(lib, nbytes=1) == 3
    for name in ("x", "w13", "w2", "ids", "probs", "y", "ws", "logits"):
        assert _few(lib, **{name: ODD}) == 5
    need = lib.moe_layer_few_tokens_workspace_size(4, 2, 8, 512, 512, BF16)
    assert need >= 4 * 2 * 512 * 2 and _few(lib, nbytes=need - 1) == 3
    assert lib.moe_layer_few_tokens_workspace_size(65, 2, 8, 512, 512, BF16) == 0
    assert lib.moe_layer_few_tokens_workspace_size(4, 2, 8, 512, 512, F32) == 0


def test_few_tokens_sizes_that_do_not_fit_shared_memory(lib):
    """The plan of very many routes and experts beside MXFP8's scales: refused with the workspace's size, not later."""
    size = lib.moe_layer_few_tokens_workspace_size
    assert size(64, 64, 8192, 512, 512, MXFP8) == 0 and _few(lib, T=64, K=64, E=8192, dtype=MXFP8) == 2
    for T, K, E in ((64, 32, 8192), (16, 128, 8192), (64, 64, 2304), (32, 128, 2304)):
        assert size(T, K, E, 512, 512, MXFP8) > 0
    for T, K in ((64, 64), (32, 128)):
        assert size(T, K, 8192, 512, 512, BF16) > 0


def _ln(lib, T=4, H=64, dtype=BF16, x=P, res=None, w=P, b=P, wdt=F32, eps=1e-5, sm=None, y=P, mean=P, rstd=P):
    return lib.moe_layer_norm(x, res, T, H, dtype, w, b, wdt, eps, sm, y, mean, rstd, None)


def _lnb(lib, T=4, H=64, dtype=BF16, dy=P, s=P, w=P, wdt=F32, mean=P, rstd=P, add=None, dx=P, dw=P, db=P, ws=P,
         nbytes=1 << 40):
    return lib.moe_layer_norm_backward(dy, s, T, H, dtype, w, wdt, mean, rstd, add, dx, dw, db, ws, nbytes, None)


def test_layer_norm(lib):
    assert _ln(lib, T=-1) == 1 and _ln(lib, H=0) == 1 and _ln(lib, dtype=MXFP8) == 1 and _ln(lib, wdt=1) == 1
    assert _ln(lib, eps=-1.0) == 1 and _ln(lib, eps=float("nan")) == 1 and _ln(lib, H=65537) == 2
    assert _ln(lib, res=P) == 1 and _ln(lib, sm=P) == 1                   # sum and residual go together
    assert _ln(lib, x=None) == 1 and _ln(lib, w=None) == 1 and _ln(lib, y=None) == 1
    assert _ln(lib, T=0, x=None, y=None) == 0
    for name in ("x", "w", "b", "y", "mean", "rstd"):
        assert _ln(lib, **{name: ODD}) == 5
    assert _lnb(lib, T=-1) == 1 and _lnb(lib, dtype=1) == 1 and _lnb(lib, H=65537) == 2
    for name in ("dy", "s", "w", "mean", "rstd", "dx"):
        assert _lnb(lib, **{name: None}) == 1
        assert _lnb(lib, **{name: ODD}) == 5
    for name in ("add", "dw", "db", "ws"):
        assert _lnb(lib, **{name: ODD}) == 5
    assert _lnb(lib, ws=None) == 3
    assert _lnb(lib, nbytes=lib.moe_layer_norm_backward_workspace_size(4, 64) - 1) == 3
    assert lib.moe_layer_norm_backward_workspace_size(-1, 64) == 0


def test_grad_norm(lib):
    def call(ptrs=(4096, 8192), counts=(10, 20), dts=(BF16, F32), outs=None, n=2, mx=1.0, eps=0.0, norm=P, ws=P,
             nbytes=1 << 30):
        a = (C.c_void_p * len(ptrs))(*ptrs)
        o = None if outs is None else (C.c_void_p * len(outs))(*outs)
        return lib.moe_grad_norm_clip(a, (C.c_longlong * len(counts))(*counts), (C.c_int * len(dts))(*dts), o, n, mx,
                                      eps, norm, ws, nbytes, None)
    assert call(n=-1) == 1 and call(mx=-1.0) == 1 and call(mx=float("nan")) == 1 and call(eps=-1.0) == 1
    assert call(norm=None) == 1 and call(counts=(10, -1)) == 1 and call(dts=(BF16, MXFP8)) == 1
    assert call(ptrs=(None, 8192)) == 1 and call(outs=(4096, None)) == 1
    assert call(counts=(10, 1 << 39)) == 2
    assert call(ws=None) == 3 and call(nbytes=lib.moe_grad_norm_workspace_size(2) - 1) == 3
    assert call(ptrs=(4097, 8192)) == 5 and call(ptrs=(4096, 8194)) == 5 and call(outs=(4096, 8193)) == 5
    assert call(norm=ODD) == 5 and call(ws=ODD) == 5
    assert lib.moe_grad_norm_workspace_size(-1) == 0
