"""Tensors, streams and the current device of the few-token layer, the norm and the clipping have to go
together: what does not is refused before the library is called. (Stand-ins for CUDA tensors: a kernel
on one device would read the other's memory.)"""
import types

import pytest
import torch

from dropless_moe_expert_router_gb300 import _lib, api

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class _Cuda(torch.Tensor):
    """A CPU tensor that says it is on the CUDA device `at`."""
    is_cuda = True


def _t(shape, dtype, at=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(_Cuda)
    t.at = at
    return t


@pytest.fixture(autouse=True)
def _no_call(monkeypatch):
    class Library:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 64

            def reached(*a):
                raise AssertionError(f"{name} was reached")
            return reached
    monkeypatch.setattr(_lib, "load", lambda: Library())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: getattr(t, "at", -1))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)


def _each_elsewhere(call, tensors):
    """call(**tensors) with one tensor at a time on another device, and on the host."""
    for name, t in tensors.items():
        for at in (1, -1):
            moved = dict(tensors)
            moved[name] = _t(t.shape, t.dtype, at)
            if at < 0:
                moved[name] = torch.zeros(t.shape, dtype=t.dtype)
            with pytest.raises(ValueError):
                call(**moved)
    with pytest.raises(AssertionError):                      # together they reach the library
        call(**tensors)


def test_layer_norm():
    T, H = 3, 8
    rows = {n: _t((T, H), BF) for n in ("x", "residual", "y", "sum")}
    _each_elsewhere(api.moe_layer_norm, dict(rows, weight=_t((H,), F32), bias=_t((H,), F32), mean=_t((T,), F32),
                                             rstd=_t((T,), F32)))
    rows = {n: _t((T, H), BF) for n in ("dy", "s", "dx_add", "dx")}
    cols = {n: _t((H,), F32) for n in ("weight", "dweight", "dbias")}
    _each_elsewhere(api.moe_layer_norm_backward, dict(rows, **cols, mean=_t((T,), F32), rstd=_t((T,), F32),
                                                      workspace=_t((64,), U8)))


def test_few_tokens():
    T, H, E, K, F = 2, 8, 4, 2, 8

    def call(x, logits, ids, probs, y, workspace, w13, w13_scales, w2, w2_scales):
        w = api.PackedWeights("mxfp8", E, H, F, w13, w13_scales, w2, w2_scales)
        return api.moe_layer_few_tokens(x, logits, w, K, ids=ids, probs=probs, y=y, workspace=workspace)
    _each_elsewhere(call, dict(x=_t((T, H), BF), logits=_t((T, E), F32), ids=_t((T, K), torch.int32), probs=_t((T, K), F32),
                               y=_t((T, H), BF), workspace=_t((64,), U8), w13=_t((E, 2 * F, H), U8),
                               w13_scales=_t((E, 2 * F, 1), U8), w2=_t((E, H, F), U8), w2_scales=_t((E, H, 1), U8)))


def test_gradient_clipping():
    def call(a, b, oa, ob, norm, workspace):
        return api.moe_grad_clip([a, b], 1.0, out=[oa, ob], norm=norm, workspace=workspace)
    _each_elsewhere(call, dict(a=_t((5,), BF), b=_t((6,), F32), oa=_t((5,), BF), ob=_t((6,), F32), norm=_t((1,), F32),
                               workspace=_t((64,), U8)))


def test_the_current_device_and_the_stream(monkeypatch):
    x, w, m = _t((3, 8), BF, 1), _t((8,), F32, 1), _t((3,), F32, 1)
    with pytest.raises(ValueError):                          # everything on cuda:1, the current device is cuda:0
        api.moe_layer_norm(x, w, y=x, mean=m, rstd=m)
    with pytest.raises(ValueError):
        api.moe_grad_clip([x, w], 1.0, norm=_t((1,), F32, 1), workspace=_t((64,), U8, 1))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(AssertionError):
        api.moe_layer_norm(x, w, y=x, mean=m, rstd=m)
    for index, refused in ((0, ValueError), (1, AssertionError)):
        with pytest.raises(refused):
            api.moe_layer_norm(x, w, y=x, mean=m, rstd=m, stream=types.SimpleNamespace(device_index=index, cuda_stream=7))
