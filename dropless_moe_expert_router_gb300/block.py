"""A pre-norm MoE block: the layer with what stands around it in a transformer.

    s = x + delta;  hn = LayerNorm(s);  logits = hn Wr^T;  delta' = MoE(hn, logits)

The block keeps the residual stream and the update apart, as a stack of blocks hands them on:
``forward`` takes (x, delta) and gives (s, delta'), and the next block's norm adds them. A
training step is ``forward``, ``backward``, ``clip_gradients``, an optimiser's update of the parameters
in place, and ``repack``; serving calls ``step`` with the few tokens of a decoding step. The router's projection is an ordinary dense product and is
left to torch; the norm, the layer, their backward passes and the clipping are the library's.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import api
from .layer import MoELayer


class MoEBlock:
    def __init__(self, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor, router: torch.Tensor,
                 norm_weight: torch.Tensor, norm_bias: Optional[torch.Tensor] = None, *, T: int, K: int,
                 eps: float = 1e-5, **layer_args):
        """Expert weights as MoELayer takes them, router [E, H] fp32, norm_weight and norm_bias [H];
        the remaining arguments are MoELayer's (precision, renorm, training, score, ...). The block keeps
        the tensors themselves; the layer also keeps packed copies of w1, w3 and w2 (``repack``)."""
        E, H, _ = w1.shape
        if tuple(router.shape) != (E, H) or router.dtype != torch.float32:
            raise ValueError("router must be [E, H] float32")
        self.layer = MoELayer(w1, w3, w2, T=T, K=K, **layer_args)
        self.router = router
        self.norm_weight, self.norm_bias, self.eps = norm_weight, norm_bias, eps
        self._saved = None
        self.gradients = None       # of every parameter, by name, after a backward

    def _norm(self, x, delta):
        o = api.moe_layer_norm(x, self.norm_weight, self.norm_bias, self.eps, residual=delta)
        return o, torch.mm(o.y.float(), self.router.t())

    def forward(self, x: torch.Tensor, delta: Optional[torch.Tensor] = None):
        """x (and delta) [T, H] bf16 -> (s [T, H], delta' [T, H], a layer-owned buffer)."""
        o, logits = self._norm(x, delta)
        out = self.layer.forward(o.y, logits)
        if self.layer.training:
            self._saved = (o, logits)
        return o.sum, out

    def step(self, x: torch.Tensor, delta: Optional[torch.Tensor] = None):
        """The block for the few tokens of a decoding step: x (and delta) [t, H], t <= 64. Steps share a
        workspace (MoELayer.forward_few) and must not overlap on the GPU."""
        o, logits = self._norm(x, delta)
        return o.sum, self.layer.forward_few(o.y, logits)

    def backward(self, ds: torch.Tensor, ddelta: torch.Tensor) -> torch.Tensor:
        """Gradients of the last training forward's outputs (s, delta') -> the gradient of s, which is
        that of x and of delta. The parameters' gradients: ``gradients``."""
        if self._saved is None:
            raise ValueError("backward wants a training layer's forward first")
        o, logits = self._saved
        dhn, dlogits, dw1, dw3, dw2 = self.layer.backward_full(o.y, logits, ddelta)
        drouter = torch.mm(dlogits.t(), o.y.float())
        dhn = torch.addmm(dhn.float(), dlogits, self.router).to(dhn.dtype)
        dsum, dnw, dnb = api.moe_layer_norm_backward(dhn, o.sum, self.norm_weight, o.mean, o.rstd, dx_add=ds)
        self.gradients = dict(w1=dw1, w3=dw3, w2=dw2, router=drouter, norm_weight=dnw)
        if self.norm_bias is not None:
            self.gradients["norm_bias"] = dnb
        return dsum

    def repack(self, stream=None) -> None:
        """After an update of w1, w3 or w2 in place: without it the kernels compute with the weights from before."""
        self.layer.repack(stream)

    def clip_gradients(self, max_norm: float) -> torch.Tensor:
        """Scale the gradients in place to a global norm of at most max_norm; the norm they had ([1] fp32
        on the device)."""
        if self.gradients is None:
            raise ValueError("clip_gradients wants a backward first")
        return api.moe_grad_clip(list(self.gradients.values()), max_norm)
