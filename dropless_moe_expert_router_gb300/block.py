"""A pre-norm MoE block: the layer with what stands around it in a transformer.

    s = x + delta;  hn = LayerNorm(s);  logits = hn Wr^T;  delta' = MoE(hn, logits)

The block keeps the residual stream and the update apart, as a stack of blocks hands them on:
``forward`` takes (x, delta) and gives (s, delta'), and the next block's norm adds them. A
training step is ``forward``, ``backward``, ``clip_gradients``, an optimiser's update of the parameters
in place, and ``repack``; serving calls ``step`` with the few tokens of a decoding step. The router's projection is an ordinary dense product and is
left to torch; the norm, the layer, their backward passes and the clipping are the library's.

A block that serves may begin with attention over a cache (``Attention``): then ``step`` is a whole decoder
block's, s' = x + delta, delta'' = Attention(LayerNorm(s')), and the MoE part as above on (s', delta'').
"""
from __future__ import annotations

from typing import Optional

import torch

from . import api
from .cache import SequenceCache
from .layer import MoELayer


class Attention:
    """Pre-norm attention of one new token per sequence over a cache. The two projections are torch's."""

    def __init__(self, qkv: torch.Tensor, out: torch.Tensor, norm_weight: torch.Tensor,
                 norm_bias: Optional[torch.Tensor] = None, *, q_heads: int, kv_heads: int, scale: Optional[float] = None,
                 window: int = 0, eps: float = 1e-5):
        """qkv [(q_heads + 2 kv_heads) * dim, H] bf16 (queries, keys, values), out [H, q_heads * dim] bf16, norm_weight and
        norm_bias [H]; scale and window are moe_paged_attention's."""
        rows, H = qkv.shape
        if kv_heads < 1 or q_heads < 1 or q_heads % kv_heads or rows % (q_heads + 2 * kv_heads):
            raise ValueError("qkv must be [(q_heads + 2 kv_heads) * dim, H], q_heads a multiple of kv_heads")
        dim = rows // (q_heads + 2 * kv_heads)
        if tuple(out.shape) != (H, q_heads * dim) or qkv.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
            raise ValueError("qkv and out must be bfloat16, out [H, q_heads * dim]")
        self.qkv, self.out = qkv, out
        self.norm_weight, self.norm_bias, self.eps = norm_weight, norm_bias, eps
        self.q_heads, self.kv_heads, self.dim, self.scale, self.window = q_heads, kv_heads, dim, scale, window

    def step(self, x: torch.Tensor, delta: Optional[torch.Tensor], cache: SequenceCache, layer: int):
        """x (and delta) [t, H], one row a slot of the cache, whose `advance` came before -> (s, delta')."""
        o = api.moe_layer_norm(x, self.norm_weight, self.norm_bias, self.eps, residual=delta)
        nq, nkv = self.q_heads, self.kv_heads
        qkv = torch.mm(o.y, self.qkv.t()).view(x.shape[0], nq + 2 * nkv, self.dim)
        cache.append(layer, qkv[:, nq:nq + nkv], qkv[:, nq + nkv:])
        heads = cache.attend(layer, qkv[:, :nq], scale=self.scale, window=self.window)
        return o.sum, torch.mm(heads.view(x.shape[0], -1), self.out.t())


class MoEBlock:
    def __init__(self, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor, router: torch.Tensor,
                 norm_weight: torch.Tensor, norm_bias: Optional[torch.Tensor] = None, *, T: int, K: int,
                 eps: float = 1e-5, attention: Optional[Attention] = None, index: int = 0, **layer_args):
        """Expert weights as MoELayer takes them, router [E, H] fp32, norm_weight and norm_bias [H];
        the remaining arguments are MoELayer's (precision, renorm, training, score, ...). The block keeps
        the tensors themselves; the layer also keeps packed copies of w1, w3 and w2 (``repack``).
        attention: what a decoder block's step begins with (serving only); index: the block's layer of the cache."""
        E, H, _ = w1.shape
        if attention is not None and (attention.qkv.shape[1] != H or layer_args.get("training")):
            raise ValueError("attention is of the block's width, and in a block that serves")
        self.attention, self.index = attention, index
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
        if self.attention is not None:
            raise ValueError("a block with attention over a cache goes by steps")
        o, logits = self._norm(x, delta)
        out = self.layer.forward(o.y, logits)
        if self.layer.training:
            self._saved = (o, logits)
        return o.sum, out

    def step(self, x: torch.Tensor, delta: Optional[torch.Tensor] = None, cache: Optional[SequenceCache] = None):
        """The block for the few tokens of a decoding step: x (and delta) [t, H], t <= 64. Steps share a
        workspace (MoELayer.forward_few) and must not overlap on the GPU. A block with attention wants the cache, and a row
        for each of its slots."""
        if (self.attention is None) != (cache is None):
            raise ValueError("a cache goes with a block that has attention")
        if cache is not None:
            x, delta = self.attention.step(x, delta, cache, self.index)
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
