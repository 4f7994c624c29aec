"""Thin Python binding of the C ABI (include/moe_gb300.h).

Each function has the name of its C entry point and only marshals arguments:
it checks devices and dtypes, allocates outputs with torch when the caller did
not pass them (from the memory of the call's stream), and hands raw pointers, sizes
and that stream, the current one unless given, to the library. Every step of the
computation runs in the library's kernels.
"""
from __future__ import annotations

import ctypes as C
from array import array
from typing import NamedTuple, Optional

import torch

from . import _lib

MOE_I16, MOE_I32, MOE_BF16, MOE_MXFP8, MOE_F32 = 0, 1, 2, 3, 4
MOE_ROUTE_RENORM = 1
MOE_PERMUTE_FUSE_MXFP8 = 2
MOE_QUANT_COLWISE = 4
MOE_DEVERR_BAD_ID = 1
MOE_DEVERR_TIMEOUT = 2


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        name = _lib.load().moe_status_string(status).decode()
        super().__init__(f"{fn} failed: {name} ({status})")
        self.status = status


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MoeError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _raw_stream(stream: Optional[torch.cuda.Stream], t: torch.Tensor) -> int:
    """The stream's handle: the given one's, or that of the current stream of t's device, which has to be the
    current device: the launch is its own."""
    dev = t.get_device()
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on cuda:{dev}, which is not the current device (torch.cuda.device)")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the stream on cuda:{stream.device_index}")
    return stream.cuda_stream


def _empty(shape, dtype: torch.dtype, device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """Uninitialised memory for a call on `stream` (None: the current one). It comes from that stream's
    memory, which follows the order of the kernels that use it: whoever gets it next, or had it before, runs
    on the same stream. What the caller enqueues on the current stream is waited for too before it goes back."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if stream == current:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _empty_like(t: torch.Tensor, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """_empty of t's shape, type and device."""
    return torch.empty_like(t) if stream is None else _empty(t.shape, t.dtype, t.device, stream)


def _at(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _want(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def _scratch(t: torch.Tensor, dev: int) -> None:
    if not (t.get_device() == dev and t.dtype is torch.uint8 and t.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{dev}, the other tensors' device")


def _on(dev: int, t: Optional[torch.Tensor], name: str) -> None:
    """t, where given, is on this CUDA device."""
    if t is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, the other tensors' device")


def _id_code(dtype: torch.dtype) -> int:
    if dtype == torch.int16:
        return MOE_I16
    if dtype == torch.int32:
        return MOE_I32
    raise ValueError("ids must be int16 or int32")


# --------------------------------------------------------------------- router
def moe_route_topk(logits: torch.Tensor, K: int, *, id_dtype=torch.int32, renorm: bool = False,
                   ids: Optional[torch.Tensor] = None, probs: Optional[torch.Tensor] = None,
                   stream=None):
    """logits [T, E] fp32 -> (ids [T, K] int16/int32, probs [T, K] fp32)."""
    _want(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    if ids is None:
        ids = _empty((T, K), id_dtype, logits.device, stream)
    if probs is None:
        probs = _empty((T, K), torch.float32, logits.device, stream)
    _want(ids, "ids", None, 2)
    _want(probs, "probs", torch.float32, 2)
    st = _lib.load().moe_route_topk(_ptr(logits), T, E, K, _ptr(ids), _id_code(ids.dtype), _ptr(probs),
                                    MOE_ROUTE_RENORM if renorm else 0, _stream(stream))
    _check("moe_route_topk", st)
    return ids, probs


def moe_route_sigmoid_topk(logits: torch.Tensor, K: int, *, expert_bias: Optional[torch.Tensor] = None,
                           id_dtype=torch.int32, renorm: bool = False, ids: Optional[torch.Tensor] = None,
                           probs: Optional[torch.Tensor] = None, stream=None):
    """logits [T, E] fp32 (+ expert_bias [E] fp32) -> (ids [T, K], probs [T, K] fp32): selection on
    sigmoid(logit) + bias, probs the sigmoid scores (renormalised over the K selected with renorm)."""
    _want(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    if expert_bias is not None:
        _want(expert_bias, "expert_bias", torch.float32, 1)
        if expert_bias.numel() != E:
            raise ValueError("expert_bias must have E entries")
    if ids is None:
        ids = _empty((T, K), id_dtype, logits.device, stream)
    if probs is None:
        probs = _empty((T, K), torch.float32, logits.device, stream)
    _want(ids, "ids", None, 2)
    _want(probs, "probs", torch.float32, 2)
    st = _lib.load().moe_route_sigmoid_topk(_ptr(logits), _ptr(expert_bias), T, E, K, _ptr(ids),
                                            _id_code(ids.dtype), _ptr(probs), MOE_ROUTE_RENORM if renorm else 0,
                                            _stream(stream))
    _check("moe_route_sigmoid_topk", st)
    return ids, probs


def moe_route_sigmoid_topk_backward(logits: torch.Tensor, ids: torch.Tensor, dprobs: torch.Tensor, *,
                                    renorm: bool = False, dlogits: Optional[torch.Tensor] = None,
                                    stream=None) -> torch.Tensor:
    """logits [T, E], ids [T, K], dprobs [T, K] -> dlogits [T, E] fp32 of the sigmoid router."""
    _want(logits, "logits", torch.float32, 2)
    _want(ids, "ids", None, 2)
    _want(dprobs, "dprobs", torch.float32, 2)
    T, E = logits.shape
    K = ids.shape[1]
    if dlogits is None:
        dlogits = _empty((T, E), torch.float32, logits.device, stream)
    _want(dlogits, "dlogits", torch.float32, 2)
    st = _lib.load().moe_route_sigmoid_topk_backward(_ptr(logits), _ptr(ids), _id_code(ids.dtype), _ptr(dprobs),
                                                     T, E, K, MOE_ROUTE_RENORM if renorm else 0, _ptr(dlogits),
                                                     _stream(stream))
    _check("moe_route_sigmoid_topk_backward", st)
    return dlogits


# -------------------------------------------------------------------- permute
class Permuted(NamedTuple):
    x_perm: torch.Tensor          # [T*K, H] bf16, or uint8 E4M3 payloads when fused
    x_perm_scales: Optional[torch.Tensor]  # [T*K, H/32] uint8 E8M0 (fused MXFP8 only)
    group_sizes: torch.Tensor     # [E] int32
    group_offsets: torch.Tensor   # [E+1] int32
    row_map: torch.Tensor         # [T, K] int32
    perm_src: torch.Tensor        # [T*K] int32


def moe_permute_workspace_size(T: int, K: int, E: int) -> int:
    return int(_lib.load().moe_permute_workspace_size(T, K, E))


def moe_permute_kernel_launches(T: int, K: int, E: int) -> int:
    return int(_lib.load().moe_permute_kernel_launches(T, K, E))


def permute_buffers(T: int, H: int, K: int, E: int, device, fuse_mxfp8: bool = False,
                    nvfp4: bool = False, stream=None) -> Permuted:
    R_cap = T * K
    dev = torch.device(device)
    if nvfp4:
        xp = _empty((R_cap, H // 2), torch.uint8, dev, stream)
        xs = _empty((R_cap, H // 16), torch.uint8, dev, stream)
    elif fuse_mxfp8:
        xp = _empty((R_cap, H), torch.uint8, dev, stream)
        xs = _empty((R_cap, H // 32), torch.uint8, dev, stream)
    else:
        xp = _empty((R_cap, H), torch.bfloat16, dev, stream)
        xs = None
    return Permuted(xp, xs, _empty(E, torch.int32, dev, stream),
                    _empty(E + 1, torch.int32, dev, stream),
                    _empty((T, K), torch.int32, dev, stream),
                    _empty(R_cap, torch.int32, dev, stream))


def moe_permute(x: torch.Tensor, ids: torch.Tensor, E: int, *, fuse_mxfp8: bool = False,
                out: Optional[Permuted] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> Permuted:
    """x [T, H] bf16, ids [T, K] -> Permuted (see the C header for each field)."""
    _want(x, "x", torch.bfloat16, 2)
    _want(ids, "ids", None, 2)
    T, H = x.shape
    K = ids.shape[1]
    if out is None:
        out = permute_buffers(T, H, K, E, x.device, fuse_mxfp8, stream=stream)
    ws_bytes = moe_permute_workspace_size(T, K, E)
    if workspace is None:
        workspace = _empty(ws_bytes, torch.uint8, x.device, stream)
    st = _lib.load().moe_permute(
        _ptr(x), T, H, _ptr(ids), _id_code(ids.dtype), K, E, _ptr(out.x_perm), _ptr(out.x_perm_scales),
        _ptr(out.group_sizes), _ptr(out.group_offsets), _ptr(out.row_map), _ptr(out.perm_src),
        MOE_PERMUTE_FUSE_MXFP8 if fuse_mxfp8 else 0, _ptr(workspace), workspace.numel(), _stream(stream))
    _check("moe_permute", st)
    return out


def moe_permute_nvfp4(x: torch.Tensor, ids: torch.Tensor, E: int, *, amax: Optional[torch.Tensor] = None,
                      out: Optional[Permuted] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None):
    """moe_permute writing NVFP4 rows: the routed tokens' amax first (-> amax [1] fp32), then the
    scatter quantises each row as it copies it (x_perm [R_cap, H/2] packed E2M1, x_perm_scales
    [R_cap, H/16] E4M3). Returns (Permuted, amax)."""
    _want(x, "x", torch.bfloat16, 2)
    _want(ids, "ids", None, 2)
    T, H = x.shape
    K = ids.shape[1]
    if out is None:
        out = permute_buffers(T, H, K, E, x.device, nvfp4=True, stream=stream)
    if amax is None:
        amax = _empty((1,), torch.float32, x.device, stream)
    ws_bytes = moe_permute_workspace_size(T, K, E)
    if workspace is None:
        workspace = _empty(ws_bytes, torch.uint8, x.device, stream)
    st = _lib.load().moe_permute_nvfp4(
        _ptr(x), T, H, _ptr(ids), _id_code(ids.dtype), K, E, _ptr(amax), _ptr(out.x_perm), _ptr(out.x_perm_scales),
        _ptr(out.group_sizes), _ptr(out.group_offsets), _ptr(out.row_map), _ptr(out.perm_src), _ptr(workspace),
        workspace.numel(), _stream(stream))
    _check("moe_permute_nvfp4", st)
    return out, amax


def moe_permute_noalloc(x: torch.Tensor, ids: torch.Tensor, E: int, *, fuse_mxfp8: bool = False,
                        out: Optional[Permuted] = None, stream=None) -> Permuted:
    """moe_permute for callers that may not allocate device memory: the library's
    static scratch array replaces the workspace (outputs are still the caller's)."""
    _want(x, "x", torch.bfloat16, 2)
    _want(ids, "ids", None, 2)
    T, H = x.shape
    K = ids.shape[1]
    if out is None:
        out = permute_buffers(T, H, K, E, x.device, fuse_mxfp8, stream=stream)
    st = _lib.load().moe_permute_noalloc(
        _ptr(x), T, H, _ptr(ids), _id_code(ids.dtype), K, E, _ptr(out.x_perm), _ptr(out.x_perm_scales),
        _ptr(out.group_sizes), _ptr(out.group_offsets), _ptr(out.row_map), _ptr(out.perm_src),
        MOE_PERMUTE_FUSE_MXFP8 if fuse_mxfp8 else 0, _stream(stream))
    _check("moe_permute_noalloc", st)
    return out


def moe_permute_noalloc_max_scratch() -> int:
    return int(_lib.load().moe_permute_noalloc_max_scratch())


# ---------------------------------------------------------------- quantiser
def colwise_scale_rows(R_cap: int, E: int) -> int:
    return E + R_cap // 32 + 1


def moe_quant_mxfp8_grouped(x: torch.Tensor, group_offsets: torch.Tensor, *, colwise: bool = False,
                            q: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                            stream=None):
    """x [R_cap, H] bf16 -> (q [R_cap, H] uint8, scales) row-wise or group-aware column-wise."""
    _want(x, "x", torch.bfloat16, 2)
    _want(group_offsets, "group_offsets", torch.int32, 1)
    R_cap, H = x.shape
    E = group_offsets.numel() - 1
    if q is None:
        q = _empty((R_cap, H), torch.uint8, x.device, stream)
    if scales is None:
        shape = (colwise_scale_rows(R_cap, E), H) if colwise else (R_cap, H // 32)
        scales = _empty(shape, torch.uint8, x.device, stream)
    st = _lib.load().moe_quant_mxfp8_grouped(_ptr(x), R_cap, H, _ptr(group_offsets), E, _ptr(q),
                                             _ptr(scales), MOE_QUANT_COLWISE if colwise else 0,
                                             _stream(stream))
    _check("moe_quant_mxfp8_grouped", st)
    return q, scales


# ------------------------------------------------------------------- combine
def moe_unpermute_combine(y_perm: torch.Tensor, row_map: torch.Tensor, probs: torch.Tensor, *,
                          y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y_perm [R_cap, H] bf16, row_map [T, K], probs [T, K] -> y [T, H] bf16."""
    _want(y_perm, "y_perm", torch.bfloat16, 2)
    _want(row_map, "row_map", torch.int32, 2)
    _want(probs, "probs", torch.float32, 2)
    T, K = row_map.shape
    H = y_perm.shape[1]
    if y is None:
        y = _empty((T, H), torch.bfloat16, y_perm.device, stream)
    st = _lib.load().moe_unpermute_combine(_ptr(y_perm), _ptr(row_map), _ptr(probs), T, K, H, _ptr(y),
                                           _stream(stream))
    _check("moe_unpermute_combine", st)
    return y


# -------------------------------------------------------------------- backward of route / permute / combine
def moe_route_topk_backward(logits: torch.Tensor, ids: torch.Tensor, dprobs: torch.Tensor, *,
                            renorm: bool = False, dlogits: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """logits [T, E] fp32, ids [T, K], dprobs [T, K] fp32 -> dlogits [T, E] fp32."""
    _want(logits, "logits", torch.float32, 2)
    _want(ids, "ids", None, 2)
    _want(dprobs, "dprobs", torch.float32, 2)
    T, E = logits.shape
    K = ids.shape[1]
    if dlogits is None:
        dlogits = _empty((T, E), torch.float32, logits.device, stream)
    _want(dlogits, "dlogits", torch.float32, 2)
    st = _lib.load().moe_route_topk_backward(_ptr(logits), _ptr(ids), _id_code(ids.dtype), _ptr(dprobs), T, E, K,
                                             MOE_ROUTE_RENORM if renorm else 0, _ptr(dlogits), _stream(stream))
    _check("moe_route_topk_backward", st)
    return dlogits


def moe_unpermute_combine_backward(dy: torch.Tensor, y_perm: torch.Tensor, row_map: torch.Tensor,
                                   probs: torch.Tensor, *, dy_perm: Optional[torch.Tensor] = None,
                                   dprobs: Optional[torch.Tensor] = None, dy_perm_q: Optional[torch.Tensor] = None,
                                   dy_perm_scales: Optional[torch.Tensor] = None, stream=None):
    """dy [T, H] bf16, y_perm [R_cap, H] bf16, row_map [T, K], probs [T, K] ->
    (dy_perm [R_cap, H] bf16, dprobs [T, K] fp32). With dy_perm_q [R_cap, H] uint8 and
    dy_perm_scales [R_cap, H/32] uint8 given, the kernel also writes the row-wise MXFP8
    codes and scales of dy_perm into them."""
    _want(dy, "dy", torch.bfloat16, 2)
    _want(y_perm, "y_perm", torch.bfloat16, 2)
    _want(row_map, "row_map", torch.int32, 2)
    _want(probs, "probs", torch.float32, 2)
    T, K = row_map.shape
    H = y_perm.shape[1]
    if dy_perm is None:
        dy_perm = _empty_like(y_perm, stream)    # rows no route maps to are not written
    if dprobs is None:
        dprobs = _empty((T, K), torch.float32, dy.device, stream)
    _want(dy_perm, "dy_perm", torch.bfloat16, 2)
    _want(dprobs, "dprobs", torch.float32, 2)
    if (dy_perm_q is None) != (dy_perm_scales is None):
        raise ValueError("dy_perm_q and dy_perm_scales go together")
    if dy_perm_q is not None:
        _want(dy_perm_q, "dy_perm_q", torch.uint8, 2)
        _want(dy_perm_scales, "dy_perm_scales", torch.uint8, 2)
        if tuple(dy_perm_q.shape) != tuple(y_perm.shape) or tuple(dy_perm_scales.shape) != (y_perm.shape[0], H // 32):
            raise ValueError("dy_perm_q must be [R_cap, H] and dy_perm_scales [R_cap, H/32]")
    st = _lib.load().moe_unpermute_combine_backward(_ptr(dy), _ptr(y_perm), _ptr(row_map), _ptr(probs), T, K, H,
                                                    _ptr(dy_perm), _ptr(dprobs),
                                                    _ptr(dy_perm_q), _ptr(dy_perm_scales), _stream(stream))
    _check("moe_unpermute_combine_backward", st)
    return dy_perm, dprobs


def moe_permute_backward(dx_perm: torch.Tensor, row_map: torch.Tensor, *, dx: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """dx_perm [R_cap, H] bf16, row_map [T, K] -> dx [T, H] bf16 (each token's rows summed)."""
    _want(dx_perm, "dx_perm", torch.bfloat16, 2)
    _want(row_map, "row_map", torch.int32, 2)
    T, K = row_map.shape
    H = dx_perm.shape[1]
    if dx is None:
        dx = _empty((T, H), torch.bfloat16, dx_perm.device, stream)
    _want(dx, "dx", torch.bfloat16, 2)
    st = _lib.load().moe_permute_backward(_ptr(dx_perm), _ptr(row_map), T, K, H, _ptr(dx), _stream(stream))
    _check("moe_permute_backward", st)
    return dx


# -------------------------------------------------------------------- expert parallelism
def moe_ep_recv_expert_ids(recv_counts: torch.Tensor, R_cap: int, *, ids: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """recv_counts [G, E_loc] int32 (rows received from each source for each local expert, on the
    device) -> ids [R_cap] int32: the local expert of each received row, -1 past them."""
    _want(recv_counts, "recv_counts", torch.int32, 2)
    G, E_loc = recv_counts.shape
    if ids is None:
        ids = _empty((R_cap,), torch.int32, recv_counts.device, stream)
    _want(ids, "ids", torch.int32, 1)
    st = _lib.load().moe_ep_recv_expert_ids(_ptr(recv_counts), G, E_loc, R_cap, _ptr(ids), _stream(stream))
    _check("moe_ep_recv_expert_ids", st)
    return ids


# -------------------------------------------------------------------- errors
def moe_get_device_errors(clear: bool = True) -> int:
    v = C.c_uint32(0)
    st = _lib.load().moe_get_device_errors(C.byref(v), 1 if clear else 0)
    if st not in (0, 6):
        _check("moe_get_device_errors", st)
    return int(v.value)


def moe_debug_bounded_wait_selftest(limit_us: int, stream=None) -> None:
    """Enqueue the bounded-wait self-test (sets MOE_DEVERR_TIMEOUT after limit_us)."""
    _check("moe_debug_bounded_wait_selftest",
           _lib.load().moe_debug_bounded_wait_selftest(int(limit_us), _stream(stream)))


def moe_route_ids_bytes(T: int, K: int, id_dtype=torch.int16) -> int:
    return int(_lib.load().moe_route_ids_bytes(T, K, _id_code(id_dtype)))


def moe_route_probs_bytes(T: int, K: int) -> int:
    return int(_lib.load().moe_route_probs_bytes(T, K))


def moe_host_mapped_pointer(t: torch.Tensor) -> Optional[int]:
    """Device address of a page-locked host tensor's data (the kernels can read and write it
    directly), or None when the tensor is not in page-locked memory the device can address."""
    if t.is_cuda or not t.is_contiguous() or t.numel() == 0:
        return None
    out = C.c_void_p()
    st = _lib.load().moe_host_mapped_pointer(C.c_void_p(t.data_ptr()), C.byref(out))
    return int(out.value) if st == 0 and out.value else None


# ------------------------------------------------------------- expert GEMMs
def _dt_code(precision: str) -> int:
    if precision == "bf16":
        return MOE_BF16
    if precision == "mxfp8":
        return MOE_MXFP8
    raise ValueError("precision must be 'bf16' or 'mxfp8'")


class PackedWeights(NamedTuple):
    precision: str
    E: int
    H: int
    F: int
    w13: torch.Tensor                 # [E, 2F, H] bf16 or uint8 (E4M3)
    w13_scales: Optional[torch.Tensor]  # [E, 2F, H/32] uint8 (MXFP8)
    w2: torch.Tensor                  # [E, H, F] bf16 or uint8
    w2_scales: Optional[torch.Tensor]   # [E, H, F/32] uint8 (MXFP8)


def _want_packed(out, kind, shapes, dev: int) -> None:
    """out is a kind of packed weights on this device, with these scalars first and these shapes (None: no
    tensor) after them."""
    n = len(out) - len(shapes[1])
    if type(out) is not kind or tuple(out[:n]) != shapes[0]:
        raise ValueError(f"out must be the {kind.__name__} of weights of this precision and size")
    for t, name, want in zip(out[n:], kind._fields[n:], shapes[1]):
        if want is None:
            continue
        if t is None:
            raise ValueError(f"out has no {name}")
        _like(t, name, want[0], want[1], dev)


def moe_prepare_weights(w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor, precision: str = "bf16",
                        stream=None, out: Optional[PackedWeights] = None) -> PackedWeights:
    """Pack logical W1, W3 [E, H, F] and W2 [E, F, H] (bf16) for the grouped GEMMs: into new buffers, or
    into those of out (packed before from weights of the same sizes that have changed since)."""
    for t, n in ((w1, "w1"), (w3, "w3"), (w2, "w2")):
        _want(t, n, torch.bfloat16, 3)
    E, H, F = w1.shape
    dev = w1.device
    fp8 = precision == "mxfp8"
    pdt = torch.uint8 if fp8 else torch.bfloat16
    if out is None:
        w13 = _empty((E, 2 * F, H), pdt, dev, stream)
        w2p = _empty((E, H, F), pdt, dev, stream)
        s13 = _empty((E, 2 * F, H // 32), torch.uint8, dev, stream) if fp8 else None
        s2 = _empty((E, H, F // 32), torch.uint8, dev, stream) if fp8 else None
        out = PackedWeights(precision, E, H, F, w13, s13, w2p, s2)
    else:
        u8 = torch.uint8
        _want_packed(out, PackedWeights, ((precision, E, H, F), (
            (pdt, (E, 2 * F, H)), (u8, (E, 2 * F, H // 32)) if fp8 else None,
            (pdt, (E, H, F)), (u8, (E, H, F // 32)) if fp8 else None)), w1.get_device())
    st = _lib.load().moe_prepare_weights(_ptr(w1), _ptr(w3), _ptr(w2), E, H, F, _dt_code(precision),
                                         _ptr(out.w13), _ptr(out.w13_scales), _ptr(out.w2), _ptr(out.w2_scales),
                                         _stream(stream))
    _check("moe_prepare_weights", st)
    return out


def moe_grouped_swiglu_gemm(x_perm: torch.Tensor, x_scales: Optional[torch.Tensor], w: PackedWeights,
                            group_offsets: torch.Tensor, *, h: Optional[torch.Tensor] = None,
                            h_scales: Optional[torch.Tensor] = None, y_perm: Optional[torch.Tensor] = None,
                            stream=None):
    """Grouped SwiGLU MLP on permuted rows -> (y_perm [R_cap, H] bf16, h, h_scales)."""
    fp8 = w.precision == "mxfp8"
    _want(x_perm, "x_perm", torch.uint8 if fp8 else torch.bfloat16, 2)
    _want(group_offsets, "group_offsets", torch.int32, 1)
    R_cap = x_perm.shape[0]
    dev = x_perm.device
    if h is None:
        h = _empty((R_cap, w.F), torch.uint8 if fp8 else torch.bfloat16, dev, stream)
    if fp8 and h_scales is None:
        h_scales = _empty((R_cap, w.F // 32), torch.uint8, dev, stream)
    if y_perm is None:
        y_perm = _empty((R_cap, w.H), torch.bfloat16, dev, stream)
    st = _lib.load().moe_grouped_swiglu_gemm(
        _ptr(x_perm), _ptr(x_scales), _ptr(w.w13), _ptr(w.w13_scales), _ptr(w.w2), _ptr(w.w2_scales),
        _dt_code(w.precision), _ptr(group_offsets), w.E, w.H, w.F, R_cap, _ptr(h), _ptr(h_scales),
        _ptr(y_perm), _stream(stream))
    _check("moe_grouped_swiglu_gemm", st)
    return y_perm, h, h_scales


def moe_grouped_gemm_up(x_perm: torch.Tensor, x_scales: Optional[torch.Tensor], w: PackedWeights,
                        group_offsets: torch.Tensor, *, h: Optional[torch.Tensor] = None,
                        h_scales: Optional[torch.Tensor] = None, ab: Optional[torch.Tensor] = None,
                        h_bf16: Optional[torch.Tensor] = None, stream=None):
    """Up projection + SwiGLU; optionally saves ab [R_cap, 2F] bf16 and (MXFP8) h_bf16 [R_cap, F]."""
    fp8 = w.precision == "mxfp8"
    R_cap = x_perm.shape[0]
    dev = x_perm.device
    if h is None:
        h = _empty((R_cap, w.F), torch.uint8 if fp8 else torch.bfloat16, dev, stream)
    if fp8 and h_scales is None:
        h_scales = _empty((R_cap, w.F // 32), torch.uint8, dev, stream)
    st = _lib.load().moe_grouped_gemm_up(
        _ptr(x_perm), _ptr(x_scales), _ptr(w.w13), _ptr(w.w13_scales), _dt_code(w.precision),
        _ptr(group_offsets), w.E, w.H, w.F, R_cap, _ptr(h), _ptr(h_scales), _ptr(ab), _ptr(h_bf16),
        _stream(stream))
    _check("moe_grouped_gemm_up", st)
    return h, h_scales


def moe_grouped_gemm_down(h: torch.Tensor, h_scales: Optional[torch.Tensor], w: PackedWeights,
                          group_offsets: torch.Tensor, *, y_perm: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Down projection y_perm = h W2[e] per group -> y_perm [R_cap, H] bf16."""
    fp8 = w.precision == "mxfp8"
    _want(h, "h", torch.uint8 if fp8 else torch.bfloat16, 2)
    _want(group_offsets, "group_offsets", torch.int32, 1)
    R_cap = h.shape[0]
    if y_perm is None:
        y_perm = _empty((R_cap, w.H), torch.bfloat16, h.device, stream)
    st = _lib.load().moe_grouped_gemm_down(
        _ptr(h), _ptr(h_scales), _ptr(w.w2), _ptr(w.w2_scales), _dt_code(w.precision), _ptr(group_offsets),
        w.E, w.H, w.F, R_cap, _ptr(y_perm), _stream(stream))
    _check("moe_grouped_gemm_down", st)
    return y_perm


# ---------------------------------------------------------------------- NVFP4
def moe_amax_bf16(x: torch.Tensor, *, valid_rows: Optional[torch.Tensor] = None, amax: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """max |x| over the rows of a bf16 matrix (over the first *valid_rows rows when that device int
    is given) -> amax [1] fp32 on the device."""
    _want(x, "x", torch.bfloat16, None)
    x2 = x.reshape(-1, x.shape[-1])
    if amax is None:
        amax = _empty((1,), torch.float32, x.device, stream)
    st = _lib.load().moe_amax_bf16(_ptr(x2), x2.shape[0], x2.shape[1], _ptr(valid_rows), _ptr(amax), _stream(stream))
    _check("moe_amax_bf16", st)
    return amax


def moe_quant_nvfp4(x: torch.Tensor, amax: torch.Tensor, *, valid_rows: Optional[torch.Tensor] = None,
                    q: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, stream=None):
    """Row-wise NVFP4 of a bf16 matrix [..., C] with the tensor encode scale of the device amax ->
    (q [..., C/2] uint8 packed E2M1, scales [..., C/16] uint8 E4M3)."""
    _want(x, "x", torch.bfloat16, None)
    C_ = x.shape[-1]
    if q is None:
        q = _empty(x.shape[:-1] + (C_ // 2,), torch.uint8, x.device, stream)
    if scales is None:
        scales = _empty(x.shape[:-1] + (C_ // 16,), torch.uint8, x.device, stream)
    rows = x.numel() // C_
    st = _lib.load().moe_quant_nvfp4(_ptr(x), rows, C_, _ptr(valid_rows), _ptr(amax), _ptr(q), _ptr(scales),
                                     _stream(stream))
    _check("moe_quant_nvfp4", st)
    return q, scales


class Nvfp4Weights(NamedTuple):
    E: int
    H: int
    F: int
    w13: torch.Tensor          # [E, 2F, H/2] packed E2M1 (the layout of PackedWeights.w13)
    w13_scales: torch.Tensor   # [E, 2F, H/16] E4M3
    w13_amax: torch.Tensor     # [1] fp32
    w2: torch.Tensor           # [E, H, F/2]
    w2_scales: torch.Tensor    # [E, H, F/16]
    w2_amax: torch.Tensor      # [1] fp32


def moe_prepare_weights_nvfp4(w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor, stream=None,
                              out: Optional[Nvfp4Weights] = None) -> Nvfp4Weights:
    """Pack the logical weights (bf16) into the grouped GEMMs' layouts and quantise each stacked tensor
    row-wise to NVFP4 along its contraction dimension, with its own amax: into new buffers, or into those of out."""
    pw = moe_prepare_weights(w1, w3, w2, "bf16", stream=stream)
    E, H, F = pw.E, pw.H, pw.F
    o = Nvfp4Weights(E, H, F, *[None] * 6) if out is None else out
    if out is not None:
        u8, f32 = torch.uint8, torch.float32
        _want_packed(out, Nvfp4Weights, ((E, H, F), (
            (u8, (E, 2 * F, H // 2)), (u8, (E, 2 * F, H // 16)), (f32, (1,)),
            (u8, (E, H, F // 2)), (u8, (E, H, F // 16)), (f32, (1,)))), w1.get_device())
    a13 = moe_amax_bf16(pw.w13, amax=o.w13_amax, stream=stream)
    q13, s13 = moe_quant_nvfp4(pw.w13, a13, q=o.w13, scales=o.w13_scales, stream=stream)
    a2 = moe_amax_bf16(pw.w2, amax=o.w2_amax, stream=stream)
    q2, s2 = moe_quant_nvfp4(pw.w2, a2, q=o.w2, scales=o.w2_scales, stream=stream)
    return Nvfp4Weights(E, H, F, q13, s13, a13, q2, s2, a2)


def moe_grouped_gemm_up_nvfp4(x_q: torch.Tensor, x_scales: torch.Tensor, x_amax: torch.Tensor, w: Nvfp4Weights,
                              group_offsets: torch.Tensor, *, h: Optional[torch.Tensor] = None,
                              h_amax: Optional[torch.Tensor] = None, ab: Optional[torch.Tensor] = None,
                              stream=None):
    """NVFP4 x [R_cap, H/2] -> (h [R_cap, F] bf16 = silu(x W1) * (x W3), h_amax [1] fp32)."""
    R_cap = x_q.shape[0]
    if h is None:
        h = _empty((R_cap, w.F), torch.bfloat16, x_q.device, stream)
    if h_amax is None:
        h_amax = _empty((1,), torch.float32, x_q.device, stream)
    st = _lib.load().moe_grouped_gemm_up_nvfp4(
        _ptr(x_q), _ptr(x_scales), _ptr(x_amax), _ptr(w.w13), _ptr(w.w13_scales), _ptr(w.w13_amax),
        _ptr(group_offsets), w.E, w.H, w.F, R_cap, _ptr(h), _ptr(h_amax), _ptr(ab), _stream(stream))
    _check("moe_grouped_gemm_up_nvfp4", st)
    return h, h_amax


def moe_grouped_gemm_down_nvfp4(h_q: torch.Tensor, h_scales: torch.Tensor, h_amax: torch.Tensor, w: Nvfp4Weights,
                                group_offsets: torch.Tensor, *, y_perm: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """NVFP4 h [R_cap, F/2] -> y_perm [R_cap, H] bf16 = h W2."""
    R_cap = h_q.shape[0]
    if y_perm is None:
        y_perm = _empty((R_cap, w.H), torch.bfloat16, h_q.device, stream)
    st = _lib.load().moe_grouped_gemm_down_nvfp4(
        _ptr(h_q), _ptr(h_scales), _ptr(h_amax), _ptr(w.w2), _ptr(w.w2_scales), _ptr(w.w2_amax),
        _ptr(group_offsets), w.E, w.H, w.F, R_cap, _ptr(y_perm), _stream(stream))
    _check("moe_grouped_gemm_down_nvfp4", st)
    return y_perm


class BwdWeights(NamedTuple):
    precision: str
    E: int
    H: int
    F: int
    w2b: torch.Tensor                   # [E, F, H] bf16 or uint8
    w2b_scales: Optional[torch.Tensor]  # [E, F, H/32]
    w13t: torch.Tensor                  # [E, H, 2F]
    w13t_scales: Optional[torch.Tensor]  # [E, H, 2F/32]


def moe_prepare_weights_bwd(w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor, precision: str = "bf16",
                            stream=None, out: Optional[BwdWeights] = None) -> BwdWeights:
    """Pack logical W1, W3 [E, H, F] and W2 [E, F, H] for the backward GEMMs: into new buffers, or into those of out."""
    for t, n in ((w1, "w1"), (w3, "w3"), (w2, "w2")):
        _want(t, n, torch.bfloat16, 3)
    E, H, F = w1.shape
    dev = w1.device
    fp8 = precision == "mxfp8"
    pdt = torch.uint8 if fp8 else torch.bfloat16
    if out is None:
        w2b = _empty((E, F, H), pdt, dev, stream)
        w13t = _empty((E, H, 2 * F), pdt, dev, stream)
        s2 = _empty((E, F, H // 32), torch.uint8, dev, stream) if fp8 else None
        s13 = _empty((E, H, 2 * F // 32), torch.uint8, dev, stream) if fp8 else None
        out = BwdWeights(precision, E, H, F, w2b, s2, w13t, s13)
    else:
        u8 = torch.uint8
        _want_packed(out, BwdWeights, ((precision, E, H, F), (
            (pdt, (E, F, H)), (u8, (E, F, H // 32)) if fp8 else None,
            (pdt, (E, H, 2 * F)), (u8, (E, H, 2 * F // 32)) if fp8 else None)), w1.get_device())
    st = _lib.load().moe_prepare_weights_bwd(_ptr(w1), _ptr(w3), _ptr(w2), E, H, F, _dt_code(precision),
                                             _ptr(out.w2b), _ptr(out.w2b_scales), _ptr(out.w13t),
                                             _ptr(out.w13t_scales), _stream(stream))
    _check("moe_prepare_weights_bwd", st)
    return out


def moe_grouped_swiglu_dgrad(dy: torch.Tensor, dy_scales: Optional[torch.Tensor], bw: BwdWeights,
                             ab: torch.Tensor, group_offsets: torch.Tensor, *, dab: Optional[torch.Tensor] = None,
                             dab_q: Optional[torch.Tensor] = None, dab_scales: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """dy [R_cap, H] (bf16 or MXFP8 codes) -> dab [R_cap, 2F] bf16 (da | db interleaved per 128).
    With dab_q [R_cap, 2F] uint8 and dab_scales [R_cap, 2F/32] uint8 given, the epilogue also
    writes the row-wise MXFP8 codes and scales of dab into them."""
    R_cap = dy.shape[0]
    if dab is None:
        dab = _empty((R_cap, 2 * bw.F), torch.bfloat16, dy.device, stream)
    if (dab_q is None) != (dab_scales is None):
        raise ValueError("dab_q and dab_scales go together")
    if dab_q is not None:
        _want(dab_q, "dab_q", torch.uint8, 2)
        _want(dab_scales, "dab_scales", torch.uint8, 2)
        if tuple(dab_q.shape) != (R_cap, 2 * bw.F) or tuple(dab_scales.shape) != (R_cap, 2 * bw.F // 32):
            raise ValueError("dab_q must be [R_cap, 2F] and dab_scales [R_cap, 2F/32]")
    st = _lib.load().moe_grouped_swiglu_dgrad(
        _ptr(dy), _ptr(dy_scales), _ptr(bw.w2b), _ptr(bw.w2b_scales), _ptr(ab), _dt_code(bw.precision),
        _ptr(group_offsets), bw.E, bw.H, bw.F, R_cap, _ptr(dab), _ptr(dab_q), _ptr(dab_scales), _stream(stream))
    _check("moe_grouped_swiglu_dgrad", st)
    return dab


def moe_grouped_gemm_dx(dab: torch.Tensor, dab_scales: Optional[torch.Tensor], bw: BwdWeights,
                        group_offsets: torch.Tensor, *, dx: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """dab [R_cap, 2F] (bf16 or MXFP8 codes) -> dx [R_cap, H] bf16."""
    R_cap = dab.shape[0]
    if dx is None:
        dx = _empty((R_cap, bw.H), torch.bfloat16, dab.device, stream)
    st = _lib.load().moe_grouped_gemm_dx(
        _ptr(dab), _ptr(dab_scales), _ptr(bw.w13t), _ptr(bw.w13t_scales), _dt_code(bw.precision),
        _ptr(group_offsets), bw.E, bw.H, bw.F, R_cap, _ptr(dx), _stream(stream))
    _check("moe_grouped_gemm_dx", st)
    return dx


def moe_grouped_transpose_kpad(R_cap: int, E: int) -> int:
    return int(_lib.load().moe_grouped_transpose_kpad(R_cap, E))


def moe_grouped_transpose(x: torch.Tensor, group_offsets: torch.Tensor, precision: str = "bf16", *,
                          R_cap: Optional[int] = None, src_rows: Optional[torch.Tensor] = None,
                          xT: Optional[torch.Tensor] = None, xT_scales: Optional[torch.Tensor] = None,
                          stream=None):
    """Group-padded transposed weight-gradient operand [C, Kpad] (bf16, or MXFP8 + scales)."""
    _want(x, "x", torch.bfloat16, 2)
    C = x.shape[1]
    if R_cap is None:
        R_cap = x.shape[0]
    E = group_offsets.numel() - 1
    kpad = moe_grouped_transpose_kpad(R_cap, E)
    fp8 = precision == "mxfp8"
    if xT is None:
        xT = _empty((C, kpad), torch.uint8 if fp8 else torch.bfloat16, x.device, stream)
    if fp8 and xT_scales is None:
        xT_scales = _empty((C, kpad // 32), torch.uint8, x.device, stream)
    st = _lib.load().moe_grouped_transpose(_ptr(x), _ptr(src_rows), R_cap, C, _ptr(group_offsets), E,
                                           _dt_code(precision), _ptr(xT), _ptr(xT_scales), _stream(stream))
    _check("moe_grouped_transpose", st)
    return xT, xT_scales


def moe_grouped_gemm_wgrad(aT: torch.Tensor, aT_scales: Optional[torch.Tensor], bT: torch.Tensor,
                           bT_scales: Optional[torch.Tensor], precision: str, group_offsets: torch.Tensor,
                           R_cap: int, *, split: bool = False, dw: Optional[torch.Tensor] = None,
                           dw2: Optional[torch.Tensor] = None, stream=None):
    """dW[e] = sum over group e's rows of a^T b, from transposed operands [M, Kpad], [N, Kpad]."""
    M, N = aT.shape[0], bT.shape[0]
    E = group_offsets.numel() - 1
    dev = aT.device
    if split:
        if dw is None:
            dw = _empty((E, M, N // 2), torch.bfloat16, dev, stream)
        if dw2 is None:
            dw2 = _empty((E, M, N // 2), torch.bfloat16, dev, stream)
    elif dw is None:
        dw = _empty((E, M, N), torch.bfloat16, dev, stream)
    st = _lib.load().moe_grouped_gemm_wgrad(
        _ptr(aT), _ptr(aT_scales), _ptr(bT), _ptr(bT_scales), _dt_code(precision), _ptr(group_offsets), E, M, N,
        R_cap, _ptr(dw), _ptr(dw2 if split else None), _stream(stream))
    _check("moe_grouped_gemm_wgrad", st)
    return (dw, dw2) if split else dw


# ---------------------------------------------------------- the layer for a few tokens
def moe_layer_few_tokens_workspace(w: PackedWeights, T: int, K: int, stream=None) -> torch.Tensor:
    """The workspace of moe_layer_few_tokens for up to T tokens (uninitialised, reusable; stream: the one of
    the first call that uses it)."""
    n = _lib.load().moe_layer_few_tokens_workspace_size(T, K, w.E, w.H, w.F, _dt_code(w.precision))
    return _empty(int(n), torch.uint8, w.w13.device, stream)


def moe_layer_few_tokens(x: torch.Tensor, logits: Optional[torch.Tensor], w: PackedWeights, K: int, *,
                         renorm: bool = False, id_dtype=torch.int32, ids: Optional[torch.Tensor] = None,
                         probs: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """The whole layer for T <= 64 tokens: x [T, H] bf16, logits [T, E] fp32 -> (y [T, H] bf16,
    ids [T, K], probs [T, K]). With logits None, ids and probs are the caller's routes instead."""
    _want(x, "x", torch.bfloat16, 2)
    T, H = x.shape
    dev = x.get_device()
    if H != w.H:
        raise ValueError(f"x must have {w.H} columns")
    if logits is not None:
        _like(logits, "logits", torch.float32, (T, w.E), dev)
    elif ids is None or probs is None:
        raise ValueError("without logits, ids and probs are inputs")
    if ids is None:
        ids = _empty((T, K), id_dtype, x.device, stream)
    else:
        _like(ids, "ids", ids.dtype, (T, K), dev)
    if probs is None:
        probs = _empty((T, K), torch.float32, x.device, stream)
    else:
        _like(probs, "probs", torch.float32, (T, K), dev)
    if y is None:
        y = _empty_like(x, stream)
    else:
        _like(y, "y", torch.bfloat16, (T, H), dev)
    if workspace is None:
        workspace = moe_layer_few_tokens_workspace(w, T, K, stream)
    else:
        _scratch(workspace, dev)
    w13, s13, w2, s2 = w.w13, w.w13_scales, w.w2, w.w2_scales
    if w13.get_device() != dev or w2.get_device() != dev or not (
            s13 is None or s13.get_device() == dev) or not (s2 is None or s2.get_device() == dev):
        raise ValueError(f"the weights must be on cuda:{dev}, x's device")
    st = _lib.load().moe_layer_few_tokens(
        x.data_ptr(), T, H, _at(logits), K, w.E, w.F, w13.data_ptr(), _at(s13), w2.data_ptr(), _at(s2),
        _dt_code(w.precision), ids.data_ptr(), _id_code(ids.dtype), probs.data_ptr(), y.data_ptr(),
        MOE_ROUTE_RENORM if renorm else 0, workspace.data_ptr(), workspace.numel(), _raw_stream(stream, x))
    _check("moe_layer_few_tokens", st)
    return y, ids, probs


# ----------------------------------------------------------------- layer norm
_FLOAT_CODES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}


def _float_code(t: torch.Tensor, name: str) -> int:
    code = _FLOAT_CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _like(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape, dev: int) -> None:
    """t, where given, is a contiguous tensor of this type and shape on this CUDA device."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        return
    _want(t, name, dtype, None)
    _on(dev, t, name)
    raise ValueError(f"{name} must be {list(shape)}")


class LayerNormed(NamedTuple):
    y: torch.Tensor                 # [T, H]
    sum: torch.Tensor               # [T, H] the normalised stream: x + residual (x itself without one)
    mean: torch.Tensor              # [T] fp32
    rstd: torch.Tensor              # [T] fp32


def moe_layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5, *,
                   residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                   sum: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                   rstd: Optional[torch.Tensor] = None, stream=None) -> LayerNormed:
    """Layer norm of x (+ residual) [T, H] bf16 or fp32 with weight (and bias) [H] bf16 or fp32."""
    _want(x, "x", None, 2)
    shape, dtype = x.shape, x.dtype
    T, H = shape
    dev = x.get_device()
    code, wcode = _float_code(x, "x"), _float_code(weight, "weight")
    _like(weight, "weight", weight.dtype, (H,), dev)
    _like(bias, "bias", weight.dtype, (H,), dev)
    _like(residual, "residual", dtype, shape, dev)
    if y is None:
        y = _empty_like(x, stream)
    else:
        _like(y, "y", dtype, shape, dev)
    if sum is not None:
        if residual is None:
            raise ValueError("sum goes with residual")
        _like(sum, "sum", dtype, shape, dev)
    elif residual is not None:
        sum = _empty_like(x, stream)
    if mean is None:
        mean = _empty(T, torch.float32, x.device, stream)
    else:
        _like(mean, "mean", torch.float32, (T,), dev)
    if rstd is None:
        rstd = _empty(T, torch.float32, x.device, stream)
    else:
        _like(rstd, "rstd", torch.float32, (T,), dev)
    st = _lib.load().moe_layer_norm(x.data_ptr(), _at(residual), T, H, code, weight.data_ptr(), _at(bias), wcode, eps,
                                    _at(sum), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _raw_stream(stream, x))
    _check("moe_layer_norm", st)
    return LayerNormed(y, x if residual is None else sum, mean, rstd)


def moe_layer_norm_backward_workspace_size(T: int, H: int) -> int:
    return int(_lib.load().moe_layer_norm_backward_workspace_size(T, H))


def moe_layer_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                            rstd: torch.Tensor, *, dx_add: Optional[torch.Tensor] = None,
                            dx: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                            dbias: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            stream=None):
    """dy, s [T, H] (s: LayerNormed.sum), mean, rstd [T] -> (dx [T, H], dweight [H], dbias [H]);
    dx_add [T, H]: the gradient that reaches s past the norm, added to dx."""
    _want(s, "s", None, 2)
    shape, dtype, wdtype = s.shape, s.dtype, weight.dtype
    T, H = shape
    dev = s.get_device()
    code, wcode = _float_code(s, "s"), _float_code(weight, "weight")
    if dy is None or mean is None or rstd is None:
        raise ValueError("dy, mean and rstd must be given")
    _like(weight, "weight", wdtype, (H,), dev)
    _like(dy, "dy", dtype, shape, dev)
    _like(mean, "mean", torch.float32, (T,), dev)
    _like(rstd, "rstd", torch.float32, (T,), dev)
    _like(dx_add, "dx_add", dtype, shape, dev)
    if dx is None:
        dx = _empty_like(s, stream)
    else:
        _like(dx, "dx", dtype, shape, dev)
    if dweight is None:
        dweight = _empty_like(weight, stream)
    else:
        _like(dweight, "dweight", wdtype, (H,), dev)
    if dbias is None:
        dbias = _empty_like(weight, stream)
    else:
        _like(dbias, "dbias", wdtype, (H,), dev)
    if workspace is None:
        workspace = _empty(moe_layer_norm_backward_workspace_size(T, H), torch.uint8, s.device, stream)
    else:
        _scratch(workspace, dev)
    st = _lib.load().moe_layer_norm_backward(dy.data_ptr(), s.data_ptr(), T, H, code, weight.data_ptr(), wcode,
                                             mean.data_ptr(), rstd.data_ptr(), _at(dx_add), dx.data_ptr(),
                                             dweight.data_ptr(), dbias.data_ptr(), workspace.data_ptr(),
                                             workspace.numel(), _raw_stream(stream, s))
    _check("moe_layer_norm_backward", st)
    return dx, dweight, dbias


# ------------------------------------------------------- gradient norm, clipping
def _grad_norm_clip(grads, outs, max_norm, eps, norm, workspace, stream):
    # (the lists can be long: each check is one pass over them)
    n = len(grads)
    devices = set(map(torch.Tensor.get_device, grads))
    if -1 in devices:
        raise ValueError("gradients must be CUDA tensors")
    dev = norm.get_device() if norm is not None else grads[0].get_device() if n else -1
    if devices and devices != {dev}:
        raise ValueError("gradients and norm must be on one device")
    if not all(map(torch.Tensor.is_contiguous, grads)):
        raise ValueError("gradients must be contiguous")
    dtypes = [t.dtype for t in grads]
    codes = [_FLOAT_CODES.get(d) for d in dtypes]
    if None in codes:
        raise ValueError("gradients must be bfloat16 or float32")
    counts = list(map(torch.Tensor.numel, grads))
    ptrs = array("q", map(torch.Tensor.data_ptr, grads))
    out_at = None
    if outs is grads:
        out_at = ptrs.buffer_info()[0]
    elif outs is not None:
        if len(outs) != n:
            raise ValueError("out must have one tensor per gradient")
        if list(map(torch.Tensor.numel, outs)) != counts or [t.dtype for t in outs] != dtypes:
            raise ValueError("outputs must have the gradients' sizes and types")
        if set(map(torch.Tensor.get_device, outs)) - {dev} or not all(map(torch.Tensor.is_contiguous, outs)):
            raise ValueError("outputs must be contiguous CUDA tensors on the gradients' device")
        optrs = array("q", map(torch.Tensor.data_ptr, outs))
        out_at = optrs.buffer_info()[0]
    if norm is None:
        if n == 0:
            raise ValueError("no gradients: pass norm, the tensor to write")
        norm = _empty(1, torch.float32, grads[0].device, stream)
    else:
        _want(norm, "norm", torch.float32, None)
        if norm.numel() != 1:
            raise ValueError("norm must hold one value")
    L = _lib.load()
    if workspace is None:
        workspace = _empty(L.moe_grad_norm_workspace_size(n), torch.uint8, norm.device, stream)
    else:
        _scratch(workspace, dev)
    counts, codes = array("q", counts), array("i", codes)
    st = L.moe_grad_norm_clip(ptrs.buffer_info()[0], counts.buffer_info()[0], codes.buffer_info()[0], out_at, n,
                              max_norm, eps, norm.data_ptr(), workspace.data_ptr(), workspace.numel(),
                              _raw_stream(stream, norm))
    _check("moe_grad_norm_clip", st)
    return norm


def moe_grad_norm(grads, *, norm: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """sqrt of the sum of squares over a list of bf16 / fp32 tensors -> norm [1] fp32 (on the device)."""
    return _grad_norm_clip(grads, None, 0.0, 0.0, norm, workspace, stream)


def moe_grad_clip(grads, max_norm: float, *, eps: float = 1e-6, out=None, norm: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scale the gradients by min(1, max_norm / (norm + eps)), norm being their global norm (1 where
    norm + eps is within max_norm, 0 and inf included): in place, or into the tensors of out. Returns the norm before clipping ([1] fp32, on the device)."""
    return _grad_norm_clip(grads, grads if out is None else out, max_norm, eps, norm, workspace, stream)
