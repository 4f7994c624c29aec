"""Refusals of the paged cache, its attention and the beam selection that need no GPU: bad shapes, types, pointers and
workspaces return a status before any CUDA call (1 invalid argument, 2 unsupported, 3 workspace, 5 alignment), and
tensors of different devices are refused before the library is called."""
import ctypes as C

import pytest
import torch

from dropless_moe_expert_router_gb300 import _lib, api

P = C.c_void_p(4096)             # stands for a buffer: never dereferenced on these paths
ODD = C.c_void_p(4097)
I16, BF16, MXFP8, F32 = 0, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from dropless_moe_expert_router_gb300 import build
    build.build()
    return _lib.load()


CACHE = dict(dtype=BF16, pages=10, heads=2, page=16, dim=64, kp=P, ks=P, vp=P, vs=P)


def _append(lib, k=P, v=P, kstride=128, vstride=128, n=3, rows=None, pos=P, table=P, S=4, M=5, **kw):
    c = dict(CACHE, **kw)
    return lib.moe_cache_append(k, v, kstride, vstride, n, rows, pos, table, S, M, c["dtype"], c["pages"], c["heads"],
                                c["page"], c["dim"], c["kp"], c["ks"], c["vp"], c["vs"], None)


def _gather(lib, k=P, v=P, n=3, rows=None, pos=P, table=P, S=4, M=5, **kw):
    c = dict(CACHE, **kw)
    return lib.moe_cache_gather(k, v, n, rows, pos, table, S, M, c["dtype"], c["pages"], c["heads"], c["page"], c["dim"],
                                c["kp"], c["ks"], c["vp"], c["vs"], None)


@pytest.mark.parametrize("call", [_append, _gather])
def test_rows(lib, call):
    assert call(lib, n=0) == 0
    assert call(lib, n=-1) == 1 and call(lib, S=-1) == 1 and call(lib, n=5) == 1          # more tokens than sequences
    for bad in (dict(dtype=F32), dict(pages=0), dict(heads=0), dict(page=0), dict(dim=0), dict(M=0), dict(kp=None), dict(vp=None)):
        assert call(lib, **bad) == 1, bad
    assert call(lib, dtype=MXFP8, ks=None) == 1 and call(lib, dtype=MXFP8, vs=None) == 1
    for bad in (dict(dim=40), dict(dim=272), dict(dtype=MXFP8, dim=48), dict(page=4097), dict(M=1 << 28),
                dict(n=(1 << 30) + 1, rows=P)):
        assert call(lib, **bad) == 2, bad
    for name in ("k", "v", "pos", "table"):
        assert call(lib, **{name: None}) == 1
        assert call(lib, **{name: ODD}) == 5
    for name in ("kp", "vp", "rows"):
        assert call(lib, **{name: ODD}) == 5
    assert call(lib, dtype=MXFP8, ks=ODD) == 5
    if call is _append:
        assert call(lib, kstride=132) == 5 and call(lib, vstride=4) == 5


def _attention(lib, q=P, stride=512, B=2, qh=8, table=P, M=5, lengths=P, scale=0.1, window=0, out=P, lse=P, ws=P, nbytes=1 << 40,
               **kw):
    c = dict(CACHE, **kw)
    return lib.moe_paged_attention(q, stride, B, qh, c["kp"], c["ks"], c["vp"], c["vs"], c["dtype"], c["pages"], c["heads"],
                                   c["page"], c["dim"], table, M, lengths, scale, window, out, lse, ws, nbytes, None)


def test_attention(lib):
    assert _attention(lib, B=0) == 0
    for bad in (dict(B=-1), dict(qh=0), dict(qh=7), dict(window=-1), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(dtype=I16), dict(M=0), dict(heads=0)):
        assert _attention(lib, **bad) == 1, bad
    for bad in (dict(B=65536), dict(qh=4096), dict(dim=24), dict(dim=512), dict(page=5000)):
        assert _attention(lib, **bad) == 2, bad
    for name in ("q", "table", "lengths", "out"):
        assert _attention(lib, **{name: None}) == 1
        assert _attention(lib, **{name: ODD}) == 5
    assert _attention(lib, lse=ODD) == 5 and _attention(lib, ws=ODD) == 5 and _attention(lib, stride=516) == 5
    assert _attention(lib, ws=None) == 3
    size = lib.moe_paged_attention_workspace_size
    assert _attention(lib, nbytes=size(2, 8, 2, 64) - 1) == 3
    assert size(65536, 8, 2, 64) == 0 and size(2, 7, 2, 64) == 0 and size(2, 8, 2, 257) == 0 and size(-1, 8, 2, 64) == 0
    assert size(0, 8, 2, 64) > 0


def _fork(lib, table=P, lengths=P, S=4, M=5, parents=P, S_new=6, pages=10, page=16, room=1, rooms=None, nt=P, nl=P, src=P, dst=P,
          used=P, ws=P, nbytes=1 << 40):
    return lib.moe_cache_fork(table, lengths, S, M, parents, S_new, pages, page, room, rooms, nt, nl, src, dst, used, ws, nbytes,
                              None)


def _compact(lib, table=P, S=4, M=5, pages=10, nt=P, src=P, dst=P, used=P, ws=P, nbytes=1 << 40):
    return lib.moe_cache_compact(table, S, M, pages, nt, src, dst, used, ws, nbytes, None)


def test_pages(lib):
    for bad in (dict(S=-1), dict(S_new=-1), dict(M=0), dict(pages=0), dict(page=0), dict(page=4097), dict(parents=None),
                dict(S_new=1 << 28), dict(M=1 << 28), dict(S_new=1 << 20, M=1 << 12, page=8)):
        assert _fork(lib, **bad) == 1, bad
    for name in ("table", "lengths", "nt", "nl", "src", "dst", "used"):
        assert _fork(lib, **{name: None}) == 1
        assert _fork(lib, **{name: ODD}) == 5
    assert _fork(lib, rooms=ODD) == 5 and _fork(lib, parents=ODD) == 5 and _fork(lib, ws=ODD) == 5 and _fork(lib, ws=None) == 3
    size = lib.moe_cache_pages_workspace_size
    assert _fork(lib, nbytes=size(10, 6) - 1) == 3
    for bad in (dict(S=-1), dict(M=0), dict(pages=0), dict(table=None), dict(nt=None), dict(src=None), dict(dst=None), dict(used=None)):
        assert _compact(lib, **bad) == 1, bad
    assert _compact(lib, S=1 << 20, M=1 << 12) == 2
    for name in ("table", "nt", "src", "dst", "used", "ws"):
        assert _compact(lib, **{name: ODD}) == 5
    assert _compact(lib, ws=None) == 3 and _compact(lib, nbytes=size(10, 0) - 1) == 3
    assert size(0, 5) == 0 and size(5, -1) == 0

    def copy(ptrs=(4096, 8192), sizes=(64, 3), m=2, src=P, dst=P, n=4, pages=5):
        return lib.moe_cache_copy_pages((C.c_void_p * len(ptrs))(*ptrs), (C.c_longlong * len(sizes))(*sizes), m, src, dst, n, pages,
                                        None)
    assert copy(n=0) == 0
    for bad in (dict(n=-1), dict(m=-1), dict(pages=0), dict(src=None), dict(dst=None), dict(ptrs=(4096, None)), dict(sizes=(64, 0))):
        assert copy(**bad) == 1, bad
    assert copy(sizes=(64, 1 << 33)) == 2 and copy(src=ODD) == 5 and copy(dst=ODD) == 5


def test_beams(lib):
    def beam(logits=P, dtype=F32, scores=P, done=None, pad=0, N=2, W=3, V=50, K=4, out=P, parents=P, tokens=P, ws=P, nbytes=1 << 40):
        return lib.moe_beam_select(logits, dtype, scores, done, pad, N, W, V, K, out, parents, tokens, ws, nbytes, None)
    assert beam(N=0) == 0
    for bad in (dict(dtype=MXFP8), dict(N=-1), dict(W=0), dict(V=0), dict(K=0), dict(V=1, K=4), dict(done=P, pad=-1), dict(done=P, pad=50)):
        assert beam(**bad) == 1, bad
    for bad in (dict(W=65), dict(V=1 << 24), dict(K=65), dict(N=1 << 23)):
        assert beam(**bad) == 2, bad
    for name in ("logits", "scores", "out", "parents", "tokens"):
        assert beam(**{name: None}) == 1
        assert beam(**{name: ODD}) == 5
    size = lib.moe_beam_select_workspace_size
    assert beam(ws=None) == 3 and beam(ws=ODD) == 5 and beam(nbytes=size(2, 3, 50, 4) - 1) == 3
    assert size(2, 65, 50, 4) == 0 and size(2, 3, 50, 65) == 0 and size(0, 3, 50, 4) > 0


def test_more_pages_than_strides_over_them_can_count(lib):
    """A stride of 8192 threads would pass 2^31 from the last pages on, and mark what lies before the workspace."""
    for pages in ((1 << 30) + 1, (1 << 31) - 1):
        assert _fork(lib, pages=pages) == 2 and _compact(lib, pages=pages) == 2


def test_more_pairs_than_their_number_can_count(lib):
    """The list's last 2048 pairs would be followed by those before its beginning."""
    one = (C.c_void_p * 1)(4096), (C.c_longlong * 1)(64)
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        assert lib.moe_cache_copy_pages(*one, 1, P, P, n, 5, None) == 2


# ------------------------------------------------------------------ devices
class _Cuda(torch.Tensor):
    """A CPU tensor that says it is on the CUDA device `at`."""
    is_cuda = True


def _t(shape, dtype, at=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(_Cuda)
    t.at = at
    return t


@pytest.fixture
def no_call(monkeypatch):
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


def test_devices(no_call):
    BF, U8, I32, FL = torch.bfloat16, torch.uint8, torch.int32, torch.float32
    pools = dict(k=_t((5, 2, 4, 32), U8), ks=_t((5, 2, 4, 1), U8), v=_t((5, 2, 4, 32), U8), vs=_t((5, 2, 4, 1), U8))

    def cache(k, ks, v, vs):
        return api.PagedCache("mxfp8", 5, 2, 4, 32, k, ks, v, vs)
    new = dict(nk=_t((3, 2, 32), BF), nv=_t((3, 2, 32), BF), table=_t((4, 2), I32), pos=_t((3,), I32), rows=_t((3,), I32))
    _each_elsewhere(lambda nk, nv, table, pos, rows, **c: api.moe_cache_append(nk, nv, cache(**c), table, pos, rows=rows),
                    dict(new, **pools))
    _each_elsewhere(lambda nk, nv, table, pos, rows, **c: api.moe_cache_gather(cache(**c), table, pos, rows=rows, k=nk, v=nv),
                    dict(new, **pools))
    att = dict(q=_t((3, 4, 32), BF), table=_t((3, 2), I32), lengths=_t((3,), I32), out=_t((3, 4, 32), BF), lse=_t((3, 4), FL),
               workspace=_t((64,), U8))
    _each_elsewhere(lambda q, table, lengths, out, lse, workspace, **c: api.moe_paged_attention(
        q, cache(**c), table, lengths, out=out, lse=lse, workspace=workspace), dict(att, **pools))

    def fork(table, lengths, parents, room, workspace, **out):
        return api.moe_cache_fork(table, lengths, parents, 5, 4, room=room, workspace=workspace, out=api.CacheFork(**{
            k[1:]: v for k, v in out.items()}))
    _each_elsewhere(fork, dict(table=_t((3, 2), I32), lengths=_t((3,), I32), parents=_t((4,), I32), room=_t((4,), I32),
                               workspace=_t((64,), U8), otable=_t((4, 2), I32), olengths=_t((4,), I32), osrc=_t((4,), I32),
                               odst=_t((4,), I32), oused=_t((1,), I32)))
    _each_elsewhere(lambda table, workspace, **out: api.moe_cache_compact(table, 5, workspace=workspace, out=api.CacheCompact(**{
        k[1:]: v for k, v in out.items()})), dict(table=_t((3, 2), I32), workspace=_t((64,), U8), otable=_t((3, 2), I32),
                                                  osrc=_t((2,), I32), odst=_t((2,), I32), oused=_t((1,), I32)))
    _each_elsewhere(lambda src, dst, **c: api.moe_cache_copy_pages(cache(**c), src, dst),
                    dict(pools, src=_t((3,), I32), dst=_t((3,), I32)))
    _each_elsewhere(lambda logits, scores, done, workspace, **out: api.moe_beam_select(
        logits, scores, 4, done=done, workspace=workspace, out=api.BeamSelected(**{k[1:]: v for k, v in out.items()})),
        dict(logits=_t((2, 3, 50), FL), scores=_t((2, 3), FL), done=_t((2, 3), torch.bool), workspace=_t((64,), U8),
             oscores=_t((2, 4), FL), oparents=_t((2, 4), I32), otokens=_t((2, 4), I32)))


@pytest.mark.parametrize("big", [1 << 32, -(1 << 32), (1 << 31), -(1 << 31) - 1])
def test_numbers_that_32_bits_do_not_hold(no_call, big):
    """big + 5 would reach the library as 5, or with another sign."""
    BF, I32, FL = torch.bfloat16, torch.int32, torch.float32
    n = big + 5 if abs(big) == 1 << 32 else big
    cache = api.PagedCache("bf16", 5, 2, 4, 32, _t((5, 2, 4, 32), BF), None, _t((5, 2, 4, 32), BF), None)
    q, table, lengths = _t((3, 4, 32), BF), _t((3, 2), I32), _t((3,), I32)
    given = dict(out=_t((3, 4, 32), BF), lse=_t((3, 4), FL), workspace=_t((64,), torch.uint8))
    if n < 0:                                                 # (above: all positions)
        with pytest.raises(ValueError):
            api.moe_paged_attention(q, cache, table, lengths, window=n, **given)
    fork = api.CacheFork(_t((3, 2), I32), *[_t((3,), I32)] * 3, _t((1,), I32))
    for pages, page_size, room in ((n, 4, 1), (5, n, 1), (5, 4, n)):
        with pytest.raises(ValueError):
            api.moe_cache_fork(table, lengths, None, pages, page_size, room=room, out=fork, workspace=given["workspace"])
    with pytest.raises(ValueError):
        api.moe_cache_compact(table, n, workspace=given["workspace"])
    logits, scores = _t((2, 3, 50), FL), _t((2, 3), FL)
    best = api.BeamSelected(_t((2, 4), FL), _t((2, 4), I32), _t((2, 4), I32))
    for K, pad in ((4, n), (n, 0)):
        with pytest.raises(ValueError):
            api.moe_beam_select(logits, scores, K, pad=pad, out=best, workspace=given["workspace"])
    for call in (lambda: api.moe_paged_attention_workspace(cache, n, 4), lambda: api.moe_paged_attention_workspace(cache, 3, n),
                 lambda: api.moe_cache_pages_workspace(n, 3, "cpu"), lambda: api.moe_cache_pages_workspace(5, n, "cpu"),
                 lambda: api.moe_beam_select_workspace(torch.zeros((2, 3, 50)), n)):
        with pytest.raises(ValueError):
            call()
