"""Memory of calls on a given stream, without a GPU: it is that stream's, and is kept until what the
current stream was given is done too. (An allocation on the current stream, dropped when the call
returns, could be handed on while the given stream's kernels still use it.)"""
import ast
import contextlib
import inspect

import torch

from dropless_moe_expert_router_gb300 import api


class _Tensor:
    def __init__(self, owner):
        self.owner, self.recorded = owner, []

    def record_stream(self, s):
        self.recorded.append(s)


def _fake(monkeypatch):
    at = ["current"]

    @contextlib.contextmanager
    def on(s):
        old, at[0] = at[0], s
        yield
        at[0] = old
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: at[0])
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: _Tensor(at[0]))
    return at


def test_memory_is_the_given_streams(monkeypatch):
    at = _fake(monkeypatch)
    t = api._empty((4,), torch.float32, "cuda", "given")
    assert t.owner == "given" and t.recorded == ["current"] and at == ["current"]
    for s in (None, "current"):
        t = api._empty((4,), torch.float32, "cuda", s)
        assert t.owner == "current" and t.recorded == []


def test_every_call_with_a_stream_allocates_there():
    tree = ast.parse(inspect.getsource(api))
    seen = 0
    for f in tree.body:
        if not isinstance(f, ast.FunctionDef) or f.name in ("_empty", "_empty_like"):
            continue
        takes = "stream" in [a.arg for a in f.args.args + f.args.kwonlyargs]
        for c in ast.walk(f):
            if not isinstance(c, ast.Call):
                continue
            name = ast.unparse(c.func)
            assert not (takes and name.startswith("torch.") and name.split(".")[-1].startswith(("empty", "zeros", "full"))), f.name
            if name in ("_empty", "_empty_like", "permute_buffers", "moe_layer_few_tokens_workspace"):
                seen += 1
                given = [ast.unparse(a) for a in c.args[-1:]] + [ast.unparse(k.value) for k in c.keywords if k.arg == "stream"]
                assert "stream" in given, f.name
    assert seen > 40
