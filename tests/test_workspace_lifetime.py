"""A workspace that the binding allocates for a call lives until the library
has been called: freed earlier, its block could be handed to another thread's
tensor before the kernels that use it are enqueued (the library is called
without the interpreter's lock).  CPU: the library is replaced by a function
that looks whether the tensor is alive, nothing is launched."""
import contextlib
import weakref

import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from zero_sharded_mixed_flatten_amd import _linear


@pytest.fixture
def made(monkeypatch):
    """weak references to the tensors that torch.empty makes from here on"""
    refs, empty = [], torch.empty

    def spy(*args, **kw):
        t = empty(*args, **kw)
        refs.append(weakref.ref(t))
        return t

    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch, "empty", spy)
    return refs


def _look(made, seen):
    def library(*args):
        seen.append([r() is not None for r in made])
        return 0
    return library


M, N, K = 40, 8, 1 << 16  # few outputs, long contractions: divided


@pytest.mark.parametrize("op", ["linear", "dgrad", "wgrad"])
def test_of_a_product(monkeypatch, made, op):
    a = torch.zeros(1, dtype=torch.bfloat16)
    tall, wide, out = a.expand(M, K), a.expand(N, K), a.expand(M, N)
    seen = []
    monkeypatch.setattr(_linear, "_torch_stream", lambda stream, device: None)
    monkeypatch.setattr(_linear, "_shape", lambda t, what: t.shape)
    monkeypatch.setattr(_linear, "_mat", lambda t, what, shape, dtype, dev: (16, shape[1]))
    library = _look(made, seen)
    monkeypatch.setattr(_linear, "_call", lambda fn, what, dev, stream, *args: library())
    if op == "linear":      # m rows of k, n outputs
        zs.zero_linear(tall, wide, out)
    elif op == "dgrad":     # the contraction is over n
        zs.zero_linear_dgrad(tall, wide.t(), out)
    else:                   # the contraction is over the rows
        zs.zero_linear_wgrad(tall.t(), wide.t(), out)
    assert seen == [[True]]


@pytest.mark.parametrize("name", ["zero_shard_reduce", "zero_shard_step", "zero_shard_step_dc",
                                  "zero_shard_step_q8", "zero_shard_step_q8_dc"])
def test_of_a_sum_of_squares(monkeypatch, made, name):
    n = 1 << 12
    lay, _ = zs.zero_flatten_layout([2 * n], 2)
    seen = []
    for f in ("_buf", "_rows", "_stream", "_torch_stream", "_consts"):
        monkeypatch.setattr(zs, f, lambda *args, **kw: None)
    monkeypatch.setattr(zs._lib, name, _look(made, seen))
    t, ss = torch.zeros(n), torch.zeros(1, dtype=torch.float64)
    hp = zs.AdamWHParams()
    if name == "zero_shard_reduce":
        zs.zero_shard_reduce(t, 2, n, n, t, sumsq=ss)
    elif "q8" in name:
        getattr(zs, name)(t, t, n, n, n, t, t, t, t, t, lay, 0, hp if name.endswith("q8") else t,
                          sumsq=ss)
    else:
        getattr(zs, name)(t, n, n, t, t, t, t.bfloat16(), lay, 0,
                          hp if name.endswith("step") else t, sumsq=ss)
    assert seen == [[True]]
