"""The README's layer example runs as written, after the step's example
whose buffers it uses; its gradient is that of autograd in 64 bits (the
stored 16-bit z, h and dz: 2^-6 in norm)."""
import os
import re

import pytest
import torch

from tests import linear_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_layer_example_runs():
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    blocks = re.findall(r"```(?:python|py)\n(.*?)```", text, flags=re.S)
    assert len(blocks) == 2
    ns = {}
    for b in blocks:
        exec(compile(b, "README.md", "exec"), ns)
    torch.cuda.synchronize()
    x, w, w2, dy = (ns[k].cpu().double() for k in ("x", "w", "w2", "dy"))
    w.requires_grad_(True)
    zz = x @ w.t()
    keep = ref.keep(*zz.shape, 0.1, 1, 1)
    h = torch.where(keep, torch.nn.functional.gelu(zz, approximate="tanh") * ref.scale32(0.1), 0.0)
    ((h @ w2.t()) * dy).sum().backward()
    got = ns["dw"].cpu().double()
    assert float((got - w.grad).norm()) <= 2.0 ** -6 * float(w.grad.norm())
    assert bool(torch.isfinite(ns["dx"]).all()) and bool((ns["row"][ns["n"] * ns["k"]:] == 0).all())
