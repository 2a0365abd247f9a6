"""The README's example of the layer norm and the Muon step runs as written,
after the two before it whose buffers it uses, and does what they say."""
import os
import re

import pytest
import torch

from tests.test_gpu_muon import check_orth, ns64

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_norm_and_muon_example_runs():
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    blocks = re.findall(r"```(?:python3|python|py)\n(.*?)```", text, flags=re.S)
    assert len(blocks) == 3
    ns = {}
    for b in blocks[:2]:
        exec(compile(b, "README.md", "exec"), ns)
    dx0, master0 = ns["dx"].clone(), ns["master"].clone()
    exec(compile(blocks[2], "README.md", "exec"), ns)
    torch.cuda.synchronize()
    n, k, lo, hi, hp = (ns[v] for v in ("n", "k", "lo", "hi", "hp"))
    x = ns["x"].double().requires_grad_(True)
    g = ns["g"].double().requires_grad_(True)
    b = ns["b"].double().requires_grad_(True)
    y = torch.nn.functional.layer_norm(x, (k,), g, b, 1e-5)
    y.backward(dx0.double())
    # fp32 sums of 16-bit inputs, one rounding of at most 2^-8 to bf16
    for got, want in ((ns["xn"], y.detach()), (ns["dx"], x.grad + ns["dstream"].double())):
        assert float((got.double() - want).norm()) <= 2.0 ** -8 * float(want.norm())
    for got, want in ((ns["dg"], g.grad), (ns["db"], b.grad)):
        assert float((got.double() - want).norm()) <= 2.0 ** -18 * float(want.norm())
    u = ns["u"][:n * k].view(n, k)
    assert int(u.count_nonzero()) > 0 and not ns["u"][:lo].any() and not ns["u"][hi:].any()
    check_orth(ns["o"][:n * k].view(n, k), ns64(u))
    step = 0.2 * max(n, k) ** 0.5 * ns["o"][lo:hi].double()
    want = master0.double()
    want[:hi - lo] = want[:hi - lo] * (1 - hp.lr * hp.weight_decay) - hp.lr * step
    assert float((ns["master"].double() - want).abs().max()) <= 2.0 ** -22
    assert torch.equal(ns["weights"][lo:hi], ns["master"][:hi - lo].to(torch.bfloat16))
