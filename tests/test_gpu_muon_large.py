"""Momentum and update of ranges as long as a shard's: from 2^20 elements on
fewer waves are kept on a CU, and beyond 2^31 a range goes out as several
launches.  Every bit against the same fp32 operations one by one."""
import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from tests.test_gpu_muon import momentum_cpu, same_bits

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("gt,n_rows", [(BF, 1), (HF, 2), (BF, 8), (BF, 13), (F, 1), (F, 3), (F, 8)])
@pytest.mark.parametrize("lead", [0, 5])
def test_momentum_of_a_million(gt, n_rows, lead):
    g = torch.Generator().manual_seed(n_rows + lead)
    n = (1 << 20) + 12345
    ld = n + 3
    grads = (torch.randn(lead + n_rows * ld, generator=g) * 1e-3).to(gt)
    mom = torch.randn(lead + n + 7, generator=g) * 1e-2
    hp = zs.AdamWHParams(beta1=0.95, grad_scale=1.0 / n_rows)
    for nesterov, ut in ((True, BF), (False, F)):
        m, u = momentum_cpu(grads[lead:].view(n_rows, ld)[:, :n], mom[lead:lead + n], hp, nesterov)
        dm, du = mom.cuda(), torch.zeros(lead + n + 7, dtype=ut, device="cuda")
        zs.zero_muon_momentum(grads.cuda()[lead:], n_rows, ld, n, dm[lead:lead + n],
                              du[lead:lead + n], hp, nesterov=nesterov)
        assert same_bits(dm[lead:lead + n], m) and same_bits(du[lead:lead + n], u.to(ut))
        assert same_bits(dm[:lead], mom[:lead]) and same_bits(dm[lead + n:], mom[lead + n:])
        assert not du[:lead].any() and not du[lead + n:].any()


@pytest.mark.parametrize("ot,wt", [(BF, BF), (HF, BF), (BF, HF)])
@pytest.mark.parametrize("lead", [0, 5])
def test_update_of_a_million(ot, wt, lead):
    g = torch.Generator().manual_seed(lead)
    n = (1 << 20) + 4321
    lay, _ = zs.zero_flatten_layout([lead + n + 9], 1)
    o = torch.randn(lead + n, generator=g).to(ot)
    w = torch.randn(lead + n, generator=g) * 0.02
    full = torch.full((lay.n_pad,), 7.0, dtype=wt, device="cuda")
    hp = zs.AdamWHParams(lr=0.02, weight_decay=0.1)
    f = lambda v: torch.tensor(v, dtype=F)  # noqa: E731
    want = w[lead:] * f(1 - 0.02 * 0.1) - f(0.02) * (f(1.5) * o[lead:].float())
    dw = w.cuda()
    zs.zero_muon_update(o.cuda()[lead:], dw[lead:], full, lay, 0, hp, update_scale=1.5,
                        shard_off=lead, length=n)
    assert same_bits(dw[lead:], want) and same_bits(dw[:lead], w[:lead])
    assert same_bits(full[lead:lead + n], want.to(wt))
    assert (full[:lead] == 7).all() and (full[lead + n:] == 7).all()


def pieces(n, size=1 << 27):
    return [slice(at, min(n, at + size)) for at in range(0, n, size)]


def same(a, b):
    it = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(it), b.view(it))


def test_ranges_of_several_launches():
    """2^31 + 4099 elements from an odd place, each piece against torch's fp32"""
    n, lead = (1 << 31) + 4099, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def fill(t, scale):
        for s in pieces(t.numel()):
            t[s] = torch.randn(t[s].shape, generator=g, device="cuda") * scale

    f = lambda v: torch.tensor(v, dtype=F, device="cuda")  # noqa: E731
    grads = torch.empty(lead + n, dtype=BF, device="cuda")
    mom, u = torch.empty(lead + n, device="cuda"), torch.zeros(lead + n + 1, dtype=BF, device="cuda")
    fill(grads, 1e-3)
    fill(mom, 1e-2)
    old = mom.clone()
    hp = zs.AdamWHParams(beta1=0.95, grad_scale=0.5, lr=0.02, weight_decay=0.1)
    zs.zero_muon_momentum(grads[lead:], 1, n, n, mom[lead:], u[lead:lead + n], hp)
    for s in pieces(n):
        s = slice(lead + s.start, lead + s.stop)
        a = grads[s].float() * f(0.5)
        m = f(0.95) * old[s] + a
        assert same(mom[s], m), s
        assert same(u[s], (a + f(0.95) * m).to(BF)), s
    assert same(mom[:lead], old[:lead]) and not u[:lead].any() and not u[lead + n:].any()

    lay, _ = zs.zero_flatten_layout([lead + n], 1)
    full = torch.zeros(lay.n_pad, dtype=BF, device="cuda")
    master = old  # as a range of weights
    before = master.clone()
    zs.zero_muon_update(u[lead:lead + n], master[lead:], full, lay, 0, hp, update_scale=1.5,
                        shard_off=lead, length=n)
    for s in pieces(n):
        s = slice(lead + s.start, lead + s.stop)
        want = before[s] * f(1 - 0.02 * 0.1) - f(0.02) * (f(1.5) * u[s].float())
        assert same(master[s], want), s
        assert same(full[s], want.to(BF)), s
    assert same(master[:lead], before[:lead]) and not full[:lead].any()
