"""The Muon step's operators on the GPU.  Momentum and update are fp32
operations in a stated order: every bit is compared with the same operations
done one by one on the CPU.  The orthogonalisation is compared with its
definition in 64 bits.

Its tolerance.  A round's operands O, Q and the high half of X are rounded to
fp16: each element is off by at most 2^-12 of its binade's top, 2^-12.3 of
itself in the root mean square, and independently, so each product is off by
that share of its norm, twice (two operands).  The first-order sum over a round
is below 4 x 2^-12.3 of the norm of what the off-diagonal products contribute,
at most twice the result's (|B| < 3, |X| <= 1.21, result ~ 1, and the diagonal
part of B is not rounded); later rounds multiply an error by the polynomial's
slope, whose magnitude at the values of the last rounds is below 2 in the
square mean.  Errors of five rounds add in squares to below 2^-9 of the
result's norm.  The output's rounding adds half a step of its type."""
import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32
USUAL = (3.4445, -4.7750, 2.0315)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------------------
# momentum, update: bit for bit


def momentum_cpu(grads, mom, hp, nesterov, s=None, clip=1.0):
    a = grads[0].float()
    for r in grads[1:]:
        a = a + r.float()
    g = a * (torch.tensor(hp.grad_scale, dtype=F) if s is None else s)
    if clip < 1.0:
        g = g * torch.tensor(clip, dtype=F)
    b = torch.tensor(hp.beta1, dtype=F)
    m = b * mom + g
    return m, (g + b * m if nesterov else m)


def same_bits(a, b):
    it = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.cpu().view(it), b.cpu().view(it))


@pytest.mark.parametrize("gt", [BF, HF, F])
@pytest.mark.parametrize("ut", [BF, HF, F])
@pytest.mark.parametrize("n_rows", [1, 2, 8, 13])
def test_momentum(gt, ut, n_rows):
    g = torch.Generator().manual_seed(n_rows)
    for n, lead, gap in ((1, 0, 0), (3, 1, 1), (1000, 0, 24), (4099, 3, 5)):
        grads = (torch.randn(lead + n_rows * (n + gap), generator=g) * 1e-3).to(gt)
        mom = torch.randn(n + 2 * lead, generator=g) * 1e-2
        hp = zs.AdamWHParams(beta1=0.95, grad_scale=1.0 / n_rows)
        dg, dm = grads.cuda(), mom.cuda()
        du = torch.zeros(n + 2 * lead, dtype=ut, device="cuda")
        view = grads[lead:].view(n_rows, n + gap)[:, :n]
        for nesterov in (True, False):
            m, u = momentum_cpu(view, dm.cpu()[lead:lead + n], hp, nesterov)
            before = dm.clone()
            zs.zero_muon_momentum(dg[lead:], n_rows, n + gap, n, dm[lead:lead + n],
                                  du[lead:lead + n], hp, nesterov=nesterov)
            assert same_bits(dm[lead:lead + n], m) and same_bits(du[lead:lead + n], u.to(ut))
            dm_out = dm.clone()
            dm_out[lead:lead + n] = before[lead:lead + n]
            assert torch.equal(dm_out, before) and not du[:lead].any() and not du[lead + n:].any()


def test_momentum_and_update_at_places_that_do_not_match():
    """each buffer at another element offset: no common alignment"""
    g = torch.Generator().manual_seed(5)
    n = 2050
    for lg, lm, lu in ((0, 1, 2), (3, 0, 1), (1, 2, 0), (2, 255, 7)):
        grads = (torch.randn(lg + 3 * n, generator=g) * 1e-3).to(BF)
        mom = torch.randn(lm + n, generator=g) * 1e-2
        hp = zs.AdamWHParams(beta1=0.95, grad_scale=1 / 3, lr=0.02)
        m, u = momentum_cpu(grads[lg:].view(3, n), mom[lm:], hp, True)
        dm, du = mom.cuda(), torch.zeros(lu + n + 1, dtype=HF, device="cuda")
        zs.zero_muon_momentum(grads.cuda()[lg:], 3, n, n, dm[lm:], du[lu:], hp)
        assert same_bits(dm[lm:], m) and same_bits(dm[:lm], mom[:lm])
        assert same_bits(du[lu:lu + n], u.to(HF)) and not du[:lu].any() and not du[lu + n:].any()
        lay, _ = zs.zero_flatten_layout([lg + n], 1)
        o = torch.randn(lu + n, generator=g).to(BF)
        full = torch.zeros(lay.n_pad, dtype=BF, device="cuda")
        want = mom[lm:] * torch.tensor(1 - 0.02 * 0.1) - \
            torch.tensor(0.02) * (torch.tensor(1.5) * o[lu:].float())
        dm = mom.cuda()
        zs.zero_muon_update(o.cuda()[lu:], dm[lm:], full, lay, 0, hp, update_scale=1.5,
                            shard_off=lg, length=n)
        assert same_bits(dm[lm:], want) and same_bits(full[lg:], want.to(BF))
        assert not full[:lg].any()


@pytest.mark.parametrize("gt", [BF, F])
@pytest.mark.parametrize("n_rows,n,gap", [(1, 33000, 0), (2, 32768, 1), (8, 70001, 0),
                                          (11, 65536, 3), (64, 40003, 0), (64, 40000, 0)])
def test_momentum_of_many_waves(gt, n_rows, n, gap):
    """rows whose lines lie at other places than the waves'; runs and what is behind the last"""
    g = torch.Generator().manual_seed(n)
    for lg, lm in ((0, 0), (7, 2)):
        grads = (torch.randn(lg + n_rows * (n + gap), generator=g) * 1e-3).to(gt)
        mom = torch.randn(lm + n + 3, generator=g) * 1e-2
        hp = zs.AdamWHParams(beta1=0.95, grad_scale=1.0 / n_rows)
        m, u = momentum_cpu(grads[lg:].view(n_rows, n + gap)[:, :n], mom[lm:lm + n], hp, True)
        dm, du = mom.cuda(), torch.zeros(n + 1, dtype=BF, device="cuda")
        zs.zero_muon_momentum(grads.cuda()[lg:], n_rows, n + gap, n, dm[lm:lm + n], du[:n], hp)
        assert same_bits(dm[lm:lm + n], m) and same_bits(du[:n], u.to(BF)) and not du[n:].any()
        assert same_bits(dm[:lm], mom[:lm]) and same_bits(dm[lm + n:], mom[lm + n:])


def test_momentum_controls():
    g = torch.Generator().manual_seed(1)
    n = 1003
    grads = (torch.randn(2, n, generator=g) * 8).to(HF)
    mom = torch.randn(n, generator=g)
    hp = zs.AdamWHParams(beta1=0.9, grad_scale=0.5)
    dg = grads.cuda()

    def fresh():
        return mom.cuda(), torch.zeros(n, dtype=BF, device="cuda")

    flag = torch.tensor([1], dtype=torch.int32, device="cuda")
    m, u = fresh()
    zs.zero_muon_momentum(dg, 2, n, n, m, u, hp, skip=flag)
    assert torch.equal(m.cpu(), mom) and not u.any()
    flag.zero_()
    scale = zs.new_loss_scale(1024.0)
    s = torch.tensor(0.5 / 1024.0, dtype=F)
    ssq = torch.tensor([4.0e6], dtype=torch.float64, device="cuda")
    norm = 4.0e6 ** 0.5 * s.double().item()
    clip = torch.tensor(0.5 / (norm + 1e-6), dtype=torch.float64).float().item()
    assert clip < 1
    consts = torch.from_numpy(zs.zero_step_consts_make(hp)).cuda()
    for kw, arg in ((dict(), 1.0), (dict(sumsq=ssq, max_norm=0.5), clip),
                    (dict(sumsq=ssq, max_norm=100.0), 1.0)):
        want = momentum_cpu(grads, mom, hp, True, s, arg)
        for call, c in ((zs.zero_muon_momentum, hp), (zs.zero_muon_momentum_dc, consts)):
            m, u = fresh()
            call(dg, 2, n, n, m, u, c, skip=flag, loss_scale=scale, **kw)
            assert same_bits(m, want[0]) and same_bits(u, want[1].to(BF))
    m, u = fresh()  # held: the constants of no step
    zs.zero_muon_momentum_dc(dg, 2, n, n, m, u, torch.full((48,), 255, dtype=torch.uint8,
                                                           device="cuda"))
    assert torch.equal(m.cpu(), mom) and not u.any()


@pytest.mark.parametrize("ot", [BF, HF])
@pytest.mark.parametrize("wt", [BF, HF])
def test_update(ot, wt):
    g = torch.Generator().manual_seed(2)
    for n, lead in ((1, 0), (7, 1), (1000, 0), (4099, 3)):
        lay, _ = zs.zero_flatten_layout([3 * (lead + n + 2)], 3)
        o = torch.randn(lead + n, generator=g).to(ot)
        w = torch.randn(lead + n, generator=g) * 0.02
        full = torch.full((lay.n_pad,), 7.0, dtype=wt, device="cuda")
        hp = zs.AdamWHParams(lr=0.02, weight_decay=0.1)
        do, dw = o.cuda(), w.cuda()
        f = lambda v: torch.tensor(v, dtype=F)  # noqa: E731
        want = w[lead:] * f(1 - 0.02 * 0.1) - f(0.02) * (f(0.2 * 7.5) * o[lead:].float())
        args = dict(update_scale=0.2 * 7.5, shard_off=lead, length=n)
        skip = torch.tensor([1], dtype=torch.int32, device="cuda")
        zs.zero_muon_update(do[lead:], dw[lead:], full, lay, 1, hp, skip=skip, **args)
        assert same_bits(dw, w) and (full == 7).all()
        zs.zero_muon_update(do[lead:], dw[lead:], full, lay, 1, hp, **args)
        at = lay.shard + lead
        assert same_bits(dw[lead:], want) and same_bits(dw[:lead], w[:lead])
        assert same_bits(full[at:at + n], want.to(wt))
        assert (full[:at] == 7).all() and (full[at + n:] == 7).all()
        consts = torch.from_numpy(zs.zero_step_consts_make(hp)).cuda()
        dw2, full2 = w.cuda(), torch.full_like(full, 7.0)
        zs.zero_muon_update_dc(do[lead:], dw2[lead:], full2, lay, 1, consts, **args)
        assert same_bits(dw2, dw) and same_bits(full2, full)
        consts.fill_(255)
        zs.zero_muon_update_dc(do[lead:], dw2[lead:], full2, lay, 1, consts, **args)
        assert same_bits(dw2, dw) and same_bits(full2, full)


# ---------------------------------------------------------------------------
# orthogonalisation


def ns64(u, steps=5, coeffs=None, eps=1e-7):
    x = u.double()
    x = x / (x.norm() + eps)
    left = x.shape[0] <= x.shape[1]
    for k in range(steps):
        a, b, c = USUAL if coeffs is None else coeffs[k]
        if left:
            g = x @ x.t().contiguous()
            x = a * x + (b * g + c * g @ g) @ x
        else:
            g = x.t().contiguous() @ x
            x = a * x + x @ (b * g + c * g @ g)
    return x


def check_orth(o, want, what=""):
    err = (o.double() - want).norm() / want.norm()
    tol = 2.0 ** -9 + torch.finfo(o.dtype).eps / 2
    assert err <= tol, f"{what}: {err:.3g} off, {tol:.3g} allowed"
    worst = (o.double() - want).abs().max() / (want.norm() / want.numel() ** 0.5)
    assert worst <= 40 * tol, f"{what}: an element is {worst:.3g} of the mean size off"


def spectrum(g, r, c, kind):
    u = torch.randn(r, c, generator=g, device="cuda") * 1e-3
    if kind == "low rank":
        k = min(4, r, c)
        u = 0.05 * u + torch.randn(r, k, generator=g, device="cuda") @ \
            torch.randn(k, c, generator=g, device="cuda") * 1e-3
    elif kind == "decay":
        u = u * torch.logspace(0, -3, c, device="cuda")
    return u


@pytest.mark.parametrize("r,c", [(1, 1), (1, 500), (500, 1), (2, 3), (7, 300), (63, 64), (64, 64),
                                 (65, 64), (64, 2000), (77, 333), (333, 77), (130, 129),
                                 (257, 520), (520, 257), (512, 512), (1100, 700), (3000, 200),
                                 (1600, 1600), (2049, 2304)])
@pytest.mark.parametrize("kind", ["flat", "low rank", "decay"])
def test_orthogonalize_sizes(r, c, kind):
    u = spectrum(gen(r * 3 + c), r, c, kind)
    o = torch.empty(r, c, dtype=BF, device="cuda")
    zs.zero_orthogonalize(u, o)
    check_orth(o, ns64(u), f"{r} x {c} {kind}")


@pytest.mark.parametrize("ut", [BF, HF, F])
@pytest.mark.parametrize("ot", [BF, HF])
@pytest.mark.parametrize("count,r,c", [(1, 40, 200), (3, 77, 333), (5, 333, 77), (17, 128, 100),
                                       (3, 300, 520)])
def test_orthogonalize_stacks(ut, ot, count, r, c):
    """types, stacks at a stride, padded rows, odd places; nothing else written"""
    g = gen(count)
    ld, lead, gap = c + 3, 5, 11
    su = r * ld + gap
    ub = torch.randn(lead + count * su, generator=g, device="cuda").to(ut)
    ob = torch.randn(lead + count * (su + 2), generator=g, device="cuda").to(ot)
    u = ub.as_strided((count, r, c), (su, ld, 1), lead)
    o = ob.as_strided((count, r, c), (su + 2, ld, 1), lead)
    keep, keep_u = ob.clone(), ub.clone()
    zs.zero_orthogonalize(u, o)
    for i in range(count):
        check_orth(o[i], ns64(u[i]), f"matrix {i}")
    first = o.clone()
    zs.zero_orthogonalize(u, o)
    assert torch.equal(first, o) and torch.equal(ub, keep_u)  # the same bits
    o.copy_(keep.as_strided((count, r, c), (su + 2, ld, 1), lead))
    assert torch.equal(ob, keep)


@pytest.mark.parametrize("steps", [1, 2, 7])
def test_orthogonalize_rounds_and_coefficients(steps):
    u = torch.randn(2, 200, 130, generator=gen(1), device="cuda")
    o = torch.empty(2, 200, 130, dtype=BF, device="cuda")
    cubic = [(1.5 + 0.01 * k, -0.5, 0.0) for k in range(steps)]
    for coeffs in (None, cubic):
        zs.zero_orthogonalize(u, o, steps=steps, coeffs=coeffs, eps=1e-3)
        for i in range(2):
            check_orth(o[i], ns64(u[i], steps, coeffs, 1e-3), f"{steps} {coeffs}")


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_orthogonalize_is_free_of_scale(scale):
    u = torch.randn(90, 150, generator=gen(2), device="cuda")
    o = torch.empty(90, 150, dtype=BF, device="cuda")
    v = u * scale  # eps below every norm but the smallest
    zs.zero_orthogonalize(v, o, eps=0.0)
    check_orth(o, ns64(v, eps=0.0), str(scale))


def test_orthogonalize_special_matrices():
    u = torch.randn(5, 70, 100, generator=gen(3), device="cuda")
    u[1, 3, 4], u[2, 0, 0], u[3] = float("inf"), float("nan"), 0.0
    o = torch.empty(5, 70, 100, dtype=BF, device="cuda")
    for shape in (lambda t: t, lambda t: t.transpose(1, 2).contiguous()):
        v, w = shape(u), shape(o)
        zs.zero_orthogonalize(v, w)
        assert w[1].isnan().all() and w[2].isnan().all() and (w[3] == 0).all()
        for i in (0, 4):
            check_orth(w[i], ns64(v[i]))
    zs.zero_orthogonalize(u, o, eps=0.0)
    assert o[3].isnan().all() and not o[4].isnan().any()
    # one strong direction: the rest still rises by the rounds' slope
    a, b = torch.randn(96, 1, generator=gen(4), device="cuda"), \
        torch.randn(1, 130, generator=gen(5), device="cuda")
    v = a @ b + 1e-4 * torch.randn(96, 130, generator=gen(6), device="cuda")
    o = torch.empty(96, 130, dtype=BF, device="cuda")
    zs.zero_orthogonalize(v, o)
    check_orth(o, ns64(v), "one direction")


def test_orthogonalize_streams_and_graphs():
    """a side stream; two graphs that share a workspace, replayed in turn with
    eager work between"""
    g = gen(7)
    u = torch.randn(4, 130, 200, generator=g, device="cuda").to(BF)
    t = torch.randn(200, 64, generator=g, device="cuda").to(BF)
    o, p = torch.zeros_like(u), torch.zeros_like(t)
    size = max(zs.zero_orthogonalize_workspace_bytes(4, 130, 200),
               zs.zero_orthogonalize_workspace_bytes(1, 200, 64))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def one():
        zs.zero_orthogonalize(u, o, workspace=ws)

    def two():
        zs.zero_orthogonalize(t, p, workspace=ws)

    one()
    want = o.clone()
    o.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    zs.zero_orthogonalize(u, o, stream=side)
    side.synchronize()
    assert torch.equal(o, want)
    graphs = []
    for f in (one, two):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        graphs.append(graph)
    for k in range(3):
        u.copy_(torch.randn(4, 130, 200, generator=g, device="cuda"))
        t.copy_(torch.randn(200, 64, generator=g, device="cuda"))
        one()
        two()
        want = o.clone(), p.clone()
        o.zero_()
        p.zero_()
        torch.cuda.synchronize()
        graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(p, want[1])


def test_the_binding_refuses_what_does_not_fit():
    u = torch.zeros(3, 8, 16, device="cuda")
    o = torch.zeros(3, 8, 16, dtype=BF, device="cuda")
    for bad in (dict(o=o.float()), dict(o=o[:2]), dict(u=u.double()), dict(u=u.transpose(1, 2)),
                dict(u=u[0, 0], o=o[0, 0]), dict(steps=0), dict(steps=33), dict(eps=-1.0),
                dict(coeffs=[USUAL] * 4), dict(coeffs=[(1.0, 2.0)] * 5), dict(u=u.cpu()),
                dict(u=u[:1].expand(3, 8, 16)),
                dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            zs.zero_orthogonalize(**{**dict(u=u, o=o), **bad})
    lay, _ = zs.zero_flatten_layout([100], 1)
    hp, w, m = zs.AdamWHParams(), torch.zeros(100, dtype=BF, device="cuda"), \
        torch.zeros(100, device="cuda")
    for bad in (dict(o=w.float()), dict(o=w[:99]), dict(weight_full=w[:99]), dict(master=w),
                dict(length=101), dict(rank=1)):
        with pytest.raises((TypeError, ValueError)):
            zs.zero_muon_update(**{**dict(o=w.clone(), master=m, weight_full=w, layout=lay, rank=0,
                                          hp=hp), **bad})
    for bad in (dict(mom=w), dict(u=w[:99]), dict(grads=w[:99]), dict(n_rows=2), dict(ld=99)):
        with pytest.raises((TypeError, ValueError)):
            zs.zero_muon_momentum(**{**dict(grads=w, n_rows=1, ld=100, length=100, mom=m,
                                            u=w.clone(), hp=hp), **bad})


@pytest.mark.parametrize("count,r,c", [(4, 2300, 2500), (5, 2304, 2304), (1, 2900, 5200),
                                       (2, 200, 9000), (1, 64, 7000), (1, 9000, 64),
                                       (300, 60, 30), (7, 64, 1024), (2, 1020, 50), (3, 120, 320),
                                       (3, 310, 100), (2, 65, 321)])
def test_orthogonalize_large(count, r, c):
    """tiles of 256 and their quarters, contractions in parts, many small ones"""
    u = torch.randn(count, r, c, generator=gen(r), device="cuda").to(BF)
    o = torch.empty_like(u)
    zs.zero_orthogonalize(u, o)
    for i in range(count):
        check_orth(o[i], ns64(u[i]), f"matrix {i}")


@pytest.mark.parametrize("r,c", [(1, 8), (9, 17), (33, 1023), (64, 1024), (1024, 63), (64, 1025),
                                 (65, 448), (127, 447), (448, 128), (100, 385), (128, 449),
                                 (449, 70)])
@pytest.mark.parametrize("ut", [BF, HF, F])
def test_orthogonalize_up_to_one_workgroups_sizes(r, c, ut):
    """the last sizes that shared memory holds and the first that it does not; rows' odd ends"""
    g = gen(r + c)
    for ot, tall_ld in ((BF, c + 1), (HF, c)):
        u = torch.randn(2, r, tall_ld, generator=g, device="cuda").to(ut)[:, :, :c]
        buf = torch.full((2, r, tall_ld + 2), 7.0, dtype=ot, device="cuda")
        o = buf[:, :, 1:c + 1]
        zs.zero_orthogonalize(u, o)
        for k in range(2):
            check_orth(o[k], ns64(u[k]), f"{r} x {c}")
        assert (buf[:, :, 0] == 7).all() and (buf[:, :, c + 1:] == 7).all()
