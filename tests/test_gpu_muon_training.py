"""Layer norm, the layer products and the Muon step together, as a training
loop runs them: a pre-norm MLP block whose parameters lie in the flat weight
buffer at odd places, fp32 gradient rows of two simulated ranks, and a step in
which the two matrices (the second one cut by the shards' border) go by their
orthogonalised momentum and the rest by AdamW."""
import math

import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from tests.test_gpu_muon import check_orth, ns64

pytestmark = pytest.mark.gpu

N_DP, MICRO, ROWS, D, F = 2, 2, 50, 96, 200
SIZES = [3, F * D, D * F, D, D]  # another parameter, W1, W2, the norm's weight and bias
FIRST, LAST = 3, 3 + 2 * F * D   # the matrices' place in the flat vector
STEPS = 3
SCALE = 0.2 * math.sqrt(F)       # of the update, the usual one
EPS = 1e-5
MUON = dict(lr=0.02, beta1=0.95, weight_decay=0.1, grad_scale=1.0 / (N_DP * MICRO))


def _setup(seed):
    g = torch.Generator().manual_seed(seed)
    lay, offs = zs.zero_flatten_layout(SIZES, N_DP)
    offs = [int(o) for o in offs]
    flat = torch.zeros(lay.n_pad)
    for o, n in zip(offs, SIZES):
        flat[o:o + n] = torch.randn(n, generator=g) * 0.1
    flat[offs[3]:offs[3] + D] += 1.0
    S = lay.shard
    assert offs[2] < S < offs[2] + D * F
    bf = dict(dtype=torch.bfloat16, device="cuda")
    dev = dict(device="cuda")

    def batch():
        return [[torch.randn(ROWS, D, generator=g).to(torch.bfloat16).cuda() for _ in range(MICRO)]
                for _ in range(N_DP)]

    st = dict(lay=lay, offs=offs, weights=flat.to(torch.bfloat16).cuda(),
              master=[flat[r * S:(r + 1) * S].cuda() for r in range(N_DP)],
              m=[torch.zeros(S, **dev) for _ in range(N_DP)],
              v=[torch.zeros(S, **dev) for _ in range(N_DP)],
              acc=torch.zeros(S, **dev), rows=torch.zeros(N_DP, lay.n_pad, **dev),
              u=torch.zeros(lay.n_pad, **bf), o=torch.zeros(lay.n_pad, **bf), x=batch(), c=batch(),
              t=zs.new_step_counter(1))
    for name, hp in (("muon", MUON), ("adam", dict(MUON, lr=1e-2, beta1=0.9))):
        st[name] = zs.new_step_consts()
        st[name + "_table"] = zs.step_consts_table([zs.AdamWHParams(step=k + 1, **hp)
                                                    for k in range(STEPS + 2)])
    st["z"], st["h"], st["dz"] = (torch.empty(ROWS, F, **bf) for _ in range(3))
    st["n"], st["y"], st["dn"], st["dx"] = (torch.empty(ROWS, D, **bf) for _ in range(4))
    st["mean"], st["rstd"] = torch.empty(ROWS, **dev), torch.empty(ROWS, **dev)
    need = [zs.zero_linear_workspace_bytes(op, ROWS, n, k) for op in range(3)
            for n, k in ((F, D), (D, F))]
    need += [zs.zero_layernorm_workspace_bytes(ROWS, D),
             zs.zero_orthogonalize_workspace_bytes(1, F, D)]
    st["ws"] = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    return st


def _param(buf, st, i, shape):
    o = st["offs"][i]
    return buf[o:o + SIZES[i]].view(*shape)


def _pieces(S, r, lo, hi):
    """the part of [lo, hi) that lies in shard r: (flat start, flat end)"""
    a, b = max(lo, r * S), min(hi, (r + 1) * S)
    return (a, b) if a < b else None


def _step(st):
    lay, offs, ws = st["lay"], st["offs"], st["ws"]
    S = lay.shard
    w1, w2 = _param(st["weights"], st, 1, (F, D)), _param(st["weights"], st, 2, (D, F))
    gw, gb = _param(st["weights"], st, 3, (D,)), _param(st["weights"], st, 4, (D,))
    for name in ("muon", "adam"):
        zs.zero_step_consts_select(st[name], st[name + "_table"], st["t"])
    for r in range(N_DP):
        row = st["rows"][r]
        for k in range(MICRO):
            x, dy = st["x"][r][k], st["c"][r][k]  # the loss is sum(c y)
            zs.zero_layernorm(x, gw, gb, st["n"], eps=EPS, mean=st["mean"], rstd=st["rstd"])
            zs.zero_linear(st["n"], w1, st["h"], act=zs.ZERO_ACT_GELU_TANH, z=st["z"],
                           workspace=ws)
            zs.zero_linear(st["h"], w2, st["y"], residual=x, workspace=ws)
            zs.zero_linear_wgrad(dy, st["h"], _param(row, st, 2, (D, F)), accumulate=k > 0,
                                 workspace=ws)
            zs.zero_linear_dgrad(dy, w2, st["dz"], act=zs.ZERO_ACT_GELU_TANH, z=st["z"],
                                 workspace=ws)
            zs.zero_linear_wgrad(st["dz"], st["n"], _param(row, st, 1, (F, D)), accumulate=k > 0,
                                 workspace=ws)
            zs.zero_linear_dgrad(st["dz"], w1, st["dn"], workspace=ws)
            zs.zero_layernorm_backward(st["dn"], x, gw, st["mean"], st["rstd"], st["dx"],
                                       residual=dy, dw=_param(row, st, 3, (D,)),
                                       db=_param(row, st, 4, (D,)), accumulate=k > 0,
                                       workspace=ws)
    for r in range(N_DP):
        a, b = _pieces(S, r, FIRST, LAST)
        zs.zero_muon_momentum_dc(st["rows"][:, a:b], N_DP, lay.n_pad, b - a,
                                 st["m"][r][a - r * S:b - r * S], st["u"][a:b], st["muon"])
    # every rank's u is here: the all-gather
    for i, shape in ((1, (F, D)), (2, (D, F))):
        zs.zero_orthogonalize(_param(st["u"], st, i, shape), _param(st["o"], st, i, shape),
                              workspace=ws)
    for r in range(N_DP):
        a, b = _pieces(S, r, FIRST, LAST)
        zs.zero_muon_update_dc(st["o"][a:b], st["master"][r][a - r * S:], st["weights"], lay, r,
                               st["muon"], update_scale=SCALE, shard_off=a - r * S, length=b - a)
        for lo, hi in ((0, FIRST), (LAST, lay.n_pad)):
            piece = _pieces(S, r, lo, hi)
            if piece is None:
                continue
            a, b = piece
            at = slice(a - r * S, b - r * S)
            zs.zero_shard_reduce(st["rows"][:, a:b], N_DP, lay.n_pad, b - a, st["acc"][at])
            zs.zero_shard_adamw_dc(st["acc"][at], st["master"][r][at], st["m"][r][at],
                                   st["v"][r][at], st["weights"], lay, r, st["adam"],
                                   shard_off=a - r * S, length=b - a)
    zs.zero_step_counter_advance(st["t"])


def _grads64(st):
    """the gradient rows by autograd in 64 bits, from the 16-bit weights"""
    flat = st["weights"].cpu().double()
    rows, dx = [], None
    for r in range(N_DP):
        w = flat.clone().requires_grad_(True)
        w1, w2 = _param(w, st, 1, (F, D)), _param(w, st, 2, (D, F))
        gw, gb = _param(w, st, 3, (D,)), _param(w, st, 4, (D,))
        loss = 0.0
        for k in range(MICRO):
            x = st["x"][r][k].cpu().double().requires_grad_(True)
            n = torch.nn.functional.layer_norm(x, (D,), gw, gb, EPS)
            h = torch.nn.functional.gelu(n @ w1.t(), approximate="tanh")
            part = (st["c"][r][k].cpu().double() * (x + h @ w2.t())).sum()
            dx, = torch.autograd.grad(part, x, retain_graph=True)
            loss = loss + part
        loss.backward()
        rows.append(w.grad)
    return torch.stack(rows), dx  # dx: of the last micro-batch of the last rank


def test_a_training_loop_has_the_gradients_of_autograd_and_the_formulas_step():
    """Gradients: the stored 16-bit n, h, z, dz and dn are each off by at most
    2^-8 of themselves, and gelu'' is below 0.8 with |z| below 6 here: every
    gradient entry's terms by at most (4 + 6 * 0.8 + 1) 2^-8 of the sum's scale
    in the worst case, and the errors of many terms average.  Held here: 2^-6
    in norm for each parameter.  The step: what the master moved by, over lr
    times the update's scale, is the orthogonalised momentum; the master's own
    rounding is 2^-24 of at most 0.8, over 0.02 SCALE = 0.056 2^-20."""
    st = _setup(1)
    S = st["lay"].shard
    mom = torch.zeros(st["lay"].n_pad)
    for step in range(1, STEPS + 1):
        want, dx = _grads64(st)
        before = torch.cat(st["master"]).cpu()
        _step(st)
        torch.cuda.synchronize()
        rows = st["rows"].cpu()
        for o, n in list(zip(st["offs"], SIZES))[1:]:
            a, b = rows[:, o:o + n].double(), want[:, o:o + n]
            assert float((a - b).norm()) <= 2.0 ** -6 * float(b.norm()), (step, o)
        assert float((st["dx"].cpu().double() - dx).norm()) <= 2.0 ** -6 * float(dx.norm())
        beta = torch.tensor(MUON["beta1"])
        g = (rows[0] + rows[1]) * torch.tensor(MUON["grad_scale"])
        mom = beta * mom + g
        u = (g + beta * mom).to(torch.bfloat16)
        assert torch.equal(st["u"][FIRST:LAST].cpu(), u[FIRST:LAST])
        after = torch.cat(st["master"]).cpu()
        moved = (before.double() * (1 - MUON["lr"] * MUON["weight_decay"]) - after) / \
            (MUON["lr"] * SCALE)
        for i, shape in ((1, (F, D)), (2, (D, F))):
            o64 = ns64(_param(u, st, i, shape))
            check_orth(_param(st["o"].cpu(), st, i, shape), o64, (step, i))
            err = (_param(moved, st, i, shape) - o64).norm() / o64.norm()
            assert err <= 2.0 ** -9 + 2.0 ** -8, (step, i, err)
        assert torch.equal(st["weights"].cpu(), after.to(torch.bfloat16))
        assert not torch.equal(before[LAST:st["lay"].n], after[LAST:st["lay"].n])
        assert S * N_DP == len(after)


def test_the_captured_loop_equals_the_eager_one():
    """one graph of the whole step, replayed with new step constants every
    time; a second, eager loop runs between the replays"""
    a, b, warm = _setup(2), _setup(2), _setup(2)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _step(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(a)
    torch.cuda.synchronize()
    for step in range(STEPS):
        graph.replay()
        torch.cuda.synchronize()
        _step(b)
        torch.cuda.synchronize()
        for k in ("rows", "weights", "u", "o", "dx", "y", "t"):
            assert torch.equal(a[k], b[k]), (step, k)
        assert all(torch.equal(x, y) for x, y in zip(a["master"] + a["m"] + a["v"],
                                                      b["master"] + b["m"] + b["v"]))
