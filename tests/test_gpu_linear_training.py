"""The layer products, the dropout and the sharded step together, as a
training loop runs them: a two-layer block whose parameters lie in the flat
weight buffer (at odd places), gradients of two micro-batches summed in place
in flat fp32 rows, one row per simulated rank, and the fused step from those
rows back into the weight buffer."""
import math

import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu

N_DP, MICRO, ROWS, D, F = 2, 2, 50, 96, 200
P = 0.2
SIZES = [3, F * D, F, D * F, D]  # an odd first parameter moves the others off alignment
STEPS = 3


def _setup(seed):
    g = torch.Generator().manual_seed(seed)
    lay, offs = zs.zero_flatten_layout(SIZES, N_DP)
    offs = [int(o) for o in offs]
    flat = torch.zeros(lay.n_pad)
    for o, n in zip(offs, SIZES):
        flat[o:o + n] = torch.randn(n, generator=g) * 0.1
    S = lay.shard
    dev = dict(device="cuda")
    st = dict(
        lay=lay, offs=offs, weights=flat.to(torch.bfloat16).cuda(),
        master=[flat[r * S:(r + 1) * S].cuda() for r in range(N_DP)],
        m=[torch.zeros(S, **dev) for _ in range(N_DP)],
        v=[torch.zeros(S, **dev) for _ in range(N_DP)],
        rows=torch.zeros(N_DP, lay.n_pad, **dev),
        x=[[torch.randn(ROWS, D, generator=g).to(torch.bfloat16).cuda() for _ in range(MICRO)]
           for _ in range(N_DP)],
        c=[[torch.randn(ROWS, D, generator=g).to(torch.bfloat16).cuda() for _ in range(MICRO)]
           for _ in range(N_DP)],
        t=zs.new_step_counter(1), consts=zs.new_step_consts(),
        table=zs.step_consts_table([zs.AdamWHParams(lr=1e-2, step=k + 1,
                                                    grad_scale=1.0 / (N_DP * MICRO))
                                    for k in range(STEPS + 2)]))
    bf = dict(dtype=torch.bfloat16, device="cuda")
    st["h"], st["z"], st["dz"] = (torch.empty(ROWS, F, **bf) for _ in range(3))
    st["y"], st["dy"] = (torch.empty(ROWS, D, **bf) for _ in range(2))
    st["ws"] = torch.empty(16 + max(zs.zero_linear_workspace_bytes(op, ROWS, n, k)
                                    for op in range(3) for n, k in ((F, D), (D, F))),
                           dtype=torch.uint8, device="cuda")
    return st


def _param(buf, st, i, shape):
    o = st["offs"][i]
    return buf[o:o + SIZES[i]].view(*shape)


def _drop(st, rank, micro):
    # a stream of its own for every rank and micro-batch, moved by the step counter
    return zs.ZeroDropout(P, seed=1234, offset=(rank * MICRO + micro) << 32, step=st["t"])


def _step(st):
    w1, b1 = _param(st["weights"], st, 1, (F, D)), _param(st["weights"], st, 2, (F,))
    w2, b2 = _param(st["weights"], st, 3, (D, F)), _param(st["weights"], st, 4, (D,))
    zs.zero_step_consts_select(st["consts"], st["table"], st["t"])
    for r in range(N_DP):
        row = st["rows"][r]
        for k in range(MICRO):
            x, c, d = st["x"][r][k], st["c"][r][k], _drop(st, r, k)
            zs.zero_linear(x, w1, st["h"], bias=b1, act=zs.ZERO_ACT_GELU, z=st["z"],
                           workspace=st["ws"])
            zs.zero_linear(st["h"], w2, st["y"], bias=b2, drop=d, residual=x, workspace=st["ws"])
            zs.zero_dropout(c, st["dy"], d)
            zs.zero_linear_wgrad(st["dy"], st["h"], _param(row, st, 3, (D, F)),
                                 db=_param(row, st, 4, (D,)), accumulate=k > 0,
                                 workspace=st["ws"])
            zs.zero_linear_dgrad(st["dy"], w2, st["dz"], act=zs.ZERO_ACT_GELU, z=st["z"],
                                 workspace=st["ws"])
            zs.zero_linear_wgrad(st["dz"], x, _param(row, st, 1, (F, D)),
                                 db=_param(row, st, 2, (F,)), accumulate=k > 0,
                                 workspace=st["ws"])
    S = st["lay"].shard
    for r in range(N_DP):
        zs.zero_shard_step_dc(st["rows"][:, r * S:(r + 1) * S], st["lay"].n_pad, S,
                              st["master"][r], st["m"][r], st["v"][r], st["weights"], st["lay"],
                              r, st["consts"])
    zs.zero_step_counter_advance(st["t"])


def _grads64(st, t):
    """the gradient rows of step t by autograd in 64 bits, from the 16-bit weights"""
    flat = st["weights"].cpu().double()
    rows = []
    for r in range(N_DP):
        w = flat.clone().requires_grad_(True)
        w1, b1 = _param(w, st, 1, (F, D)), _param(w, st, 2, (F,))
        w2, b2 = _param(w, st, 3, (D, F)), _param(w, st, 4, (D,))
        loss = 0.0
        for k in range(MICRO):
            x, c = st["x"][r][k].cpu().double(), st["c"][r][k].cpu().double()
            z = x @ w1.t() + b1
            h = 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
            keep = ref.keep(ROWS, D, P, 1234, ((r * MICRO + k) << 32) + t)
            y = x + torch.where(keep, (h @ w2.t() + b2) * ref.scale32(P), 0.0)
            loss = loss + (c * y).sum()
        loss.backward()
        rows.append(w.grad)
    return torch.stack(rows)


def test_a_training_loop_has_the_gradients_of_autograd():
    """The stored 16-bit h, dy, z and dz are each off by at most 2^-8 of
    themselves, and gelu'' is below 0.8 with |z| below 6 here: every gradient
    entry's terms by at most (2 + 6 * 0.8 + 1) 2^-8 of the sum's scale in the
    worst case, and the errors of many terms average.  Held here: 2^-6 in norm
    for each parameter."""
    st = _setup(1)
    for step in range(1, STEPS + 1):
        want = _grads64(st, step)
        before = [m.clone() for m in st["master"]]
        _step(st)
        torch.cuda.synchronize()
        got = st["rows"].cpu().double()
        for o, n in list(zip(st["offs"], SIZES))[1:]:
            a, b = got[:, o:o + n], want[:, o:o + n]
            assert float((a - b).norm()) <= 2.0 ** -6 * float(b.norm()), (step, o)
        assert bool((got[:, :3] == 0).all()) and bool((got[:, st["lay"].n:] == 0).all())
        # the weights are the cast of the stepped master
        flat = torch.cat(st["master"])
        assert torch.equal(st["weights"], flat.to(torch.bfloat16))
        assert all(not torch.equal(a, b) for a, b in zip(before, st["master"]))
    assert int(st["t"].item()) == STEPS + 1


def test_the_captured_loop_equals_the_eager_one():
    """one graph of the whole step, replayed, with a new mask and new step
    constants every time; a second, eager loop runs between the replays"""
    a, b = _setup(2), _setup(2)
    warm = _setup(2)
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
        assert torch.equal(a["rows"], b["rows"]) and torch.equal(a["weights"], b["weights"])
        assert all(torch.equal(x, y) for x, y in zip(a["master"] + a["m"] + a["v"],
                                                      b["master"] + b["m"] + b["v"]))
