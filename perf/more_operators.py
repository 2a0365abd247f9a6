"""Layer norm on the flat buffers and the Muon step of a shard: the cases they
are measured on, their plain forms and their definitions in 64 bits.

Between two steps a rank normalises activations with weights that lie in the
flat 16-bit buffer, and writes their gradients into the flat row; at the step,
the matrices' momentum is orthogonalised before it is applied to the shard.
Five operators:

  layernorm           y = (x - mean) rstd w + b over each row of x,
                      rstd = 1 / sqrt(var + eps); mean and rstd kept for
                      the backward pass on request
  layernorm_backward  with h = (x - mean) rstd and g = dy w:
                      dx = residual + rstd (g - mean(g) - h mean(g h)),
                      dw (+)= sum over rows of dy h, db (+)= that of dy
  muon_momentum       a = the sum of the ranks' rows, g = a s,
                      mom = beta mom + g, u = mom or (Nesterov) g + beta mom
  orthogonalize       X = u / (|u| + eps); five times
                      A = X X^T, X = a X + (b A + c A A) X; o = X
  muon_update         w = w (1 - lr decay) - lr (k o), and its 16-bit cast

`own` False: elementary torch operations in 32 bits.  `own` True: the calls
a user makes of zero_sharded_mixed_flatten_amd.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

_NORM = dict(op="layernorm", type="bf16", x="same", y="same", bias=True, stats=True, pad=0, lead=0)
_NORM_B = dict(op="layernorm_backward", type="bf16", x="same", dy="same", grad="f32",
               residual=True, micro=1, pad=0, lead=0)
_ORTH = dict(op="orthogonalize", type="bf16", count=1, pad=0, lead=0)
_MOM = dict(op="muon_momentum", rows="bf16", u="bf16", n_dp=8, nesterov=True, lead=0)
_UPD = dict(op="muon_update", o="bf16", weights="bf16", lead=0)

_COEFFS = (3.4445, -4.7750, 2.0315)
_STEPS = 5
_EPS_ORTH = 1e-7
_EPS_NORM = 1e-5


def listed():
    return [
        # one new token of the GPT-2-XL list: latency
        dict(_NORM, name="norm_token_gpt2xl", m=1, n=1600, stats=False),
        # training, 7B list's width: a 32-bit residual stream in, the products' 16-bit input out
        dict(_NORM, name="norm_train_7b_f32_stream", m=16384, n=4096, x="f32"),
        # training, GPT-2-XL list: the gradient joins the residual stream's, fp32 rows
        dict(_NORM_B, name="norm_back_gpt2xl", m=8192, n=1600),
        # two micro-batches of a ragged fp16 sequence at odd places, 16-bit rows
        dict(_NORM_B, name="norm_back_ragged", m=1023, n=6401, type="f16", dy="f32", grad="same",
             residual=False, micro=2, pad=3, lead=5),
        # one projection of the GPT-2-XL list
        dict(_ORTH, name="orth_gpt2xl_proj", rows=1600, cols=1600),
        # a layer's four attention matrices of the 7B list, one behind the other
        dict(_ORTH, name="orth_7b_attention", count=4, rows=4096, cols=4096),
        # the 7B list's tall MLP matrix, momentum in 32 bits: the largest
        dict(_ORTH, name="orth_7b_up_f32", rows=11008, cols=4096, type="f32"),
        # small odd matrices of three layers, padded rows, an odd place
        dict(_ORTH, name="orth_ragged", count=3, rows=77, cols=333, type="f16", pad=3, lead=5),
        # the 7B list's MLP matrix, eight ranks' bf16 rows
        dict(_MOM, name="momentum_7b_up", length=11008 * 4096),
        # an odd piece of a shard from a 32-bit accumulator
        dict(_MOM, name="momentum_piece", length=100003, rows="f32", n_dp=1, u="f32",
             nesterov=False, lead=1),
        # the update of the same matrix
        dict(_UPD, name="update_7b_up", length=11008 * 4096),
        # an odd piece, fp16 weights
        dict(_UPD, name="update_piece", length=100003, weights="f16", lead=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layernorm", "layernorm_backward", "orthogonalize", "orthogonalize",
                     "muon_momentum", "muon_update"])
    most_bytes = max(work(c)["bytes"] for c in listed())
    most_flops = max(work(c)["flops"] for c in listed())
    while True:
        pad, lead = rng.choice([0, 0, 8, 3]), rng.choice([0, 0, 0, 8, 5])
        if op in ("layernorm", "layernorm_backward"):
            # one token to a long batch; rows from a small model's to beyond the lists'
            m, n = 1 if rng.random() < 0.1 else _log(rng, 1, 32768), _log(rng, 32, 16384)
            if rng.random() < 0.5:  # widths are mostly round
                n = -(-n // 64) * 64
            t = rng.choice(["bf16", "bf16", "f16"])
            if op == "layernorm":
                case = dict(_NORM, type=t, x=rng.choice(["same", "f32"]),
                            y=rng.choice(["same", "same", "f32"]), bias=rng.random() < 0.7,
                            stats=rng.random() < 0.7)
            else:
                case = dict(_NORM_B, type=t, x=rng.choice(["same", "f32"]),
                            dy=rng.choice(["same", "same", "f32"]),
                            grad=rng.choice(["f32", "same"]), residual=rng.random() < 0.6,
                            micro=rng.choice([1, 1, 2]))
            case.update(m=m, n=n, pad=pad, lead=lead)
        elif op == "orthogonalize":
            # a head's block to the lists' largest matrices, one to a stack of layers
            r, c = _log(rng, 8, 11008), _log(rng, 8, 11008)
            if rng.random() < 0.5:
                r, c = -(-r // 64) * 64, -(-c // 64) * 64
            case = dict(_ORTH, type=rng.choice(["bf16", "bf16", "f16", "f32"]),
                        count=rng.choice([1, 1, 2, 4, 12, 48]), rows=r, cols=c, pad=pad, lead=lead)
        elif op == "muon_momentum":
            case = dict(_MOM, length=_log(rng, 1000, 48000000), rows=rng.choice(["bf16", "f16", "f32"]),
                        u=rng.choice(["bf16", "bf16", "f16", "f32"]), n_dp=rng.choice([1, 2, 8, 64]),
                        nesterov=rng.random() < 0.7, lead=lead)
        else:
            case = dict(_UPD, length=_log(rng, 1000, 48000000), o=rng.choice(["bf16", "f16"]),
                        weights=rng.choice(["bf16", "f16"]), lead=lead)
        w = work(case)
        if w["flops"] <= most_flops and w["bytes"] <= most_bytes:
            return case


def _size(t):
    return 4 if t == "f32" else 2


def _of(case, key):
    return case["type"] if case[key] == "same" else case[key]


def work(case):
    op = case["op"]
    if op == "layernorm":
        m, n = case["m"], case["n"]
        b = m * n * (_size(_of(case, "x")) + _size(_of(case, "y"))) + \
            2 * n * (2 if case["bias"] else 1) + (8 * m if case["stats"] else 0)
        return {"bytes": b, "flops": 8 * m * n}
    if op == "layernorm_backward":
        m, n, k = case["m"], case["n"], case["micro"]
        x = _size(_of(case, "x"))
        b = m * n * (x * (3 if case["residual"] else 2) + _size(_of(case, "dy"))) + 2 * n + 8 * m
        g = 2 * n * _size(_of(case, "grad"))
        return {"bytes": k * b + (2 * k - 1) * g, "flops": k * 16 * m * n}
    if op == "orthogonalize":
        r, c = sorted((case["rows"], case["cols"]))
        # A and A A are symmetric: half of their products
        return {"bytes": case["count"] * r * c * (_size(case["type"]) + 2),
                "flops": case["count"] * _STEPS * (3 * r * r * c + r * r * r)}
    n = case["length"]
    if op == "muon_momentum":
        return {"bytes": n * (case["n_dp"] * _size(case["rows"]) + 8 + _size(case["u"])),
                "flops": n * (case["n_dp"] + 4)}
    return {"bytes": n * (2 + 8 + 2), "flops": 4 * n}


# ---------------------------------------------------------------------------
# inputs


class _Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def flat(self, count, scale, dtype):
        """count values of N(0, scale), made in pieces to keep the fp32 draws small."""
        t = torch.empty(count, dtype=dtype, device="cuda")
        for at in range(0, count, 1 << 26):
            c = min(1 << 26, count - at)
            t[at:at + c] = torch.randn(c, generator=self.g, device="cuda") * scale
        return t

    def rows(self, m, n, pad, scale, dtype):
        """an [m][n] view of rows n + pad apart"""
        return self.flat(m * (n + pad), scale, dtype).view(m, n + pad)[:, :n]


def _empty_rows(m, n, pad, dtype):
    return torch.empty(m * (n + pad), dtype=dtype, device="cuda").view(m, n + pad)[:, :n]


def _activations(g, case):
    """a residual stream: channels of unequal size, a few of them large, and a mean"""
    m, n = case["m"], case["n"]
    x = g.rows(m, n, case["pad"], 1.0, _TYPES[_of(case, "x")])
    size = torch.exp(0.5 * g.flat(n, 1.0, torch.float32))
    size[::97] *= 10.0
    x.mul_(size.to(x.dtype)).add_(0.25)
    return x


def _affine(g, n, lead, t):
    """the norm's weight and bias in the flat weight buffer"""
    buf = g.flat(lead + 2 * n, 0.1, t)
    buf[lead:lead + n] += 1.0
    return buf[lead:lead + n], buf[lead + n:lead + 2 * n]


def _stack(buf, lead, case, ld):
    """count matrices one behind the other from element lead on"""
    return buf.as_strided((case["count"], case["rows"], case["cols"]),
                          (case["rows"] * ld, ld, 1), lead)


def prepare(case, seed):
    g = _Maker(seed)
    op = case["op"]
    s = {"case": case}
    if op == "layernorm":
        m, n = case["m"], case["n"]
        s["x"] = _activations(g, case)
        s["w"], s["b"] = _affine(g, n, case["lead"], _TYPES[case["type"]])
        if not case["bias"]:
            s["b"] = None
        s["y"] = _empty_rows(m, n, case["pad"], _TYPES[_of(case, "y")])
        s["mean"], s["rstd"] = (torch.empty(m, device="cuda") for _ in range(2)) \
            if case["stats"] else (None, None)
    elif op == "layernorm_backward":
        m, n, lead = case["m"], case["n"], case["lead"]
        t = _TYPES[case["type"]]
        s["w"], _ = _affine(g, n, lead, t)
        s["micro"] = []
        for _ in range(case["micro"]):
            x = _activations(g, case)
            # what the forward call left
            var, mean = torch.var_mean(x.float(), 1, unbiased=False)
            s["micro"].append(dict(
                x=x, mean=mean, rstd=1 / torch.sqrt(var + _EPS_NORM),
                dy=g.rows(m, n, case["pad"], 1.0, _TYPES[_of(case, "dy")]),
                residual=g.rows(m, n, case["pad"], 1.0, x.dtype) if case["residual"] else None,
                dx=_empty_rows(m, n, case["pad"], x.dtype)))
        # the flat gradient row: other parameters, the weight's place, the bias's
        row = torch.zeros(lead + 2 * n, dtype=_TYPES[_of(case, "grad")], device="cuda")
        s["dw"], s["db"] = row[lead:lead + n], row[lead + n:]
    elif op == "orthogonalize":
        r, c, k = case["rows"], case["cols"], case["count"]
        ld = c + case["pad"]
        t = _TYPES[case["type"]]
        # momentum: noise and a few strong directions
        u = _stack(g.flat(case["lead"] + k * r * ld, 1e-3, t), case["lead"], case, ld)
        for i in range(k):
            a, b = (g.flat(n * 8, 1.0, torch.float32) for n in (r, c))
            u[i] += ((a.view(r, 8) * 1e-3) @ b.view(8, c)).to(t)
        s["u"] = u
        s["o"] = _stack(torch.empty(case["lead"] + k * r * ld, dtype=torch.bfloat16, device="cuda"),
                        case["lead"], case, ld)
    elif op == "muon_momentum":
        n, lead = case["length"], case["lead"]
        # the ranks' rows of the shard, as the reduce-scatter delivers them
        s["grads"] = g.flat(lead + case["n_dp"] * n, 1e-3, _TYPES[case["rows"]])[lead:].view(
            case["n_dp"], n)
        s["mom"] = g.flat(lead + n, 1e-2, torch.float32)[lead:]
        s["u"] = torch.empty(lead + n, dtype=_TYPES[case["u"]], device="cuda")[lead:]
    else:
        n, lead = case["length"], case["lead"]
        s["o"] = g.flat(lead + n, 0.016, _TYPES[case["o"]])[lead:]
        s["master"] = g.flat(lead + n, 0.02, torch.float32)[lead:]
        s["weights"] = torch.zeros(lead + n, dtype=_TYPES[case["weights"]], device="cuda")
        # 0.2 sqrt(larger side): the usual update's size
        s["lr"], s["decay"], s["k"] = 3e-4, 0.1, 0.2 * math.sqrt(11008)
    if op == "muon_momentum":
        s["beta"], s["scale"] = 0.95, 1.0 / case["n_dp"]
    if own:
        import zero_sharded_mixed_flatten_amd as zs
        if op == "layernorm_backward":
            nbytes = zs.zero_layernorm_workspace_bytes(case["m"], case["n"])
        elif op == "orthogonalize":
            nbytes = zs.zero_orthogonalize_workspace_bytes(case["count"], case["rows"],
                                                           case["cols"])
        else:
            nbytes = 0
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None
        if op == "muon_momentum":
            s["hp"] = zs.AdamWHParams(beta1=s["beta"], grad_scale=s["scale"])
        elif op == "muon_update":
            s["hp"] = zs.AdamWHParams(lr=s["lr"], weight_decay=s["decay"])
            # this shard is the buffer's only one
            s["layout"] = zs.zero_flatten_layout([case["lead"] + case["length"]], 1)[0]
    return s


# ---------------------------------------------------------------------------
# the plain forms: 32 bits, elementary operations


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + _EPS_NORM)
    y = d * rstd * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    y = y.to(s["y"].dtype)
    return (y, mean[:, 0], rstd[:, 0]) if s["mean"] is not None else (y,)


def _plain_norm_backward(s):
    w, dw, db, dxs = s["w"].float(), None, None, []
    for b in s["micro"]:
        dy, rstd = b["dy"].float(), b["rstd"][:, None]
        h = (b["x"].float() - b["mean"][:, None]) * rstd
        g = dy * w
        dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        if b["residual"] is not None:
            dx = b["residual"].float() + dx
        dxs.append(dx.to(b["dx"].dtype))
        a, c = (dy * h).sum(0), dy.sum(0)  # each micro-batch's sum is rounded to the row's type
        dw = (a if dw is None else dw.float() + a).to(s["dw"].dtype)
        db = (c if db is None else db.float() + c).to(s["dw"].dtype)
    return (dxs, dw, db)


def _plain_orthogonalize(s):
    x = s["u"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + _EPS_ORTH)
    a, b, c = _COEFFS
    for _ in range(_STEPS):
        gram = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16)


def _plain(s):
    op = s["case"]["op"]
    if op == "layernorm":
        return _plain_norm(s)
    if op == "layernorm_backward":
        return _plain_norm_backward(s)
    if op == "orthogonalize":
        return _plain_orthogonalize(s)
    if op == "muon_momentum":
        g = s["grads"].float().sum(0) * s["scale"]
        s["mom"].mul_(s["beta"]).add_(g)
        u = g + s["beta"] * s["mom"] if s["case"]["nesterov"] else s["mom"]
        return (s["mom"], u.to(s["u"].dtype))
    s["master"].mul_(1 - s["lr"] * s["decay"]).sub_(s["lr"] * (s["k"] * s["o"].float()))
    return (s["master"], s["master"].to(s["weights"].dtype))


# ---------------------------------------------------------------------------
# the framework's calls


def _calls(s):
    import zero_sharded_mixed_flatten_amd as zs
    case = s["case"]
    op = case["op"]
    if op == "layernorm":
        zs.zero_layernorm(s["x"], s["w"], s["b"], s["y"], eps=_EPS_NORM, mean=s["mean"],
                          rstd=s["rstd"])
        return (s["y"], s["mean"], s["rstd"]) if s["mean"] is not None else (s["y"],)
    if op == "layernorm_backward":
        for i, b in enumerate(s["micro"]):
            zs.zero_layernorm_backward(b["dy"], b["x"], s["w"], b["mean"], b["rstd"], b["dx"],
                                       residual=b["residual"], dw=s["dw"], db=s["db"],
                                       accumulate=i > 0, workspace=s["workspace"])
        return ([b["dx"] for b in s["micro"]], s["dw"], s["db"])
    if op == "orthogonalize":
        zs.zero_orthogonalize(s["u"], s["o"], steps=_STEPS, eps=_EPS_ORTH,
                              workspace=s["workspace"])
        return s["o"]
    n, lead = case["length"], case["lead"]
    if op == "muon_momentum":
        zs.zero_muon_momentum(s["grads"], case["n_dp"], n, n, s["mom"], s["u"], s["hp"],
                              nesterov=case["nesterov"])
        return (s["mom"], s["u"])
    zs.zero_muon_update(s["o"], s["master"], s["weights"], s["layout"], 0, s["hp"],
                        update_scale=s["k"], shard_off=lead, length=n)
    return (s["master"], s["weights"][lead:])


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_orthogonalize(u):
    """X after k rounds is P_k X_0 with P_k a polynomial of A_0 = X_0 X_0^T, and so is A_k"""
    out = torch.empty(u.shape, dtype=torch.float64, device=u.device)
    a, b, c = _COEFFS
    for i in range(u.shape[0]):
        x = u[i].double()
        flip = x.shape[0] > x.shape[1]
        x = (x.t() if flip else x).contiguous()
        x = x / (torch.linalg.vector_norm(x) + _EPS_ORTH)
        p, gram = None, x @ x.t().contiguous()
        for _ in range(_STEPS):
            f = b * gram + c * gram @ gram
            f.diagonal().add_(a)
            gram = f @ gram @ f
            gram = 0.5 * (gram + gram.t())
            p = f if p is None else f @ p
        y = p @ x
        out[i] = y.t() if flip else y
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "layernorm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = torch.rsqrt(var + _EPS_NORM)
        y = rstd[:, None] * (s["w"].double() * x) - (rstd * mean)[:, None] * s["w"].double()
        if s["b"] is not None:
            y += s["b"].double()
        return (y, mean, rstd) if case["stats"] else (y,)
    if op == "layernorm_backward":
        n, dxs = case["n"], []
        dw = torch.zeros(n, dtype=torch.float64, device="cuda")
        db = torch.zeros_like(dw)
        for b in s["micro"]:
            dy, r = b["dy"].double(), b["rstd"].double()
            c = b["x"].double() - b["mean"].double()[:, None]
            dw += torch.mv(torch.mul(dy, c).t(), r)
            db += torch.mv(dy.t(), torch.ones_like(r))
            w = s["w"].double()
            s1, s2 = torch.mv(dy, w), torch.mv(dy * c, w)
            dx = r[:, None] * (dy * w) - (r * s1 / n)[:, None] - c * (r ** 3 * s2 / n)[:, None]
            dxs.append(dx if b["residual"] is None else dx + b["residual"].double())
        return (dxs, dw, db)
    if op == "orthogonalize":
        return _exact_orthogonalize(s["u"])
    if op == "muon_momentum":
        g = torch.zeros(case["length"], dtype=torch.float64, device="cuda")
        for row in s["grads"]:
            g += row
        g *= s["scale"]
        mom = torch.add(g, s["mom"].double(), alpha=s["beta"])
        return (mom, torch.add(g, mom, alpha=s["beta"]) if case["nesterov"] else mom)
    w = s["master"].double()
    w = w - s["lr"] * (s["decay"] * w + s["k"] * s["o"].double())
    return (w, w)
