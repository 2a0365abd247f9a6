"""The layer products on the flat 16-bit buffers and the counter-based
dropout: the cases they are measured on, their plain forms and their
definitions in 64 bits.

A parameter's matrix is read where the all-gather leaves it, in the flat
weight buffer, and its gradient is written where the reduce-scatter takes it
from, in a flat gradient row; both start at whatever element the flat layout
gives the parameter.  Four operators:

  linear   y = residual + D(act(z)),  z = x W^T + b      (and z itself)
  dgrad    dx = residual + D(act'(z) * (dy W))
  wgrad    dW (+)= dy^T x,  db (+)= sum over rows of dy   (micro-batches)
  dropout  y = residual + D(x)

D keeps an element when 16 bits of Philox4x32-10 are at least T =
rint(65536 p) and multiplies it by 65536 / (65536 - T); a dropped element is
0 whatever it was.  The generator's counter is (column block, row, stream
low, stream high) and its key the seed: the block of column c is
(c // 32) * 4 + (c % 16) // 4, and of that block's four words column c takes
word c % 4, its low half when c % 32 < 16, else its high half.  The stream
is the call's offset plus a step counter in device memory, so that a
captured graph draws a new mask at every replay.

`own` False: elementary torch operations in 32 bits.  `own` True: the calls
a user makes of zero_sharded_mixed_flatten_amd.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

_LINEAR = dict(op="linear", type="bf16", out="same", bias=False, act="none", p=0.0,
               residual=False, keep_z=False, pad=0, lead=0)
_DGRAD = dict(op="dgrad", type="bf16", out="same", act="none", p=0.0, residual=False, pad=0,
              lead=0)
_WGRAD = dict(op="wgrad", type="bf16", grad="f32", bias=False, micro=1, pad=0, lead=0)
_DROPOUT = dict(op="dropout", type="bf16", p=0.1, residual=False, pad=0)


def listed():
    return [
        # one new token through the GPT-2-XL list's first MLP matrix: latency and the
        # weight's bytes
        dict(_LINEAR, name="linear_token_gpt2xl_up", m=1, n=6400, k=1600, bias=True,
             act="gelu_tanh"),
        # a batch of 16 new tokens through the 7B list's down matrix
        dict(_LINEAR, name="linear_16_tokens_7b_down", m=16, n=4096, k=11008, residual=True),
        # training, GPT-2-XL list, MLP up: bias, GELU, the pre-activation kept for backward
        dict(_LINEAR, name="linear_gpt2xl_up_train", m=8192, n=6400, k=1600, bias=True,
             act="gelu_tanh", keep_z=True),
        # training, 7B list's down matrix with dropout and the residual: the largest product
        dict(_LINEAR, name="linear_7b_down_train", m=8192, n=4096, k=11008, residual=True, p=0.1),
        # logits of a short fp16 batch over an odd vocabulary, at an odd place of the buffer
        dict(_LINEAR, name="linear_logits_ragged", m=333, n=50257, k=1600, type="f16", out="f32",
             lead=5),
        # backward through the GPT-2-XL list's MLP down matrix into GELU's input
        dict(_DGRAD, name="dgrad_gpt2xl_down", m=8192, n=1600, k=6400, act="gelu_tanh"),
        # a short ragged fp16 sequence: SiLU, dropout, padded rows
        dict(_DGRAD, name="dgrad_ragged", m=77, n=2001, k=1333, type="f16", act="silu", p=0.2,
             pad=3, lead=1),
        # weight gradient of the 7B list's MLP over two micro-batches, summed in fp32 rows
        dict(_WGRAD, name="wgrad_7b_accumulated", m=4096, n=11008, k=4096, micro=2),
        # weight and bias gradient of the GPT-2-XL list's projection, in bf16 rows
        dict(_WGRAD, name="wgrad_gpt2xl_proj", m=4096, n=1600, k=1600, grad="same", bias=True),
        # dropout of one token's row
        dict(_DROPOUT, name="dropout_token", m=1, n=1600, p=0.1),
        # dropout of a training batch's activations into the residual stream
        dict(_DROPOUT, name="dropout_train_residual", m=16384, n=4096, residual=True),
        # an fp32 batch of odd shape with padded rows
        dict(_DROPOUT, name="dropout_f32_ragged", m=2047, n=6401, type="f32", p=0.5, pad=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "dgrad", "wgrad", "dropout"])
    most = work(listed()[3])
    while True:
        m = 1 if rng.random() < 0.1 else _log(rng, 1, 16384)
        n, k = _log(rng, 48, 50257), _log(rng, 48, 12288)
        if rng.random() < 0.5:  # layers are mostly round, but not all of them
            n, k = -(-n // 64) * 64, -(-k // 64) * 64
        pad, lead = rng.choice([0, 0, 8, 3]), rng.choice([0, 0, 0, 8, 5])
        if op == "linear":
            case = dict(_LINEAR, type=rng.choice(["bf16", "bf16", "f16"]),
                        out=rng.choice(["same", "same", "f32"]), bias=rng.random() < 0.5,
                        act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                        p=rng.choice([0.0, 0.0, 0.1, 0.35]), residual=rng.random() < 0.5,
                        keep_z=rng.random() < 0.3)
        elif op == "dgrad":
            case = dict(_DGRAD, type=rng.choice(["bf16", "bf16", "f16"]),
                        out=rng.choice(["same", "same", "f32"]),
                        act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                        p=rng.choice([0.0, 0.0, 0.1, 0.35]), residual=rng.random() < 0.3)
        elif op == "wgrad":
            case = dict(_WGRAD, type=rng.choice(["bf16", "bf16", "f16"]),
                        grad=rng.choice(["f32", "same"]), bias=rng.random() < 0.5,
                        micro=rng.choice([1, 1, 2]))
        else:
            case = dict(_DROPOUT, type=rng.choice(["bf16", "f16", "f32"]),
                        p=rng.choice([0.05, 0.1, 0.5, 0.9]), residual=rng.random() < 0.5)
            lead = 0
            k = 0
        case.update(m=m, n=n, pad=pad)
        if op != "dropout":
            case.update(k=k, lead=lead)
        w = work(case)
        if w["flops"] <= most["flops"] and w["bytes"] <= 1.2e9:
            return case


def work(case):
    m, n, op = case["m"], case["n"], case["op"]
    e = 4 if case["type"] == "f32" else 2
    if op == "dropout":
        return {"bytes": m * n * e * (3 if case["residual"] else 2), "flops": 2 * m * n}
    k = case["k"]
    if op == "wgrad":
        g = 4 if case["grad"] == "f32" else 2
        first = m * n * 2 + m * k * 2 + (n * k + (n if case["bias"] else 0)) * g
        later = first + (n * k + (n if case["bias"] else 0)) * g
        return {"bytes": first + (case["micro"] - 1) * later,
                "flops": 2 * m * n * k * case["micro"]}
    o = 4 if case["out"] == "f32" else 2
    rows_in, rows_out = (m * k, m * n) if op == "linear" else (m * n, m * k)
    b = 2 * (rows_in + n * k) + rows_out * o * (2 if case["residual"] else 1)
    if op == "linear":
        b += 2 * (n if case["bias"] else 0) + 2 * (rows_out if case["keep_z"] else 0)
    elif case["act"] != "none":
        b += 2 * rows_out
    return {"bytes": b, "flops": 2 * m * n * k}


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


def prepare(case, seed):
    g = _Maker(seed)
    m, n, pad, op = case["m"], case["n"], case["pad"], case["op"]
    t = _TYPES[case["type"]]
    s = {"case": case}
    if op == "dropout":
        s["x"] = g.rows(m, n, pad, 1.0, t)
        s["residual"] = g.rows(m, n, pad, 1.0, t) if case["residual"] else None
        s["y"] = _empty_rows(m, n, pad, t)
    elif op in ("linear", "dgrad"):
        k, lead = case["k"], case["lead"]
        out = torch.float32 if case["out"] == "f32" else t
        # the flat weight buffer: other parameters, the matrix, its bias
        weights = g.flat(lead + n * k + n, 0.02, t)
        s["w"] = weights[lead:lead + n * k].view(n, k)
        if op == "linear":
            s["x"] = g.rows(m, k, pad, 1.0, t)
            s["bias"] = weights[lead + n * k:] if case["bias"] else None
            s["residual"] = g.rows(m, n, pad, 1.0, out) if case["residual"] else None
            s["y"] = _empty_rows(m, n, pad, out)
            s["z"] = _empty_rows(m, n, pad, t) if case["keep_z"] else None
        else:
            s["dy"] = g.rows(m, n, pad, 1.0, t)
            s["z"] = g.rows(m, k, pad, 1.0, t) if case["act"] != "none" else None
            s["residual"] = g.rows(m, k, pad, 1.0, out) if case["residual"] else None
            s["dx"] = _empty_rows(m, k, pad, out)
    else:
        k, lead = case["k"], case["lead"]
        gt = torch.float32 if case["grad"] == "f32" else t
        s["dy"] = [g.rows(m, n, pad, 1.0, t) for _ in range(case["micro"])]
        s["x"] = [g.rows(m, k, pad, 1.0, t) for _ in range(case["micro"])]
        row = torch.zeros(lead + n * k + n, dtype=gt, device="cuda")  # the flat gradient row
        s["dw"] = row[lead:lead + n * k].view(n, k)
        s["db"] = row[lead + n * k:] if case["bias"] else None
    if case.get("p"):
        s["seed"], s["offset"] = (0x9E3779B97F4A7C15 * (seed + 1)) % (1 << 63), 1000 * seed
        s["step"] = torch.tensor([7 + seed % 5], dtype=torch.int64, device="cuda")
    if own:
        import zero_sharded_mixed_flatten_amd as zs
        s["drop"] = zs.ZeroDropout(p=case["p"], seed=s["seed"], offset=s["offset"],
                                   step=s["step"]) if case.get("p") else None
        if op != "dropout":
            which = {"linear": zs.ZERO_LINEAR, "dgrad": zs.ZERO_LINEAR_DGRAD,
                     "wgrad": zs.ZERO_LINEAR_WGRAD}[op]
            s["act"] = {"none": zs.ZERO_ACT_NONE, "relu": zs.ZERO_ACT_RELU,
                        "gelu": zs.ZERO_ACT_GELU, "gelu_tanh": zs.ZERO_ACT_GELU_TANH,
                        "silu": zs.ZERO_ACT_SILU}[case.get("act", "none")]
            s["workspace"] = torch.empty(zs.zero_linear_workspace_bytes(which, m, n, case["k"]),
                                         dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the plain forms: 32 bits, elementary operations

_M0, _M1 = 0xD2511F53, 0xCD9E8D57
_W0, _W1 = 0x9E3779B9, 0xBB67AE85


def _mul32(a, c):
    """high and low 32 bits of a * c, a an int64 tensor of 32-bit values"""
    lo, hi = a * (c & 0xFFFF), a * (c >> 16)            # each below 2^48
    mid = (lo >> 16) + (hi & 0xFFFFFFFF)                # (a c) >> 16, its low parts
    return (((hi >> 32) << 16) + (mid >> 16)) & 0xFFFFFFFF, \
        ((mid << 16) | (lo & 0xFFFF)) & 0xFFFFFFFF


def _keep(m, n, p, seed, stream):
    """True where D keeps the element, for rows 0..m-1 and columns 0..n-1"""
    groups = -(-n // 32)
    c0 = torch.arange(groups * 4, device="cuda").view(1, -1).expand(m, -1)
    c1 = torch.arange(m, device="cuda").view(-1, 1).expand(-1, groups * 4)
    c2 = (stream & 0xFFFFFFFF).expand(m, groups * 4)
    c3 = (stream >> 32).expand(m, groups * 4)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mul32(c0, _M0)
        h1, l1 = _mul32(c2, _M1)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + _W0) & 0xFFFFFFFF, (k1 + _W1) & 0xFFFFFFFF
    words = torch.stack([c0, c1, c2, c3], -1).view(m, groups, 1, 16)  # [group][block][word]
    u = torch.cat([words & 0xFFFF, words >> 16], 2).reshape(m, groups * 32)[:, :n]
    return u >= _threshold(p)


def _threshold(p):
    return min(65535, int(round(p * 65536)))


def _drop(v, s):
    p = s["case"].get("p")
    if not p:
        return v
    keep = _keep(v.shape[0], v.shape[1], p, s["seed"], s["step"] + s["offset"])
    scale = 65536.0 / (65536 - _threshold(p))
    return torch.where(keep, v * scale, torch.zeros_like(v))


def _act(v, name):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _act_grad(v, name):
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + \
            v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * c * (1 + 3 * 0.044715 * v * v)
    sg = 1 / (1 + torch.exp(-v))
    return sg * (1 + v * (1 - sg))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "dropout":
        y = _drop(s["x"].float(), s)
        if s["residual"] is not None:
            y = s["residual"].float() + y
        return y.to(s["y"].dtype)
    if op == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _drop(_act(z, case["act"]), s)
        if s["residual"] is not None:
            y = s["residual"].float() + y
        return (y.to(s["y"].dtype), z.to(s["z"].dtype) if s["z"] is not None else None)
    if op == "dgrad":
        d = s["dy"].float() @ s["w"].float()
        if case["act"] != "none":
            d = d * _act_grad(s["z"].float(), case["act"])
        d = _drop(d, s)
        if s["residual"] is not None:
            d = s["residual"].float() + d
        return d.to(s["dx"].dtype)
    dw = db = None
    for dy, x in zip(s["dy"], s["x"]):  # each micro-batch's sum is rounded to the row's type
        w = dy.float().t() @ x.float()
        b = dy.float().sum(0)
        dw = (w if dw is None else dw.float() + w).to(s["dw"].dtype)
        db = (b if db is None else db.float() + b).to(s["dw"].dtype)
    return (dw, db if s["db"] is not None else None)


# ---------------------------------------------------------------------------
# the framework's calls


def _calls(s):
    import zero_sharded_mixed_flatten_amd as zs
    op = s["case"]["op"]
    if op == "dropout":
        zs.zero_dropout(s["x"], s["y"], s["drop"], residual=s["residual"])
        return s["y"]
    if op == "linear":
        zs.zero_linear(s["x"], s["w"], s["y"], bias=s["bias"], act=s["act"], drop=s["drop"],
                       residual=s["residual"], z=s["z"], workspace=s["workspace"])
        return (s["y"], s["z"])
    if op == "dgrad":
        zs.zero_linear_dgrad(s["dy"], s["w"], s["dx"], act=s["act"], z=s["z"], drop=s["drop"],
                             residual=s["residual"], workspace=s["workspace"])
        return s["dx"]
    for i, (dy, x) in enumerate(zip(s["dy"], s["x"])):
        zs.zero_linear_wgrad(dy, x, s["dw"], db=s["db"], accumulate=i > 0,
                             workspace=s["workspace"])
    return (s["dw"], s["db"])


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _philox_words(c, key):
    """Philox4x32-10 of counter arrays c (four uint64 arrays of 32-bit values)"""
    mask = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    key = [key & 0xFFFFFFFF, key >> 32]
    for r in range(10):
        p0, p1 = c[0] * np.uint64(_M0), c[2] * np.uint64(_M1)
        c = [(p1 >> s32) ^ c[1] ^ np.uint64((key[0] + r * _W0) & 0xFFFFFFFF), p1 & mask,
             (p0 >> s32) ^ c[3] ^ np.uint64((key[1] + r * _W1) & 0xFFFFFFFF), p0 & mask]
    return c


def _factor64(m, n, case, s):
    """0 or 1 / (1 - T / 65536) for every element, float64 on the host"""
    t = _threshold(case["p"])
    stream = s["offset"] + int(s["step"].item())
    blocks = (n + 31) // 32 * 4
    out = np.zeros((m, n))
    for r0 in range(0, m, 2048):
        rows = np.arange(r0, min(m, r0 + 2048), dtype=np.uint64)[:, None]
        b = np.arange(blocks, dtype=np.uint64)[None, :]
        zero = np.zeros((len(rows), blocks), np.uint64)
        w = _philox_words([zero + b, zero + rows, zero + np.uint64(stream & 0xFFFFFFFF),
                           zero + np.uint64(stream >> 32)], s["seed"])
        for word in range(4):
            for half in range(2):
                u = (w[word] >> np.uint64(16 * half)) & np.uint64(0xFFFF)
                col = np.arange(blocks) // 4 * 32 + 16 * half + np.arange(blocks) % 4 * 4 + word
                ok = col < n
                out[r0:r0 + len(rows), col[ok]] = (u[:, ok] >= np.uint64(t)) / (1 - t / 65536)
    return torch.from_numpy(out).cuda()


def _act64(z, name):
    """(act(z), act'(z)) in float64"""
    one = torch.ones_like(z)
    if name == "none":
        return z, one
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        return z * torch.sigmoid(z), torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    if name == "gelu":
        phi = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)   # 0.5 (1 + tanh(u / 2)) = sigmoid(u)
    sg = torch.sigmoid(u)
    du = math.sqrt(8 / math.pi) * (1 + 0.134145 * z * z)
    return z * sg, sg + z * sg * torch.sigmoid(-u) * du


def exact(case, seed):
    s = prepare(case, seed)
    op, m = case["op"], case["m"]
    if op == "wgrad":
        dw = sum(dy.double().t() @ x.double() for dy, x in zip(s["dy"], s["x"]))
        db = sum(dy.double().sum(0) for dy in s["dy"]) if case["bias"] else None
        return (dw, db)
    z = None
    if op == "dropout":
        v = s["x"].double()
    elif op == "linear":
        z = s["x"].double() @ s["w"].double().t()
        if case["bias"]:
            z = z + s["bias"].double()
        v = _act64(z, case["act"])[0]
    else:
        v = s["dy"].double() @ s["w"].double()
        if case["act"] != "none":
            v = v * _act64(s["z"].double(), case["act"])[1]
    if case["p"]:
        v = v * _factor64(m, v.shape[1], case, s)
    if case["residual"]:
        v = v + s["residual"].double()
    return (v, z if case["keep_z"] else None) if op == "linear" else v
