"""Measured cases of the linear-layer operators: the products of a layer with
their epilogues, the layer's backward pass, the 8-bit saved activations it
reads, and the same products grouped by expert.

``run`` computes each operator in its plain form (elementary torch operations
in fp32, rounded once) or, where ``own`` is true, through the library.

Definitions (t tokens, n output features, k input features, e the group that
token t belongs to):

    z[t,n]  = sum_k x[t,k] w[e,n,k] + bias[e,n]
    y[t,n]  = act(z[t,n]) + residual[t,n]
    dz[t,n] = dy[t,n] act'(z[t,n])
    dx[t,k] = sum_n dz[t,n] w[e,n,k]
    dw[e,n,k] = sum_{t in e} dz[t,n] x[t,k]      db[e,n] = sum_{t in e} dz[t,n]

An activation saved in 8 bits holds, for each row and each run of ``block``
columns, scale = amax / 127 and code = rint(v * (127 / amax)); what it gives
back is bf16(code * scale), and the backward pass computes with that value.
"""

import math
import random

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # one token through a key projection: latency, and the weight's bytes
        dict(name="forward, one token", op="forward", tokens=1, inputs=8192, outputs=1024, groups=1,
             act="none", bias=True, residual=False, save=0),
        # an attention output projection of 2,880 columns with bias, onto the residual stream
        dict(name="forward, 2049 tokens", op="forward", tokens=2049, inputs=4096, outputs=2880, groups=1,
             act="none", bias=True, residual=True, save=0),
        # a 70B model's gate projection in training, its input to the activation saved in 8 bits
        dict(name="forward, 8192 tokens", op="forward", tokens=8192, inputs=8192, outputs=28672, groups=1,
             act="silu", bias=False, residual=False, save=128),
        # saving and restoring the activations of a short ragged batch
        dict(name="save, 1000 x 2880", op="save", tokens=1000, inputs=2880, save=64),
        # ... and of a long one
        dict(name="save, 16384 x 8192", op="save", tokens=16384, inputs=8192, save=128),
        # a low-rank query projection on a short sequence, gradients in fp32
        dict(name="backward, 77 tokens", op="backward", tokens=77, inputs=7168, outputs=1536, groups=1,
             act="none", bias=True, saved=0, wide=True),
        # a small model's feed-forward layer with bias, from bf16 activations
        dict(name="backward, 4001 tokens", op="backward", tokens=4001, inputs=2880, outputs=5760, groups=1,
             act="gelu", bias=True, saved=0, wide=False),
        # the 70B gate projection's backward pass from 8-bit activations
        dict(name="backward, 8192 tokens, 8 bits", op="backward", tokens=8192, inputs=8192, outputs=28672, groups=1,
             act="silu", bias=False, saved=128, wide=False),
        # single tokens of 64 sequences routed to 32 experts with biases
        dict(name="experts forward, 64 tokens", op="forward", tokens=64, inputs=2880, outputs=5760, groups=32,
             act="none", bias=True, residual=False, save=0),
        # a training batch over 32 experts of 2,048 x 7,168
        dict(name="experts forward, 16384 tokens", op="forward", tokens=16384, inputs=7168, outputs=2048, groups=32,
             act="silu", bias=False, residual=False, save=128),
        # few tokens for each expert, with biases
        dict(name="experts backward, 500 tokens", op="backward", tokens=500, inputs=2880, outputs=2880, groups=16,
             act="none", bias=True, saved=0, wide=True),
        # the training batch's backward pass from 8-bit activations
        dict(name="experts backward, 16384 tokens", op="backward", tokens=16384, inputs=7168, outputs=2048, groups=32,
             act="silu", bias=False, saved=128, wide=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def features(hi):
        n = max(8, spread(64, hi) // 8 * 8)
        return n + rng.randint(1, 7) if rng.random() < 0.15 else n

    op = rng.choice(("forward", "forward", "backward", "backward", "save"))
    if op == "save":
        return dict(op=op, tokens=spread(1, 16384), inputs=features(8192), save=rng.choice((32, 64, 128)))
    groups = rng.choice((1, 1, rng.randint(2, 64)))
    tokens = spread(1, 8192)
    inputs, outputs = features(8192), features(8192 if groups == 1 else 4096)
    act = rng.choice(ACTS)
    c = dict(op=op, tokens=tokens, inputs=inputs, outputs=outputs, groups=groups, act=act, bias=rng.random() < 0.5)
    if op == "forward":
        return dict(c, residual=rng.random() < 0.5, save=rng.choice((0, 0, 32, 64, 128)))
    return dict(c, saved=rng.choice((0, 32, 64, 128)), wide=act == "none" and rng.random() < 0.5)


def lengths(case):
    """Tokens of each group: ragged, about one group in eight empty."""
    tokens, groups = case["tokens"], case["groups"]
    if groups == 1:
        return [tokens]
    r = random.Random(tokens * 8191 + groups * 131 + case["inputs"])
    share = [0.0 if r.random() < 0.125 else math.exp(0.6 * r.gauss(0, 1)) for _ in range(groups)]
    share[r.randrange(groups)] = 1.0
    total, at, edges = sum(share), 0.0, [0]
    for s in share:
        at += s
        edges.append(int(round(tokens * at / total)))
    return [b - a for a, b in zip(edges, edges[1:])]


# ---------------------------------------------------------------------------
# what a program has in hand

def pack_plain(v, block):
    """fp32 values [rows, cols] -> (codes as fp32, scales): each row's runs of `block` columns."""
    rows, cols = v.shape
    runs = F.pad(v, (0, -cols % block)).reshape(rows, -1, block)
    amax = runs.abs().amax(-1, keepdim=True)
    up = torch.where(amax < 2.0 ** -100, 2.0 ** 64, 1.0)
    codes = torch.where(amax > 0, torch.round(runs * up * (127.0 / (amax * up))), torch.zeros_like(runs))
    return codes.reshape(rows, -1)[:, :cols], (amax / 127.0).squeeze(-1)


def restore_plain(codes, scales, block):
    """bf16(code * scale), in fp32."""
    wide = scales.repeat_interleave(block, 1)[:, :codes.shape[1]]
    return (codes.float() * wide).to(torch.bfloat16).float()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def bf16(v):
        return v.to(torch.bfloat16)

    T, K = case["tokens"], case["inputs"]
    s = dict(case=case)
    # activations: some channels are many times the others
    x = bf16(normal(T, K) * torch.exp(0.8 * normal(K)))
    if case["op"] == "save":
        b = case["save"]
        s.update(x=x, codes=torch.empty(T, K, dtype=torch.int8, device=DEV),
                 scales=torch.empty(T, -(-K // b), dtype=torch.float32, device=DEV), out=torch.empty_like(x))
        return s
    N, E = case["outputs"], case["groups"]
    s["w"] = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        s["w"][e] = bf16(normal(N, K) * (K ** -0.5))
    if E == 1:
        s["w"] = s["w"][0]
        s["offsets"] = None
    else:
        n = lengths(case)
        s["offsets"] = torch.tensor([sum(n[:e]) for e in range(E + 1)], dtype=torch.int64, device=DEV)
        s["longest"] = max(n)  # the plain form's padded batch
    s["bias"] = bf16(0.2 * (normal(E, N) if E > 1 else normal(N))) if case["bias"] else None
    if case["op"] == "forward":
        b = case["save"]
        s.update(x=x, residual=bf16(normal(T, N)) if case["residual"] else None,
                 y=torch.empty(T, N, dtype=torch.bfloat16, device=DEV))
        if b:
            s.update(codes=torch.empty(T, N, dtype=torch.int8, device=DEV),
                     scales=torch.empty(T, -(-N // b), dtype=torch.float32, device=DEV),
                     z=torch.empty(T, N, dtype=torch.bfloat16, device=DEV))
        return s
    # gradients: small, of another size in each row
    s["dy"] = bf16(1e-3 * normal(T, N) * torch.exp(0.5 * normal(T, 1)))
    z = bf16(1.5 * normal(T, N)) if case["act"] != "none" else None
    b = case["saved"]
    for key, v in (("x", x), ("z", z)):
        if b and v is not None:
            codes, scales = pack_plain(v.float(), b)
            s[key] = (codes.to(torch.int8), scales)
        else:
            s[key] = v
    grad = torch.float32 if case["wide"] else torch.bfloat16
    s.update(dx=torch.empty(T, K, dtype=torch.bfloat16, device=DEV), dw=torch.empty_like(s["w"], dtype=grad),
             db=torch.empty((E, N) if E > 1 else (N,), dtype=grad, device=DEV) if case["bias"] else None)
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"save": own_save, "forward": own_forward, "backward": own_backward}[op](s)
    return {"save": plain_save, "forward": plain_forward, "backward": plain_backward}[op](s)


def own_save(s):
    import ragged_shard_optimizer_amd as ve
    q = ve.Act8(s["codes"], s["scales"], s["case"]["save"])
    ve.act8_pack(s["x"], q)
    ve.act8_unpack(q, s["out"])
    return {"restored": s["out"], "scales": s["scales"]}


def own_forward(s):
    import ragged_shard_optimizer_amd as ve
    c = s["case"]
    q = ve.Act8(s["codes"], s["scales"], c["save"]) if c["save"] else None
    ve.linear_forward(s["x"], s["w"], s["y"], bias=s["bias"], activation=c["act"], residual=s["residual"], z8=q,
                      offsets=s["offsets"])
    if q is None:
        return {"y": s["y"]}
    ve.act8_unpack(q, s["z"])
    return {"y": s["y"], "z": s["z"]}


def own_backward(s):
    import ragged_shard_optimizer_amd as ve
    c = s["case"]
    x, z = (ve.Act8(*s[k], c["saved"]) if isinstance(s[k], tuple) else s[k] for k in ("x", "z"))
    ve.linear_backward(s["dy"], s["w"], x=x, z=z, activation=c["act"], dx=s["dx"], dw=s["dw"], dbias=s["db"],
                       offsets=s["offsets"])
    return {"dx": s["dx"], "dw": s["dw"]} if s["db"] is None else {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def act_plain(name, z):
    if name == "relu":
        return torch.clamp_min(z, 0)
    if name == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope_plain(name, z):
    if name == "relu":
        return (z > 0).float()
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def padded(s, v):
    """Rows [T, C] of ragged groups -> [groups, longest, C], zeros behind each group's rows."""
    off = s["offsets"]
    at = torch.arange(s["longest"], device=DEV)
    inside = at < (off[1:] - off[:-1])[:, None]
    rows = (off[:-1, None] + at).clamp_max(v.shape[0] - 1)
    return v[rows] * inside[..., None]


def joined(s, v, tokens):
    """The rows of padded groups, in token order."""
    t = torch.arange(tokens, device=DEV)
    e = torch.searchsorted(s["offsets"][1:], t, right=True)
    return v[e, t - s["offsets"][e]]


def plain_save(s):
    b = s["case"]["save"]
    codes, scales = pack_plain(s["x"].float(), b)
    return {"restored": restore_plain(codes, scales, b).to(torch.bfloat16), "scales": scales}


def plain_forward(s):
    c, w = s["case"], s["w"].float()
    if s["offsets"] is None:
        z = s["x"].float() @ w.t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
    else:
        z = torch.bmm(padded(s, s["x"].float()), w.transpose(1, 2))
        if s["bias"] is not None:
            z = z + s["bias"].float()[:, None]
        z = joined(s, z, c["tokens"])
    y = act_plain(c["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if not c["save"]:
        return {"y": y.to(torch.bfloat16)}
    return {"y": y.to(torch.bfloat16),
            "z": restore_plain(*pack_plain(z, c["save"]), c["save"]).to(torch.bfloat16)}


def plain_backward(s):
    c, w = s["case"], s["w"].float()
    x, z = (restore_plain(*s[k], c["saved"]) if isinstance(s[k], tuple) else None if s[k] is None else s[k].float()
            for k in ("x", "z"))
    dz = s["dy"].float()
    if z is not None:
        dz = dz * slope_plain(c["act"], z)
    if s["offsets"] is None:
        dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    else:
        p = padded(s, dz)
        dx = joined(s, torch.bmm(p, w), c["tokens"])
        dw, db = torch.bmm(p.transpose(1, 2), padded(s, x)), p.sum(1)
    out = {"dx": dx.to(torch.bfloat16), "dw": dw.to(s["dw"].dtype)}
    if s["db"] is not None:
        out["db"] = db.to(s["db"].dtype)
    return out


# ---------------------------------------------------------------------------
# the definition in 64 bits, and what a pass cannot do without

def exact(case, seed):
    s = prepare(case, seed)

    def saved(v, block):
        """(codes * scale rounded to bf16, scale) of 64-bit values, run by run."""
        out, scales = torch.empty_like(v), []
        for a in range(0, v.shape[1], block):
            run_ = v[:, a:a + block]
            m = run_.abs().max(1, keepdim=True).values
            step = m / 127
            q = torch.where(m > 0, torch.round(run_ * (127 / torch.where(m > 0, m, 1.0))), 0.0)
            out[:, a:a + block] = (q * step).to(torch.bfloat16).double()
            scales.append(step[:, 0])
        return out, torch.stack(scales, 1)

    def value(v):
        if not isinstance(v, tuple):
            return v.double()
        codes, scales = v[0].double(), v[1].double()
        for j in range(scales.shape[1]):
            codes[:, j * case["saved"]:(j + 1) * case["saved"]] *= scales[:, j:j + 1]
        return codes.to(torch.bfloat16).double()

    if case["op"] == "save":
        restored, scales = saved(s["x"].double(), case["save"])
        return {"restored": restored, "scales": scales}
    edges = [0]
    for n in lengths(case):
        edges.append(edges[-1] + n)
    parts = list(zip(range(case["groups"]), edges, edges[1:]))
    weight = lambda e: (s["w"] if case["groups"] == 1 else s["w"][e]).double()  # noqa: E731
    name = case["act"]
    if case["op"] == "forward":
        z = torch.zeros(case["tokens"], case["outputs"], dtype=torch.float64, device=DEV)
        for e, a, b in parts:
            z[a:b] = torch.mm(s["x"][a:b].double(), weight(e).t())
            if case["bias"]:
                z[a:b] += (s["bias"] if case["groups"] == 1 else s["bias"][e]).double()
        if name == "relu":
            y = z.clamp(min=0)
        elif name == "gelu":
            y = z * torch.special.ndtr(z)
        elif name == "gelu_tanh":
            y = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        elif name == "silu":
            y = z * torch.sigmoid(z)
        else:
            y = z.clone()
        if case["residual"]:
            y += s["residual"].double()
        return {"y": y, "z": saved(z, case["save"])[0]} if case["save"] else {"y": y}
    x, dz = value(s["x"]), s["dy"].double()
    if name != "none":
        z = value(s["z"])
        if name == "relu":
            dz = torch.where(z > 0, dz, torch.zeros_like(dz))
        elif name == "gelu":
            dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        elif name == "gelu_tanh":
            u = 2 * math.sqrt(2 / math.pi)
            q = torch.sigmoid(u * (z + 0.044715 * z ** 3))
            dz = dz * (q + z * q * (1 - q) * u * (1 + 3 * 0.044715 * z * z))
        else:
            q = torch.sigmoid(z)
            dz = dz * (q + z * q * (1 - q))
    dx = torch.zeros(case["tokens"], case["inputs"], dtype=torch.float64, device=DEV)
    dw = torch.zeros(case["groups"], case["outputs"], case["inputs"], dtype=torch.float64, device=DEV)
    db = torch.zeros(case["groups"], case["outputs"], dtype=torch.float64, device=DEV)
    for e, a, b in parts:
        if b > a:
            dx[a:b] = torch.mm(dz[a:b], weight(e))
            dw[e] = torch.mm(dz[a:b].t(), x[a:b])
            db[e] = dz[a:b].sum(0)
    out = {"dx": dx, "dw": dw if case["groups"] > 1 else dw[0]}
    if case["bias"]:
        out["db"] = db if case["groups"] > 1 else db[0]
    return out


def work(case):
    T, K = case["tokens"], case["inputs"]

    def saved(cols, block):  # bytes of one activation matrix: bf16, or codes and scales
        return T * (cols + 4 * -(-cols // block)) if block else 2 * T * cols

    if case["op"] == "save":
        return {"bytes": 2 * T * K + 2 * saved(K, case["save"]) + 2 * T * K, "flops": 0}
    N, n = case["outputs"], lengths(case)
    used = sum(v > 0 for v in n)
    weights = 2 * used * N * K + (2 * used * N if case["bias"] else 0)
    if case["op"] == "forward":
        moved = 2 * T * K + weights + 2 * T * N * (2 if case["residual"] else 1)
        if case["save"]:
            moved += 2 * saved(N, case["save"]) + 2 * T * N
        return {"bytes": moved, "flops": 2 * T * N * K}
    grad = 4 if case["wide"] else 2
    moved = 2 * T * N + 2 * used * N * K + 2 * T * K + saved(K, case["saved"]) + grad * case["groups"] * N * K
    if case["act"] != "none":
        moved += saved(N, case["saved"])
    if case["bias"]:
        moved += grad * case["groups"] * N
    return {"bytes": moved, "flops": 4 * T * N * K}
