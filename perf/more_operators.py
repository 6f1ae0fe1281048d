"""Measured cases of the operators around a layer of experts: tokens sorted by
expert and brought back, with their gradients, matrices packed in 8-bit
floating point, and a linear layer's products on such matrices.

``run`` computes each operator in its plain form (elementary torch operations
in fp32, rounded once) or, where ``own`` is true, through the library.

Definitions (T tokens, k slots a token, E experts, C columns):

    sort     slots (t, j) in the order of their expert, then of t k + j;
             position[t,j] is a slot's place, -1 where the expert is not in
             [0, E); offsets[e] the first place of expert e
    gather   rows[position[t,j]] = x[t]            dx[t] = sum_j drows[position[t,j]]
    combine  y[t] = sum_j weights[t,j] rows[position[t,j]] + residual[t]
             drows[position[t,j]] = weights[t,j] dy[t]
             dweights[t,j] = sum_c dy[t,c] rows[position[t,j],c]
    pack     a block of values v with largest magnitude a: e the smallest
             whole number >= -127 with a <= MAX 2^e (MAX = 448 for E4M3,
             57344 for E5M2), code = the format's nearest value to v 2^-e;
             blocks are runs of 128 columns of a row, runs of 128 rows of a
             group (the transposed matrix), or 128 x 128 (weights)
    forward  y[t,n] = act(sum_k x[t,k] w[e,n,k] + bias[e,n])
    backward dx[t,k] = sum_n dy[t,n] w[e,n,k]      dw[e,n,k] = sum_{t in e} dy[t,n] x[t,k]

with x, w and dy the values that the packed matrices stand for.
"""

import math
import random

import torch

own = False

DEV = "cuda"
FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # eight sequences' single tokens to 8 of 256 experts: latency
        dict(name="dispatch, 8 tokens", op="dispatch", tokens=8, cols=7168, experts=256, slots=8, bits=16, dropped=False,
             grad=False),
        # a ragged prompt to 4 of 128 experts, packed on the way, some slots over capacity
        dict(name="dispatch, 2049 tokens, 8 bits", op="dispatch", tokens=2049, cols=2880, experts=128, slots=4, bits=8,
             dropped=True, grad=False),
        # a training batch to 8 of 256 experts and its gradient back
        dict(name="dispatch + grad, 4096 tokens", op="dispatch", tokens=4096, cols=7168, experts=256, slots=8, bits=16,
             dropped=False, grad=True),
        # single tokens of 64 sequences back onto the residual stream
        dict(name="combine, 64 tokens", op="combine", tokens=64, cols=2880, experts=128, slots=4, residual=True,
             dropped=False, grad=False),
        # the training batch back, with both gradients
        dict(name="combine + grads, 4096 tokens", op="combine", tokens=4096, cols=7168, experts=256, slots=8,
             residual=False, dropped=False, grad=True),
        # a short batch's activations for the forward and the weight gradient's product
        dict(name="pack, 500 x 2880", op="pack", tokens=500, cols=2880, groups=16, format="e4m3"),
        # 16 experts' projections for forward and backward products, once a step
        dict(name="pack, 16 weights", op="weights", groups=16, outputs=2048, inputs=7168),
        # one token through a key projection: latency, and the weight's bytes
        dict(name="forward, one token", op="forward", tokens=1, inputs=8192, outputs=1024, groups=1, act="none",
             bias=True, z=False),
        # 64 sequences' single tokens, 8 slots each, on 64 of the experts
        dict(name="experts forward, 512 rows", op="forward", tokens=512, inputs=7168, outputs=2048, groups=64,
             act="none", bias=False, z=False),
        # a 70B model's gate projection in training
        dict(name="forward, 8192 tokens", op="forward", tokens=8192, inputs=8192, outputs=28672, groups=1, act="silu",
             bias=False, z=True),
        # a short batch over 16 experts, the gradient in the format of the wider range
        dict(name="experts backward, 777 rows", op="backward", tokens=777, inputs=2880, outputs=2880, groups=16,
             format="e5m2", wide=True),
        # a training batch over 32 experts of 2,048 x 7,168
        dict(name="experts backward, 16384 rows", op="backward", tokens=16384, inputs=7168, outputs=2048, groups=32,
             format="e4m3", wide=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def features(hi):
        n = max(8, spread(64, hi) // 8 * 8)
        return n + rng.randint(1, 7) if rng.random() < 0.2 else n

    op = rng.choice(("dispatch", "combine", "pack", "weights", "forward", "forward", "backward", "backward"))
    if op in ("dispatch", "combine"):
        experts = spread(2, 256)
        slots = min(experts, rng.randint(1, 8))
        c = dict(op=op, tokens=spread(1, 32768 // slots), cols=features(7168), experts=experts, slots=slots,
                 dropped=rng.random() < 0.3, grad=rng.random() < 0.5)
        if op == "dispatch":
            return dict(c, bits=rng.choice((16, 8)))
        return dict(c, residual=rng.random() < 0.5)
    if op == "pack":
        return dict(op=op, tokens=spread(1, 8192), cols=features(8192), groups=rng.choice((1, rng.randint(2, 64))),
                    format=rng.choice(tuple(FORMATS)))
    if op == "weights":
        return dict(op=op, groups=rng.randint(1, 16), outputs=features(4096), inputs=features(4096))
    groups = rng.choice((1, 1, rng.randint(2, 64)))
    c = dict(op=op, tokens=spread(1, 8192), inputs=features(8192), outputs=features(8192 if groups == 1 else 4096),
             groups=groups)
    if op == "forward":
        act = rng.choice(("none", "none", "silu", "gelu", "relu"))
        return dict(c, act=act, bias=rng.random() < 0.5, z=act != "none" and rng.random() < 0.5)
    return dict(c, format=rng.choice(tuple(FORMATS)), wide=rng.random() < 0.5)


def lengths(case):
    """Tokens of each group: ragged, about one group in eight empty."""
    tokens, groups = case["tokens"], case["groups"]
    if groups == 1:
        return [tokens]
    r = random.Random(tokens * 8191 + groups * 131)
    share = [0.0 if r.random() < 0.125 else math.exp(0.6 * r.gauss(0, 1)) for _ in range(groups)]
    share[r.randrange(groups)] = 1.0
    total, at, edges = sum(share), 0.0, [0]
    for s in share:
        at += s
        edges.append(int(round(tokens * at / total)))
    return [b - a for a, b in zip(edges, edges[1:])]


def up(n, to):
    return -(-n // to) * to


def columns(case):
    """Columns of a transposed matrix of tokens: each group's are whole runs of 128."""
    tokens = case["tokens"]
    return (tokens + 127 * min(case["groups"], tokens)) // 128 * 128


# ---------------------------------------------------------------------------
# matrices in 8 bits: codes [rows, cols] whose rows start on 16 bytes and end
# in zeros, scale exponents (plus 127) [ceil(cols / 128), ceil(rows / block)]
# whose rows start on 4 bytes

def buffers(rows, cols, block=1, format="e4m3", groups=None):
    lead = () if groups is None else (groups,)
    codes = torch.zeros(*lead, rows, up(cols, 16), dtype=torch.uint8, device=DEV).view(FORMATS[format][0])
    scales = torch.zeros(*lead, -(-cols // 128), up(-(-rows // block), 4), dtype=torch.uint8, device=DEV)
    return codes[..., :cols], scales[..., :-(-rows // block)]


def power(exponent):
    """2^(exponent - 127) for whole numbers in [1, 254]."""
    return (exponent << 23).view(torch.float32)


def blocked(v, block):
    """fp32 [rows, cols] -> [row blocks, block, column runs, 128], zeros behind the ends."""
    rows, cols = v.shape
    p = torch.zeros(up(rows, block), up(cols, 128), dtype=v.dtype, device=v.device)
    p[:rows, :cols] = v
    return p.view(-1, block, p.shape[1] // 128, 128)


def pack_plain(v, block=1, format="e4m3"):
    """fp32 [rows, cols] -> (codes [rows, cols] in the format, exponents [runs, row blocks])."""
    dtype, most = FORMATS[format]
    rows, cols = v.shape
    b = blocked(v, block)
    amax = b.abs().amax((1, 3), keepdim=True)
    frac, exp = torch.frexp(amax)  # amax = frac 2^exp, frac in [0.5, 1)
    top = math.frexp(most)
    e = exp - top[1] + (frac > top[0])
    e = torch.where(amax > 0, (e + 127).clamp_min(0), torch.zeros_like(e)).to(torch.int32)
    codes = (b * power(254 - e)).reshape(-1, b.shape[2] * 128)[:rows, :cols].to(dtype)
    return codes, e[:, 0, :, 0].t().to(torch.uint8)


def restore_plain(codes, exponents, block=1):
    """The values that packed matrices stand for, in fp32 (an exponent of 0: half of 2^-126)."""
    e = exponents.t().to(torch.int32)
    s = power(e.clamp_min(1)) * torch.where(e > 0, 1.0, 0.5)
    rows, cols = codes.shape
    s = s.repeat_interleave(block, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return codes.to(torch.float32) * s


def fill(q, v, block=1, format="e4m3"):
    codes, scales = pack_plain(v, block, format)
    q[0].view(torch.uint8).copy_(codes.view(torch.uint8))
    q[1].copy_(scales)


def places(case):
    """Column of each token in the transposed matrix."""
    at, cols = 0, []
    for n in lengths(case):
        cols += range(at, at + n)
        at += up(n, 128)
    return torch.tensor(cols, dtype=torch.int64, device=DEV)


# ---------------------------------------------------------------------------
# what a program has in hand

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def bf16(v):
        return v.to(torch.bfloat16)

    def rows(n, cols):  # some channels are many times the others
        return bf16(normal(n, cols) * torch.exp(0.8 * normal(cols)))

    def grads(n, cols):  # small, of another size in each row
        return bf16(1e-3 * normal(n, cols) * torch.exp(0.5 * normal(n, 1)))

    op, s = case["op"], dict(case=case)
    if op in ("dispatch", "combine"):
        T, C, E, k = case["tokens"], case["cols"], case["experts"], case["slots"]
        # a router's choice: experts of unequal popularity, no expert twice for a token
        logits = normal(T, E) + 0.7 * normal(E)
        s["ids"] = torch.topk(logits, k, dim=1).indices
        if case["dropped"]:
            s["ids"] = torch.where(torch.rand(T, k, generator=g, device=DEV) < 0.03, -1, s["ids"])
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
        s["position"] = torch.zeros(T, k, dtype=torch.int32, device=DEV)
        if op == "dispatch":
            s["x"] = rows(T, C)
            s["rows"] = torch.zeros(T * k, C, dtype=torch.bfloat16, device=DEV)
            if case["bits"] == 8:
                s["rows8"] = buffers(T * k, C)
            if case["grad"]:
                s["drows"], s["dx"] = grads(T * k, C), torch.zeros(T, C, dtype=torch.bfloat16, device=DEV)
            return s
        s["offsets"], s["position"] = sort_plain(s["ids"], E)
        s["weights"] = torch.softmax(normal(T, k), 1)
        s["rows"] = rows(T * k, C)
        s["residual"] = rows(T, C) if case["residual"] else None
        s["y"] = torch.zeros(T, C, dtype=torch.bfloat16, device=DEV)
        if case["grad"]:
            s.update(dy=grads(T, C), drows=torch.zeros(T * k, C, dtype=torch.bfloat16, device=DEV),
                     dweights=torch.zeros(T, k, device=DEV))
        return s
    if op == "weights":
        E, N, K = case["groups"], case["outputs"], case["inputs"]
        s["w"] = bf16(normal(E, N, K) * (K ** -0.5) * torch.exp(0.3 * normal(E, N, 1)))
        s["w8"], s["w8_t"] = buffers(N, K, 128, groups=E), buffers(K, N, 128, groups=E)
        s["out"], s["out_t"] = torch.zeros_like(s["w"]), torch.zeros(E, K, N, dtype=torch.bfloat16, device=DEV)
        return s
    T, E = case["tokens"], case["groups"]
    s["lengths"] = lengths(case)
    edges = [sum(s["lengths"][:e]) for e in range(E + 1)]
    s["offsets"] = torch.tensor(edges, dtype=torch.int64, device=DEV) if E > 1 else None
    if op == "pack":
        C = case["cols"]
        s["x"], s["places"] = rows(T, C), places(case)
        s["x8"] = buffers(T, C, format=case["format"])
        s["x8_t"] = buffers(C, columns(case), format=case["format"])
        s["out"] = torch.zeros(T, C, dtype=torch.bfloat16, device=DEV)
        s["out_t"] = torch.zeros(C, columns(case), dtype=torch.bfloat16, device=DEV)
        return s
    K, N = case["inputs"], case["outputs"]

    def weights(n, k):
        q = buffers(n, k, 128, groups=E if E > 1 else None)
        for e in range(E):
            fill(q if E == 1 else (q[0][e], q[1][e]), bf16(normal(n, k) * (K ** -0.5)).float(), 128)
        return q

    if op == "forward":
        s["x8"], s["w8"] = buffers(T, K), weights(N, K)
        fill(s["x8"], rows(T, K).float())
        s["bias"] = bf16(0.2 * (normal(E, N) if E > 1 else normal(N))) if case["bias"] else None
        s["y"] = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV)
        s["z"] = torch.zeros_like(s["y"]) if case["z"] else None
        return s
    f, C = case["format"], columns(case)
    s["dy8"], s["dy8_t"], s["x8_t"] = buffers(T, N, format=f), buffers(N, C, format=f), buffers(K, C)
    dy, at = grads(T, N).float(), places(case)
    fill(s["dy8"], dy, format=f)
    for key, v, fmt in (("dy8_t", dy, f), ("x8_t", rows(T, K).float(), "e4m3")):
        wide = torch.zeros(v.shape[1], C, device=DEV)
        wide[:, at] = v.t()
        fill(s[key], wide, format=fmt)
    s["w8_t"] = weights(K, N)
    s["dx"] = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    grad = torch.float32 if case["wide"] else torch.bfloat16
    s["dw"] = torch.zeros(*((E,) if E > 1 else ()), N, K, dtype=grad, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    return globals()[("own_" if own else "plain_") + s["case"]["op"]](s)


def own_dispatch(s):
    import ragged_shard_optimizer_amd as ve
    c = s["case"]
    ve.expert_sort(s["ids"], s["offsets"], s["position"])
    if c["bits"] == 8:
        q = ve.Fp8(*s["rows8"])
        ve.expert_gather(s["x"], s["position"], q)
        ve.fp8_unpack(q, s["rows"])
    else:
        ve.expert_gather(s["x"], s["position"], s["rows"])
    out = {"offsets": s["offsets"], "position": s["position"], "rows": s["rows"]}
    if c["grad"]:
        ve.expert_combine(s["drows"], s["position"], s["dx"])
        out["dx"] = s["dx"]
    return out


def own_combine(s):
    import ragged_shard_optimizer_amd as ve
    ve.expert_combine(s["rows"], s["position"], s["y"], weights=s["weights"], residual=s["residual"])
    if not s["case"]["grad"]:
        return {"y": s["y"]}
    ve.expert_combine_backward(s["dy"], s["position"], rows=s["rows"], weights=s["weights"], drows=s["drows"],
                               dweights=s["dweights"])
    return {"y": s["y"], "drows": s["drows"], "dweights": s["dweights"]}


def own_pack(s):
    import ragged_shard_optimizer_amd as ve
    q, t = ve.Fp8(*s["x8"]), ve.Fp8(*s["x8_t"])
    ve.fp8_pack(s["x"], q, t, offsets=s["offsets"])
    ve.fp8_unpack(q, s["out"])
    ve.fp8_unpack(t, s["out_t"])
    return {"rows": s["out"], "columns": s["out_t"]}


def own_weights(s):
    import ragged_shard_optimizer_amd as ve
    q, t = ve.Fp8(*s["w8"], block_rows=128), ve.Fp8(*s["w8_t"], block_rows=128)
    ve.fp8_pack_weight(s["w"], q, t)
    ve.fp8_unpack(q, s["out"])
    ve.fp8_unpack(t, s["out_t"])
    return {"w": s["out"], "w_t": s["out_t"]}


def own_forward(s):
    import ragged_shard_optimizer_amd as ve
    ve.fp8_linear_forward(ve.Fp8(*s["x8"]), ve.Fp8(*s["w8"], block_rows=128), s["y"], bias=s["bias"],
                          activation=s["case"]["act"], z=s["z"], offsets=s["offsets"])
    return {"y": s["y"]} if s["z"] is None else {"y": s["y"], "z": s["z"]}


def own_backward(s):
    import ragged_shard_optimizer_amd as ve
    ve.fp8_linear_backward(dy=ve.Fp8(*s["dy8"]), w_t=ve.Fp8(*s["w8_t"], block_rows=128), dx=s["dx"],
                           dy_t=ve.Fp8(*s["dy8_t"]), x_t=ve.Fp8(*s["x8_t"]), dw=s["dw"], offsets=s["offsets"])
    return {"dx": s["dx"], "dw": s["dw"]}


def sort_plain(ids, experts):
    T, k = ids.shape
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=DEV)
    bounds = torch.arange(experts + 1, device=DEV)
    offsets = torch.searchsorted(key[order], bounds)
    position = torch.where(key < experts, place, -1).to(torch.int32)
    return offsets, position.view(T, k)


def rows_of(v, position):
    """[T, k, C] in fp32: the rows at the positions, zeros for those of no row."""
    there = position >= 0
    return v[position.clamp_min(0).long()].float() * there[..., None]


def plain_dispatch(s):
    c, x = s["case"], s["x"]
    offsets, position = sort_plain(s["ids"], c["experts"])
    if c["bits"] == 8:
        x = restore_plain(*pack_plain(x.float())).to(torch.bfloat16)
    out = torch.zeros(c["tokens"] * c["slots"] + 1, c["cols"], dtype=torch.bfloat16, device=DEV)
    at = torch.where(position >= 0, position, c["tokens"] * c["slots"]).long()
    out[at.reshape(-1)] = x[:, None].expand(-1, c["slots"], -1).reshape(-1, c["cols"])
    res = {"offsets": offsets, "position": position, "rows": out[:-1]}
    if c["grad"]:
        res["dx"] = rows_of(s["drows"], position).sum(1).to(torch.bfloat16)
    return res


def plain_combine(s):
    c, position, w = s["case"], s["position"], s["weights"]
    r = rows_of(s["rows"], position)
    y = (r * w[..., None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if not c["grad"]:
        return {"y": y.to(torch.bfloat16)}
    dy = s["dy"].float()
    drows = torch.zeros(c["tokens"] * c["slots"] + 1, c["cols"], dtype=torch.bfloat16, device=DEV)
    at = torch.where(position >= 0, position, c["tokens"] * c["slots"]).long()
    drows[at.reshape(-1)] = (w[..., None] * dy[:, None]).to(torch.bfloat16).reshape(-1, c["cols"])
    return {"y": y.to(torch.bfloat16), "drows": drows[:-1], "dweights": (r * dy[:, None]).sum(-1)}


def plain_pack(s):
    c, x = s["case"], s["x"].float()
    f = c["format"]
    wide = torch.zeros(c["cols"], columns(c), device=DEV)
    wide[:, s["places"]] = x.t()
    return {"rows": restore_plain(*pack_plain(x, format=f)).to(torch.bfloat16),
            "columns": restore_plain(*pack_plain(wide, format=f)).to(torch.bfloat16)}


def plain_weights(s):
    w = [restore_plain(*pack_plain(v.float(), 128), 128).to(torch.bfloat16) for v in s["w"]]
    return {"w": torch.stack(w), "w_t": torch.stack([v.t() for v in w])}


def parts(s):
    at = 0
    for e, n in enumerate(s["lengths"]):
        yield e, at, at + n
        at += n


def act_plain(name, z):
    if name == "relu":
        return torch.clamp_min(z, 0)
    if name == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def one(q, e, groups):
    return q if groups == 1 else (q[0][e], q[1][e])


def plain_forward(s):
    c = s["case"]
    x = restore_plain(*s["x8"])
    z = torch.empty(c["tokens"], c["outputs"], device=DEV)
    for e, a, b in parts(s):
        if b > a:
            z[a:b] = x[a:b] @ restore_plain(*one(s["w8"], e, c["groups"]), 128).t()
            if s["bias"] is not None:
                z[a:b] += (s["bias"] if c["groups"] == 1 else s["bias"][e]).float()
    y = act_plain(c["act"], z).to(torch.bfloat16)
    return {"y": y} if s["z"] is None else {"y": y, "z": z.to(torch.bfloat16)}


def plain_backward(s):
    c = s["case"]
    dy, dy_t, x_t = restore_plain(*s["dy8"]), restore_plain(*s["dy8_t"]), restore_plain(*s["x8_t"])
    dx = torch.empty(c["tokens"], c["inputs"], device=DEV)
    dw = torch.zeros(c["groups"], c["outputs"], c["inputs"], device=DEV)
    at = 0
    for e, a, b in parts(s):
        n = up(b - a, 128)
        if b > a:
            dx[a:b] = dy[a:b] @ restore_plain(*one(s["w8_t"], e, c["groups"]), 128).t()
            dw[e] = dy_t[:, at:at + n] @ x_t[:, at:at + n].t()
        at += n
    dw = dw.to(s["dw"].dtype)
    return {"dx": dx.to(torch.bfloat16), "dw": dw[0] if c["groups"] == 1 else dw}


# ---------------------------------------------------------------------------
# the definition in 64 bits, and what a pass cannot do without

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def packed(v, block, format):
        """Restored values of 64-bit v, run by run."""
        dtype, most = FORMATS[format]
        out = torch.empty_like(v)
        step = 1 if block == 1 else block
        for a in range(0, v.shape[1], 128):
            strip = v[:, a:a + 128]
            if block == 1:
                m = strip.abs().max(1).values
            else:
                m = torch.stack([strip[r:r + step].abs().max() for r in range(0, v.shape[0], step)])
                m = m.repeat_interleave(step)[:v.shape[0]]
            e = torch.ceil(torch.log2(torch.where(m > 0, m, 1.0) / most))
            e = torch.where(m * torch.exp2(-e) > most, e + 1, e)  # the logarithm's rounding
            e = torch.where(m * torch.exp2(1 - e) <= most, e - 1, e).clamp(min=-127)
            up_ = torch.exp2(-e)[:, None]
            # the format's nearest value, ties to even
            y = strip * up_
            bits, low = (3, -6) if format == "e4m3" else (2, -14)
            x = torch.floor(torch.log2(torch.where(y != 0, y.abs(), 1.0))).clamp(min=low)
            grid = torch.exp2(x - bits)
            out[:, a:a + 128] = torch.round(y / grid) * grid / up_
        return out

    def value(q, block=1):
        codes, e = q[0].double(), q[1].double()
        for j in range(e.shape[0]):
            f = torch.exp2(e[j] - 127).repeat_interleave(block)[:codes.shape[0], None]
            codes[:, j * 128:(j + 1) * 128] *= f
        return codes

    if op in ("dispatch", "combine"):
        T, k, E, C = case["tokens"], case["slots"], case["experts"], case["cols"]
        ids = s["ids"].cpu().reshape(-1).tolist()
        lists = [[] for _ in range(E)]
        for slot, e in enumerate(ids):
            if 0 <= e < E:
                lists[e].append(slot)
        order = [slot for group in lists for slot in group]
        edges = [0]
        for group in lists:
            edges.append(edges[-1] + len(group))
        place = [-1] * (T * k)
        for i, slot in enumerate(order):
            place[slot] = i
        n = len(order)
        position = torch.tensor(place, dtype=torch.int32, device=DEV).view(T, k)
        slots = torch.tensor(order, dtype=torch.int64, device=DEV)
        token = slots // k

        def back(v):  # [n, C] in sorted order -> sums by token
            y = torch.zeros(T, C, dtype=torch.float64, device=DEV)
            where = torch.tensor(place, dtype=torch.int64, device=DEV).view(T, k)
            for j in range(k):
                hit = where[:, j] >= 0
                y[hit] += v[where[hit, j]]
            return y

        if op == "dispatch":
            x = s["x"].double()
            if case["bits"] == 8:
                x = packed(x, 1, "e4m3")
            rows = torch.zeros(T * k, C, dtype=torch.float64, device=DEV)
            rows[:n] = x[token]
            out = {"offsets": torch.tensor(edges, dtype=torch.int64, device=DEV), "position": position, "rows": rows}
            if case["grad"]:
                out["dx"] = back(s["drows"].double())
            return out
        w = s["weights"].double().reshape(-1)[slots]
        rows = s["rows"].double()[:n]
        y = back(rows * w[:, None])
        if case["residual"]:
            y += s["residual"].double()
        if not case["grad"]:
            return {"y": y}
        dy = s["dy"].double()[token]
        drows = torch.zeros(T * k, C, dtype=torch.float64, device=DEV)
        drows[:n] = dy * w[:, None]
        dweights = torch.zeros(T * k, dtype=torch.float64, device=DEV)
        dweights[slots] = torch.linalg.vecdot(dy, rows)
        return {"y": y, "drows": drows, "dweights": dweights.view(T, k)}
    if op == "weights":
        w = torch.stack([packed(v.double(), 128, "e4m3") for v in s["w"]])
        return {"w": w, "w_t": w.transpose(1, 2)}
    if op == "pack":
        x = s["x"].double()
        wide = torch.zeros(case["cols"], columns(case), dtype=torch.float64, device=DEV)
        a = at = 0
        for n in lengths(case):
            wide[:, at:at + n] = x[a:a + n].t()
            a, at = a + n, at + up(n, 128)
        return {"rows": packed(x, 1, case["format"]), "columns": packed(wide, 1, case["format"])}
    T, K, N, E = case["tokens"], case["inputs"], case["outputs"], case["groups"]
    weight = lambda q, e: value(q if E == 1 else (q[0][e], q[1][e]), 128)  # noqa: E731
    edges = [0]
    for n in lengths(case):
        edges.append(edges[-1] + n)
    if op == "forward":
        x, z = value(s["x8"]), torch.zeros(T, N, dtype=torch.float64, device=DEV)
        for e in range(E):
            a, b = edges[e], edges[e + 1]
            if b > a:
                z[a:b] = torch.mm(x[a:b], weight(s["w8"], e).t())
                if case["bias"]:
                    z[a:b] += (s["bias"] if E == 1 else s["bias"][e]).double()
        name = case["act"]
        if name == "relu":
            y = z.clamp(min=0)
        elif name == "gelu":
            y = z * torch.special.ndtr(z)
        elif name == "silu":
            y = z * torch.sigmoid(z)
        else:
            y = z
        return {"y": y, "z": z} if case["z"] else {"y": y}
    dy, dy_t, x_t = value(s["dy8"]), value(s["dy8_t"]), value(s["x8_t"])
    dx = torch.zeros(T, K, dtype=torch.float64, device=DEV)
    dw = torch.zeros(E, N, K, dtype=torch.float64, device=DEV)
    at = 0
    for e in range(E):
        a, b = edges[e], edges[e + 1]
        n = up(b - a, 128)
        if b > a:
            dx[a:b] = torch.mm(dy[a:b], weight(s["w8_t"], e).t())
            dw[e] = torch.mm(dy_t[:, at:at + n], x_t[:, at:at + n].t())
        at += n
    return {"dx": dx, "dw": dw if E > 1 else dw[0]}


def work(case):
    op = case["op"]

    def packed(rows, cols, block=1):  # bytes of codes and scales
        return rows * cols + -(-rows // block) * -(-cols // 128)

    if op in ("dispatch", "combine"):
        T, C, k = case["tokens"], case["cols"], case["slots"]
        index, rows = 4 * T * k, 2 * T * k * C
        if op == "dispatch":
            moved = 8 * T * k + index + 8 * (case["experts"] + 1) + 2 * T * C + rows
            if case["bits"] == 8:
                moved += 2 * packed(T * k, C)
            flops = 0
            if case["grad"]:
                moved, flops = moved + rows + 2 * T * C + index, T * k * C
            return {"bytes": moved, "flops": flops}
        moved, flops = rows + 2 * index + 2 * T * C * (2 if case["residual"] else 1), 2 * T * k * C
        if case["grad"]:
            moved, flops = moved + 2 * rows + 2 * T * C + 3 * index, flops + 3 * T * k * C
        return {"bytes": moved, "flops": flops}
    if op == "pack":
        T, C, t = case["tokens"], case["cols"], columns(case)
        return {"bytes": 2 * T * C + 2 * (packed(T, C) + packed(C, t)) + 2 * T * C + 2 * C * t, "flops": 0}
    if op == "weights":
        E, N, K = case["groups"], case["outputs"], case["inputs"]
        return {"bytes": 6 * E * N * K + 2 * E * (packed(N, K, 128) + packed(K, N, 128)), "flops": 0}
    T, K, N = case["tokens"], case["inputs"], case["outputs"]
    n = lengths(case)
    used = sum(v > 0 for v in n)
    if op == "forward":
        moved = packed(T, K) + used * packed(N, K, 128) + 2 * T * N * (2 if case["z"] else 1)
        return {"bytes": moved + (2 * used * N if case["bias"] else 0), "flops": 2 * T * N * K}
    t = sum(up(v, 128) for v in n)
    moved = packed(T, N) + used * packed(K, N, 128) + 2 * T * K + packed(N, t) + packed(K, t)
    return {"bytes": moved + (4 if case["wide"] else 2) * case["groups"] * N * K, "flops": 4 * T * N * K}
