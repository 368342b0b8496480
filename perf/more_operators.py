"""Workloads of the gated experts: the router, the gated feed-forward block with its gradients, checkpoints in 8 bits.

A mixture-of-experts layer chooses k experts for every token, runs the tokens' rows through each chosen expert's
gated block h = act(g) u with [g u] = xs [Wg Wu]^T, and, in training, keeps what the way back needs:

  topk         spmm_topk: the k largest logits of each token and their softmax weights (spmm_topk_grad, the gradient
               of the logits, in the cases that ask for it)
  gated        spmm_experts_gated: both projections, the activation and the product, on rows sorted by expert
  gated_train  the same, saving [g u], then the way back: spmm_gated_grad (gradient of [g u]) and the gradients of
               the rows and of the weights.  save 16: [g u] in the rows' type; save 8: [g u] and the rows are kept
               as 8-bit checkpoints and read from them
  rows8        spmm_pack_rows + spmm_unpack_rows: a checkpoint of rows written in 8 bits and read back

``run`` computes each in a plain form (``own`` false: elementary torch operations in 32 bits) or by the library's
entry points (``own`` true).

A checkpoint in 8 bits: 16 consecutive values of a row share a power of two 2^e, the smallest (from 2^-126) for
which all of them round to integers q of at most 127 in magnitude; x is held as q 2^e, q = x 2^-e rounded half to even.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
IDT = {"i32": torch.int32, "i64": torch.int64}
GROUP = 16


def listed():
    return [
        # the router of one decoding step of 16 sequences over 128 experts: launch latency
        dict(name="topk_decode", op="topk", T=16, E=128, k=8, dt="bf16", idt="i64", renorm=True, masked=0.0, grad=False),
        # a training step's router over 256 experts, logits in 32 bits, and its gradient
        dict(name="topk_train", op="topk", T=16384, E=256, k=8, dt="f32", idt="i64", renorm=True, masked=0.0, grad=True),
        # an odd number of experts, some of them closed to a token, weights of the softmax over all experts
        dict(name="topk_masked", op="topk", T=5003, E=60, k=6, dt="f16", idt="i32", renorm=False, masked=0.3, grad=True),
        # one decoded token of a single sequence through a gated block of 64 experts
        dict(name="gated_token", op="gated", T=1, k=8, E=64, K=2048, N=768, dt="bf16", act="silu", drop=0.0),
        # one decoding step of 32 sequences: bound by reading the weights
        dict(name="gated_decode", op="gated", T=32, k=8, E=128, K=4096, N=1280, dt="bf16", act="silu", drop=0.0),
        # a prompt batch: bound by the tensor cores
        dict(name="gated_prefill", op="gated", T=8192, k=4, E=32, K=4096, N=2048, dt="bf16", act="silu", drop=0.0),
        # a training step that keeps [g u] in 16 bits, odd row counts, some choices dropped
        dict(name="gated_train_16", op="gated_train", T=4093, k=4, E=16, K=3584, N=1280, dt="bf16", act="silu", drop=0.01, save=16),
        # a training step with checkpoints in 8 bits, fp16
        dict(name="gated_train_8", op="gated_train", T=8191, k=2, E=8, K=4096, N=1792, dt="f16", act="gelu_tanh", drop=0.0, save=8),
        # a small fine-tuning batch with checkpoints in 8 bits: few rows per expert, ragged sizes
        dict(name="gated_train_small", op="gated_train", T=301, k=3, E=12, K=1032, N=528, dt="bf16", act="gelu", drop=0.3, save=8),
        # a layer's rows of a prompt-sized batch, kept in 8 bits and read back
        dict(name="rows8_layer", op="rows8", rows=32768, cols=4096, dt="bf16"),
        # rows in 32 bits of an odd length: the last group of a row is short
        dict(name="rows8_odd", op="rows8", rows=1537, cols=2051, dt="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["topk", "gated", "gated", "gated_train", "gated_train", "rows8"])
    dt = rng.choice(["bf16", "f16", "f32"])
    if op == "topk":
        E = _log(rng, 2, 512)
        k = min(rng.randint(1, 8), E)
        T = min(_log(rng, 1, 32768), 16384 * 256 * 4 // (E * SIZE[dt]))
        return dict(op=op, T=T, E=E, k=k, dt=dt, idt=rng.choice(["i32", "i64"]), renorm=rng.random() < 0.5,
                    masked=rng.choice([0.0, 0.0, 0.3]), grad=rng.random() < 0.6)
    if op == "rows8":
        cols = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            cols = max(16, cols // 16 * 16)
        return dict(op=op, rows=min(_log(rng, 1, 65536), 32768 * 4096 * 2 // (cols * SIZE[dt])), cols=cols, dt=dt)
    E, K, N = _log(rng, 2, 128), _log(rng, 256, 4096) // 8 * 8, _log(rng, 128, 2048) // 16 * 16
    k = min(rng.randint(1, 8), E)
    case = dict(op=op, k=k, K=K, N=N, dt=rng.choice(["bf16", "f16"]), act=rng.choice(["silu", "gelu", "gelu_tanh"]),
                drop=rng.choice([0.0, 0.01]))
    if op == "gated":
        case["E"] = max(k, min(E, 128 * 4096 * 1280 // (K * N)))
        case["T"] = min(_log(rng, 1, 8192), max(1, 32768 * 4096 * 2048 // (k * K * N)))
    else:
        case["E"] = max(k, min(E, 32 * 4096 * 1792 // (K * N)))
        case["T"] = min(_log(rng, 16, 8192), max(1, 16372 * 3584 * 1280 // (k * K * N)))
        case["save"] = rng.choice([16, 8])
    return case


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return g


def _normal(g, shape, dt, scale=1.0):
    """Normal values of the type, drawn in pieces so that no 32-bit copy of a large operand is held."""
    out = torch.empty(shape, dtype=dt, device="cuda")
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 27):
        piece = flat[a:a + (1 << 27)]
        piece.copy_(torch.randn(piece.numel(), generator=g, device="cuda") * scale)
    return out


def _experts_of(case, g):
    """ids[T][k]: each token's k distinct experts, the experts of unequal popularity, some choices dropped (-1)."""
    T, k, E = case["T"], case["k"], case["E"]
    pop = torch.randn(E, generator=g, device="cuda") * 0.4
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)))
    ids = torch.topk(pop + noise, k, dim=1).indices
    if case["drop"]:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["drop"], -1, ids)
    return ids


def _plan(ids, E):
    """A layer's route, built once and used by every product after it: order, pos and offsets as the library keeps
    them, and for the plain form's batched products the slot of each kept row in E x most rows."""
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    count = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum(count, 0)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=flat.device)
    pos = torch.where(key < E, place, -1).view(ids.shape)
    most, kept = int(count.max()), int(offsets[-1])
    expert = key[order][:kept]
    slot = expert * most + torch.arange(kept, device=flat.device) - offsets[expert]
    return dict(order=order.int(), pos=pos.int(), offsets=offsets.int(), slot=slot, most=most, kept=kept)


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DT[case["dt"]]
    s = dict(case=case)
    if op == "topk":
        T, E = case["T"], case["E"]
        # some experts are preferred; close to a training step's logits
        pop = torch.randn(E, generator=g, device="cuda")
        s["logits"] = (torch.randn(T, E, generator=g, device="cuda") * 1.5 + pop).to(dt)
        if case["masked"]:
            s["logits"].masked_fill_(torch.rand(T, E, generator=g, device="cuda") < case["masked"], -math.inf)
            if T > 3:
                s["logits"][T - T // 4:T - T // 4 + 2] = -math.inf  # tokens that no expert may take
        s["dw"] = torch.randn(T, case["k"], generator=g, device="cuda") if case["grad"] else None
        return s
    if op == "rows8":
        # activations: columns of unequal size, a few far larger than the rest
        size = torch.exp(torch.randn(case["cols"], generator=g, device="cuda"))
        s["x"] = _normal(g, (case["rows"], case["cols"]), dt)
        s["x"].mul_(size.to(dt))
        return s
    s["plan"] = _plan(_experts_of(case, g), case["E"])
    R, K, N, E = case["T"] * case["k"], case["K"], case["N"], case["E"]
    s["xs"] = _normal(g, (R, K), dt)
    s["W"] = _normal(g, (E, 2 * N, K), dt, K ** -0.5)
    if op == "gated_train":
        s["dh"] = _normal(g, (R, N), dt, 0.1)
    return s


# ---------------------------------------------------------------- one pass

def _run_own(s):
    import sparse_dense_matrix_spmm_gb300 as spmm
    case, op = s["case"], s["case"]["op"]
    if op == "topk":
        ids, w = spmm.spmm_topk(s["logits"], case["k"], renorm=case["renorm"], id_dtype=IDT[case["idt"]])
        if not case["grad"]:
            return [ids, w]
        return [ids, w, spmm.spmm_topk_grad(s["logits"], ids, w, s["dw"], renorm=case["renorm"])]
    if op == "rows8":
        return [spmm.spmm_unpack_rows(spmm.spmm_pack_rows(s["x"]))]
    p, act = s["plan"], case["act"]
    R = spmm.Route(case["T"], case["k"], case["E"], p["order"], p["pos"], p["offsets"])
    if op == "gated":
        return [spmm.spmm_experts_gated(R, s["xs"], s["W"], act=act)]
    if case["save"] == 8:
        xs = spmm.spmm_pack_rows(s["xs"])
        h, gu = spmm.spmm_experts_gated(R, s["xs"], s["W"], act=act, save="packed")
    else:
        xs = s["xs"]
        h, gu = spmm.spmm_experts_gated(R, xs, s["W"], act=act, save="rows")
    dgu, dxs, dW = spmm.spmm_experts_gated_grad(R, s["dh"], xs, s["W"], gu, act=act)
    return [h, dgu, dxs, dW]


def _act(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * 0.5 ** 0.5))
    return 0.5 * x * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (x + 0.044715 * x * x * x)))


def _act_grad(x, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return s * (1.0 + x * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(x * 0.5 ** 0.5)) + x * torch.exp(-0.5 * x * x) * (0.5 / math.pi) ** 0.5
    t = torch.tanh((2.0 / math.pi) ** 0.5 * (x + 0.044715 * x * x * x))
    return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * (2.0 / math.pi) ** 0.5 * (1.0 + 3 * 0.044715 * x * x)


def _two_to(e):
    """2^e in 32 bits for whole e from -126 to 127, exactly."""
    return ((e + 127) << 23).view(torch.float32)


def _rows8(x):
    """The values that a checkpoint of x holds, in 32 bits.  The exponent of a group's largest magnitude comes from its
    bits: 127.5 of 128 parts and more round to 128, so the exponent is that of the magnitude plus 2^-7 of its binade."""
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    wide = torch.zeros(rows, groups * GROUP, device=x.device)
    wide[:, :cols] = x.float()
    wide = wide.view(rows, groups, GROUP)
    bits = wide.abs().amax(2, keepdim=True).view(torch.int32)
    e = (((bits + (1 << 16)) >> 23) - 127 - 6).clamp(-126, 121)
    q = torch.round(wide * _two_to(-e)).clamp(-127, 127)
    return (q * _two_to(e)).view(rows, groups * GROUP)[:, :cols]


def run(s):
    if own:
        return _run_own(s)
    case, op = s["case"], s["case"]["op"]
    dt = DT[case["dt"]]
    if op == "topk":
        k, x = case["k"], s["logits"].float()
        top, ids = torch.sort(x, dim=1, descending=True, stable=True)  # equal logits keep the order of their experts
        top, ids = top[:, :k], ids[:, :k]
        live = top > -math.inf
        most = torch.where(live[:, :1], top[:, :1], 0.0)
        p = torch.where(live, torch.exp(top - most), 0.0)
        full = torch.exp(x - most)
        total = (p if case["renorm"] else full).sum(1, keepdim=True)
        w = torch.where(live, p / total, 0.0)
        out = [torch.where(live, ids, -1).to(IDT[case["idt"]]), w]
        if not case["grad"]:
            return out
        dw = torch.where(live, s["dw"], 0.0)
        dot = (w * dw).sum(1, keepdim=True)
        chosen = torch.zeros_like(x).scatter_(1, ids, w * dw)
        if case["renorm"]:
            d = chosen - torch.zeros_like(x).scatter_(1, ids, w * dot)
        else:
            d = chosen - torch.where(total > 0, full / total, 0.0) * dot
        return out + [d.to(dt)]
    if op == "rows8":
        return [_rows8(s["x"]).to(dt)]
    E, K, N = case["E"], case["K"], case["N"]
    xs, p = s["xs"], s["plan"]
    slot, most, kept = p["slot"], p["most"], p["kept"]

    def padded(rows):  # kept rows in E x most, zeros between
        out = torch.zeros(E * most, rows.shape[1], device=rows.device)
        out[slot] = rows[:kept].float()
        return out.view(E, most, rows.shape[1])

    def back(batch, rows):  # and out again, zero rows past the kept ones
        out = torch.zeros(rows, batch.shape[2], device=batch.device)
        out[:kept] = batch.reshape(E * most, batch.shape[2])[slot]
        return out

    W = s["W"].float()
    gu = back(torch.bmm(padded(xs), W.transpose(1, 2)), xs.shape[0])
    h = (_act(gu[:, :N], case["act"]) * gu[:, N:]).to(dt)
    if op == "gated":
        return [h]
    if case["save"] == 8:
        gu, xs = _rows8(gu), _rows8(xs)
    else:
        gu = gu.to(dt).float()
    dh = torch.zeros(xs.shape[0], N, device=xs.device)
    dh[:kept] = s["dh"][:kept].float()
    g, u = gu[:, :N], gu[:, N:]
    # the gradient of [g u] is a result of its own, in the rows' type, and the products after it read that
    dgu = torch.cat([dh * u * _act_grad(g, case["act"]), dh * _act(g, case["act"])], 1).to(dt)
    d = padded(dgu)
    dxs = back(torch.bmm(d, W), xs.shape[0]).to(dt)
    dW = torch.bmm(d.transpose(1, 2), padded(xs)).to(dt)
    return [h, dgu, dxs, dW]


# ---------------------------------------------------------------- what a pass cannot do without

def _experts_reached(case):
    """Experts that T tokens with k choices of E reach, on average (equal popularity)."""
    return case["E"] * (1.0 - (1.0 - case["k"] / case["E"]) ** case["T"])


def work(case):
    op, b = case["op"], SIZE[case["dt"]]
    if op == "topk":
        T, E, k, ib = case["T"], case["E"], case["k"], 4 if case["idt"] == "i32" else 8
        # logits read; ids and weights written; for the gradient dw read and the logits' gradient written
        return {"bytes": T * E * b + T * k * (ib + 4) + (T * k * 4 + T * E * b if case["grad"] else 0), "flops": 0}
    if op == "rows8":
        # rows read, the checkpoint (a byte a value, a byte a group) written and read, rows written
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * b + 2 * (n + case["rows"] * -(-case["cols"] // GROUP)), "flops": 0}
    R, K, N, E = case["T"] * case["k"], case["K"], case["N"], case["E"]
    used = _experts_reached(case)
    if op == "gated":
        return {"bytes": int((R * (K + N) + used * 2 * N * K) * b), "flops": 4 * R * N * K}
    # xs, dh and the used weights read; h, the gradient of [g u], dxs and every expert's gradient written
    return {"bytes": int((2 * R * K + 4 * R * N + (used + E) * 2 * N * K) * b), "flops": 12 * R * N * K}


# ---------------------------------------------------------------- the definition in 64 bits

def _unit(e):
    """2^e in 64 bits, exactly (torch.pow is not), as a column."""
    return ((e.long() + 1023) << 52).view(torch.float64)[:, None]


def _held(x):
    """What an 8-bit checkpoint of x (64 bits) holds: group by group, the power of two found by trying."""
    rows, cols = x.shape
    out = torch.empty_like(x)
    for a in range(0, cols, GROUP):
        v = x[:, a:a + GROUP]
        e = torch.floor(torch.log2(v.abs().amax(1).clamp(min=2.0 ** -140))) - 8
        for _ in range(4):  # from too small upwards, one at a time
            q = torch.round(v / _unit(e))
            e = torch.where(q.abs().amax(1) > 127, e + 1, e)
        unit = _unit(e.clamp(-126, 121))
        out[:, a:a + GROUP] = torch.round(v / unit).clamp(-127, 127) * unit
    return out


def _exact_topk(case, s):
    T, E, k = case["T"], case["E"], case["k"]
    x = s["logits"].double()
    ids = torch.full((T, k), -1, dtype=torch.int64, device=x.device)
    w = torch.zeros(T, k, dtype=torch.float64, device=x.device)
    grad = torch.zeros(T, E, dtype=torch.float64, device=x.device)
    lower = torch.ones(E, E, dtype=torch.bool, device=x.device).triu(1).t()  # [e, f]: f comes before e
    step = max(1, (1 << 27) // (E * E))
    for a in range(0, T, step):
        v = x[a:a + step]
        # an expert's rank: how many are larger, or equal and before it
        rank = ((v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & lower)).sum(2)
        taken = (rank < k) & (v > -math.inf)
        t, e = taken.nonzero(as_tuple=True)
        ids[a + t, rank[t, e]] = e
        weight = torch.where(taken if case["renorm"] else torch.ones_like(taken), v, -math.inf)
        top = weight.amax(1, keepdim=True)
        p = torch.where(top > -math.inf, torch.exp(weight - torch.where(top > -math.inf, top, 0.0)), 0.0)
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        w[a + t, rank[t, e]] = p[t, e]
        if case["grad"]:
            dp = torch.zeros_like(v)
            dp[t, e] = s["dw"][a + t, rank[t, e]].double()
            grad[a:a + step] = p * (dp - (p * dp).sum(1, keepdim=True))
    return [ids.to(IDT[case["idt"]]), w] + ([grad] if case["grad"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "topk":
        return _exact_topk(case, s)
    if op == "rows8":
        return [_held(s["x"].double())]
    K, N, E, act, dt = case["K"], case["N"], case["E"], case["act"], DT[case["dt"]]
    R = case["T"] * case["k"]
    if (4 if op == "gated" else 12) * R * K * N > 6e12:
        return None
    starts = s["plan"]["offsets"].tolist()
    f64 = dict(dtype=torch.float64, device="cuda")
    h, dgu, dxs = torch.zeros(R, N, **f64), torch.zeros(R, 2 * N, **f64), torch.zeros(R, K, **f64)
    dW = torch.zeros(E, 2 * N, K, **f64) if op == "gated_train" else None
    half, pi = 0.5, math.pi
    for e in range(E):
        a, b = starts[e], starts[e + 1]
        if a == b:
            continue
        x, w = s["xs"][a:b].double(), s["W"][e].double()
        gu = torch.einsum("rk,nk->rn", x, w)
        for saved in (False, True):
            if saved and op == "gated":
                continue
            if saved:
                gu = _held(gu) if case["save"] == 8 else gu.to(dt).double()
            g, u = gu[:, :N], gu[:, N:]
            if act == "silu":
                f = torch.sigmoid(g)
                df = f + g * f * (1 - f)
            elif act == "gelu":
                f = half * torch.erfc(-g / math.sqrt(2))
                df = f + g * torch.exp(-half * g.square()) / math.sqrt(2 * pi)
            else:
                z = math.sqrt(2 / pi) * (g + 0.044715 * g.pow(3))
                f = torch.sigmoid(2 * z)
                df = f + g * 2 * f * (1 - f) * math.sqrt(2 / pi) * (1 + 0.134145 * g.square())
            if not saved:
                h[a:b] = g * f * u
                continue
            d = s["dh"][a:b].double()
            dgu[a:b, :N], dgu[a:b, N:] = d * u * df, d * g * f
        if op == "gated_train":
            # asked of the gradient of [g u] as a program holds it: rounded to the rows' type
            d = dgu[a:b].to(dt).double()
            dxs[a:b] = torch.einsum("rn,nk->rk", d, w)
            dW[e] = torch.einsum("rn,rk->nk", d, _held(x) if case["save"] == 8 else x)
    return [h] if op == "gated" else [h, dgu, dxs, dW]
