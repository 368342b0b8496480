"""Workloads of the one-hot operators: routing tokens to experts and back, embedding lookup, the experts' products.

A mixture of experts and an embedding table multiply by sparse matrices whose rows are one-hot: token t's
choice j of expert e, or token t's vocabulary row v.  The library stores such a matrix by its sorted rows
(``Route``: ``order``, ``pos``, ``offsets``) and multiplies with it:

  route     spmm_build_route + spmm_dispatch: tokens sorted by expert, their rows copied into that order
  combine   spmm_combine + spmm_combine_grad: rows brought back with weights, and the gradient of that
            (spmm_dispatch_grad, the gradient of the way there, in the cases that ask for it)
  embed     spmm_embed: table rows by token id, scaled
  embed_grad  spmm_build_route + spmm_embed_grad: the table's dense gradient, summed over sorted tokens
  experts   spmm_experts: the block-diagonal product of the sorted rows with the experts' weights
  experts_grad  spmm_experts_grad: gradients of the rows and of the weights

``run`` computes each in a plain form (``own`` false: elementary torch operations in 32 bits, rounded once) or
by the library's entry points (``own`` true).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
IDT = {"i32": torch.int32, "i64": torch.int64}


def listed():
    return [
        # one decoding step of 16 sequences through a layer of 128 experts, 8 per token: launch latency
        dict(name="route_decode", op="route", T=16, k=8, E=128, H=4096, dt="bf16", idt="i64", drop=0.0),
        # a prompt batch of 16384 tokens through the same layer, one choice in a hundred dropped by capacity
        dict(name="route_prefill", op="route", T=16384, k=8, E=128, H=4096, dt="bf16", idt="i64", drop=0.01),
        # a small fine-tuning batch in 32 bits, a row length that no vector of four divides
        dict(name="route_odd_f32", op="route", T=1537, k=3, E=60, H=2051, dt="f32", idt="i32", drop=0.05),
        # the way back of the decoding step, forward only
        dict(name="combine_decode", op="combine", T=16, k=8, E=128, H=4096, dt="bf16", idt="i64", drop=0.0, grad=False),
        # a training step's way back and both gradients, fp16, 4 experts per token
        dict(name="combine_train", op="combine", T=16384, k=4, E=64, H=3584, dt="f16", idt="i64", drop=0.01, grad=True),
        # embedding of one decoding step of 8 sequences
        dict(name="embed_decode", op="embed", T=8, V=131072, H=4096, dt="bf16", idt="i64", pad=0.0, scale=1.0),
        # embedding of a padded prompt batch, scaled by sqrt(H)
        dict(name="embed_prefill", op="embed", T=32768, V=131072, H=4096, dt="bf16", idt="i64", pad=0.1, scale=64.0),
        # gradient of the table in a training step, bf16, as many rows as a large vocabulary has
        dict(name="embed_grad_large", op="embed_grad", T=32768, V=131072, H=4096, dt="bf16", idt="i64", pad=0.1, scale=64.0),
        # gradient of a smaller table with an odd vocabulary, in 32 bits
        dict(name="embed_grad_f32", op="embed_grad", T=8191, V=50021, H=1600, dt="f32", idt="i32", pad=0.0, scale=1.0),
        # the experts' up projection in one decoding step of 16 sequences: bound by reading the weights
        dict(name="experts_decode", op="experts", T=16, k=8, E=128, K=4096, N=1536, dt="bf16", drop=0.0),
        # the same product for a prompt batch: bound by the tensor cores
        dict(name="experts_prefill", op="experts", T=8192, k=4, E=32, K=4096, N=2048, dt="bf16", drop=0.0),
        # its backward pass in a training step, both gradients, odd row counts, some choices dropped
        dict(name="experts_grad_train", op="experts_grad", T=4093, k=4, E=16, K=3584, N=2560, dt="bf16", drop=0.01),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "combine", "embed", "embed_grad", "experts", "experts_grad"])
    idt = rng.choice(["i32", "i64"])
    if op in ("route", "combine"):
        E, H = _log(rng, 2, 512), _log(rng, 64, 8192)
        if rng.random() < 0.7:
            H = max(8, H // 8 * 8)
        k = min(rng.randint(1, 8), E)
        dt = rng.choice(["bf16", "f16", "f32"])
        room = 16384 * 4 * 3584 // (k * H * SIZE[dt] // 2)
        T = min(_log(rng, 1, 32768), max(1, room))
        case = dict(op=op, T=T, k=k, E=E, H=H, dt=dt, idt=idt, drop=rng.choice([0.0, 0.0, 0.01, 0.3]))
        if op == "combine":
            case["grad"] = rng.random() < 0.6
        return case
    if op in ("embed", "embed_grad"):
        H, V = _log(rng, 64, 8192), _log(rng, 1000, 200000)
        if rng.random() < 0.7:
            H = max(8, H // 8 * 8)
        dt = rng.choice(["bf16", "f16", "f32"])
        V = max(1000, min(V, 131072 * 4096 * 2 // (H * SIZE[dt])))
        T = min(_log(rng, 1, 32768), max(1, 32768 * 4096 * 2 // (H * SIZE[dt])))
        return dict(op=op, T=T, V=V, H=H, dt=dt, idt=idt, pad=rng.choice([0.0, 0.1]),
                    scale=rng.choice([1.0, 0.125, math.sqrt(H)]))
    E, K, N = _log(rng, 2, 128), _log(rng, 256, 4096) // 8 * 8, _log(rng, 256, 4096) // 8 * 8
    k = min(rng.randint(1, 8), E)
    E = max(k, min(E, 128 * 4096 * 1536 // (K * N)))
    flops = 32768 * 4096 * 2048 if op == "experts" else 16372 * 3584 * 2560
    T = min(_log(rng, 1, 8192), max(1, flops // (k * K * N)))
    if op == "experts_grad":
        E = max(k, min(E, 64 * 4096 * 1536 // (K * N)))
    return dict(op=op, T=T, k=k, E=E, K=K, N=N, dt=rng.choice(["bf16", "f16"]), drop=rng.choice([0.0, 0.01]))


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
    pop = torch.randn(E, generator=g, device="cuda") * 0.7
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)))
    top = torch.topk(pop + noise, k, dim=1)
    w = torch.softmax(top.values, dim=1).contiguous()
    ids = top.indices
    if case["drop"]:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["drop"], -1, ids)
    return ids.to(IDT[case.get("idt", "i64")]).contiguous(), w


def _tokens_of(case, g):
    """Token ids, a few very frequent and most rare (log-uniform rank, ranks spread over the vocabulary); -1 pads."""
    T, V = case["T"], case["V"]
    rank = (torch.exp(torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * math.log(V + 1)) - 1).long()
    place = torch.randperm(V, generator=g, device="cuda")
    ids = place[rank.clamp_(0, V - 1)]
    if case["pad"]:
        n = int(T * case["pad"])
        if n:
            ids[T - n:] = -1
    return ids.to(IDT[case["idt"]]).contiguous()


def _plan(ids, E):
    """The route of ids by torch: order, pos and offsets as the plain form keeps them."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(E + 1, dtype=torch.int64, device=flat.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum(count[:E], 0)
    place = torch.empty_like(order)
    place.scatter_(0, order, torch.arange(order.numel(), device=flat.device))
    pos = torch.where(key < E, place, -1)
    return order, pos.view(ids.shape), offsets


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DT[case["dt"]]
    s = dict(case=case)
    if op == "route":
        s["ids"], _ = _experts_of(case, g)
        s["x"] = _normal(g, (case["T"], case["H"]), dt)
    elif op == "combine":
        s["ids"], s["w"] = _experts_of(case, g)
        R = case["T"] * case["k"]
        s["ys"] = _normal(g, (R, case["H"]), dt)
        s["dy"] = _normal(g, (case["T"], case["H"]), dt, 0.1) if case["grad"] else None
    elif op == "embed":
        s["ids"] = _tokens_of(case, g)
        s["table"] = _normal(g, (case["V"], case["H"]), dt, 0.02)
    elif op == "embed_grad":
        s["ids"] = _tokens_of(case, g)
        s["dy"] = _normal(g, (case["T"], case["H"]), dt, 0.1)
    else:
        s["ids"], _ = _experts_of(case, g)
        R, K, N, E = case["T"] * case["k"], case["K"], case["N"], case["E"]
        s["xs"] = _normal(g, (R, K), dt)
        s["W"] = _normal(g, (E, N, K), dt, K ** -0.5)
        s["dys"] = _normal(g, (R, N), dt, 0.1) if op == "experts_grad" else None
    # a layer's route is built once and used by every product after it; the plain form of the experts'
    # products also keeps its offsets on the host, so that it waits for nothing
    if op in ("combine", "experts", "experts_grad"):
        if own:
            import sparse_dense_matrix_spmm_gb300 as spmm
            s["route"] = spmm.spmm_build_route(s["ids"], case["E"])
        else:
            order, pos, offsets = _plan(s["ids"], case["E"])
            s["route"] = (order, pos, offsets)
            s["starts"] = offsets.tolist()
    return s


# ---------------------------------------------------------------- one pass

def _run_own(s):
    import sparse_dense_matrix_spmm_gb300 as spmm
    case, op = s["case"], s["case"]["op"]
    if op == "route":
        R = spmm.spmm_build_route(s["ids"], case["E"])
        return [R.order, R.pos, R.offsets, spmm.spmm_dispatch(R, s["x"])]
    if op == "combine":
        y = spmm.spmm_combine(s["route"], s["ys"], s["w"])
        if not case["grad"]:
            return [y]
        dys, dw = spmm.spmm_combine_grad(s["route"], s["dy"], s["ys"], s["w"])
        return [y, dys, dw, spmm.spmm_dispatch_grad(s["route"], dys)]
    if op == "embed":
        return [spmm.spmm_embed(s["table"], s["ids"], case["scale"])]
    if op == "embed_grad":
        R = spmm.spmm_build_route(s["ids"], case["V"])
        return [spmm.spmm_embed_grad(R, s["dy"], case["scale"])]
    if op == "experts":
        return [spmm.spmm_experts(s["route"], s["xs"], s["W"])]
    return list(spmm.spmm_experts_grad(s["route"], s["dys"], s["xs"], s["W"]))


def _rows_back(pos, rows, w):
    """sum_j w[t, j] rows[pos[t, j]] in 32 bits, nothing for a dropped choice."""
    y = torch.zeros(pos.shape[0], rows.shape[1], device=rows.device)
    for j in range(pos.shape[1]):
        p = pos[:, j]
        part = rows[p.clamp(min=0)].float()
        if w is not None:
            part *= w[:, j, None]
        y += torch.where(p[:, None] >= 0, part, 0.0)
    return y


def run(s):
    if own:
        return _run_own(s)
    case, op = s["case"], s["case"]["op"]
    dt = DT[case["dt"]]
    if op == "route":
        order, pos, offsets = _plan(s["ids"], case["E"])
        live = torch.arange(order.numel(), device=order.device) < offsets[-1]
        xs = torch.where(live[:, None], s["x"][order // case["k"]].float(), 0.0).to(dt)
        return [order.int(), pos.int(), offsets.int(), xs]
    if op == "combine":
        order, pos, offsets = s["route"]
        k = case["k"]
        y = _rows_back(pos, s["ys"], s["w"]).to(dt)
        if not case["grad"]:
            return [y]
        live = torch.arange(order.numel(), device=order.device) < offsets[-1]
        dys = s["dy"][order // k].float() * s["w"].reshape(-1)[order][:, None]
        dys = torch.where(live[:, None], dys, 0.0).to(dt)
        dw = torch.stack([torch.where(pos[:, j] >= 0, (s["dy"].float() * s["ys"][pos[:, j].clamp(min=0)].float()).sum(1), 0.0)
                          for j in range(k)], dim=1)
        return [y, dys, dw, _rows_back(pos, dys, None).to(dt)]
    ids = s["ids"].long()
    if op == "embed":
        rows = s["table"][ids.clamp(min=0)].float() * case["scale"]
        return [torch.where(ids[:, None] >= 0, rows, 0.0).to(dt)]
    if op == "embed_grad":
        d = torch.zeros(case["V"], case["H"], device=ids.device)
        d.index_add_(0, ids.clamp(min=0), torch.where(ids[:, None] >= 0, s["dy"].float(), 0.0))
        return [(d * case["scale"]).to(dt)]
    starts, E = s["starts"], case["E"]
    xs, W = s["xs"], s["W"]
    if op == "experts":
        ys = torch.zeros(xs.shape[0], case["N"], dtype=dt, device=xs.device)
        for e in range(E):
            a, b = starts[e], starts[e + 1]
            if b > a:
                ys[a:b] = (xs[a:b].float() @ W[e].float().t()).to(dt)
        return [ys]
    dxs, dW = torch.zeros_like(xs), torch.zeros_like(W)
    for e in range(E):
        a, b = starts[e], starts[e + 1]
        if b > a:
            d = s["dys"][a:b].float()
            dxs[a:b] = (d @ W[e].float()).to(dt)
            dW[e] = (d.t() @ xs[a:b].float()).to(dt)
    return [dxs, dW]


# ---------------------------------------------------------------- what a pass cannot do without

def _experts_reached(case):
    """Experts that T tokens with k choices of E reach, on average (equal popularity)."""
    return case["E"] * (1.0 - (1.0 - case["k"] / case["E"]) ** case["T"])


def _rows_reached(T, V):
    """Distinct vocabulary rows of T tokens, on average: rank r has probability log((r + 2) / (r + 1)) / log(V + 1)."""
    n, r, c = 0.0, 0, T / math.log(V + 1)
    while r < V:
        step = min(max(1, r // 50), V - r)  # ranks r .. r + step - 1 are alike
        n += step * (1.0 - math.exp(-c * math.log((r + step + 1) / (r + 1)) / step))
        r += step
    return n


def work(case):
    op, b = case["op"], SIZE[case["dt"]]
    T = case["T"]
    if op in ("route", "combine"):
        R, H, ib = T * case["k"], case["H"], 4 if case["idt"] == "i32" else 8
        if op == "route":
            return {"bytes": R * (ib + 8) + 4 * (case["E"] + 1) + (T + R) * H * b, "flops": 0}
        fwd = R * 8 + (R + T) * H * b
        if not case["grad"]:
            return {"bytes": fwd, "flops": 2 * R * H}
        # ys, dy, w and pos read; y, dys, dw and dx written
        return {"bytes": R * 12 + (2 * R + 3 * T) * H * b, "flops": 6 * R * H}
    if op in ("embed", "embed_grad"):
        H, V, ib = case["H"], case["V"], 4 if case["idt"] == "i32" else 8
        live = T - int(T * case["pad"])
        if op == "embed":
            return {"bytes": int(T * ib + (_rows_reached(live, V) + T) * H * b), "flops": live * H}
        return {"bytes": T * ib + live * H * b + V * H * b, "flops": live * H + V * H}
    R, K, N, E = T * case["k"], case["K"], case["N"], case["E"]
    used = _experts_reached(case)
    if op == "experts":
        return {"bytes": int((R * (K + N) + used * N * K) * b), "flops": 2 * R * N * K}
    # xs, dys and the used weights read; dxs and every expert's gradient written
    return {"bytes": int((2 * R * K + R * N + (used + E) * N * K) * b), "flops": 4 * R * N * K}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """Row by row and key by key from the formulas, in 64 bits: one index list per expert or vocabulary row."""
    s = prepare(case, seed)
    op = case["op"]
    ids = s["ids"].cpu().reshape(-1).tolist()
    n_keys = case["V"] if op in ("embed", "embed_grad") else case["E"]
    lists = {}
    for f, v in enumerate(ids):
        if 0 <= v < n_keys:
            lists.setdefault(v, []).append(f)
    if op == "embed":
        i = torch.tensor([v if v >= 0 else 0 for v in ids], device="cuda")
        keep = torch.tensor([[1.0] if v >= 0 else [0.0] for v in ids], dtype=torch.float64, device="cuda")
        return [s["table"].index_select(0, i).double() * case["scale"] * keep]
    if op == "embed_grad":
        dy = s["dy"].double()
        out = torch.zeros(case["V"], case["H"], dtype=torch.float64, device="cuda")
        keys = sorted(lists)
        if keys:
            # sums of consecutive sorted rows as differences of a running total would lose bits: rows are added
            # by rank instead, the i-th token of every vocabulary row together
            depth = max(len(lists[v]) for v in keys)
            if depth > 4000:
                keep = [v for v in keys if len(lists[v]) > 64]
                for v in keep:
                    out[v] = dy.index_select(0, torch.tensor(lists[v], device="cuda")).sum(0)
                keys = [v for v in keys if len(lists[v]) <= 64]
                depth = max((len(lists[v]) for v in keys), default=0)
            for i in range(depth):
                keys = [v for v in keys if len(lists[v]) > i]
                out[torch.tensor(keys, device="cuda")] += dy.index_select(0, torch.tensor([lists[v][i] for v in keys], device="cuda"))
        return [out * case["scale"]]
    k, E, R = case["k"], case["E"], len(ids)
    order, offsets = [], [0]
    for e in range(E):
        order += lists.get(e, [])
        offsets.append(len(order))
    live = len(order)
    pos = [-1] * R
    for p, f in enumerate(order):
        pos[f] = p
    order += [f for f in range(R) if pos[f] < 0]
    where = torch.tensor(order, device="cuda")
    if op == "route":
        xs = s["x"].index_select(0, where // k).double()
        xs[live:] = 0
        return [where.int(), torch.tensor(pos, dtype=torch.int32, device="cuda").view(-1, k),
                torch.tensor(offsets, dtype=torch.int32, device="cuda"), xs]
    if op == "combine":
        ys, w = s["ys"].double(), s["w"].double().reshape(-1)
        tok = where[:live] // k
        y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        y.index_add_(0, tok, ys[:live] * w[where[:live], None])
        if not case["grad"]:
            return [y]
        dy = s["dy"].double()
        dys = torch.zeros_like(ys)
        dys[:live] = dy.index_select(0, tok) * w[where[:live], None]
        dw = torch.zeros(R, dtype=torch.float64, device="cuda")
        dw[where[:live]] = (dy.index_select(0, tok) * ys[:live]).sum(1)
        # the gradient of the way there is asked of dys as a program holds it: rounded to the rows' type
        dx = torch.zeros_like(y).index_add_(0, tok, dys[:live].to(DT[case["dt"]]).double())
        return [y, dys, dw.view(-1, k), dx]
    K, N, dt = case["K"], case["N"], torch.float64
    if 4 * R * K * N > 3e12:
        return None
    xs = s["xs"]
    ys = torch.zeros(R, N, dtype=dt, device="cuda") if op == "experts" else None
    dxs = torch.zeros(R, K, dtype=dt, device="cuda") if op == "experts_grad" else None
    dW = torch.zeros(E, N, K, dtype=dt, device="cuda") if op == "experts_grad" else None
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        w, x = s["W"][e].double(), xs[a:b].double()
        if op == "experts":
            ys[a:b] = torch.einsum("rk,nk->rn", x, w)
        else:
            d = s["dys"][a:b].double()
            dxs[a:b] = torch.einsum("rn,nk->rk", d, w)
            dW[e] = torch.einsum("rn,rk->nk", d, x)
    return [ys] if op == "experts" else [dxs, dW]
