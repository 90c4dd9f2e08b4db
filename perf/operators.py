"""Cases of the mixture-of-experts and 4-bit-weight operators: their inputs,
their plain forms in 32 bits, their values in 64 bits, and the calls of this
package that compute them.

Four operators, told apart by a case's "op":

* ``route``: the k largest logits of each token, their softmax gates, and the
  order of the chosen (token, choice) slots sorted by expert; with ``train``
  also the gradient of the logits.
* ``permute``: rows of tokens into expert order and the gated sum back; with
  ``train`` also the gradients of both.
* ``grouped``: one matrix product per expert over ragged groups of rows
  (``form`` "rows"), or each expert's weight gradient (``form`` "grad").
* ``w4``: rows times 4-bit weights with a scale (and zero point) per group.
"""
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a server: 16 tokens choose 8 of 128 experts
        {"name": "route_decode", "op": "route", "T": 16, "E": 128, "k": 8, "type": "bf16",
         "norm": True, "train": False, "masked": 0},
        # a training batch with padding tokens, and the gradient of its router
        {"name": "route_train", "op": "route", "T": 32768, "E": 256, "k": 8, "type": "f32",
         "norm": True, "train": True, "masked": 1000},
        # the same decode step's rows to their experts and back
        {"name": "permute_decode", "op": "permute", "T": 16, "k": 8, "H": 4096, "E": 128,
         "type": "bf16", "train": False, "masked": 0},
        # a training batch's rows there and back, forward and backward
        {"name": "permute_train", "op": "permute", "T": 16384, "k": 4, "H": 4096, "E": 64,
         "type": "bf16", "train": True, "masked": 500},
        # a decode step: 64 rows over 48 of 64 experts, one or two rows each
        {"name": "grouped_decode", "op": "grouped", "form": "rows", "E": 64, "active": 48,
         "R": 64, "K": 4096, "N": 2048, "type": "bf16", "out": "bf16", "order": "nk"},
        # a short prompt on an odd width, weights stored N-contiguous (the
        # order in which an input gradient reads a K-contiguous weight)
        {"name": "grouped_odd", "op": "grouped", "form": "rows", "E": 8, "active": 7,
         "R": 1000, "K": 1000, "N": 1000, "type": "f16", "out": "f16", "order": "kn"},
        # a training batch through the experts' first weight
        {"name": "grouped_batch", "op": "grouped", "form": "rows", "E": 32, "active": 32,
         "R": 32768, "K": 4096, "N": 4096, "type": "bf16", "out": "bf16", "order": "nk"},
        # the weight gradient of a batch, one expert without a row
        {"name": "grouped_wgrad", "op": "grouped", "form": "grad", "E": 32, "active": 31,
         "R": 16384, "K": 2048, "N": 4096, "type": "bf16", "out": "bf16", "order": ""},
        # one token through a 4096 x 4096 projection
        {"name": "w4_token", "op": "w4", "E": 1, "active": 1, "R": 1, "K": 4096, "N": 4096,
         "group": 128, "type": "bf16", "zeros": False},
        # a decode batch of 16 through an 8192 x 8192 projection, asymmetric
        {"name": "w4_batch", "op": "w4", "E": 1, "active": 1, "R": 16, "K": 8192, "N": 8192,
         "group": 64, "type": "f16", "zeros": True},
        # the decode step's rows through 4-bit experts
        {"name": "w4_experts", "op": "w4", "E": 64, "active": 40, "R": 64, "K": 4096, "N": 2048,
         "group": 128, "type": "bf16", "zeros": False},
        # a wide output layer: 4 rows against 32768 x 8192
        {"name": "w4_wide", "op": "w4", "E": 1, "active": 1, "R": 4, "K": 8192, "N": 32768,
         "group": 128, "type": "bf16", "zeros": True},
    ]


def _log(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, int(low * (high / low) ** rng.random() + 0.5)))


def _width(rng, low, high):
    """A row length: mostly a multiple of 64, some of 8, a few odd."""
    n = _log(rng, low, high)
    how = rng.random()
    if how < 0.6:
        return max(low, n // 64 * 64)
    return max(low, n // 8 * 8) if how < 0.85 else n | 1


def draw(rng: random.Random):
    op = rng.choice(["route", "permute", "grouped", "grouped", "w4", "w4"])
    if op == "route":
        E = _log(rng, 8, 512)
        T = _log(rng, 1, min(32768, 32768 * 256 // E))
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, 8), "type": rng.choice(list(TYPES)),
                "norm": rng.random() < 0.6, "train": rng.random() < 0.5,
                "masked": rng.choice([0, T // 16])}
    if op == "permute":
        H, k = _width(rng, 64, 8192), rng.randint(1, 8)
        T = _log(rng, 1, min(16384, 16384 * 4 * 4096 // (k * H)))
        return {"op": op, "T": T, "k": k, "H": H, "E": _log(rng, 8, 256),
                "type": rng.choice(["f16", "bf16", "f32"]) if H <= 4096 else "bf16",
                "train": rng.random() < 0.5, "masked": rng.choice([0, T // 16])}
    if op == "grouped":
        K, N = _width(rng, 64, 8192), _width(rng, 64, 8192)
        E = _log(rng, 1, max(1, min(128, 32 * 4096 * 4096 // (K * N))))
        R = _log(rng, 1, min(32768, 32768 * 4096 * 4096 // (K * N)))
        form = rng.choice(["rows", "rows", "grad"])
        return {"op": op, "form": form, "E": E, "active": min(R, max(1, E - rng.randint(0, E // 2))),
                "R": R, "K": K, "N": N, "type": rng.choice(["f16", "bf16"]),
                "out": rng.choice(["f16", "bf16"]),
                "order": "" if form == "grad" else rng.choice(["nk", "kn"])}
    K, N = 32 * _log(rng, 8, 512), _width(rng, 64, 32768)
    E = 1 if rng.random() < 0.6 else _log(rng, 2, 128)
    E = max(1, min(E, 8192 * 32768 // (K * N)))
    R = _log(rng, 1, 16 if E == 1 else 64)
    return {"op": op, "E": E, "active": min(R, max(1, E - rng.randint(0, E // 2))), "R": R, "K": K,
            "N": N, "group": rng.choice([32, 64, 128]), "type": rng.choice(["f16", "bf16"]),
            "zeros": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs
def _counts(g, E, active, R):
    """Group sizes: R rows over `active` of E experts, at least one each and
    within about a factor of three of one another."""
    share = torch.rand(active, generator=g) + 0.5
    edges = (share.cumsum(0) / share.sum() * (R - active)).round().long()
    n = torch.diff(edges, prepend=torch.zeros(1, dtype=torch.long)) + 1
    n[-1] += R - int(n.sum())
    counts = torch.zeros(E, dtype=torch.long)
    counts[torch.randperm(E, generator=g)[:active]] = n
    return counts


def _offsets(counts):
    return torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).to(torch.int32).cuda()


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": case}
    made = {"route": _prepare_route, "permute": _prepare_permute, "grouped": _prepare_grouped,
            "w4": _prepare_w4}[case["op"]]
    made(s, case, gen, host)
    if own:
        s["plan"] = _plan(s, case)
    return s


def _prepare_route(s, c, gen, host):
    T, E, k = c["T"], c["E"], min(c["k"], c["E"])
    dt = TYPES[c["type"]]
    x = _normal(gen, (T, E), torch.float32, 2.0)
    if c["masked"]:
        # padding tokens (nothing to choose) and tokens with few experts left
        x[torch.randperm(T, generator=host)[:c["masked"]].cuda()] = float("-inf")
        few = torch.randperm(T, generator=host)[:c["masked"]].cuda()
        x[few] = x[few].masked_fill(torch.rand((len(few), E), generator=gen, device="cuda") < 0.9,
                                    float("-inf"))
    s["k"], s["logits"] = k, x.to(dt)
    i32 = dict(dtype=torch.int32, device="cuda")
    s["experts"], s["gates"] = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
    s["offsets"] = torch.empty(E + 1, **i32)
    s["row_slot"], s["slot_row"] = torch.empty(T * k, **i32), torch.empty((T, k), **i32)
    if c["train"]:
        s["dgates"] = _normal(gen, (T, k), torch.float32)
        s["dlogits"] = torch.empty_like(s["logits"])


def _prepare_permute(s, c, gen, host):
    T, k, H, E = c["T"], c["k"], c["H"], c["E"]
    dt = TYPES[c["type"]]
    experts = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :k].reshape(-1)
    gates = torch.rand((T, k), generator=gen, device="cuda")
    if c["masked"]:
        out = torch.randperm(T, generator=host)[:c["masked"]].cuda()
        experts.view(T, k)[out] = E
        gates[out] = 0
    order = experts.argsort(stable=True)
    rows = int((experts < E).sum())
    position = torch.empty_like(order)
    position[order] = torch.arange(T * k, device="cuda")
    s["slot_row"] = torch.where(position < rows, position, -1).to(torch.int32).view(T, k)
    order[rows:] = -1
    s["row_slot"], s["gates"] = order.to(torch.int32), gates
    s["X"], s["Ys"] = _normal(gen, (T, H), dt), _normal(gen, (T * k, H), dt)
    s["Xs"], s["Y"] = torch.empty_like(s["Ys"]), torch.empty_like(s["X"])
    if c["train"]:
        s["dY"], s["dXs"] = _normal(gen, (T, H), dt), _normal(gen, (T * k, H), dt)
        s["dYs"], s["dX"] = torch.empty_like(s["Ys"]), torch.empty_like(s["X"])
        s["dgates"] = torch.empty_like(gates)


def _prepare_grouped(s, c, gen, host):
    E, R, K, N, dt = c["E"], c["R"], c["K"], c["N"], TYPES[c["type"]]
    counts = _counts(host, E, c["active"], R)
    s["most"], s["offsets"] = int(counts.max()), _offsets(counts)
    s["A"] = _normal(gen, (R, K), dt)
    if c["form"] == "grad":
        s["B"] = _normal(gen, (R, N), dt)
        s["D"] = torch.empty((E, K, N), dtype=TYPES[c["out"]], device="cuda")
        return
    shape = (E, N, K) if c["order"] == "nk" else (E, K, N)
    s["B"] = torch.empty(shape, dtype=dt, device="cuda").normal_(0, K ** -0.5, generator=gen)
    s["B"] = s["B"].transpose(1, 2) if c["order"] == "nk" else s["B"]
    s["D"] = torch.empty((R, N), dtype=TYPES[c["out"]], device="cuda")


def _prepare_w4(s, c, gen, host):
    E, R, K, N, dt = c["E"], c["R"], c["K"], c["N"], TYPES[c["type"]]
    G = -(-K // c["group"])
    counts = _counts(host, E, c["active"], R)
    s["most"], s["offsets"] = int(counts.max()), (_offsets(counts) if E > 1 else None)
    s["X"] = _normal(gen, (R, K), dt)
    s["W"] = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s["scales"] = ((torch.rand((E, N, G), generator=gen, device="cuda") + 0.5) *
                   (0.2 * K ** -0.5)).to(dt)
    s["zeros"] = (torch.randint(4, 12, (E, N, G), generator=gen, device="cuda", dtype=torch.uint8)
                  if c["zeros"] else None)
    s["D"] = torch.empty((R, N), dtype=dt, device="cuda")


# ---------------------------------------------------------------- this package's calls
def _plan(s, c):
    import dense_tiled_gemm_02_gb300 as gemm
    if c["op"] == "route":
        return gemm.Route.like(s["logits"], s["k"], normalize=c["norm"])
    if c["op"] == "grouped":
        return gemm.GroupedGemm.like(s["A"], s["B"], s["offsets"], None, s["D"])
    if c["op"] == "w4":
        return gemm.W4Gemm.like(s["X"], s["W"], s["scales"], s["zeros"], s["offsets"], s["D"],
                                group=c["group"])
    return gemm.Permute.like(s["X"], s["slot_row"])


def _run_own(s, c):
    plan = s["plan"]
    if c["op"] == "route":
        plan.run(s["logits"], s["experts"], s["gates"], s["offsets"], s["row_slot"], s["slot_row"])
        out = [s["experts"], s["gates"], s["offsets"], s["row_slot"], s["slot_row"]]
        if c["train"]:
            plan.backward(s["logits"], s["experts"], s["gates"], s["dgates"], s["dlogits"])
            out.append(s["dlogits"])
        return out
    if c["op"] == "permute":
        plan.gather(s["X"], s["row_slot"], s["slot_row"], s["Xs"])
        plan.combine(s["Ys"], s["slot_row"], s["gates"], s["Y"])
        out = [s["Xs"], s["Y"]]
        if c["train"]:
            plan.combine_backward(s["dY"], s["Ys"], s["row_slot"], s["slot_row"], s["gates"],
                                  s["dYs"], s["dgates"])
            plan.combine(s["dXs"], s["slot_row"], None, s["dX"])
            out += [s["dYs"], s["dgates"], s["dX"]]
        return out
    if c["op"] == "grouped":
        plan.run(s["A"], s["B"], s["offsets"], None, s["D"])
        return s["D"]
    plan.run(s["X"], s["W"], s["scales"], s["zeros"], s["offsets"], s["D"])
    return s["D"]


# ---------------------------------------------------------------- the plain forms
def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"route": _plain_route, "permute": _plain_permute, "grouped": _plain_grouped,
            "w4": _plain_w4}[c["op"]](s, c)


def _plain_route(s, c):
    T, E, k = c["T"], c["E"], s["k"]
    x = s["logits"].float()
    top, experts = torch.sort(x, dim=1, descending=True, stable=True)
    top, experts = top[:, :k], experts[:, :k]
    chosen = top > float("-inf")
    high = top[:, :1].clamp_min(torch.finfo(torch.float32).min)
    ex = torch.exp(top - high)
    total = ex.sum(1, keepdim=True) if c["norm"] else torch.exp(x - high).sum(1, keepdim=True)
    gates = torch.where(chosen, ex / total, 0.0)
    key = torch.where(chosen, experts, E).reshape(-1)
    order = key.argsort(stable=True)
    slot_row = torch.empty_like(order)
    rows = torch.arange(T * k, device=x.device)
    slot_row[order] = rows
    counts = torch.zeros(E + 2, device=x.device, dtype=torch.long)
    offsets = counts.scatter_add_(0, key + 1, torch.ones_like(key)).cumsum(0)[:E + 1]
    order = torch.where(rows < offsets[E], order, -1)
    slot_row = torch.where(key < E, slot_row, -1)
    i32 = torch.int32
    out = [torch.where(chosen, experts, -1).to(i32), gates, offsets.to(i32), order.to(i32),
           slot_row.to(i32).view(T, k)]
    if c["train"]:
        dg = s["dgates"]
        mean = (gates * dg).sum(1, keepdim=True)
        if c["norm"]:
            dx = torch.zeros_like(x).scatter_(1, experts, gates * (dg - mean))
        else:
            p = torch.exp(x - high) / total
            p = torch.where(x > float("-inf"), p, 0.0)
            dx = (-p * mean).scatter_add_(1, experts, gates * dg)
        out.append(dx.to(s["logits"].dtype))
    return out


def _plain_permute(s, c):
    T, k = c["T"], c["k"]
    dt = s["X"].dtype
    row_slot, slot_row, gates = s["row_slot"].long(), s["slot_row"].long(), s["gates"]
    routed = (slot_row >= 0)[:, :, None]
    live = (row_slot >= 0)[:, None]
    token = row_slot.clamp_min(0) // k
    at = slot_row.clamp_min(0)
    Xs = torch.where(live, s["X"][token], 0.0).to(dt)
    back = torch.where(routed, s["Ys"][at].float(), 0.0)
    Y = (gates[:, :, None] * back).sum(1).to(dt)
    if not c["train"]:
        return [Xs, Y]
    dYf = s["dY"].float()
    gate = gates.reshape(-1)[row_slot.clamp_min(0)]
    dYs = torch.where(live, gate[:, None] * dYf[token], 0.0).to(dt)
    dgates = (dYf[:, None, :] * back).sum(2)
    dX = torch.where(routed, s["dXs"][at].float(), 0.0).sum(1).to(dt)
    return [Xs, Y, dYs, dgates, dX]


def _places(s, R):
    """Of each row: the rank of its expert among those with rows, and its place in the group."""
    off = s["offsets"].long()
    r = torch.arange(R, device=off.device)
    e = torch.searchsorted(off, r, right=True) - 1
    rank = (off[1:] > off[:-1]).long().cumsum(0) - 1
    return e, rank[e], r - off[e]


def _padded(x, rank, place, active, most):
    """[active, most, width] fp32 with each row at (rank, place), zeros elsewhere."""
    out = torch.zeros((active, most, x.shape[1]), dtype=torch.float32, device=x.device)
    out[rank, place] = x.float()
    return out


def _plain_grouped(s, c):
    A, B, R, n, most = s["A"], s["B"], c["R"], c["active"], s["most"]
    off = s["offsets"].long()
    ids = torch.argsort((off[1:] == off[:-1]).long(), stable=True)[:n]
    e, rank, place = _places(s, R)
    a = _padded(A, rank, place, n, most)
    if c["form"] == "grad":
        b = _padded(B, rank, place, n, most)
        D = torch.zeros((c["E"], c["K"], c["N"]), dtype=s["D"].dtype, device=A.device)
        D[ids] = torch.bmm(a.transpose(1, 2), b).to(D.dtype)
        return D
    return torch.bmm(a, B[ids].float())[rank, place].to(s["D"].dtype)


def _plain_w4(s, c):
    E, R, K, N, g = c["E"], c["R"], c["K"], c["N"], c["group"]
    X, W, scales, zeros = s["X"], s["W"], s["scales"], s["zeros"]
    if E > 1:
        off = s["offsets"].long()
        ids = torch.argsort((off[1:] == off[:-1]).long(), stable=True)[:c["active"]]
        W, scales, zeros = W[ids], scales[ids], None if zeros is None else zeros[ids]
    q = torch.stack([W & 15, W >> 4], dim=3).view(len(W), N, K).float()
    z = 8.0 if zeros is None else zeros.float().repeat_interleave(g, 2)[:, :, :K]
    w = (q - z) * scales.float().repeat_interleave(g, 2)[:, :, :K]
    if E == 1:
        return torch.matmul(X.float(), w[0].t()).to(X.dtype)
    e, rank, place = _places(s, R)
    x = _padded(X, rank, place, c["active"], s["most"])
    return torch.bmm(x, w.transpose(1, 2))[rank, place].to(X.dtype)


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "permute": _exact_permute, "grouped": _exact_grouped,
            "w4": _exact_w4}[case["op"]](s, case)


def _exact_route(s, c):
    """Only the gates and the logits' gradient are computed numbers."""
    x, k = s["logits"].double(), s["k"]
    val, idx = torch.topk(x, k, dim=1)
    none = torch.isinf(val) & (val < 0)
    full = torch.softmax(torch.where(torch.isinf(x).all(1, keepdim=True), 0.0, x), 1)
    full = torch.where(torch.isinf(x), 0.0, full)
    gates = full.gather(1, idx)
    if c["norm"]:
        gates = gates / gates.sum(1, keepdim=True).clamp_min(1e-300)
    gates = torch.where(none, 0.0, gates)
    out = [None, gates, None, None, None]
    if c["train"]:
        # equal 16-bit logits may be chosen in another order here, which pairs
        # them with other entries of dgates: no value then
        if c["type"] != "f32":
            return out + [None]
        dg = s["dgates"].double()
        d = torch.zeros_like(x).scatter_(1, idx, torch.where(none, 0.0, dg))
        p = torch.zeros_like(x).scatter_(1, idx, gates) if c["norm"] else full
        out.append(p * (d - (p * d).sum(1, keepdim=True)))
    return out


def _exact_permute(s, c):
    T, k, H = c["T"], c["k"], c["H"]
    slot = s["slot_row"].long().view(-1)
    live = torch.nonzero(slot >= 0)[:, 0]
    token, row, gate = live // k, slot[live], s["gates"].double().view(-1)[live]
    X, Ys = s["X"].double(), s["Ys"].double()
    Xs = torch.zeros_like(Ys)
    Xs[row] = X[token]
    Y = torch.zeros_like(X).index_add_(0, token, Ys[row] * gate[:, None])
    if not c["train"]:
        return [Xs, Y]
    dY = s["dY"].double()
    dYs = torch.zeros_like(Ys)
    dYs[row] = dY[token] * gate[:, None]
    dgates = torch.zeros(T * k, dtype=torch.float64, device=X.device)
    dgates[live] = torch.einsum("rh,rh->r", dY[token], Ys[row])
    dX = torch.zeros_like(X).index_add_(0, token, s["dXs"].double()[row])
    return [Xs, Y, dYs, dgates.view(T, k), dX]


def _exact_grouped(s, c):
    off = s["offsets"].tolist()
    A, B = s["A"], s["B"]
    D = torch.zeros(s["D"].shape, dtype=torch.float64, device=A.device)
    for e in range(c["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        if c["form"] == "grad":
            D[e] = A[a:b].double().t() @ B[a:b].double()
        else:
            D[a:b] = A[a:b].double() @ B[e].double()
    return D


def _exact_w4(s, c):
    off = [0, c["R"]] if s["offsets"] is None else s["offsets"].tolist()
    K, N, g = c["K"], c["N"], c["group"]
    D = torch.zeros((c["R"], N), dtype=torch.float64, device=s["X"].device)
    where = torch.arange(K, device=s["X"].device) // g
    for e in range(c["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        w = torch.empty((N, K), dtype=torch.float64, device=s["X"].device)
        w[:, 0::2] = s["W"][e] % 16
        w[:, 1::2] = s["W"][e] // 16
        w -= 8 if s["zeros"] is None else s["zeros"][e][:, where]
        w *= s["scales"][e].double()[:, where]
        D[a:b] = s["X"][a:b].double() @ w.t()
    return D


# ---------------------------------------------------------------- compulsory work
def work(c):
    if c["op"] == "route":
        T, E, k, b = c["T"], c["E"], min(c["k"], c["E"]), BYTES[c["type"]]
        n = T * E * b + 16 * T * k + 4 * (E + 1)
        # the gradient reads dgates and writes every logit's; over all E it
        # also needs the logits, read already
        return {"bytes": n + (T * E * b + 4 * T * k if c["train"] else 0),
                "flops": (6 if c["train"] else 2) * T * E}
    if c["op"] == "permute":
        T, k, H, b = c["T"], c["k"], c["H"], BYTES[c["type"]]
        row, slots = H * b, 12 * T * k
        # X, Ys read, Xs, Y written; then dY, dXs read, dYs, dX written (Ys
        # is the forward pass's own)
        n = 2 * T * row + 2 * T * k * row + slots
        return {"bytes": n + (2 * T * row + 2 * T * k * row + 4 * T * k if c["train"] else 0),
                "flops": (6 if c["train"] else 2) * T * k * H}
    R, K, N, n = c["R"], c["K"], c["N"], c["active"]
    b = BYTES[c["type"]]
    flops = 2 * R * K * N
    if c["op"] == "grouped":
        if c["form"] == "grad":
            return {"bytes": R * (K + N) * b + c["E"] * K * N * BYTES[c["out"]] + 4 * (c["E"] + 1),
                    "flops": flops}
        return {"bytes": R * K * b + n * K * N * b + R * N * BYTES[c["out"]] + 4 * (c["E"] + 1),
                "flops": flops}
    G = -(-K // c["group"])
    return {"bytes": n * N * (K // 2 + G * (b + (1 if c["zeros"] else 0))) + R * (K + N) * b,
            "flops": flops}
