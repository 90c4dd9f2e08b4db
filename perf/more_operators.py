"""Cases of the operators on rows held in 8 bits: their inputs, their plain
forms in 32 bits, their values in 64 bits, and the calls of this package that
compute them.

Four kinds, told apart by a case's "op":

* ``norm``: a residual's addition and the root-mean-square norm of each token,
  out in the tokens' type or (``out`` "i8") in 8 bits with a scale a token; with
  ``train`` also the gradients, from the rows or (``held``) from their 8 bits.
* ``rows8``: rows to 8 bits and back, with a power of two for every 32 values
  (``block`` 32) or one scale a row (``block`` 0).
* ``grad``: an expert's (or one layer's) weight gradient from rows held in 8
  bits.
* ``i8``: rows times weights, both of 8-bit integers, with a scale for each
  token and each output, dense or grouped by expert.
"""
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-6
BLOCK = 32


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a server: 16 tokens become the next product's operand
        {"name": "norm_token", "op": "norm", "T": 16, "H": 4096, "type": "bf16", "residual": True,
         "out": "i8", "train": False, "held": False},
        # a training batch's norm, forward and backward
        {"name": "norm_train", "op": "norm", "T": 16384, "H": 4096, "type": "bf16",
         "residual": True, "out": "x", "train": True, "held": False},
        # its backward pass from rows kept in 8 bits since the forward pass
        {"name": "norm_held", "op": "norm", "T": 16384, "H": 4096, "type": "bf16",
         "residual": True, "out": "", "train": True, "held": True},
        # a prompt of odd length and width, no residual
        {"name": "norm_odd", "op": "norm", "T": 1023, "H": 1001, "type": "f16", "residual": False,
         "out": "i8", "train": False, "held": False},
        # a training batch's rows kept for the backward pass, and read back
        {"name": "rows8_save", "op": "rows8", "T": 16384, "H": 4096, "type": "bf16", "block": 32},
        # a prompt's rows as an operand: odd width, one scale a row
        {"name": "rows8_odd", "op": "rows8", "T": 999, "H": 2047, "type": "f16", "block": 0},
        # 32 experts' weight gradients from 16384 kept rows
        {"name": "grad_experts", "op": "grad", "E": 32, "active": 32, "R": 16384, "K": 2048,
         "N": 4096, "type": "bf16"},
        # one layer's weight gradient from a batch of odd length
        {"name": "grad_dense", "op": "grad", "E": 1, "active": 1, "R": 8191, "K": 4096, "N": 4096,
         "type": "bf16"},
        # one token through a layer of 8-bit weights
        {"name": "i8_token", "op": "i8", "E": 1, "active": 1, "R": 1, "K": 4096, "N": 4096,
         "type": "bf16"},
        # a decode batch
        {"name": "i8_batch", "op": "i8", "E": 1, "active": 1, "R": 64, "K": 8192, "N": 8192,
         "type": "f16"},
        # a decode step's rows through 8-bit experts
        {"name": "i8_experts", "op": "i8", "E": 64, "active": 40, "R": 64, "K": 4096, "N": 2048,
         "type": "bf16"},
        # a long prompt through a square layer
        {"name": "i8_prompt", "op": "i8", "E": 1, "active": 1, "R": 8192, "K": 8192, "N": 8192,
         "type": "bf16"},
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
    op = rng.choice(["norm", "norm", "rows8", "grad", "i8", "i8", "i8"])
    if op == "norm":
        H = _width(rng, 64, 16384)
        T = _log(rng, 1, min(32768, 16384 * 4096 // H))
        residual = rng.random() < 0.6
        how = rng.choice(["i8", "x", "train", "held"])
        # 8 bits are an operand of 16-bit models: which of two values is the
        # nearer is a matter of fp32's last bits
        kind = rng.choice(["f16", "bf16"] if how == "i8" else list(TYPES))
        return {"op": op, "T": T, "H": H, "type": kind, "residual": residual,
                "out": {"i8": "i8", "x": "x", "train": "x", "held": ""}[how],
                "train": how in ("train", "held"), "held": how == "held"}
    if op == "rows8":
        H = _width(rng, 64, 16384)
        block = rng.choice([0, 32])
        return {"op": op, "T": _log(rng, 1, min(32768, 16384 * 4096 // H)), "H": H,
                "type": rng.choice(list(TYPES) if block else ["f16", "bf16"]), "block": block}
    K, N = _width(rng, 64, 8192), _width(rng, 64, 8192)
    if op == "grad":
        E = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, min(64, 32 * 2048 * 4096 // (K * N))))
        R = _log(rng, 1, min(32768, 16384 * 4096 * 4096 // (K * N)))
        return {"op": op, "E": E, "active": min(R, max(1, E - rng.randint(0, E // 2))), "R": R,
                "K": K, "N": N, "type": rng.choice(["f16", "bf16"])}
    E = 1 if rng.random() < 0.6 else _log(rng, 2, max(2, min(128, 64 * 4096 * 4096 // (K * N))))
    R = _log(rng, 1, min(8192, 8192 * 8192 * 4096 // (K * N)))
    return {"op": op, "E": E, "active": min(R, max(1, E - rng.randint(0, E // 2))), "R": R, "K": K,
            "N": N, "type": rng.choice(list(TYPES))}


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


def _rows(gen, T, H, dtype):
    """Activations: a few channels are an order of magnitude larger."""
    x = torch.randn((T, H), generator=gen, device="cuda")
    wide = torch.rand(H, generator=gen, device="cuda") < 0.01
    return (x * torch.where(wide, 12.0, 1.0)).to(dtype)


def _ints(gen, shape):
    """Integers as rows of normal values leave them: the largest of a row near 127."""
    x = torch.empty(shape, device="cuda").normal_(0, 33.0, generator=gen)
    return x.round_().clamp_(-127, 127).to(torch.int8)


def _blocks(H):
    return -(-H // BLOCK)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": case}
    made = {"norm": _prepare_norm, "rows8": _prepare_rows8, "grad": _prepare_grad,
            "i8": _prepare_i8}[case["op"]]
    made(s, case, gen, host)
    if own:
        _plan(s, case)
    return s


def _prepare_norm(s, c, gen, host):
    T, H, dt = c["T"], c["H"], TYPES[c["type"]]
    f32 = dict(dtype=torch.float32, device="cuda")
    s["x"] = _rows(gen, T, H, dt)
    s["weight"] = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(dt)
    s["residual"] = _rows(gen, T, H, dt) if c["residual"] else None
    s["h"] = torch.empty_like(s["x"]) if c["residual"] else None
    s["y"] = torch.empty((T, H), dtype=torch.int8 if c["out"] == "i8" else dt, device="cuda")
    s["scales"] = torch.empty(T, **f32) if c["out"] == "i8" else None
    s["values"] = torch.empty_like(s["x"])
    if c["train"]:
        s["rstd"], s["dweight"] = torch.empty(T, **f32), torch.empty(H, **f32)
        s["dy"] = torch.randn((T, H), generator=gen, device="cuda").to(dt)
        s["dresidual"] = (torch.randn((T, H), generator=gen, device="cuda").to(dt)
                          if c["residual"] else None)
        s["dx"] = torch.empty_like(s["x"])
    if c["held"]:  # what the forward pass kept: h in 8 bits, the norm's factor
        s["h8"] = _ints(gen, (T, H))
        s["exponents"] = torch.randint(119, 123, (T, _blocks(H)), generator=gen, device="cuda",
                                       dtype=torch.uint8)
        s["rstd"] = 1 + torch.rand(T, generator=gen, device="cuda")


def _prepare_rows8(s, c, gen, host):
    T, H = c["T"], c["H"]
    s["X"] = _rows(gen, T, H, TYPES[c["type"]])
    s["q"] = torch.empty((T, H), dtype=torch.int8, device="cuda")
    s["scales"] = (torch.empty((T, _blocks(H)), dtype=torch.uint8, device="cuda") if c["block"]
                   else torch.empty(T, dtype=torch.float32, device="cuda"))
    s["values"] = torch.empty_like(s["X"])


def _prepare_grad(s, c, gen, host):
    E, R, K, N, dt = c["E"], c["R"], c["K"], c["N"], TYPES[c["type"]]
    counts = _counts(host, E, c["active"], R)
    s["counts"] = counts.tolist()
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long),
                              counts.cumsum(0)]).to(torch.int32).cuda()
    s["q"] = _ints(gen, (R, K))
    s["exponents"] = torch.randint(119, 123, (R, _blocks(K)), generator=gen, device="cuda",
                                   dtype=torch.uint8)
    s["B"] = torch.randn((R, N), generator=gen, device="cuda").to(dt)
    s["D"] = torch.empty((E, K, N), dtype=dt, device="cuda")


def _prepare_i8(s, c, gen, host):
    E, R, K, N = c["E"], c["R"], c["K"], c["N"]
    counts = _counts(host, E, c["active"], R)
    s["counts"] = counts.tolist()
    s["offsets"] = None if E == 1 else torch.cat([torch.zeros(1, dtype=torch.long),
                                                  counts.cumsum(0)]).to(torch.int32).cuda()
    s["X"], s["W"] = _ints(gen, (R, K)), _ints(gen, (E, N, K))
    s["x_scales"] = 0.02 + 0.02 * torch.rand(R, generator=gen, device="cuda")
    s["w_scales"] = (1 + torch.rand((E, N), generator=gen, device="cuda")) / (33.0 * K ** 0.5)
    s["D"] = torch.empty((R, N), dtype=TYPES[c["type"]], device="cuda")


# ---------------------------------------------------------------- this package's calls
def _plan(s, c):
    import dense_tiled_gemm_02_gb300 as gemm
    if c["op"] == "norm":
        s["plan"] = gemm.RmsNorm.like(s["x"], s["weight"], s["y"], scales=s["scales"],
                                      residual=s["residual"], h=s["h"], eps=EPS)
        if c["out"] == "i8":
            s["rows"] = gemm.Rows8.like(s["values"], s["y"], s["scales"])
    elif c["op"] == "rows8":
        s["plan"] = gemm.Rows8.like(s["X"], s["q"], s["scales"])
    elif c["op"] == "grad":
        s["plan"] = gemm.Rows8Grad.like(s["q"], s["exponents"], s["B"], s["offsets"], None, s["D"])
    else:
        s["plan"] = gemm.I8Gemm.like(s["X"], s["x_scales"], s["W"], s["w_scales"], s["offsets"],
                                     s["D"])


def _run_own(s, c):
    plan = s["plan"]
    if c["op"] == "norm":
        out = []
        if c["out"]:
            plan.run(s["x"], s["weight"], s["y"], scales=s["scales"], residual=s["residual"],
                     h=s["h"], rstd=s.get("rstd"))
            out = [s["h"]] if c["residual"] else []
        if c["out"] == "x":
            out.append(s["y"])
        elif c["out"] == "i8":
            s["rows"].unpack(s["y"], s["scales"], s["values"])
            out += [s["values"], s["scales"]]
        if c["train"]:
            h = s["h8"] if c["held"] else s["h"] if c["residual"] else s["x"]
            plan.backward(s["dy"], h, s["weight"], s["rstd"], s["dx"], s["dweight"],
                          dresidual=s["dresidual"], exponents=s.get("exponents"))
            out += [s["dx"], s["dweight"]]
        return out
    if c["op"] == "rows8":
        plan.pack(s["X"], s["q"], s["scales"])
        plan.unpack(s["q"], s["scales"], s["values"])
        return [s["values"]] if c["block"] else [s["values"], s["scales"]]
    if c["op"] == "grad":
        plan.run(s["q"], s["exponents"], s["B"], s["offsets"], None, s["D"])
        return s["D"]
    plan.run(s["X"], s["x_scales"], s["W"], s["w_scales"], s["offsets"], s["D"])
    return s["D"]


# ---------------------------------------------------------------- the plain forms
def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"norm": _plain_norm, "rows8": _plain_rows8, "grad": _plain_grad,
            "i8": _plain_i8}[c["op"]](s, c)


def _widened(q, exponents):
    """The values of 8-bit rows with a power of two for every block of 32."""
    power = torch.exp2(exponents.float() - 127).repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return q.float() * power


def _plain_norm(s, c):
    x, w, dt = s["x"], s["weight"].float(), s["x"].dtype
    out = []
    if c["held"]:
        h, rstd = _widened(s["h8"], s["exponents"]), s["rstd"][:, None]
    else:
        h = x
        if c["residual"]:
            h = (x.float() + s["residual"].float()).to(dt)
            out.append(h)
        h = h.float()
        rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
        y = h * rstd * w
        if c["out"] == "i8":
            scale = y.abs().amax(1, keepdim=True) / 127
            q = torch.round(y / scale)
            out += [(q * scale).to(dt), scale[:, 0]]
        else:
            out.append(y.to(dt))
    if c["train"]:
        dy = s["dy"].float()
        g = dy * w
        normed = h * rstd
        dx = rstd * (g - normed * (g * normed).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dresidual"].float()
        out += [dx.to(dt), (dy * normed).sum(0)]
    return out


def _plain_rows8(s, c):
    X, (T, H) = s["X"].float(), s["X"].shape
    if not c["block"]:
        scale = X.abs().amax(1, keepdim=True) / 127
        return [(torch.round(X / scale) * scale).to(s["X"].dtype), scale[:, 0]]
    x = torch.nn.functional.pad(X, (0, -H % BLOCK)).view(T, -1, BLOCK)
    # amax = m 2^k with m in [1/2, 1): 127 steps of 2^(k - 7) reach m <= 127/128
    m, k = torch.frexp(x.abs().amax(2, keepdim=True))
    step = torch.exp2((k - 7 + (m > 127 / 128).int()).float())
    return [(torch.round(x / step) * step).view(T, -1)[:, :H].to(s["X"].dtype)]


def _places(off, R):
    """Of each row: the rank of its expert among those with rows, and its place in the group."""
    off = off.long()
    r = torch.arange(R, device=off.device)
    e = torch.searchsorted(off, r, right=True) - 1
    rank = (off[1:] > off[:-1]).long().cumsum(0) - 1
    return rank[e], r - off[e]


def _padded(x, rank, place, active, most):
    """[active, most, width] fp32 with each row at (rank, place), zeros elsewhere."""
    out = torch.zeros((active, most, x.shape[1]), dtype=torch.float32, device=x.device)
    out[rank, place] = x.float()
    return out


def _with_rows(off, active):
    """The experts that have rows, in their order."""
    return torch.argsort((off[1:] == off[:-1]).long(), stable=True)[:active]


def _plain_grad(s, c):
    n, most = c["active"], max(s["counts"])
    rank, place = _places(s["offsets"], c["R"])
    a = _padded(_widened(s["q"], s["exponents"]), rank, place, n, most)
    b = _padded(s["B"], rank, place, n, most)
    D = torch.zeros((c["E"], c["K"], c["N"]), dtype=s["D"].dtype, device=a.device)
    D[_with_rows(s["offsets"], n)] = torch.bmm(a.transpose(1, 2), b).to(D.dtype)
    return D


def _plain_i8(s, c):
    X, W, dt = s["X"], s["W"], s["D"].dtype
    if c["E"] == 1:
        sums = torch.matmul(X.float(), W[0].float().t())
        return (sums * s["x_scales"][:, None] * s["w_scales"]).to(dt)
    n, off = c["active"], s["offsets"]
    ids = _with_rows(off, n)
    rank, place = _places(off, c["R"])
    x = _padded(X, rank, place, n, max(s["counts"]))
    sums = torch.bmm(x, W[ids].float().transpose(1, 2))[rank, place]
    return (sums * s["x_scales"][:, None] * s["w_scales"][ids[rank]]).to(dt)


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rows8": _exact_rows8, "grad": _exact_grad,
            "i8": _exact_i8}[case["op"]](s, case)


def _in_steps(v, step):
    """Multiples of step nearest to v, ties to even; zero where step is."""
    return torch.where(step > 0, torch.round(v / step.clamp_min(1e-300)), 0.0) * step


def _held(s, name):
    power = torch.exp2(s["exponents"].float() - 127).double()
    return s[name].double() * power.repeat_interleave(BLOCK, 1)[:, :s[name].shape[1]]


def _exact_norm(s, c):
    w, out = s["weight"].double(), []
    if c["held"]:
        h, rstd = _held(s, "h8"), s["rstd"].double()
    else:
        h = s["x"]
        if c["residual"]:
            h = (s["x"].double() + s["residual"].double()).to(h.dtype)
            out.append(h.double())
        h = h.double()
        rstd = (h.square().sum(1) / c["H"] + EPS).rsqrt()
        y = torch.einsum("th,t,h->th", h, rstd, w)
        if c["out"] == "i8":
            step = y.abs().max(1).values / 127
            out += [_in_steps(y, step[:, None]), step]
        else:
            out.append(y)
    if c["train"]:
        dy = s["dy"].double()
        dot = torch.einsum("th,h,th->t", dy, w, h)
        dx = dy * w * rstd[:, None] - h * (rstd ** 3 * dot / c["H"])[:, None]
        if c["residual"]:
            dx = dx + s["dresidual"].double()
        out += [dx, torch.einsum("th,th,t->h", dy, h, rstd)]
    return out


def _exact_rows8(s, c):
    X = s["X"].double()
    if not c["block"]:
        step = X.abs().max(1).values / 127
        return [_in_steps(X, step[:, None]), step]
    parts = []
    for x in X.split(BLOCK, 1):
        top = x.abs().max(1, keepdim=True).values
        # in 32 bits exp2 is exact at whole numbers (pow in 64 is not); and a
        # logarithm may come out just above a whole one
        step = torch.exp2(torch.ceil(torch.log2(top / 127)).float()).double()
        step = torch.where(63.5 * step >= top, step / 2, step)
        parts.append(_in_steps(x, step))
    return [torch.cat(parts, 1)]


def _exact_grad(s, c):
    a, b, at = _held(s, "q"), s["B"].double(), 0
    D = torch.zeros((c["E"], c["K"], c["N"]), dtype=torch.float64, device=a.device)
    for e, n in enumerate(s["counts"]):
        D[e] = a[at:at + n].t() @ b[at:at + n]
        at += n
    return D


def _exact_i8(s, c):
    at, parts = 0, []
    for e, n in enumerate(s["counts"]):
        if n:
            x = s["X"][at:at + n].double() * s["x_scales"][at:at + n, None].double()
            parts.append(x @ (s["W"][e].double() * s["w_scales"][e, :, None].double()).t())
        at += n
    return torch.cat(parts)


# ---------------------------------------------------------------- work
def work(case):
    c, op = case, case["op"]
    if op == "norm":
        n, b = c["T"] * c["H"], BYTES[c["type"]]
        move = 0
        if c["out"]:
            move += n * (b + (2 * b if c["residual"] else 0) + (1 if c["out"] == "i8" else b))
        if c["train"]:
            move += n * (2 * b + (b if c["residual"] else 0))
            move += n * (1 + 1 / BLOCK) if c["held"] else n * b
        return {"bytes": move, "flops": n * (6 + (12 if c["train"] else 0))}
    if op == "rows8":
        n, b = c["T"] * c["H"], BYTES[c["type"]]
        s = n / BLOCK if c["block"] else 4 * c["T"]
        return {"bytes": 2 * (n * (b + 1) + s), "flops": 4 * n}
    R, K, N, b = c["R"], c["K"], c["N"], BYTES[c["type"]]
    if op == "grad":
        return {"bytes": R * K * (1 + 1 / BLOCK) + R * N * b + c["E"] * K * N * b,
                "flops": 2 * R * K * N}
    return {"bytes": R * K + c["active"] * N * (K + 4) + R * (N * b + 4), "flops": 2 * R * K * N}
