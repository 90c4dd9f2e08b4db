"""The operators on 8-bit rows on the GPU, against their formulas in 64 bits.

Tolerances.  With u = 2**-24, half a step of fp32: each rounded fp32 operation
is off by u of its result, so a sum of n terms by at most n u of the sum S of
their magnitudes, and an expression of a few more operations by that many u
more.  Products on the tensor cores: the accumulation truncates, 2 u an
addition.  One rounding to the output's type adds half its step (2**-8 of the
result in bf16, 2**-11 in fp16), or half the least subnormal.  Whole numbers
(exponents, integers of block rows, sums of integer products) are equal;
integers of scaled rows are the nearest ones up to the roundings of the ratio.
"""
from __future__ import annotations

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg
from gpu_helpers import forced_plan

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF_STEP = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}
EPS = 1e-6


def rnd(shape, dtype=F32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def ints(shape, seed=0, low=-128, high=128):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, high, shape, generator=g, dtype=torch.int8).cuda()


def near(got, ref, slack, what=""):
    """|got - ref| within slack and one rounding to got's type; NaN where ref is."""
    dt = got.dtype
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    off = (got - ref).abs() - (slack + HALF_STEP[dt] * (ref.abs() + slack) + TINY[dt])
    off = off[~torch.isnan(off)]
    assert off.numel() == 0 or float(off.max()) <= 0, f"{what}: {float(off.max())} over the bound"


def done(op, code=pkg.GEMM_OK):
    assert op.status() == code
    op.close()


def strided(t, pad):
    """The same rows, `pad` elements of something else between them."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), 77, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


# ---------------------------------------------------------------- norm
def norm_ref(x, residual, w, eps=EPS):
    """(h in x's type, rstd, y) of the formula in 64 bits."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    hd = h.double()
    rstd = 1 / torch.sqrt((hd * hd).mean(1) + eps)
    return h, rstd, hd * rstd[:, None] * w.double()


NORM_SIZES = [(1, 1), (3, 7), (16, 64), (5, 200), (7, 256), (2, 1001), (700, 1024), (33, 2048),
              (300, 4096), (2, 4096), (1, 16384), (160, 16384), (5, 40000), (700, 33), (64, 20001)]


@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm(T, H, dtype, with_residual):
    x = rnd((T, H), dtype, 1, 3.0)
    res = rnd((T, H), dtype, 2) if with_residual else None
    w = rnd((H,), F32 if H % 2 else dtype, 3)
    h = torch.empty_like(x) if with_residual else None
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, residual=res, h=h, eps=EPS)
    op.run(x, w, y, residual=res, h=h, rstd=rstd)
    done(op)
    h_ref, r_ref, y_ref = norm_ref(x, res, w)
    if with_residual:
        assert torch.equal(h, h_ref)
    # a sum of H positive terms, then five operations
    near(rstd, r_ref, (H + 5) * U * r_ref, "rstd")
    near(y, y_ref, (H + 8) * U * y_ref.abs(), "y")


@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_to_8_bits(T, H, dtype):
    x, res, w = rnd((T, H), dtype, 1, 3.0), rnd((T, H), dtype, 2), rnd((H,), dtype, 3)
    x[0] = 0
    res[0] = 0  # a row of zeros
    h, y = torch.empty_like(x), torch.empty((T, H), dtype=torch.int8, device="cuda")
    scales = torch.empty(T, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, scales=scales, residual=res, h=h, eps=EPS)
    op.run(x, w, y, scales=scales, residual=res, h=h)
    done(op)
    h_ref, r_ref, y_ref = norm_ref(x, res, w)
    assert torch.equal(h, h_ref)
    top = y_ref.abs().amax(1)
    near(scales, top / 127, (H + 9) * U * top / 127, "scales")
    # 127 h w / max |h w|: five roundings, of a ratio of at most 127
    hw = h_ref.double() * w.double()
    ratio = 127 * hw / hw.abs().amax(1, keepdim=True).clamp_min(1e-300)
    assert float((y.double() - ratio).abs().max()) <= 0.5 + 127 * 6 * U
    assert int(y.abs().max()) <= 127 and not y[0].any() and float(scales[0]) == 0


def backward_ref(dy, h, w, rstd, dres):
    dy, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    H = h.shape[1]
    g = dy * w
    c = r * r / H * (g * h).sum(1, keepdim=True)
    size = r * (g.abs() + h.abs() * (r * r / H * (g * h).abs().sum(1, keepdim=True)))
    dx = r * (g - h * c)
    if dres is not None:
        dx, size = dx + dres.double(), size + dres.double().abs()
    return dx, size, (dy * h * r).sum(0), (dy * h * r).abs().sum(0)


def held(T, H, seed):
    """Random block rows and their values."""
    q = ints((T, H), seed, -127, 128)
    e = ints((T, -(-H // 32)), seed + 1, 119, 124).to(torch.uint8)
    return q, e, q.double() * 2.0 ** (e.cpu().double() - 127).cuda().repeat_interleave(32, 1)[:, :H]


@pytest.mark.parametrize("T,H", NORM_SIZES + [(3000, 72)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("in_8_bits", [False, True])
def test_norm_backward(T, H, dtype, in_8_bits):
    x, w, dy = rnd((T, H), dtype, 1, 2.0), rnd((H,), dtype, 3), rnd((T, H), dtype, 4)
    dres = rnd((T, H), dtype, 5) if T % 2 else None
    rstd = rnd((T,), F32, 6).abs() + 0.5
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    op = pkg.RmsNorm.like(x, w, torch.empty_like(x), eps=EPS)
    if in_8_bits:
        q, e, h = held(T, H, 7)
        op.backward(dy, q, w, rstd, dx, dw, dresidual=dres, exponents=e)
    else:
        h = x
        op.backward(dy, h, w, rstd, dx, dw, dresidual=dres)
    done(op)
    dx_ref, size, dw_ref, dw_size = backward_ref(dy, h, w, rstd, dres)
    near(dx, dx_ref, (H + 12) * U * size, "dx")
    near(dw, dw_ref, (T + 4) * U * dw_size, "dweight")


def test_norm_gradients_are_the_differences():
    """The gradient of a function of (x, residual, weight) against central
    differences of the forward pass in 64 bits."""
    T, H = 4, 48
    x, res, w = rnd((T, H), F32, 1), rnd((T, H), F32, 2), rnd((H,), F32, 3)
    dy, dh = rnd((T, H), F32, 4), rnd((T, H), F32, 5)
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, residual=res, h=h, eps=EPS)
    op.run(x, w, y, residual=res, h=h, rstd=rstd)
    op.backward(dy, h, w, rstd, dx, dw, dresidual=dh)
    done(op)

    def loss(x, w):
        hd = x + res.double()
        r = 1 / torch.sqrt((hd * hd).mean(1, keepdim=True) + EPS)
        return float((hd * r * w * dy.double()).sum() + (hd * dh.double()).sum())

    xd, wd, d = x.double(), w.double(), 1e-5
    for i in [(0, 0), (1, 5), (3, 47), (2, 20)]:
        e = torch.zeros_like(xd)
        e[i] = d
        assert abs((loss(xd + e, wd) - loss(xd - e, wd)) / (2 * d) - float(dx[i])) < 1e-4
        e = torch.zeros_like(wd)
        e[i[1]] = d
        assert abs((loss(xd, wd + e) - loss(xd, wd - e)) / (2 * d) - float(dw[i[1]])) < 1e-4


@pytest.mark.parametrize("H,pad", [(256, 8), (256, 3), (1000, 24), (77, 5)])
@pytest.mark.parametrize("out", ["x", "i8"])
def test_norm_strides_and_places(H, pad, out):
    """Rows with gaps, which stay as they were; h over x."""
    T, dtype = 21, BF16
    x, res, w = rnd((T, H), dtype, 1), rnd((T, H), dtype, 2), rnd((H,), dtype, 3)
    xs, rs = strided(x, pad), strided(res, pad + 8)
    y = strided(torch.zeros((T, H), dtype=torch.int8 if out == "i8" else dtype, device="cuda"), pad)
    scales = torch.empty(T, device="cuda") if out == "i8" else None
    rstd = torch.empty(T, device="cuda")
    op = pkg.RmsNorm.like(xs, w, y, scales=scales, residual=rs, h=xs, eps=EPS)
    op.run(xs, w, y, scales=scales, residual=rs, h=xs, rstd=rstd)
    h_ref, r_ref, y_ref = norm_ref(x, res, w)
    assert torch.equal(xs, h_ref)
    near(rstd, r_ref, (H + 5) * U * r_ref)
    for t in (xs, y):
        edge = t.as_strided((T, pad), (t.stride(0), 1), t.storage_offset() + H)
        assert bool((edge[:-1] == 77).all())
    if out == "x":
        near(y, y_ref, (H + 8) * U * y_ref.abs())
        dy = strided(rnd((T, H), dtype, 5), pad)
        dres, dx, dw = strided(res, pad), strided(res, pad), torch.empty(H, device="cuda")
        op.backward(dy, xs, w, rstd, dx, dw, dresidual=dres)
        dx_ref, size, dw_ref, dw_size = backward_ref(dy, h_ref, w, rstd, res)
        near(dx, dx_ref, (H + 12) * U * size)
        near(dw, dw_ref, (T + 4) * U * dw_size)
        edge = dx.as_strided((T, pad), (dx.stride(0), 1), dx.storage_offset() + H)
        assert bool((edge[:-1] == 77).all())
    done(op)


def test_norm_backward_in_place():
    T, H = 50, 512
    x, w, dy, dres = (rnd((T, H), BF16, 1), rnd((H,), BF16, 3), rnd((T, H), BF16, 4),
                      rnd((T, H), BF16, 5))
    rstd, dw = rnd((T,), F32, 6).abs() + 0.5, torch.empty(H, device="cuda")
    op = pkg.RmsNorm.like(x, w, torch.empty_like(x), eps=EPS)
    outs = []
    for place in ("dx", "dy", "dresidual"):
        a, b = dy.clone(), dres.clone()
        dx = {"dx": torch.empty_like(x), "dy": a, "dresidual": b}[place]
        op.backward(a, x, w, rstd, dx, dw, dresidual=b)
        outs.append((dx.clone(), dw.clone()))
    done(op)
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])


def test_norm_of_values_that_are_not_finite():
    T, H = 6, 320
    x, w = rnd((T, H), BF16, 1), rnd((H,), BF16, 2)
    x[1, 7], x[2, 9], x[3, 319] = float("inf"), float("nan"), float("-inf")
    y, scales = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, scales=scales, eps=EPS)
    op.run(x, w, y, scales=scales)
    done(op)
    assert torch.isfinite(scales).tolist() == [True, False, False, False, True, True]
    assert not y[1:4].any() and y[0].any()
    y = torch.empty_like(x)
    op = pkg.RmsNorm.like(x, w, y, eps=EPS)
    op.run(x, w, y)
    done(op)
    assert torch.isfinite(y).all(1).tolist() == [True, False, False, False, True, True]


# ---------------------------------------------------------------- rows to 8 bits
def blocks_ref(X):
    """(q, exponents, values) by integer arithmetic on the CPU in 64 bits."""
    X = X.cpu()
    least = -24 if X.dtype == F16 else -127
    T, H = X.shape
    x = torch.nn.functional.pad(X.double(), (0, -H % 32)).view(T, -1, 32)
    top = x.abs().amax(2)
    bad = ~torch.isfinite(x).all(2)
    m, k = torch.frexp(torch.where(bad, 1.0, top))
    e = (k - 7 + (m > 127 / 128).int()).clamp_min(least)
    e = torch.where(top == 0, torch.full_like(e, least), e)
    q = torch.where(bad[:, :, None], 0.0, torch.round(torch.ldexp(x, -e[:, :, None])))
    v = torch.ldexp(q, e[:, :, None].expand_as(q))
    big = torch.finfo(X.dtype).max
    v = torch.where(bad[:, :, None], float("nan"), v.clamp(-big, big))
    e = torch.where(bad, 255, e + 127)
    flat = lambda t: t.reshape(T, -1)[:, :H]  # noqa: E731
    return flat(q).to(torch.int8), e.to(torch.uint8), flat(v).to(X.dtype)


ROWS = [(1, 1), (3, 31), (2, 32), (5, 33), (4, 64), (1, 48), (9, 1000), (33, 1024), (700, 96),
        (64, 4096), (2, 20001)]


@pytest.mark.parametrize("T,H", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pad", [0, 5, 16])
def test_block_rows(T, H, dtype, pad):
    g = torch.Generator().manual_seed(H)
    # blocks of very different sizes, ties among them
    size = torch.exp2(torch.randint(-12, 12, (T, H), generator=g).float())
    X = (torch.randn((T, H), generator=g) * size).to(dtype).cuda()
    X = strided(X, pad) if pad else X
    q, e = pkg.Rows8.empty(X)
    q = strided(q, pad) if pad else q
    back = strided(torch.zeros_like(X), pad) if pad else torch.empty_like(X)
    op = pkg.Rows8.like(X, q, e)
    op.pack(X, q, e)
    op.unpack(q, e, back)
    done(op)
    q_ref, e_ref, v_ref = blocks_ref(X)
    assert torch.equal(e.cpu(), e_ref)
    assert torch.equal(q.cpu(), q_ref)
    assert torch.equal(back.cpu(), v_ref)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_block_rows_at_the_ends_of_the_range(dtype):
    f = torch.finfo(dtype)
    least = {BF16: 2.0 ** -133, F16: 2.0 ** -24, F32: 2.0 ** -149}[dtype]
    rows = torch.zeros(12, 64)
    rows[1, 3] = float("nan")
    rows[2, 5], rows[2, 40] = float("inf"), 1.0
    rows[3, :32], rows[3, 32:] = f.max, -f.max
    rows[4] = least
    rows[5, 0], rows[5, 1:] = f.tiny, f.tiny / 4
    rows[6, 0], rows[6, 1] = 127.0, 0.5     # 127 is a whole step, and a tie to even (0)
    rows[7, 0], rows[7, 1] = 127.0, 1.5     # a tie to 2
    rows[8, 0], rows[8, 1] = 127.5, 1.0     # above 127: two a step
    rows[9, 63] = -least
    rows[10] = float("-inf")
    rows[11, ::2] = 3.0
    X = rows.to(dtype).cuda()
    q, e = pkg.Rows8.empty(X)
    back = torch.empty_like(X)
    op = pkg.Rows8.like(X, q, e)
    op.pack(X, q, e)
    op.unpack(q, e, back)
    done(op)
    q_ref, e_ref, v_ref = blocks_ref(X)
    assert torch.equal(e.cpu(), e_ref)
    assert torch.equal(q.cpu(), q_ref)
    assert torch.equal(torch.isnan(back).cpu(), torch.isnan(v_ref))
    ok = ~torch.isnan(v_ref)
    assert torch.equal(back.cpu()[ok], v_ref[ok])


@pytest.mark.parametrize("T,H", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pad", [0, 5])
def test_scaled_rows(T, H, dtype, pad):
    X = rnd((T, H), dtype, 1, 4.0)
    X[-1] = 0 if T > 1 else X[-1]
    X = strided(X, pad) if pad else X
    q, s = pkg.Rows8.empty(X, block=False)
    back = strided(torch.zeros_like(X), pad) if pad else torch.empty_like(X)
    op = pkg.Rows8.like(X, q, s)
    op.pack(X, q, s)
    op.unpack(q, s, back)
    done(op)
    top = X.float().abs().amax(1)
    # divided in 64 bits: by a number, torch multiplies with a rounded 1 / 127 on the GPU
    assert torch.equal(s, (top.double() / 127).float())
    ratio = 127 * X.double() / top.double().clamp_min(1e-300)[:, None]
    assert float((q.double() - ratio).abs().max()) <= 0.5 + 127 * 3 * U
    near(back, q.double() * s.double()[:, None], U * (q.double() * s.double()[:, None]).abs())


def test_scaled_rows_of_odd_values():
    X = torch.zeros(7, 64, device="cuda")
    X[0, 1], X[1, 2], X[2, 3] = float("nan"), float("inf"), float("-inf")
    X[3] = 1e-40
    X[3, 0] = -1e-38
    X[4] = 3e38
    X[5] = 2.0 ** -149
    q, s = pkg.Rows8.empty(X, block=False)
    back = torch.empty_like(X)
    op = pkg.Rows8.like(X, q, s)
    op.pack(X, q, s)
    op.unpack(q, s, back)
    done(op)
    assert torch.isfinite(s).tolist() == [False] * 3 + [True] * 4
    assert not q[:3].any() and torch.isnan(back[:3]).all()
    assert int(q[3, 0]) == -127 and int(q[3, 1]) == 1 and (q[4] == 127).all() and not q[6].any()
    assert torch.isfinite(back[3:]).all()


# ---------------------------------------------------------------- gradients from block rows
COUNTS = {
    "one": [1],
    "mixed": [0, 1, 33, 0, 256, 31, 32, 257, 0],
    "long": [600, 5, 129],
    "none": [0, 0, 0],
}


def offsets_of(counts, first=0):
    return torch.tensor([first] + list(counts)).cumsum(0).to(torch.int32).cuda()


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N,dtype,out,with_c,pad", [
    (64, 128, BF16, BF16, False, 0),
    (328, 200, F16, F16, True, 8),
    (72, 136, BF16, F32, True, 3),
    (33, 61, BF16, BF16, False, 0),
    (1, 300, F16, F32, False, 0),
])
def test_grad(counts, K, N, dtype, out, with_c, pad):
    counts = COUNTS[counts]
    E, R = len(counts), sum(counts)
    off = offsets_of(counts)
    q, e, A = held(max(R, 1), K, 1)
    q, e, A = q[:R], e[:R], A[:R]
    q = strided(q, pad) if pad else q
    B = rnd((max(R, 1), N), dtype, 4)[:R]
    C = rnd((E, K, N), out, 5) if with_c else None
    D = torch.full((E, K, N), 7.0, dtype=out, device="cuda")
    op = pkg.Rows8Grad.like(q, e, B, off, C, D)
    op.run(q, e, B, off, C, D)
    done(op)
    at = 0
    for i, n in enumerate(counts):
        a, b = A[at:at + n], B[at:at + n].double()
        ref, S = a.t() @ b, a.abs().t() @ b.abs()
        if C is not None:
            ref, S = ref + C[i].double(), S + C[i].double().abs()
        near(D[i], ref, 2 * (n + 1) * U * S, f"expert {i}")
        at += n


@pytest.mark.parametrize("R,K,N", [(0, 64, 64), (1, 8, 8), (777, 200, 136), (4096, 512, 768)])
def test_grad_dense(R, K, N):
    q, e, A = held(max(R, 1), K, 1)
    q, e, A, B = q[:R], e[:R], A[:R], rnd((max(R, 1), N), BF16, 4)[:R]
    D = torch.full((1, K, N), 7.0, device="cuda")
    op = pkg.Rows8Grad.like(q, e, B, None, None, D)
    op.run(q, e, B, None, None, D)
    done(op)
    near(D[0], A.t() @ B.double(), 2 * R * U * (A.abs().t() @ B.double().abs()))


def test_grad_of_one_expert_keeps_from_the_others():
    """NaN rows (a block that was not finite) reach their own expert alone, and
    rows of no expert none."""
    off = offsets_of([40, 40, 40], first=8)
    q, e, A = held(140, 64, 1)
    B = rnd((140, 64), BF16, 2)
    e[50, 1] = 255                      # expert 1
    e[3], e[130] = 255, 255             # of none
    B[4], B[135] = float("nan"), float("inf")
    D = torch.zeros((3, 64, 64), dtype=BF16, device="cuda")
    op = pkg.Rows8Grad.like(q, e, B, off, None, D)
    op.run(q, e, B, off, None, D)
    done(op)
    for i in (0, 2):
        r = slice(8 + 40 * i, 48 + 40 * i)
        a, b = A[r], B[r].double()
        near(D[i], a.t() @ b, 82 * U * (a.abs().t() @ b.abs()))
    assert torch.isnan(D[1, 32:]).all() and torch.isfinite(D[1, :32]).all()


def test_grad_reports_offsets_that_decrease():
    q, e, _ = held(20, 32, 1)
    B, D = rnd((20, 32), BF16, 2), torch.zeros((2, 32, 32), device="cuda")
    off = torch.tensor([0, 15, 10], dtype=torch.int32, device="cuda")
    op = pkg.Rows8Grad.like(q, e, B, off, None, D)
    op.run(q, e, B, off, None, D)
    assert op.status() == pkg.GEMM_ERR_INVALID_ARG
    done(op)


# ---------------------------------------------------------------- scaled products
def i8_check(counts, K, N, out, seed=0, x=None, w=None, pad=0, first=0, plan=None, scale=1.0):
    E, R = len(counts), sum(counts)
    off = offsets_of(counts, first) if E > 1 or first else None
    rows = R + 2 * first
    X = ints((max(rows, 1), K), seed + 1)[:rows] if x is None else x
    W = ints((E, N, K), seed + 2) if w is None else w
    if pad:
        X = strided(X, pad)
        wide = torch.full((E, N, K + pad), 99, dtype=torch.int8, device="cuda")
        wide[:, :, :K] = W
        W = wide[:, :, :K]
    xs, ws = rnd((rows,), F32, seed + 3).abs() * scale, rnd((E, N), F32, seed + 4) * K ** -0.5 / 64
    D = torch.full((rows, N), 7.0, dtype=out, device="cuda")
    if pad:
        D = strided(D, pad)
    with forced_plan(plan):
        op = pkg.I8Gemm.like(X, xs, W, ws, off, D)
    op.run(X, xs, W, ws, off, D)
    done(op)
    at = first
    for i, n in enumerate(counts):
        r = slice(at, at + n)
        a, b = X[r].double(), W[i].double()
        s = xs[r, None].double() * ws[i].double()
        ref = a @ b.t() * s
        # exact below 2^24, which K up to 1024 stays within; else K u of the magnitudes
        slack = 4 * U * ref.abs()
        if K > 1024:
            slack = slack + K * U * (a.abs() @ b.abs().t()) * s.abs()
        near(D[r], ref, slack, f"expert {i}")
        at += n
    assert bool((D[:first] == 7).all()) and bool((D[at:] == 7).all())
    return D


SIZES = [(64, 16), (64, 64), (128, 256), (1000, 264), (33, 61), (1, 1), (15, 7), (17, 130),
         (4096, 512), (272, 1040)]


# the few-rows kernel; tensor-core tiles of 64 and of 128 rows, shared by clusters where they are few,
# and by the schedule; CTA pairs over widened operands
PLANS = ["tiles=0,wide=0", "tiles=1,wide=0,tall=0", "tiles=1,wide=0,tall=1",
         "tiles=1,wide=0,tall=0,csk=0", "tiles=1,wide=0,tall=1,csk=0", "wide=1"]


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("R", [1, 2, 8, 9, 16, 17, 40, 64, 65, 130, 300])
@pytest.mark.parametrize("K,N", SIZES)
def test_i8_dense(R, K, N, plan):
    i8_check([R], K, N, [BF16, F16, F32][(R + K) % 3], seed=R + K, plan=plan)


@pytest.mark.parametrize("R,K,N", [(1, 640, 320), (16, 640, 320), (17, 640, 320), (64, 8192, 512),
                                   (600, 512, 512), (1500, 2048, 2304), (4000, 256, 4096)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_i8_as_planned(R, K, N, out):
    """Without a forced plan; more tiles than CTAs, and tiles shared by several."""
    i8_check([R], K, N, out)


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("counts", [[1, 0, 2, 0, 0, 1, 3, 0, 1, 0, 0, 0, 0, 0, 0, 1, 2],
                                    [0, 1, 33, 0, 256, 31, 32, 257, 0], [600, 5, 129], [0, 0, 0],
                                    [9, 20, 0, 17]])
@pytest.mark.parametrize("K,N,out", [(64, 128, BF16), (200, 328, F16), (1000, 264, F32),
                                     (33, 61, BF16), (2048, 96, BF16)])
def test_i8_experts(counts, K, N, out, plan):
    i8_check(counts, K, N, out, plan=plan)


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("counts", [[3], [70], [5, 0, 90, 33]])
@pytest.mark.parametrize("K,N,pad", [(128, 64, 16), (128, 64, 1), (100, 33, 12), (513, 72, 7)])
def test_i8_strides_and_rows_of_no_expert(counts, K, N, pad, plan):
    i8_check(counts, K, N, BF16, pad=pad, plan=plan)
    i8_check(counts, K, N, F16, pad=pad, first=5, plan=plan)


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("R", [1, 16, 64, 200])
def test_i8_extremes(R, plan):
    """Every value -128 and every product 2^14: 1024 of them are 2^24, exactly."""
    K, N = 1024, 160
    x = torch.full((R, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
    i8_check([R], K, N, F32, x=x, w=w, plan=plan)
    w[:, ::2] = 127
    x[:, 1::2] = 127
    i8_check([R], K, N, F32, x=x, w=w, plan=plan)


@pytest.mark.parametrize("plan", PLANS[1:])
@pytest.mark.parametrize("flag", [pkg.GEMM_DEBUG_SKIP_FIRST_FILL, pkg.GEMM_DEBUG_SKIP_ONE_FILL])
@pytest.mark.parametrize("counts", [[700], [40] * 20])
def test_i8_after_a_timeout(plan, flag, counts):
    """A wait that runs out is reported, and the next call starts afresh."""
    R, K, N = sum(counts), 1536, 1000
    off = offsets_of(counts) if len(counts) > 1 else None
    X, W = ints((R, K), 1), ints((len(counts), N, K), 2)
    xs, ws = torch.ones(R, device="cuda"), torch.ones((len(counts), N), device="cuda")
    D = torch.zeros((R, N), device="cuda")
    with forced_plan(plan):
        op = pkg.I8Gemm.like(X, xs, W, ws, off, D)
    op.run(X, xs, W, ws, off, D)
    assert op.status() == pkg.GEMM_OK
    first = D.clone()
    for timeout_ns in (1_000_000, 10_000_000):
        op.debug_set(flag, timeout_ns)
        op.run(X, xs, W, ws, off, D)
        assert op.status() == pkg.GEMM_ERR_DEVICE_TIMEOUT
        op.debug_set(0)
        D.fill_(7.0)
        op.run(X, xs, W, ws, off, D)
        assert op.status() == pkg.GEMM_OK
        assert torch.equal(D, first)
    op.close()


@pytest.mark.parametrize("R", [1, 33])
def test_i8_scales_that_are_not_finite(R):
    """A row's or an output's scale reaches nothing else."""
    K, N = 64, 48
    X, W = ints((R, K), 1), ints((1, N, K), 2)
    xs, ws = torch.ones(R, device="cuda"), torch.ones((1, N), device="cuda")
    xs[0], ws[0, 5] = float("nan"), float("inf")
    D = pkg.i8_matmul(X, xs, W, ws, out_dtype=F32)
    assert torch.isnan(D[0]).all()
    keep = [n for n in range(N) if n != 5]
    assert torch.equal(D[1:][:, keep], (X[1:].double() @ W[0].double().t()).float()[:, keep])


def test_i8_without_k_is_zero():
    D = torch.full((3, 8), 7.0, device="cuda")
    X, W = torch.empty((3, 0), dtype=torch.int8, device="cuda"), torch.empty((1, 8, 0), dtype=torch.int8, device="cuda")
    op = pkg.I8Gemm.like(X, torch.ones(3, device="cuda"), W, torch.ones((1, 8), device="cuda"), None, D)
    op.run(X, torch.ones(3, device="cuda"), W, torch.ones((1, 8), device="cuda"), None, D)
    done(op)
    assert not D.any()


def test_i8_reports_offsets_that_decrease():
    X, W = ints((20, 64), 1), ints((2, 32, 64), 2)
    xs, ws = torch.ones(20, device="cuda"), torch.ones((2, 32), device="cuda")
    D = torch.zeros((20, 32), device="cuda")
    off = torch.tensor([0, 30, 10], dtype=torch.int32, device="cuda")
    op = pkg.I8Gemm.like(X, xs, W, ws, off, D)
    op.run(X, xs, W, ws, off, D)
    assert op.status() == pkg.GEMM_ERR_INVALID_ARG
    done(op)


# ---------------------------------------------------------------- together
def test_a_layer_from_norm_to_gradient():
    """The norm's 8-bit rows go to the product; the rows kept in 8 bits give the
    weight's and the norm's gradients."""
    T, H, F = 130, 256, 192
    x, res, g = rnd((T, H), BF16, 1), rnd((T, H), BF16, 2), rnd((H,), BF16, 3)
    W, ws = ints((1, F, H), 4), rnd((1, F), F32, 5).abs() / 900
    h, y8, s = torch.empty_like(x), torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    D = torch.empty((T, F), dtype=BF16, device="cuda")
    norm = pkg.RmsNorm.like(x, g, y8, scales=s, residual=res, h=h, eps=EPS)
    product = pkg.I8Gemm.like(y8, s, W, ws, None, D)
    norm.run(x, g, y8, scales=s, residual=res, h=h)
    product.run(y8, s, W, ws, None, D)
    ref = y8.double() @ W[0].double().t() * s.double()[:, None] * ws[0].double()
    near(D, ref, 4 * U * ref.abs())
    # training: what the norm gave is kept in 8 bits, and so is h
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    train = pkg.RmsNorm.like(x, g, y, residual=res, h=h, eps=EPS)
    train.run(x, g, y, residual=res, h=h, rstd=rstd)
    keep = pkg.Rows8.like(y, *pkg.Rows8.empty(y))
    (qy, ey), (qh, eh) = pkg.Rows8.empty(y), pkg.Rows8.empty(h)
    keep.pack(y, qy, ey)
    keep.pack(h, qh, eh)
    dD, dW = rnd((T, F), BF16, 6), torch.empty((1, H, F), dtype=F32, device="cuda")
    grad = pkg.Rows8Grad.like(qy, ey, dD, None, None, dW)
    grad.run(qy, ey, dD, None, None, dW)
    _, _, yv = blocks_ref(y)
    yv = yv.double().cuda()
    near(dW[0], yv.t() @ dD.double(), 2 * T * U * (yv.abs().t() @ dD.double().abs()))
    dy, dx, dg = rnd((T, H), BF16, 7), torch.empty_like(x), torch.empty(H, device="cuda")
    train.backward(dy, qh, g, rstd, dx, dg, dresidual=res, exponents=eh)
    _, _, hv = blocks_ref(h)
    dx_ref, size, dg_ref, dg_size = backward_ref(dy, hv.cuda(), g, rstd, res)
    near(dx, dx_ref, (H + 12) * U * size)
    near(dg, dg_ref, (T + 4) * U * dg_size)
    for op in (norm, product, train, keep, grad):
        done(op)


@pytest.mark.parametrize("plan", PLANS)
def test_i8_experts_with_most_of_the_rows(plan):
    """Few rows an expert on average, but one has nearly all of them."""
    i8_check([0] * 20 + [150] + [0] * 30 + [1] + [0] * 12, 256, 136, BF16, plan=plan)


def test_i8_many_rows_without_k():
    """More rows than a grid's second dimension has blocks of eight."""
    R = 8 * 70000
    D = torch.full((R, 8), 7.0, dtype=BF16, device="cuda")
    X = torch.empty((R, 0), dtype=torch.int8, device="cuda")
    W = torch.empty((1, 8, 0), dtype=torch.int8, device="cuda")
    xs, ws = torch.ones(R, device="cuda"), torch.ones((1, 8), device="cuda")
    op = pkg.I8Gemm.like(X, xs, W, ws, None, D)
    op.run(X, xs, W, ws, None, D)
    done(op)
    assert not D.any()
