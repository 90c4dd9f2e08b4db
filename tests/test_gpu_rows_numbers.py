"""The operators on 8-bit rows on the GPU where a value lies between two answers
or near the ends of its type's range.

Integers of scaled rows are the nearest to 127 v / max |v| rounded to fp32, ties to
even, and compared for equality: in 64 bits 127 v is exact, and the quotient of two
numbers of 24 bits is a middle of two integers or off one by more than 2^-53 of it.
Of 16-bit values the rounding to fp32 changes nothing, and is left out.
Tolerances otherwise are those of test_gpu_rows.py: u = 2^-24 a rounded fp32
operation, and half a step of the output's type.
"""
from __future__ import annotations

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg
from gpu_helpers import forced_plan
from test_gpu_rows import (BF16, EPS, F16, F32, HALF_STEP, PLANS, TINY, U, backward_ref, done, ints,
                           near, offsets_of, rnd, strided)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- integers of scaled rows
def nearest_integers(v):
    """Those of rows v (any type), on the CPU in 64 bits; zeros for a row of zeros."""
    short, v = v.dtype != F32, v.cpu().double()
    top = v.abs().amax(1, keepdim=True)
    quotient = torch.where(top > 0, 127 * v / top.clamp_min(1e-300), 0.0)
    return torch.round(quotient if short else quotient.float()).to(torch.int8)


def rows_with_ties(T, H, dtype, seed):
    """Rows in which about half of the values lie at or, in fp32, next to the middle of
    two steps: c (n + 1/2) beside the largest, 127 c, or what is nearest to (n + 1/2)
    largest / 127; of sizes spread over the type's range."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(1, {BF16: 2, F16: 16, F32: 2 ** 16}[dtype], (T, 1), generator=g).double()
    middle = torch.randint(-126, 126, (T, H), generator=g) + 0.5
    rows = c * middle
    other = torch.randn((T, H), generator=g).double() * 30 * c
    rows = torch.where(torch.rand((T, H), generator=g) < 0.5, rows, other.clamp(-120 * c, 120 * c))
    top = 127 * c
    if dtype == F32:  # every second row has any largest value
        odd = torch.arange(T)[:, None] % 2 == 1
        some = (1 + torch.rand((T, 1), generator=g)).double()
        beside = torch.randint(-1, 2, (T, H), generator=g).double()
        value = (some * middle / 127).float()
        value = value.double() + beside * 2.0 ** (torch.frexp(value)[1].double() - 24)
        rows, top = torch.where(odd, value, rows), torch.where(odd, some, top)
    rows[:, H // 2] = top[:, 0] * torch.where(torch.rand(T, generator=g) < 0.5, 1.0, -1.0)
    low, high = {BF16: (-120, 118), F16: (-12, 4), F32: (-110, 108)}[dtype]
    rows = rows * 2.0 ** torch.linspace(low, high, T).round().double()[:, None]
    return rows.to(dtype).cuda()


WIDTHS = [(1, 1), (9, 64), (33, 1000), (200, 2047), (3, 4096), (170, 4096), (5, 40001), (3, 65536)]


@pytest.mark.parametrize("T,H", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pad", [0, 5])
def test_scaled_rows_have_the_nearest_integers(T, H, dtype, pad):
    X = rows_with_ties(T, H, dtype, H)
    X = strided(X, pad) if pad else X
    q, s = pkg.Rows8.empty(X, block=False)
    op = pkg.Rows8.like(X, q, s)
    op.pack(X, q, s)
    done(op)
    assert torch.equal(q.cpu(), nearest_integers(X))


@pytest.mark.parametrize("T,H", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("weights", ["ones", "any"])
@pytest.mark.parametrize("pad", [0, 5])
def test_norm_to_the_nearest_integers(T, H, dtype, weights, pad):
    """Those of h w, whose product is rounded to fp32 where it has more bits."""
    low, high = (2.0 ** -60, 2.0 ** 60) if dtype != F16 else (0, float("inf"))
    x = rows_with_ties(T, H, dtype, H)
    keep = (x.abs().amax(1) > low) & (x.abs().amax(1) < high)
    x[~keep] = 0  # (the ends of the range have a test of their own)
    x = strided(x, pad) if pad else x
    w = torch.ones(H, dtype=dtype, device="cuda") if weights == "ones" else rnd((H,), dtype, 3)
    y, scales = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, scales=scales, eps=EPS)
    op.run(x, w, y, scales=scales)
    done(op)
    assert torch.equal(y.cpu(), nearest_integers(x.cpu().float() * w.cpu().float()))


# ---------------------------------------------------------------- scaled rows back
def test_scaled_rows_back_from_scales_of_either_sign():
    """What rounds past the largest finite value comes back as that, by negative
    scales too."""
    for dtype in (F16, BF16, F32):
        top = torch.finfo(dtype).max
        s = torch.tensor([1.0, -1.0, 0.01, -0.01, 0.0, -0.0, 1e-3, -1e-3], device="cuda") * top
        q = ints((8, 96), 3, -127, 128)
        q[:, 0], q[:, 1] = 127, -127
        X = torch.empty((8, 96), dtype=dtype, device="cuda")
        op = pkg.Rows8.like(X, q, s)
        op.unpack(q, s, X)
        done(op)
        want = (q.double() * s.double()[:, None]).clamp(-top, top)
        assert bool(torch.isfinite(X).all())
        near(X, want, U * want.abs())


# ---------------------------------------------------------------- norm at the ends of the range
def norm_of_any_size(h, w, eps):
    """(rstd, y) in 64 bits."""
    h = h.double()
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    return rstd, h * rstd[:, None] * w.double()


# a row's size, as the exponent of two; at the last of them rstd is below fp32's normal range
SIZES = [-126, -120, -80, -64, -50, -40, 40, 60, 64, 70, 100, 120, 126]
RANGE_WIDTHS = [64, 1001, 2048, 4096, 8200, 40000, 40001]


def rows_of_sizes(H, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.rand((len(SIZES), H), generator=g) + 0.5) * torch.where(
        torch.rand((len(SIZES), H), generator=g) < 0.5, 1.0, -1.0)
    return (x * torch.exp2(torch.tensor(SIZES, dtype=torch.float64))[:, None]).to(dtype).cuda()


@pytest.mark.parametrize("H", RANGE_WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("eps", [0.0, EPS, 2.0 ** -100, 1e30])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_of_rows_of_any_size(H, dtype, eps, with_residual):
    """Neither the squares nor their sum leave fp32's range unseen."""
    x, w = rows_of_sizes(H, dtype, H), rnd((H,), dtype, 3)
    res = torch.zeros_like(x) if with_residual else None
    h = torch.empty_like(x) if with_residual else None
    y, rstd = torch.empty_like(x), torch.empty(len(SIZES), device="cuda")
    op = pkg.RmsNorm.like(x, w, y, residual=res, h=h, eps=eps)
    op.run(x, w, y, residual=res, h=h, rstd=rstd)
    done(op)
    r_ref, y_ref = norm_of_any_size(x, w, op.desc.eps)
    if with_residual:
        assert torch.equal(h, x)
    # (rstd's least step is 2^-149, half of it what h multiplies)
    near(rstd, r_ref, (H + 8) * U * r_ref, "rstd")
    near(y, y_ref, (H + 12) * U * y_ref.abs() + 2.0 ** -150 * (x.double() * w.double()).abs(), "y")


@pytest.mark.parametrize("H", RANGE_WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("eps", [0.0, EPS])
@pytest.mark.parametrize("size", [-100, -60, 0, 60, 100])
def test_norm_to_8_bits_of_rows_and_weights_of_any_size(H, dtype, eps, size):
    """h w may leave fp32's range where y does not."""
    x, w = rows_of_sizes(H, dtype, H), (rnd((H,), F32, 3) * 2.0 ** size).to(dtype)
    y, scales = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(x), device="cuda")
    op = pkg.RmsNorm.like(x, w, y, scales=scales, eps=eps)
    op.run(x, w, y, scales=scales)
    done(op)
    r_ref, y_ref = norm_of_any_size(x, w, op.desc.eps)
    top = y_ref.abs().amax(1)
    # two roundings of what may be below the normal range, then divided by 127
    near(scales, top / 127, (H + 12) * U * top / 127 + 2 * 2.0 ** -150, "scales")
    ratio = 127 * y_ref / top[:, None]
    assert float((y.double() - ratio).abs().max()) <= 0.5 + 127 * 3 * U


@pytest.mark.parametrize("H", [64, 1001, 4096, 40001])
@pytest.mark.parametrize("dtype,size", [(BF16, -128), (BF16, -133), (F32, -128), (F32, -140), (F32, -149)])
def test_norm_of_rows_below_the_normal_range(H, dtype, size):
    """rstd is infinite in fp32, y is not."""
    g = torch.Generator().manual_seed(H)
    x = torch.randint(-3, 4, (5, H), generator=g).double() * 2.0 ** size
    x[:, 0] = 2.0 ** size
    x, w = x.to(dtype).cuda(), rnd((H,), dtype, 3)
    y, rstd = torch.empty_like(x), torch.empty(5, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, eps=0.0)
    op.run(x, w, y, rstd=rstd)
    done(op)
    r_ref, y_ref = norm_of_any_size(x, w, 0.0)
    near(y, y_ref, (H + 12) * U * y_ref.abs(), "y")
    fits = r_ref < torch.finfo(F32).max
    near(rstd[fits], r_ref[fits], (H + 8) * U * r_ref[fits], "rstd")
    assert bool(torch.isinf(rstd[~fits]).all())
    y, scales = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, scales=scales, eps=0.0)
    op.run(x, w, y, scales=scales)
    done(op)
    near(scales, y_ref.abs().amax(1) / 127, (H + 12) * U * y_ref.abs().amax(1) / 127, "scales")


def test_norm_of_zeros_and_what_is_not_finite_beside_large_rows():
    H = 320
    x = rows_of_sizes(H, BF16, 1)
    x[1], x[3, 7], x[9, 5], x[11, 300] = 0, float("inf"), float("nan"), float("-inf")
    w = rnd((H,), BF16, 2)
    y, rstd = torch.empty_like(x), torch.empty(len(x), device="cuda")
    op = pkg.RmsNorm.like(x, w, y, eps=0.0)
    op.run(x, w, y, rstd=rstd)
    done(op)
    r_ref, y_ref = norm_of_any_size(x, w, 0.0)
    assert torch.equal(torch.isnan(y), torch.isnan(y_ref))  # (of zeros: 0 / 0)
    assert torch.equal(torch.isinf(rstd), torch.isinf(r_ref))
    assert torch.equal(rstd == 0, r_ref == 0)
    y, scales = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(x), device="cuda")
    op = pkg.RmsNorm.like(x, w, y, scales=scales, eps=EPS)
    op.run(x, w, y, scales=scales)
    done(op)
    bad = [3, 9, 11]
    assert torch.isfinite(scales).logical_not().nonzero().flatten().tolist() == bad
    assert not y[bad].any() and not y[1].any() and float(scales[1]) == 0


@pytest.mark.parametrize("H", [64, 1001, 4096, 8200, 16392, 40001])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kept", ["rows", "8 bits"])
def test_norm_gradients_of_rows_of_any_size(H, dtype, kept):
    """The forward pass's own rstd, from rows or from their 8 bits."""
    x, w = rows_of_sizes(H, dtype, H), rnd((H,), dtype, 3)
    T = len(x)
    dy, dres = rnd((T, H), dtype, 4), rnd((T, H), dtype, 5)
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, eps=0.0)
    op.run(x, w, y, rstd=rstd)
    rows, exponents, h = x, None, x.double()
    if kept == "8 bits":
        rows, exponents = pkg.Rows8.empty(x)
        pkg.Rows8.like(x, rows, exponents).pack(x, rows, exponents)
        step = torch.exp2(exponents.cpu().double() - 127).cuda().repeat_interleave(32, 1)[:, :H]
        h = rows.double() * step
    op.backward(dy, rows, w, rstd, dx, dw, dresidual=dres, exponents=exponents)
    done(op)
    dx_ref, size, dw_ref, dw_size = backward_ref(dy, h, w, rstd, dres)
    # below the normal range a rounding is 2^-150 instead of relative: of h r, whose
    # error w dy and the sum over the row pass on, and of r times what it multiplies
    r = rstd.double()[:, None]
    low = 4 * 2.0 ** -150 * (1 + r * (1 + (dy.double() * w.double()).abs().amax(1, keepdim=True)) * 8)
    fits = (dx_ref.abs() + size) < torch.finfo(dtype).max
    near(torch.where(fits, dx, torch.zeros_like(dx)), torch.where(fits, dx_ref, 0.0),
         torch.where(fits, (H + 12) * U * size + low, 0.0), "dx")
    near(dw, dw_ref, (T + 4) * U * dw_size + T * 2.0 ** -140, "dweight")
    assert bool(torch.isfinite(dw).all())


# ---------------------------------------------------------------- the gradients' wait
@pytest.mark.parametrize("flag", [pkg.GEMM_DEBUG_SKIP_FIRST_FILL, pkg.GEMM_DEBUG_SKIP_ONE_FILL])
@pytest.mark.parametrize("T,H", [(3, 64), (2000, 256), (700, 1001), (5000, 4096)])
@pytest.mark.parametrize("in_8_bits", [False, True])
@pytest.mark.parametrize("with_dresidual", [False, True])
def test_norm_gradients_after_a_timeout(flag, T, H, in_8_bits, with_dresidual):
    """A wait that runs out is reported, and the next call starts afresh."""
    x, w, dy = rnd((T, H), BF16, 1), rnd((H,), BF16, 2), rnd((T, H), BF16, 3)
    dres = rnd((T, H), BF16, 4) if with_dresidual else None
    rstd, dx, dw = rnd((T,), F32, 5).abs() + 0.5, torch.empty_like(x), torch.empty(H, device="cuda")
    rows, exponents = x, None
    if in_8_bits:
        rows, exponents = pkg.Rows8.empty(x)
        pkg.Rows8.like(x, rows, exponents).pack(x, rows, exponents)
    op = pkg.RmsNorm.like(x, w, torch.empty_like(x), eps=EPS)

    def run():
        op.backward(dy, rows, w, rstd, dx, dw, dresidual=dres, exponents=exponents)
        return op.status()

    assert run() == pkg.GEMM_OK
    first = dx.clone(), dw.clone()
    for timeout_ns in (1_000_000, 10_000_000):
        op.debug_set(flag, timeout_ns)
        assert run() == pkg.GEMM_ERR_DEVICE_TIMEOUT
        op.debug_set(0)
        dx.fill_(7.0)
        dw.fill_(7.0)
        assert run() == pkg.GEMM_OK
        assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])
    op.close()


# ---------------------------------------------------------------- scales of a product
@pytest.mark.parametrize("counts", [[1], [8], [20], [70], [3, 0, 40, 9]])
@pytest.mark.parametrize("out", [F32, BF16])
def test_i8_scales_the_same_in_every_form(counts, out):
    """The sum times the row's scale, then times the output's: where the scales'
    product would leave fp32's range, and the same bits in every form."""
    R, K, N, E = sum(counts), 1000, 136, len(counts)
    off = offsets_of(counts) if E > 1 else None
    X, W = ints((R, K), 1), ints((E, N, K), 2)
    X[0] = 0  # a sum of zero
    pairs = torch.tensor([(1e-25, 1e-18), (1e20, 1e25), (3e-20, 2e-24), (0.01, 0.02)])
    xs = pairs[torch.arange(R) % 4, 0].cuda() * (1 + rnd((R,), F32, 3).abs())
    ws = pairs[torch.arange(N) % 4, 1].cuda() * (1 + rnd((E, N), F32, 4).abs())
    got = []
    for plan in PLANS:
        D = torch.empty((R, N), dtype=out, device="cuda")
        with forced_plan(plan):
            op = pkg.I8Gemm.like(X, xs, W, ws, off, D)
        op.run(X, xs, W, ws, off, D)
        done(op)
        got.append(D)
    at = 0
    for e, n in enumerate(counts):
        r = slice(at, at + n)
        sums = X[r].double() @ W[e].double().t()
        first = (sums.float() * xs[r, None]).double()  # the sums are exact
        ref = first * ws[e].double()
        fits = ref.abs() < torch.finfo(out).max
        d = got[0][r].double()
        off_by = (d - ref).abs() - (U * ref.abs() + 2.0 ** -150) * 2 - HALF_STEP[out] * ref.abs() - TINY[out]
        assert not bool((off_by[fits] > 0).any())
        assert not d[sums == 0].any()
        at += n
    for D, plan in zip(got[1:], PLANS[1:]):
        assert torch.equal(D, got[0]), plan


# ---------------------------------------------------------------- forms of a product
@pytest.mark.parametrize("E,R,N,K,form", [
    (1, 8, 4096, 4096, "rows"), (1, 64, 4096, 4096, "tiles"), (1, 4096, 4096, 1024, "tiles"),
    (1, 8192, 256, 2048, "tiles"), (1, 8192, 2048, 512, "tiles"), (1, 8192, 8192, 256, "wide"),
    (8, 49152, 512, 256, "wide"), (8, 49152, 128, 256, "tiles"), (64, 64, 512, 256, "rows"),
])
def test_i8_form_by_rows_and_outputs(E, R, N, K, form):
    """Both operands are widened where there are many rows and tiles enough for all SMs."""
    X = torch.zeros((R, K), dtype=torch.int8, device="cuda")
    W = torch.zeros((E, N, K), dtype=torch.int8, device="cuda")
    xs, ws = torch.ones(R, device="cuda"), torch.ones((E, N), device="cuda")
    off = offsets_of([R // E] * E) if E > 1 else None
    D = torch.empty((R, N), dtype=BF16, device="cuda")
    op = pkg.I8Gemm.like(X, xs, W, ws, off, D)
    assert f"form={form} " in op.plan()
    op.close()
