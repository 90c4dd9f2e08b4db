"""The expert and 4-bit-weight operators on the GPU, against their formulas in
64 bits.

Tolerances, per element of a sum of n products with S = sum of their
magnitudes: every fp32 addition (in the tensor core too, where it truncates)
is off by at most 2**-23 of the partial sum, and the partial sums are at most
S, so the sum is within n * 2**-23 * S; the one rounding to D's type adds half
a unit in the last place (2**-9 of the result in bf16, 2**-12 in fp16, 2**-25
below its normal range).  Softmax gates: two exponentials and a division of
two ulp each and a sum of n terms, n + 8 units of 2**-23.  Whole numbers are
equal.
"""
from __future__ import annotations

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg
from gpu_helpers import forced_plan

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
HALF_ULP = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -133, F32: 2.0 ** -149}


def rnd(shape, dtype=F32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def near(got, ref, S, n, what=""):
    """got within the bound above of ref (fp64), NaN where ref is NaN."""
    dt = got.dtype
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    bound = n * 2.0 ** -23 * S + HALF_ULP[dt] * (ref.abs() + n * 2.0 ** -23 * S) + TINY[dt]
    off = (got - ref).abs() - bound
    off = off[~torch.isnan(off)]
    assert off.numel() == 0 or float(off.max()) <= 0, f"{what}: {float(off.max())} over the bound"


def offsets_of(counts, first=0):
    c = torch.tensor([first] + list(counts)).cumsum(0)
    return c.to(torch.int32).cuda()


def done(op, code=pkg.GEMM_OK):
    assert op.status() == code
    op.close()


# ---------------------------------------------------------------- grouped products
COUNTS = {
    "one": [1],
    "mixed": [0, 1, 33, 0, 256, 31, 32, 257, 0],
    "long": [600, 5, 129],
    "decode": [1, 0, 2, 0, 0, 1, 3, 0, 1, 0, 0, 0, 0, 0, 0, 1, 2],
    "none": [0, 0, 0],
}


def grouped_ref(A, B, off, C, grad):
    """(values, magnitudes) of the formula in fp64, NaN-free rows only where written."""
    off = off.tolist()
    E = len(off) - 1
    A, B = A.double(), B.double()
    if grad:
        D = torch.zeros((E, A.shape[1], B.shape[1]), dtype=torch.float64, device="cuda")
    else:
        D = torch.zeros((A.shape[0], B.shape[2]), dtype=torch.float64, device="cuda")
    S = torch.zeros_like(D)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        a, b = (A[r].t(), B[r]) if grad else (A[r], B[e])
        at = e if grad else r
        D[at] = a @ b
        S[at] = a.abs() @ b.abs()
    if C is not None:
        D += C.double()
        S += C.double().abs()
    return D, S


@pytest.mark.parametrize("plan", ["wide=0", "wide=1"])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N,dtype,out,order,with_c", [
    (64, 128, BF16, BF16, "nk", False),
    (200, 328, F16, F16, "kn", True),     # K and N end inside a tile
    (136, 72, BF16, F32, "kn", False),
    (1000, 264, F16, BF16, "nk", True),
    (33, 61, BF16, BF16, "nk", False),    # rows off the 16-byte grid: workspace copies
    (61, 33, F16, F32, "kn", True),
    (1, 1, BF16, F16, "nk", False),
    (8, 8, BF16, BF16, "kn", False),
])
def test_grouped_rows(plan, counts, K, N, dtype, out, order, with_c):
    counts = COUNTS[counts]
    E, R = len(counts), sum(counts)
    off = offsets_of(counts)
    A = rnd((max(R, 1), K), dtype, 1)[:R]
    B = rnd((E, N, K) if order == "nk" else (E, K, N), dtype, 2)
    B = B.transpose(1, 2) if order == "nk" else B
    C = rnd((R, N), out, 3) if with_c else None
    D = torch.full((R, N), 7.0, dtype=out, device="cuda")
    with forced_plan(plan):
        op = pkg.GroupedGemm.like(A, B, off, C, D)
    op.run(A, B, off, C, D)
    done(op)
    ref, S = grouped_ref(A, B, off, C, False)
    near(D, ref, S, K + 1)


@pytest.mark.parametrize("plan", ["wide=0", "wide=1"])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N,dtype,out,with_c", [
    (64, 128, BF16, BF16, False),
    (328, 200, F16, F16, True),
    (72, 136, BF16, F32, True),
    (33, 61, BF16, BF16, False),
    (1, 300, F16, F32, False),
])
def test_grouped_grad(plan, counts, K, N, dtype, out, with_c):
    counts = COUNTS[counts]
    E, R = len(counts), sum(counts)
    off = offsets_of(counts)
    A, B = rnd((max(R, 1), K), dtype, 1)[:R], rnd((max(R, 1), N), dtype, 2)[:R]
    C = rnd((E, K, N), out, 3) if with_c else None
    D = torch.full((E, K, N), 7.0, dtype=out, device="cuda")
    with forced_plan(plan):
        op = pkg.GroupedGemm.like(A, B, off, C, D)
    op.run(A, B, off, C, D)
    done(op)
    ref, S = grouped_ref(A, B, off, C, True)
    near(D, ref, S, max(counts) + 1)


@pytest.mark.parametrize("plan", ["wide=0", "wide=1"])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("K,N", [(96, 136), (40, 300)])
def test_grouped_rows_outside_and_nan_neighbours(plan, grad, K, N):
    """Rows before offsets[0] and past offsets[E] are NaN, as are the whole
    of expert 1 and the padding of every stride: no NaN reaches the others,
    and no row or column outside D is written."""
    counts, first, tail, pad = [37, 20, 300, 5], 3, 9, 8
    E, R = len(counts), first + sum(counts) + tail
    off = offsets_of(counts, first)
    nan = float("nan")

    def padded(shape, dtype, seed):
        t = torch.full((*shape[:-1], shape[-1] + pad), nan, dtype=dtype, device="cuda")
        t[..., :shape[-1]] = rnd(shape, dtype, seed)
        return t[..., :shape[-1]]

    A = padded((R, K), BF16, 1)
    A[:first] = nan
    A[R - tail:] = nan
    bad = slice(int(off[1]), int(off[2]))
    if grad:
        B = padded((R, N), BF16, 2)
        B[:first] = nan
        B[R - tail:] = nan
        A[bad] = nan
        whole = torch.full((E, K, N + pad), 7.0, dtype=BF16, device="cuda")
    else:
        B = padded((E, K, N), BF16, 2)
        B[1] = nan
        whole = torch.full((R, N + pad), 7.0, dtype=BF16, device="cuda")
    D = whole[..., :N]
    with forced_plan(plan):
        op = pkg.GroupedGemm.like(A, B, off, None, D)
    op.run(A, B, off, None, D)
    done(op)
    ref, S = grouped_ref(torch.nan_to_num(A), torch.nan_to_num(B), off, None, grad)
    assert bool((whole[..., N:] == 7).all())
    if grad:
        assert bool(torch.isnan(D[1]).all())
        keep = [0, 2, 3]
        near(D[keep], ref[keep], S[keep], max(counts))
    else:
        assert bool((D[:first] == 7).all()) and bool((D[R - tail:] == 7).all())
        assert bool(torch.isnan(D[bad]).all())
        rows = torch.arange(R, device="cuda")
        keep = (rows >= first) & (rows < R - tail) & ((rows < bad.start) | (rows >= bad.stop))
        near(D[keep], ref[keep], S[keep], K)


def test_grouped_k_zero_and_c_in_place():
    off = offsets_of([2, 0, 3])
    A, B = torch.zeros(5, 0, dtype=BF16, device="cuda"), torch.zeros(3, 0, 16, dtype=BF16,
                                                                     device="cuda")
    C = rnd((5, 16), F32, 1)
    D = C.clone()
    op = pkg.GroupedGemm.like(A, B, off, D, D)
    op.run(A, B, off, D, D)
    done(op)
    assert torch.equal(D, C)
    # accumulation over two calls, D read as C
    A, B = rnd((5, 24), BF16, 2), rnd((5, 40), BF16, 3)
    D = torch.zeros((3, 24, 40), device="cuda")
    op = pkg.GroupedGemm.like(A, B, off, D, D)
    op.run(A, B, off, D, D)
    op.run(A, B, off, D, D)
    done(op)
    ref, S = grouped_ref(A, B, off, None, True)
    near(D, 2 * ref, 2 * S, 8)


@pytest.mark.parametrize("plan", ["wide=0", "wide=1"])
@pytest.mark.parametrize("grad", [False, True])
def test_grouped_long_sums_are_shared_between_units(plan, grad):
    """Fewer tiles than units and a long sum: its pieces are added in one
    order, whoever is last, so every call gives the same bits."""
    counts = [3000, 0, 1111] if grad else [70, 0, 300]
    R, K, N = sum(counts), (96 if grad else 5000), 200
    off = offsets_of(counts)
    A = rnd((R, K), BF16, 1)
    B = rnd((R, N) if grad else (3, K, N), BF16, 2)
    D = torch.zeros((3, K, N) if grad else (R, N), device="cuda")
    with forced_plan(plan):
        op = pkg.GroupedGemm.like(A, B, off, None, D)
    op.run(A, B, off, None, D)
    ref, S = grouped_ref(A, B, off, None, grad)
    near(D, ref, S, max(counts) if grad else K)
    first = D.clone()
    for _ in range(5):
        op.run(A, B, off, None, D)
        assert torch.equal(D, first)
    done(op)


def test_grouped_long_groups_and_many_experts():
    """Every tile count: 1024 experts with 0 to 3 rows, and one long group."""
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 4, (1024,), generator=g).tolist()
    counts[700] = 2100
    off = offsets_of(counts)
    A, B = rnd((sum(counts), 72), BF16, 1), rnd((1024, 136, 72), BF16, 2).transpose(1, 2)
    D = torch.empty((sum(counts), 136), dtype=BF16, device="cuda")
    op = pkg.GroupedGemm.like(A, B, off, None, D)
    op.run(A, B, off, None, D)
    done(op)
    ref, S = grouped_ref(A, B, off, None, False)
    near(D, ref, S, 72)


def test_grouped_offsets_change_between_calls_on_another_stream():
    A, B = rnd((400, 128), BF16, 1), rnd((6, 128, 192), BF16, 2)
    D = torch.zeros((400, 192), dtype=BF16, device="cuda")
    off = offsets_of([0] * 6)
    op = pkg.GroupedGemm.like(A, B, off, None, D)
    side = torch.cuda.Stream()
    for counts in ([400, 0, 0, 0, 0, 0], [1, 99, 100, 0, 150, 50], [0, 0, 0, 0, 0, 3]):
        torch.cuda.synchronize()
        D.fill_(0)
        torch.cuda.current_stream().synchronize()
        with torch.cuda.stream(side):
            # the offsets come from work on the same stream
            off.copy_(offsets_of(counts))
            op.run(A, B, off, None, D)
        assert op.status(side) == pkg.GEMM_OK
        ref, S = grouped_ref(A, B, off, None, False)
        near(D, ref, S, 128)
    op.close()


def test_grouped_reports_bad_offsets_and_stays_usable():
    A, B = rnd((64, 64), BF16, 1), rnd((3, 64, 64), BF16, 2)
    D = torch.zeros((64, 64), dtype=BF16, device="cuda")
    good = offsets_of([10, 20, 34])
    op = pkg.GroupedGemm.like(A, B, good, None, D)
    for bad in ([0, 40, 20, 64], [0, 10, 20, 65], [-1, 10, 20, 64]):
        op.run(A, B, torch.tensor(bad, dtype=torch.int32, device="cuda"), None, D)
        assert op.status() == pkg.GEMM_ERR_INVALID_ARG
    op.run(A, B, good, None, D)
    done(op)
    ref, S = grouped_ref(A, B, good, None, False)
    near(D, ref, S, 64)


def test_grouped_bounded_wait_reports_timeout_and_stays_usable():
    A, B = rnd((300, 256), BF16, 1), rnd((2, 256, 256), BF16, 2)
    D = torch.zeros((300, 256), dtype=BF16, device="cuda")
    off = offsets_of([100, 200])
    op = pkg.GroupedGemm.like(A, B, off, None, D)
    op.debug_set(pkg.GEMM_DEBUG_SKIP_FIRST_FILL, 50_000_000)
    op.run(A, B, off, None, D)
    assert op.status() == pkg.GEMM_ERR_DEVICE_TIMEOUT
    op.debug_set(0)
    op.run(A, B, off, None, D)
    done(op)
    ref, S = grouped_ref(A, B, off, None, False)
    near(D, ref, S, 256)


def test_grouped_refuses_misaligned_bases_and_other_tensors():
    buf = torch.zeros(64 * 64 + 8, dtype=BF16, device="cuda")
    A, B = buf[1:1 + 64 * 64].view(64, 64), rnd((2, 64, 64), BF16, 2)
    D = torch.zeros((64, 64), dtype=BF16, device="cuda")
    off = offsets_of([32, 32])
    op = pkg.GroupedGemm.like(A, B, off, None, D)
    with pytest.raises(pkg.GemmError) as e:
        op.run(A, B, off, None, D)
    assert e.value.code == pkg.GEMM_ERR_MISALIGNED
    with pytest.raises(ValueError, match="D: planned"):
        op.run(A, B, off, None, torch.zeros((64, 65), dtype=BF16, device="cuda"))
    with pytest.raises(ValueError, match="without C"):
        op.run(A, B, off, D, D)
    op.close()


def test_grouped_gradients_agree_with_differences():
    """dA and dB of L = <G, A B_e> from the operator, against centred
    differences of L computed from the operator's own fp32 products: L is
    bilinear, so a difference is exact but for rounding."""
    counts = [5, 0, 11]
    off, R, K, N = offsets_of(counts), 16, 24, 32
    A, B, G = rnd((R, K), BF16, 1), rnd((3, K, N), BF16, 2), rnd((R, N), BF16, 3)
    dA = pkg.grouped_matmul(G, B.transpose(1, 2), off, out_dtype=F32)
    dB = torch.empty((3, K, N), device="cuda")
    pkg.grouped_matmul(A, G, off, D=dB)

    def loss(a, b):
        return float((pkg.grouped_matmul(a, b, off, out_dtype=F32).double() * G.double()).sum())

    base = 2.0 ** -16 * float((A.double().abs().sum() * B.double().abs().max() *
                               G.double().abs().max()))
    for r, k in ((0, 0), (4, 23), (15, 7)):
        hi, lo = A.clone(), A.clone()
        hi[r, k] = A[r, k] + 1
        lo[r, k] = A[r, k] - 1
        step = float(hi[r, k].double() - lo[r, k].double())
        assert abs((loss(hi, B) - loss(lo, B)) / step - float(dA[r, k])) <= base
    for e, k, n in ((0, 3, 5), (1, 0, 0), (2, 23, 31)):
        hi, lo = B.clone(), B.clone()
        hi[e, k, n] = B[e, k, n] + 1
        lo[e, k, n] = B[e, k, n] - 1
        step = float(hi[e, k, n].double() - lo[e, k, n].double())
        assert abs((loss(A, hi) - loss(A, lo)) / step - float(dB[e, k, n])) <= base


# ---------------------------------------------------------------- 4-bit weights
def w4_ref(X, q, scales, zeros, off, group):
    E, N, K = q.shape
    off = [0, X.shape[0]] if off is None else off.tolist()
    where = torch.arange(K, device="cuda") // group
    D = torch.zeros((X.shape[0], N), dtype=torch.float64, device="cuda")
    S = torch.zeros_like(D)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        z = 8.0 if zeros is None else zeros[e].double()[:, where]
        w = (q[e].double() - z) * scales[e].double()[:, where]
        D[r], S[r] = X[r].double() @ w.t(), X[r].double().abs() @ w.abs().t()
    return D, S


@pytest.mark.parametrize("R", [1, 3, 8, 9, 16, 17, 32, 45])
@pytest.mark.parametrize("K,N,group,dtype,scale,out,zeros", [
    (128, 64, 128, BF16, BF16, BF16, False),
    (4096, 48, 128, F16, F16, F16, True),
    (160, 33, 32, BF16, F32, F32, True),     # N ends inside a tile
    (1056, 17, 64, F16, F16, F32, False),    # the last group is half one
    (288, 1, 256, BF16, BF16, F16, True),
    (32, 130, 32, F16, F32, BF16, False),
    (96, 40, 128, BF16, BF16, BF16, True),   # less than one group
])
def test_w4_dense(R, K, N, group, dtype, scale, out, zeros):
    G = -(-K // group)
    g = torch.Generator().manual_seed(R + K)
    q = torch.randint(0, 16, (1, N, K), generator=g).cuda()
    W, X = pkg.pack_w4(q), rnd((R, K), dtype, 1)
    s = (rnd((1, N, G), F32, 2).abs() * 0.1 + 0.01).to(scale)
    z = torch.randint(0, 16, (1, N, G), generator=g).to(torch.uint8).cuda() if zeros else None
    D = torch.full((R, N), 7.0, dtype=out, device="cuda")
    op = pkg.W4Gemm.like(X, W, s, z, None, D, group)
    op.run(X, W, s, z, None, D)
    done(op)
    ref, S = w4_ref(X, q, s, z, None, group)
    near(D, ref, S, K + 1)


def test_w4_gives_the_same_bits_every_time():
    R, K, N, group = 5, 16384, 300, 64
    q = torch.randint(0, 16, (1, N, K), generator=torch.Generator().manual_seed(2)).cuda()
    W, X = pkg.pack_w4(q), rnd((R, K), BF16, 1)
    s = (rnd((1, N, K // group), F32, 2).abs() * 0.1 + 0.01).to(BF16)
    D = torch.zeros((R, N), device="cuda")
    op = pkg.W4Gemm.like(X, W, s, None, None, D, group)
    op.run(X, W, s, None, None, D)
    ref, S = w4_ref(X, q, s, None, None, group)
    near(D, ref, S, K + 1)
    first = D.clone()
    for _ in range(5):
        op.run(X, W, s, None, None, D)
        assert torch.equal(D, first)
    done(op)


@pytest.mark.parametrize("counts", [[0, 1, 0, 2, 0, 0, 9], [1], [3, 0, 40, 17, 0, 1], [0, 0, 0]])
@pytest.mark.parametrize("K,N,group,zeros", [(256, 72, 64, True), (512, 33, 128, False),
                                             (544, 130, 32, True)])
def test_w4_experts(counts, K, N, group, zeros):
    E, first, tail, G = len(counts), 2, 3, -(-K // group)
    R, off = first + sum(counts) + tail, offsets_of(counts, first)
    g = torch.Generator().manual_seed(K)
    q = torch.randint(0, 16, (E, N, K), generator=g).cuda()
    W, X = pkg.pack_w4(q), rnd((R, K + 8), BF16, 1)[:, :K]
    X[:first] = float("nan")
    X[first + sum(counts):] = float("nan")
    s = (rnd((E, N, G), F32, 2).abs() * 0.1 + 0.01).to(BF16)
    z = torch.randint(0, 16, (E, N, G), generator=g).to(torch.uint8).cuda() if zeros else None
    whole = torch.full((R, N + 3), 7.0, dtype=BF16, device="cuda")
    D = whole[:, :N]
    op = pkg.W4Gemm.like(X, W, s, z, off, D, group)
    op.run(X, W, s, z, off, D)
    done(op)
    live = slice(first, first + sum(counts))
    ref, S = w4_ref(torch.nan_to_num(X), q, s, z, off, group)
    near(D[live], ref[live], S[live], K + 1)
    assert bool((D[:first] == 7).all()) and bool((D[live.stop:] == 7).all())
    assert bool((whole[:, N:] == 7).all())


def test_w4_specials_and_bad_offsets():
    """An infinite activation gives infinities (or NaN where q is the zero
    point), a NaN only its own row; offsets out of range set the status."""
    K, N = 128, 16
    q = torch.randint(0, 16, (1, N, K), generator=torch.Generator().manual_seed(1)).cuda()
    W, s = pkg.pack_w4(q), torch.ones((1, N, 1), dtype=BF16, device="cuda")
    X = rnd((3, K), BF16, 1)
    X[0, 5], X[1, 7] = float("inf"), float("nan")
    inf = float("inf")
    want = torch.where(q[0, :, 5] == 8, float("nan"), torch.where(q[0, :, 5] > 8, inf, -inf))
    D = pkg.w4_matmul(X, W, s)
    assert torch.equal(torch.nan_to_num(D[0].double(), nan=3.0),
                       torch.nan_to_num(want.double(), nan=3.0))
    assert bool(torch.isnan(D[1]).all()) and bool(torch.isfinite(D[2]).all())
    off = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    op = pkg.W4Gemm.like(X, W, s, None, off, D, 128)
    op.run(X, W, s, None, off, D)
    done(op, pkg.GEMM_ERR_INVALID_ARG)


# ---------------------------------------------------------------- routing
def route_ref(x, k, normalize):
    """The formula in fp64 on the host."""
    T, E = x.shape
    v = x.double().cpu()
    key = torch.where(torch.isnan(v), float("inf"), v)
    # NaN above +inf: sort by (is NaN, value) with stable falling sorts
    order = key.argsort(dim=1, descending=True, stable=True)
    nan = torch.isnan(v).gather(1, order).to(torch.int8).argsort(dim=1, descending=True, stable=True)
    order = order.gather(1, nan)[:, :k]
    val = v.gather(1, order)
    none = val == float("-inf")
    top = torch.where(none[:, :1], 0.0, val[:, :1])
    ex = torch.where(none, 0.0, torch.exp(val - top))
    total = ex.sum(1, keepdim=True) if normalize else torch.exp(v - top).sum(1, keepdim=True)
    gates = torch.where(none, 0.0, ex / total)
    experts = torch.where(none, -1, order)
    flat = experts.reshape(-1)
    rows = torch.where(flat < 0, E, flat).argsort(stable=True)
    n = int((flat >= 0).sum())
    offsets = torch.cat([torch.zeros(1, dtype=torch.long),
                         torch.bincount(flat[flat >= 0], minlength=E).cumsum(0)])
    slot_row = torch.full((T * k,), -1)
    slot_row[rows[:n]] = torch.arange(n)
    row_slot = rows.clone()
    row_slot[n:] = -1
    return experts, gates, offsets, row_slot, slot_row.view(T, k)


def check_route(x, k, normalize):
    op = pkg.Route.like(x, k, normalize)
    outs = op.outputs()
    for o in outs:
        o.fill_(77)
    op.run(x, *outs)
    assert op.status() == pkg.GEMM_OK
    ref = route_ref(x, k, normalize)
    for i, name in ((0, "experts"), (2, "offsets"), (3, "row_slot"), (4, "slot_row")):
        assert torch.equal(outs[i].cpu().long(), ref[i]), name
    n = x.shape[1] + 8
    near(outs[1], ref[1].cuda(), ref[1].cuda(), n, "gates")
    return op, outs, ref


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (7, 33, 5), (64, 128, 8), (64, 1024, 32),
                                   (65, 64, 2), (500, 96, 4), (3000, 256, 8), (1111, 513, 3),
                                   (40000, 16, 1)])
@pytest.mark.parametrize("dtype,normalize", [(F32, True), (BF16, False), (F16, True)])
def test_route(T, E, k, dtype, normalize):
    # 16-bit logits tie often; a tenth of them are masked, and some rows wholly
    x = rnd((T, E), dtype, T + E, 2.0)
    g = torch.Generator().manual_seed(T)
    x[(torch.rand((T, E), generator=g) < 0.1).cuda()] = float("-inf")
    x[(torch.rand(T, generator=g) < 0.05).cuda()] = float("-inf")
    op, outs, ref = check_route(x, k, normalize)
    again = op.outputs()
    op.run(x, *again)
    for a, b in zip(outs, again):
        assert torch.equal(a, b)
    done(op)


def test_route_ties_specials_and_strides():
    ninf, inf, nan = float("-inf"), float("inf"), float("nan")
    lowest = torch.finfo(F32).min
    rows = torch.tensor([
        [0.0, -0.0, 0.0, -0.0, 0.0, 0.0],       # all equal: 0, 1, 2
        [ninf] * 6,                              # nothing to choose
        [ninf, 1.0, ninf, ninf, ninf, ninf],     # one choice
        [lowest, lowest, ninf, lowest, 0, 0],    # a mask of the lowest value is chosen last
        [1.0, nan, 2.0, nan, 3.0, 0.0],          # NaN first; its gates are NaN
        [lowest] * 6,
    ])
    wide = torch.full((6, 9), 50.0)
    wide[:, :6] = rows
    for normalize in (True, False):
        op, outs, _ = check_route(wide.cuda()[:, :6], 3, normalize)
        assert outs[0][0].tolist() == [0, 1, 2] and outs[0][4].tolist() == [1, 3, 4]
        assert outs[0][1].tolist() == [-1, -1, -1] and float(outs[1][1].sum()) == 0
        op.close()
    x = rows.cuda()
    x[0, 3] = inf
    op = pkg.Route.like(x, 2)
    outs = op.outputs()
    op.run(x, *outs)
    done(op)
    assert outs[0][0].tolist() == [3, 0]  # an infinite logit comes first


def test_route_no_tokens():
    x = torch.zeros((0, 8), device="cuda")
    op = pkg.Route.like(x, 2)
    outs = op.outputs()
    outs[2].fill_(5)
    op.run(x, *outs)
    done(op)
    assert outs[2].tolist() == [0] * 9


@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (50, 40, 8), (300, 700, 5)])
@pytest.mark.parametrize("dtype,normalize", [(F32, True), (F32, False), (BF16, False), (F16, True)])
def test_route_backward(T, E, k, dtype, normalize):
    x = rnd((T, E), dtype, 3, 2.0)
    x[0, E // 2:] = float("-inf")
    op, outs, _ = check_route(x, k, normalize)
    dg = rnd((T, k), F32, 4)
    dx = torch.full_like(x, 7.0)
    op.backward(x, outs[0], outs[1], dg, dx)
    done(op)
    experts = outs[0].long().cpu()
    v = x.double().cpu()
    p = torch.softmax(v, 1)
    chosen = torch.zeros_like(p).scatter_(1, experts.clamp_min(0), (experts >= 0).double())
    if normalize:
        p = p * chosen / (p * chosen).sum(1, keepdim=True)
    d = torch.zeros_like(p).scatter_add_(1, experts.clamp_min(0),
                                         torch.where(experts >= 0, dg.double().cpu(), 0.0))
    s = (p * d).sum(1, keepdim=True)
    ref = (p * (d - s)).cuda()
    # p is within n units, s within n + k more of its magnitudes
    size = (p * (d.abs() + (p * d.abs()).sum(1, keepdim=True))).cuda()
    near(dx, ref, size, 2 * E + 32)


def test_route_backward_agrees_with_differences():
    """Centred differences, in fp64, of L = sum(gates * dg)."""
    x, k, h = rnd((3, 12), F32, 9), 4, 1e-5
    dg = rnd((3, k), F32, 10)
    for normalize in (True, False):
        op, outs, ref = check_route(x, k, normalize)
        dx = torch.empty_like(x)
        op.backward(x, outs[0], outs[1], dg, dx)
        done(op)
        w = dg.double().cpu()
        for t, e in ((0, int(outs[0][0, 0])), (1, int(outs[0][1, 3])), (2, 5)):
            side = []
            for d in (h, -h):
                y = x.double().cpu().clone()
                y[t, e] += d
                side.append(float((route_ref(y, k, normalize)[1] * w).sum()))
            assert abs((side[0] - side[1]) / (2 * h) - float(dx[t, e])) < 1e-5


# ---------------------------------------------------------------- row movement
def routing(T, k, E, drop, seed):
    g = torch.Generator().manual_seed(seed)
    experts = torch.rand((T, E), generator=g).argsort(1)[:, :k].reshape(-1)
    experts[torch.rand(T * k, generator=g) < drop] = E
    order = experts.argsort(stable=True)
    n = int((experts < E).sum())
    slot_row = torch.full((T * k,), -1)
    slot_row[order[:n]] = torch.arange(n)
    order[n:] = -1
    return order.to(torch.int32).cuda(), slot_row.to(torch.int32).view(T, k).cuda()


@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (5, 2, 64), (33, 8, 4096), (100, 3, 77), (17, 10, 2056),
                                   (9, 32, 136), (700, 4, 264)])
@pytest.mark.parametrize("dtype,drop", [(BF16, 0.0), (F16, 0.3), (F32, 0.1), (BF16, 1.0)])
def test_permute(T, k, H, dtype, drop):
    row_slot, slot_row = routing(T, k, max(k, 8), drop, T)
    nan = float("nan")
    pad = torch.full((T, H + 8), nan, dtype=dtype, device="cuda")
    pad[:, :H] = rnd((T, H), dtype, 1)
    X = pad[:, :H]
    Ys, gates = rnd((T * k, H), dtype, 2), rnd((T, k), F32, 3)
    live = row_slot.long() >= 0
    Ys[~live] = nan        # rows of no slot are not read
    gates[slot_row < 0] = nan
    Xs, Y = torch.full_like(Ys, 7.0), torch.full((T, H + 8), 7.0, dtype=dtype, device="cuda")
    op = pkg.Permute.like(X, slot_row)
    op.gather(X, row_slot, slot_row, Xs)
    want = torch.where(live[:, None], X[row_slot.long().clamp_min(0) // k], 0.0)
    assert torch.equal(Xs, want.to(dtype))
    op.combine(Ys, slot_row, gates, Y[:, :H])
    routed = (slot_row >= 0)[:, :, None]
    rows = torch.where(routed, Ys[slot_row.long().clamp_min(0)].double(), 0.0)
    g = torch.where(slot_row >= 0, gates, 0.0).double()[:, :, None]
    near(Y[:, :H], (g * rows).sum(1), (g * rows).abs().sum(1), k + 1)
    assert bool((Y[:, H:] == 7).all())
    dYs, dgates = torch.full_like(Ys, 7.0), torch.full_like(gates, 7.0)
    dY = X
    op.combine_backward(dY, Ys, row_slot, slot_row, gates, dYs, dgates)
    prod = dY.double()[:, None, :] * rows
    near(dgates, prod.sum(2), prod.abs().sum(2), H + 1)
    token = row_slot.long().clamp_min(0) // k
    flat = g.reshape(-1)[row_slot.long().clamp_min(0)][:, None]
    want = torch.where(live[:, None], flat * dY.double()[token], 0.0)
    near(dYs, want, want.abs(), 2)
    op.combine(Ys, slot_row, None, Y[:, :H])
    near(Y[:, :H], rows.sum(1), rows.abs().sum(1), k)
    done(op)


def test_permute_reports_bad_rows():
    row_slot, slot_row = routing(4, 2, 8, 0.0, 1)
    X = rnd((4, 64), BF16, 1)
    Xs = torch.zeros((8, 64), dtype=BF16, device="cuda")
    op = pkg.Permute.like(X, slot_row)
    bad = slot_row.clone()
    bad[1, 1] = 8
    op.gather(X, row_slot, bad, Xs)
    assert op.status() == pkg.GEMM_ERR_INVALID_ARG
    op.gather(X, row_slot, slot_row, Xs)
    done(op)


# ---------------------------------------------------------------- together
def test_expert_layer_matches_the_dense_formula():
    """Route, gather, grouped product, combine: the same as every expert's
    product of every token, weighted by its gate."""
    T, E, k, H, N = 90, 12, 3, 128, 72
    x, W = rnd((T, H), BF16, 1), rnd((E, H, N), BF16, 2, H ** -0.5)
    logits = rnd((T, E), F32, 3)
    route = pkg.Route.like(logits, k)
    experts, gates, offsets, row_slot, slot_row = route.outputs()
    route.run(logits, experts, gates, offsets, row_slot, slot_row)
    perm = pkg.Permute.like(x, slot_row)
    xs = torch.empty((T * k, H), dtype=BF16, device="cuda")
    perm.gather(x, row_slot, slot_row, xs)
    ys = pkg.grouped_matmul(xs, W, offsets)
    out = pkg.Permute.like(torch.empty((T, N), dtype=BF16, device="cuda"), slot_row)
    y = torch.empty((T, N), dtype=BF16, device="cuda")
    out.combine(ys, slot_row, gates, y)
    every = torch.einsum("th,ehn->ten", x.double(), W.double())
    g = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    g.scatter_(1, experts.long(), gates.double())
    ref = (g[:, :, None] * every).sum(1)
    mag = (g[:, :, None] * torch.einsum("th,ehn->ten", x.double().abs(), W.double().abs())).sum(1)
    # ys is rounded once more, to bf16: half an ulp of each product
    off = (y.double() - ref).abs()
    assert bool((off <= 2.0 ** -8 * (ref.abs() + (g[:, :, None] * every).abs().sum(1) + 1e-30)
                 + 2.0 ** -14 * mag).all())
    for op in (route, perm, out):
        done(op)


def test_route_nan_of_either_sign_comes_first():
    x = torch.zeros((3, 40))
    x[0, 7], x[0, 31] = float("nan"), float("inf")
    x[1, 39] = torch.tensor(-0x400000, dtype=torch.int32).view(F32)  # NaN with its sign bit set
    x[1, 2] = 3.0
    x[2] = float("nan")
    for dtype in (F32, F16, BF16):
        op = pkg.Route.like(x.to(dtype).cuda(), 2)
        outs = op.outputs()
        op.run(x.to(dtype).cuda(), *outs)
        done(op)
        assert outs[0].tolist() == [[7, 31], [39, 2], [0, 1]]
        assert bool(torch.isnan(outs[1][2]).all())
