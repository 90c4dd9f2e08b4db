"""Calls of the expert and 4-bit-weight operators at the edges of their
protocols: staging buffers under many ragged tiles, streams, timeouts, and
values that must not be looked at.  Bounds as in test_gpu_experts."""
from __future__ import annotations

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg
from gpu_helpers import forced_plan
from test_gpu_experts import BF16, F16, done, grouped_ref, near, offsets_of, rnd, w4_ref

pytestmark = pytest.mark.gpu


def ragged_counts(E, low, high, seed):
    """Group sizes of which few are a multiple of 32."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, high, (E,), generator=g).tolist()


# ---------------------------------------------------------------- grouped products
@pytest.mark.parametrize("K,N,dtype,order", [(8, 520, BF16, "nk"), (64, 1032, F16, "kn"),
                                             (200, 768, BF16, "nk")])
def test_grouped_ragged_tiles_share_staging_buffers(K, N, dtype, order):
    """Short sums, many tiles a CTA pair, and groups that end inside a box of
    32 rows: boxes stored by TMA and boxes stored by the threads take turns in
    the staging buffers, and a buffer is not written before its store has read
    it."""
    counts = ragged_counts(120, 200, 300, K) + [1, 31, 33, 0, 257, 289, 513]
    E, R = len(counts), sum(counts)
    off = offsets_of(counts)
    A = rnd((R, K), dtype, 1)
    B = rnd((E, N, K) if order == "nk" else (E, K, N), dtype, 2)
    B = B.transpose(1, 2) if order == "nk" else B
    D = torch.full((R, N), 7.0, dtype=dtype, device="cuda")
    with forced_plan("wide=1"):
        op = pkg.GroupedGemm.like(A, B, off, None, D)
    assert "wide=1" in op.plan()
    ref, S = grouped_ref(A, B, off, None, False)
    first = None
    for _ in range(20):
        D.fill_(7.0)
        op.run(A, B, off, None, D)
        if first is None:
            first = D.clone()
            near(D, ref, S, K)
        assert torch.equal(D, first)
    done(op)


# ---------------------------------------------------------------- streams
def busy(milliseconds=30):
    """Work on the current stream that takes about that long."""
    torch.cuda._sleep(int(milliseconds * 2e6))


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("K,N", [(61, 1000), (5000, 264)])  # copied rows; sums shared by units
def test_grouped_first_run_on_a_side_stream(K, N, grad):
    """A handle made while the default stream is busy is ready for a stream
    that does not wait for it."""
    counts = [70, 0, 300]
    off, R = offsets_of(counts), sum(counts)
    A = rnd((R, K), BF16, 1)
    B = rnd((R, N) if grad else (3, K, N), BF16, 2)
    D = torch.zeros((3, K, N) if grad else (R, N), device="cuda")
    ref, S = grouped_ref(A, B, off, None, grad)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    op = pkg.GroupedGemm.like(A, B, off, None, D)
    op.run(A, B, off, None, D, stream=side)
    assert op.status(side) == pkg.GEMM_OK
    side.synchronize()
    with torch.cuda.stream(side):
        got = D.clone()
    torch.cuda.synchronize()
    near(got, ref, S, max(counts) if grad else K)
    op.run(A, B, off, None, D, stream=side)  # nothing was cleared late
    torch.cuda.synchronize()
    assert torch.equal(D, got)
    done(op)


def test_route_first_run_on_a_side_stream():
    x = rnd((5000, 90), torch.float32, 1)
    op = pkg.Route.like(x, 3)
    want = op.outputs()
    op.run(x, *want)
    done(op)
    outs = tuple(torch.empty_like(o) for o in want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    op = pkg.Route.like(x, 3)
    op.run(x, *outs, stream=side)
    assert op.status(side) == pkg.GEMM_OK
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    op.close()


@pytest.mark.parametrize("raw", [False, True])
def test_new_results_on_a_given_stream(raw):
    """grouped_matmul and w4_matmul with `stream`: the zeros of a new result
    do not arrive after the product."""
    off = offsets_of([30, 0, 50], first=2)
    A, B = rnd((90, 128), BF16, 1), rnd((3, 128, 72), BF16, 2)
    ref, S = grouped_ref(A, B, off, None, False)
    q = torch.randint(0, 16, (3, 72, 128), generator=torch.Generator().manual_seed(3)).cuda()
    W, s = pkg.pack_w4(q), rnd((3, 72, 1), BF16, 4)
    wref, wS = w4_ref(A, q, s, None, off, 128)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    torch.cuda.synchronize()
    busy()
    D = pkg.grouped_matmul(A, B, off, stream=stream)
    torch.cuda.synchronize()
    near(D, ref, S, 128)
    busy()
    D = pkg.w4_matmul(A, W, s, None, off, 128, stream=stream)
    torch.cuda.synchronize()
    near(D, wref, wS, 129)
    assert bool((D[:2] == 0).all()) and bool((D[82:] == 0).all())


# ---------------------------------------------------------------- timeouts
@pytest.mark.parametrize("plan", ["wide=0", "wide=1"])
@pytest.mark.parametrize("grad", [False, True])
def test_grouped_shared_sums_after_a_timeout(plan, grad):
    """One unit gives up a wait while the others finish their pieces of the
    tiles they share with it: once that is reported, the next calls are right."""
    counts = [3000, 0, 1111] if grad else [70, 0, 300]
    R, K, N = sum(counts), (96 if grad else 5000), 200
    off = offsets_of(counts)
    A = rnd((R, K), BF16, 1)
    B = rnd((R, N) if grad else (3, K, N), BF16, 2)
    D = torch.zeros((3, K, N) if grad else (R, N), device="cuda")
    ref, S = grouped_ref(A, B, off, None, grad)
    with forced_plan(plan):
        op = pkg.GroupedGemm.like(A, B, off, None, D)
    for _ in range(3):
        op.debug_set(pkg.GEMM_DEBUG_SKIP_ONE_FILL, 20_000_000)
        op.run(A, B, off, None, D)
        assert op.status() == pkg.GEMM_ERR_DEVICE_TIMEOUT
        op.debug_set(0)
        for _ in range(3):
            D.fill_(7.0)
            op.run(A, B, off, None, D)
            assert op.status() == pkg.GEMM_OK
            near(D, ref, S, max(counts) if grad else K)
    op.close()


@pytest.mark.parametrize("plan", ["wide=0", "wide=1"])
@pytest.mark.parametrize("flag", [pkg.GEMM_DEBUG_SKIP_FIRST_FILL, pkg.GEMM_DEBUG_SKIP_ONE_FILL])
@pytest.mark.parametrize("out", [BF16, torch.float32])
def test_grouped_timeout_among_empty_groups(plan, flag, out):
    """Empty groups need no wait, so pieces of them are still handed out when a
    wait has run out: every warp of the kernel ends all the same."""
    counts = ([40] + [0] * 9 + [70] + [0] * 3) * 6
    E, R, K, N = len(counts), sum(counts), 136, 264
    off = offsets_of(counts)
    A, B = rnd((R, K), BF16, 1), rnd((R, N), BF16, 2)
    D = torch.zeros((E, K, N), dtype=out, device="cuda")
    ref, S = grouped_ref(A, B, off, None, True)
    with forced_plan(plan):
        op = pkg.GroupedGemm.like(A, B, off, None, D)
    for timeout_ns in (1_000_000, 3_000_000, 10_000_000):
        op.debug_set(flag, timeout_ns)
        op.run(A, B, off, None, D)
        assert op.status() == pkg.GEMM_ERR_DEVICE_TIMEOUT
        op.debug_set(0)
        D.fill_(7.0)
        op.run(A, B, off, None, D)
        assert op.status() == pkg.GEMM_OK
        near(D, ref, S, max(counts))
    op.close()


# ---------------------------------------------------------------- row movement
@pytest.mark.parametrize("H", [64, 77])
@pytest.mark.parametrize("bad", [12, 1000, -2, -2 ** 31])
def test_permute_rows_with_a_bad_slot_are_zeros(H, bad):
    """row_slot outside [-1, T * k) counts as -1 and sets the status, in the
    gather and in the gated sum's gradient."""
    T, k = 4, 3
    row_slot = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0)
    slot_row = row_slot.clone().view(T, k)  # its own inverse
    row = 7
    slot_row.view(-1)[int(row_slot[row])] = -1
    row_slot[row] = bad
    X, Ys, gates = rnd((T, H), BF16, 1), rnd((T * k, H), BF16, 2), rnd((T, k), torch.float32, 3)
    out, dgates = torch.full_like(Ys, 7.0), torch.empty_like(gates)
    op = pkg.Permute.like(X, slot_row)
    op.gather(X, row_slot, slot_row, out)
    assert op.status() == pkg.GEMM_ERR_INVALID_ARG
    live = torch.arange(T * k, device="cuda") != row
    token = row_slot.long().clamp(0, T * k - 1) // k
    assert bool((out[row] == 0).all()) and torch.equal(out[live], X[token[live]])
    out.fill_(7.0)
    op.combine_backward(X, Ys, row_slot, slot_row, gates, out, dgates)
    assert op.status() == pkg.GEMM_ERR_INVALID_ARG
    assert bool((out[row] == 0).all()) and not bool((out[live] == 7).all())
    row_slot[row] = -1
    op.gather(X, row_slot, slot_row, out)
    op.combine_backward(X, Ys, row_slot, slot_row, gates, out, dgates)
    done(op)


# ---------------------------------------------------------------- 4-bit weights
@pytest.mark.parametrize("R", [1, 12, 32])
@pytest.mark.parametrize("K,group", [(32, 32), (64, 64), (96, 32), (128, 128), (320, 64),
                                     (384, 128), (160, 128)])
def test_w4_infinite_scale_of_the_last_group(K, group, R):
    """The last group's scale is applied to its sum alone: an infinite one
    gives infinities (its sum is not zero), and nothing past K turns them into
    NaN."""
    N, G = 40, -(-K // group)
    q = torch.full((1, N, K), 12).cuda()
    W, s = pkg.pack_w4(q), torch.ones((1, N, G), dtype=F16, device="cuda")
    s[0, ::2, -1] = float("inf")
    X = rnd((R, K), F16, 1).abs() + 0.5
    D = pkg.w4_matmul(X, W, s, group=group, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert bool((D[:, ::2] == float("inf")).all())
    near(D[:, 1::2], 4 * X.double().sum(1, keepdim=True).expand(R, N // 2),
         4 * X.double().sum(1, keepdim=True).expand(R, N // 2), K + 1)


@pytest.mark.parametrize("plan", ["wide=0", "wide=1"])
@pytest.mark.parametrize("K,ld,order", [(24, 32, "nk"), (25, 25, "nk"), (24, 1, "kn"), (24, 8, "kn")])
def test_grouped_single_column(plan, K, ld, order):
    counts = [5, 0, 70]
    off, E, R = offsets_of(counts), 3, 75
    A = rnd((R, K), BF16, 1)
    B = (rnd((E, 1, ld), BF16, 2)[:, :, :K].transpose(1, 2) if order == "nk" else
         rnd((E, K, ld), BF16, 2)[:, :, :1])
    D = torch.full((R, 1), 7.0, device="cuda")
    with forced_plan(plan):
        op = pkg.GroupedGemm.like(A, B, off, None, D)
    op.run(A, B, off, None, D)
    done(op)
    ref, S = grouped_ref(A, B, off, None, False)
    near(D, ref, S, K)


# ---------------------------------------------------------------- handles
def test_plan_strings_are_whole():
    logits = torch.zeros((100_000, 1024), dtype=BF16, device="cuda")
    slot_row = torch.zeros((100_000, 32), dtype=torch.int32, device="cuda")
    X = torch.zeros((100_000, 8), dtype=BF16, device="cuda")
    off = offsets_of([0] * 1024)
    A, B = X[:, :8], torch.zeros((1024, 8, 16), dtype=BF16, device="cuda")
    D = torch.zeros((100_000, 16), dtype=BF16, device="cuda")
    W = torch.zeros((1024, 16, 16), dtype=torch.uint8, device="cuda")
    s = torch.zeros((1024, 16, 1), dtype=BF16, device="cuda")
    for op, want in (
            (pkg.Route.like(logits, 32), "route T=100000 E=1024 k=32 blocks="),
            (pkg.Permute.like(X, slot_row), "permute T=100000 k=32 H=8"),
            (pkg.GroupedGemm.like(A, B, off, None, D), "grouped form=rows E=1024 R=100000 K=8 N=16 "),
            (pkg.W4Gemm.like(torch.zeros((100_000, 32), dtype=BF16, device="cuda"), W, s, None, off,
                             D, 32), "w4 E=1024 R=100000 K=32 N=16 group=32 zeros=0")):
        assert op.plan().startswith(want), op.plan()
        assert pkg.load().gemm_op_plan_string(op.handle, None, 0) == len(op.plan())
        done(op)
