"""Handles made while the default stream is busy, run at once on a stream that
does not wait for it.  Bounds as in test_gpu_experts."""
from __future__ import annotations

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg
from gpu_helpers import forced_plan
from test_gpu_experts import BF16, near, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,plan", [
    (1, 4096, 4096, None),                                # decode: counters of column blocks
    (512, 1280, 1024, "pair=1,bn=256,tail=1,grid=8"),     # stream-K: flags of the partial sums
    (300, 520, 201, None),                                # operands copied to aligned rows
])
def test_first_run_on_a_side_stream(M, N, K, plan):
    A, B = rnd((M, K), BF16, 1), rnd((N, K), BF16, 2).t()
    D = torch.zeros((M, N), dtype=BF16, device="cuda")
    ref, S = A.double() @ B.double(), A.double().abs() @ B.double().abs()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(60_000_000)  # some 30 ms
    with forced_plan(plan):
        g = pkg.Gemm.like(A, B, None, D)
    for _ in range(3):
        g.run(A, B, None, D, side)
    assert g.status(side) == pkg.GEMM_OK
    with torch.cuda.stream(side):
        got = D.clone()
    torch.cuda.synchronize()
    near(got, ref, S, K)
    g.run(A, B, None, D, side)  # nothing was cleared late
    torch.cuda.synchronize()
    assert torch.equal(D, got)
    assert g.status(side) == pkg.GEMM_OK
    g.close()


def test_matmul_add_on_a_given_stream():
    """A new D may get memory whose last use the current stream has yet to
    run: it is not written after the product."""
    A, B = rnd((200, 256), BF16, 1), rnd((256, 136), BF16, 2)
    ref, S = A.double() @ B.double(), A.double().abs() @ B.double().abs()
    side = torch.cuda.Stream()
    old = torch.empty((200, 136), dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(60_000_000)
    old.fill_(9.0)
    del old
    D = pkg.matmul_add(A, B, stream=side)
    torch.cuda.synchronize()
    near(D, ref, S, 256)
