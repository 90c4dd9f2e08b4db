"""The CTA-pair kernel's staged stores where some chunks of a tile leave by
TMA and others by rows, over many tiles of short sums a CTA pair: a staging
buffer is not written before its store has read it.  Bounds as in
test_gpu_experts."""
from __future__ import annotations

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg
from gpu_helpers import forced_plan
from test_gpu_experts import BF16, F16, near, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,dtype,plan", [
    (2048, 2016, 64, BF16, "pair=1,bn=224,grid=8"),   # half a chunk ends each tile
    (2000, 1000, 128, F16, "pair=1,bn=224,grid=8"),
    (4096, 299, 64, BF16, "pair=1,bn=256,grid=8"),    # a chunk crosses N off the 16-byte grid
])
def test_chunks_by_tma_and_by_rows_share_staging_buffers(M, N, K, dtype, plan):
    A, B = rnd((M, K), dtype, 1), rnd((N, K), dtype, 2).t()
    D = torch.zeros((M, -(-N // 8) * 8), dtype=dtype, device="cuda")[:, :N]
    with forced_plan(plan):
        g = pkg.Gemm.like(A, B, None, D)
    assert "pair=1" in g.plan() and plan.split(",")[1] in g.plan(), g.plan()
    ref, S = A.double() @ B.double(), A.double().abs() @ B.double().abs()
    first = None
    for _ in range(20):
        D.fill_(7.0)
        g.run(A, B, None, D)
        if first is None:
            first = D.clone()
            near(D, ref, S, K)
        assert torch.equal(D, first)
    assert g.status(torch.cuda.current_stream()) == pkg.GEMM_OK
    g.close()
