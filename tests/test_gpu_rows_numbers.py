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
from test_gpu_rows import (BF16, EPS, F16, F32, done, rnd, strided)

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
