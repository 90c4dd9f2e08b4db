"""Refusals of the operators on 8-bit rows beyond those of test_rows_abi.py; on the
CPU, which every check comes before."""
from __future__ import annotations

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg
from test_rows_abi import grad_operands


@pytest.mark.parametrize("change", [
    dict(B=torch.zeros(8, dtype=torch.bfloat16)),
    dict(B=torch.zeros(1, 8, 32, dtype=torch.bfloat16)),
    dict(D=torch.zeros(())),
    dict(D=torch.zeros(64, 32)),
    dict(D=torch.zeros(1, 2, 64, 32)),
])
def test_grad_like_refuses_operands_of_other_dimensions(change):
    with pytest.raises(ValueError, match="do not give D"):
        pkg.Rows8Grad.like(**{**grad_operands(), **change})
