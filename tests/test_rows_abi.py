"""Refusals of the operators on 8-bit rows: descriptions that the host rejects
before any device is needed, and the Python binding's checks."""
from __future__ import annotations

import ctypes

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg

INVALID, UNSUPPORTED = pkg.GEMM_ERR_INVALID_ARG, pkg.GEMM_ERR_UNSUPPORTED
BF16, F16, F32, I8, I32 = (pkg.GEMM_BF16, pkg.GEMM_F16, pkg.GEMM_F32, pkg.GEMM_I8, pkg.GEMM_I32)

NORM = dict(T=4, H=64, type=BF16, weight_type=BF16, y_type=BF16, residual=1, eps=1e-6, ldx=0,
            ldr=0, ldh=0, ldy=0)
ROWS8 = dict(T=4, H=64, type=BF16, block=32, ldx=0, ldq=0)
GRAD = dict(E=2, R=8, K=64, N=32, b_type=BF16, c_type=0, d_type=F32, ldq=0, ldb=0, ldc=0, ldd=0)
PRODUCT = dict(E=1, R=4, K=64, N=32, d_type=BF16, ldx=0, ldw=0, ldd=0)
OPS = {"norm": ("gemm_norm_create", pkg.NormDesc, NORM),
       "rows8": ("gemm_rows8_create", pkg.Rows8Desc, ROWS8),
       "grad": ("gemm_rows8_grad_create", pkg.Rows8GradDesc, GRAD),
       "i8": ("gemm_i8_create", pkg.I8Desc, PRODUCT)}


def create(op, **kw):
    name, cls, base = OPS[op]
    h = ctypes.c_void_p()
    desc = cls(**{**base, **kw})
    rc = getattr(pkg.load(), name)(ctypes.byref(h), ctypes.byref(desc))
    if h.value:
        pkg.load().gemm_op_destroy(h)
    return rc


@pytest.mark.parametrize("op,kw,code", [
    ("norm", dict(T=-1), INVALID), ("norm", dict(H=-1), INVALID), ("norm", dict(ldx=63), INVALID),
    ("norm", dict(ldr=63), INVALID), ("norm", dict(ldh=1), INVALID), ("norm", dict(ldy=63), INVALID),
    ("norm", dict(eps=-1.0), INVALID), ("norm", dict(eps=float("nan")), INVALID),
    ("norm", dict(eps=float("inf")), INVALID), ("norm", dict(H=2 ** 31), INVALID),
    ("norm", dict(type=I8), UNSUPPORTED), ("norm", dict(weight_type=F16), UNSUPPORTED),
    ("norm", dict(y_type=F32), UNSUPPORTED), ("norm", dict(y_type=I32), UNSUPPORTED),
    ("rows8", dict(T=-1), INVALID), ("rows8", dict(H=-1), INVALID), ("rows8", dict(block=16), INVALID),
    ("rows8", dict(block=64), INVALID), ("rows8", dict(ldq=63), INVALID),
    ("rows8", dict(ldx=63), INVALID), ("rows8", dict(type=I32), UNSUPPORTED),
    ("grad", dict(E=0), INVALID), ("grad", dict(E=1025), INVALID), ("grad", dict(R=-1), INVALID),
    ("grad", dict(K=-1), INVALID), ("grad", dict(N=-1), INVALID), ("grad", dict(ldq=63), INVALID),
    ("grad", dict(ldb=31), INVALID), ("grad", dict(ldd=31), INVALID),
    ("grad", dict(b_type=F32), UNSUPPORTED), ("grad", dict(d_type=I8), UNSUPPORTED),
    ("grad", dict(c_type=BF16), UNSUPPORTED),  # not D's
    ("i8", dict(E=0), INVALID), ("i8", dict(E=1025), INVALID), ("i8", dict(R=-1), INVALID),
    ("i8", dict(K=2 ** 17), INVALID), ("i8", dict(K=-1), INVALID), ("i8", dict(N=2 ** 30), INVALID),
    ("i8", dict(E=1024, N=2 ** 21), INVALID), ("i8", dict(ldx=63), INVALID),
    ("i8", dict(ldw=63), INVALID), ("i8", dict(ldd=31), INVALID), ("i8", dict(d_type=I32), UNSUPPORTED),
])
def test_create_rejects_bad_descriptions(op, kw, code):
    assert create(op, **kw) == code


@pytest.mark.parametrize("op", OPS)
def test_create_without_gpu_reports_no_device(op):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert create(op) == pkg.GEMM_ERR_NO_DEVICE


def test_null_handles_and_arguments_are_refused():
    lib = pkg.load()
    assert lib.gemm_norm_run(*[None] * 9) == INVALID
    assert lib.gemm_norm_backward(*[None] * 10) == INVALID
    assert lib.gemm_rows8_pack(*[None] * 5) == INVALID
    assert lib.gemm_rows8_unpack(*[None] * 5) == INVALID
    assert lib.gemm_rows8_grad_run(*[None] * 8) == INVALID
    assert lib.gemm_i8_run(*[None] * 8) == INVALID
    for name, _, _ in OPS.values():
        assert getattr(lib, name)(None, None) == INVALID


def norm_operands(T=4, H=64, dtype=torch.bfloat16):
    new = lambda *s, dtype=dtype: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return dict(x=new(T, H), weight=new(H), y=new(T, H), residual=new(T, H), h=new(T, H))


@pytest.mark.parametrize("change,match", [
    (dict(weight=torch.zeros(63, dtype=torch.bfloat16)), "weight must be 64"),
    (dict(weight=torch.zeros(64, dtype=torch.float16)), "neither x's"),
    (dict(weight=torch.zeros(128, dtype=torch.bfloat16)[::2]), "contiguous"),
    (dict(y=torch.zeros(4, 63, dtype=torch.bfloat16)), "y must be"),
    (dict(y=torch.zeros(4, 64)), "y must be"),
    (dict(y=torch.zeros(4, 64, dtype=torch.int8)), "scales go with"),
    (dict(scales=torch.zeros(4)), "scales go with"),
    (dict(y=torch.zeros(4, 64, dtype=torch.int8), scales=torch.zeros(5)), "scales must be"),
    (dict(y=torch.zeros(4, 64, dtype=torch.int8), scales=torch.zeros(4).double()), "scales must be"),
    (dict(h=None), "go together"), (dict(residual=None), "go together"),
    (dict(residual=torch.zeros(4, 64)), "residual must have"),
    (dict(h=torch.zeros(3, 64, dtype=torch.bfloat16)), "h must have"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(x=torch.zeros(4, 128, dtype=torch.bfloat16)[:, ::2]), "row-major"),
    (dict(residual=torch.zeros(4, 64, dtype=torch.bfloat16, device="meta")), "residual is on meta"),
    ({}, "CUDA"),
])
def test_norm_like_refuses(change, match):
    with pytest.raises(ValueError, match=match):
        pkg.RmsNorm.like(**{**norm_operands(), **change})


@pytest.mark.parametrize("q,scales,match", [
    (torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4), "q must be int8"),
    (torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4), "q must be int8"),
    (torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 3, dtype=torch.uint8), "scales must be"),
    (torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2), "scales must be"),
    (torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8), "CUDA"),
    (torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4), "CUDA"),
    (torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, device="meta"), "scales is on meta"),
])
def test_rows8_like_refuses(q, scales, match):
    with pytest.raises(ValueError, match=match):
        pkg.Rows8.like(torch.zeros(4, 64), q, scales)


def grad_operands(E=2, R=8, K=64, N=32):
    return dict(q=torch.zeros(R, K, dtype=torch.int8),
                exponents=torch.zeros(R, -(-K // 32), dtype=torch.uint8),
                B=torch.zeros(R, N, dtype=torch.bfloat16),
                offsets=torch.zeros(E + 1, dtype=torch.int32), C=None, D=torch.zeros(E, K, N))


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros(8, 64)), "q must be int8"),
    (dict(exponents=torch.zeros(8, 1, dtype=torch.uint8)), "exponents must be"),
    (dict(exponents=torch.zeros(8, 2, dtype=torch.int8)), "exponents must be"),
    (dict(B=torch.zeros(7, 32, dtype=torch.bfloat16)), "do not give D"),
    (dict(D=torch.zeros(2, 32, 64)), "do not give D"),
    (dict(offsets=None), "offsets are needed"),
    (dict(offsets=torch.zeros(3)), "offsets must be"),
    (dict(offsets=torch.zeros(2, dtype=torch.int32)), "offsets must be"),
    (dict(C=torch.zeros(2, 64, 32, dtype=torch.bfloat16)), "C must have"),
    (dict(B=torch.zeros(8, 32, dtype=torch.int32)), "element type"),
    (dict(D=torch.zeros(2, 64, 64)[:, :, ::2]), "stack of row-major"),
    (dict(B=torch.zeros(8, 32, dtype=torch.bfloat16, device="meta")), "B is on meta"),
    ({}, "CUDA"),
])
def test_grad_like_refuses(change, match):
    with pytest.raises(ValueError, match=match):
        pkg.Rows8Grad.like(**{**grad_operands(), **change})


def product_operands(E=2, R=4, K=64, N=32):
    return dict(X=torch.zeros(R, K, dtype=torch.int8), x_scales=torch.zeros(R),
                W=torch.zeros(E, N, K, dtype=torch.int8), w_scales=torch.zeros(E, N),
                offsets=torch.zeros(E + 1, dtype=torch.int32), D=torch.zeros(R, N))


@pytest.mark.parametrize("change,match", [
    (dict(X=torch.zeros(4, 64)), "X must be int8"),
    (dict(W=torch.zeros(2, 32, 63, dtype=torch.int8)), "W must be int8"),
    (dict(W=torch.zeros(32, 64, dtype=torch.int8)), "W must be int8"),
    (dict(W=torch.zeros(2, 32, 64, dtype=torch.uint8)), "W must be int8"),
    (dict(W=torch.zeros(2, 64, 32, dtype=torch.int8).transpose(1, 2)), "stack of row-major"),
    (dict(x_scales=torch.zeros(3)), "x_scales must be"),
    (dict(w_scales=torch.zeros(2, 32, dtype=torch.bfloat16)), "w_scales must be"),
    (dict(D=torch.zeros(4, 31)), "D must be"),
    (dict(D=torch.zeros(4, 32, dtype=torch.int32)), "element type"),
    (dict(offsets=None), "offsets are needed"),
    (dict(offsets=torch.zeros(3, dtype=torch.int64)), "offsets must be"),
    (dict(w_scales=torch.zeros(2, 32, device="meta")), "w_scales is on meta"),
    ({}, "CUDA"),
])
def test_i8_like_refuses(change, match):
    with pytest.raises(ValueError, match=match):
        pkg.I8Gemm.like(**{**product_operands(), **change})
