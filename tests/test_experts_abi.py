"""Refusals of the expert and 4-bit-weight operators: descriptions that the
host rejects before any device is needed, and the Python binding's checks."""
from __future__ import annotations

import ctypes

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg
from dense_tiled_gemm_02_gb300 import experts

INVALID, UNSUPPORTED, MISALIGNED = (pkg.GEMM_ERR_INVALID_ARG, pkg.GEMM_ERR_UNSUPPORTED,
                                    pkg.GEMM_ERR_MISALIGNED)
BF16, F16, F32 = pkg.GEMM_BF16, pkg.GEMM_F16, pkg.GEMM_F32


def create(name, desc):
    h = ctypes.c_void_p()
    rc = getattr(pkg.load(), name)(ctypes.byref(h), ctypes.byref(desc))
    if h.value:
        pkg.load().gemm_op_destroy(h)
    return rc


def fields(cls, base, kw):
    return cls(**{**base, **kw})


ROUTE = dict(T=4, E=8, k=2, type=F32, normalize=1, ld=0)
PERMUTE = dict(T=4, H=64, k=2, type=BF16, ld_tokens=0, ld_rows=0)
GROUPED = dict(form=0, E=4, R=16, K=64, N=64, ab_type=BF16, c_type=0, d_type=BF16, layout_b=0,
               lda=0, ldb=0, ldc=0, ldd=0)
W4 = dict(E=1, group=32, has_zeros=0, R=1, K=64, N=64, x_type=BF16, scale_type=BF16, d_type=BF16,
          ldx=0, ldd=0)


@pytest.mark.parametrize("name,cls,base,kw,code", [
    ("gemm_route_create", pkg.RouteDesc, ROUTE, dict(T=-1), INVALID),
    ("gemm_route_create", pkg.RouteDesc, ROUTE, dict(E=0), INVALID),
    ("gemm_route_create", pkg.RouteDesc, ROUTE, dict(E=1025), INVALID),
    ("gemm_route_create", pkg.RouteDesc, ROUTE, dict(k=9), INVALID),      # more than E
    ("gemm_route_create", pkg.RouteDesc, ROUTE, dict(E=64, k=33), INVALID),
    ("gemm_route_create", pkg.RouteDesc, ROUTE, dict(ld=7), INVALID),
    ("gemm_route_create", pkg.RouteDesc, ROUTE, dict(T=2 ** 31), INVALID),
    ("gemm_route_create", pkg.RouteDesc, ROUTE, dict(type=pkg.GEMM_I8), UNSUPPORTED),
    ("gemm_permute_create", pkg.PermuteDesc, PERMUTE, dict(H=-1), INVALID),
    ("gemm_permute_create", pkg.PermuteDesc, PERMUTE, dict(k=0), INVALID),
    ("gemm_permute_create", pkg.PermuteDesc, PERMUTE, dict(ld_rows=63), INVALID),
    ("gemm_permute_create", pkg.PermuteDesc, PERMUTE, dict(type=pkg.GEMM_I32), UNSUPPORTED),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(form=2), INVALID),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(E=0), INVALID),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(R=-1), INVALID),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(lda=63), INVALID),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(ldd=8), INVALID),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(layout_b=2), INVALID),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(E=1024, K=2 ** 21), INVALID),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(ab_type=F32), UNSUPPORTED),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(d_type=pkg.GEMM_I32), UNSUPPORTED),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(c_type=F32), UNSUPPORTED),  # not D's
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED, dict(form=1, layout_b=1), UNSUPPORTED),
    ("gemm_w4_create", pkg.W4Desc, W4, dict(group=48), INVALID),
    ("gemm_w4_create", pkg.W4Desc, W4, dict(group=0), INVALID),
    ("gemm_w4_create", pkg.W4Desc, W4, dict(K=72), INVALID),
    ("gemm_w4_create", pkg.W4Desc, W4, dict(ldx=32), INVALID),
    ("gemm_w4_create", pkg.W4Desc, W4, dict(x_type=F32), UNSUPPORTED),
    ("gemm_w4_create", pkg.W4Desc, W4, dict(scale_type=pkg.GEMM_I8), UNSUPPORTED),
    ("gemm_w4_create", pkg.W4Desc, W4, dict(ldx=68), MISALIGNED),
])
def test_create_rejects_bad_descriptions(name, cls, base, kw, code):
    assert create(name, fields(cls, base, kw)) == code


@pytest.mark.parametrize("name,cls,base", [
    ("gemm_route_create", pkg.RouteDesc, ROUTE), ("gemm_permute_create", pkg.PermuteDesc, PERMUTE),
    ("gemm_grouped_create", pkg.GroupedDesc, GROUPED), ("gemm_w4_create", pkg.W4Desc, W4)])
def test_create_without_gpu_reports_no_device(name, cls, base):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert create(name, fields(cls, base, {})) == pkg.GEMM_ERR_NO_DEVICE


def test_null_handles_are_refused():
    lib = pkg.load()
    assert lib.gemm_route_run(None, None, None, None, None, None, None, None) == INVALID
    assert lib.gemm_permute_gather(None, None, None, None, None, None) == INVALID
    assert lib.gemm_grouped_run(None, None, None, None, None, None, None) == INVALID
    assert lib.gemm_w4_run(None, None, None, None, None, None, None, None) == INVALID
    assert lib.gemm_op_status(None, None) == INVALID
    assert lib.gemm_op_workspace_bytes(None) == -1
    assert lib.gemm_op_destroy(None) == pkg.GEMM_OK


def test_like_rejects_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.Route.like(x, 2)
    offsets = torch.zeros(3, dtype=torch.int32)
    A, B = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="do not give D"):
        pkg.GroupedGemm.like(A, B, offsets, None, torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="stack of row-major"):
        pkg.GroupedGemm.like(A, torch.zeros(2, 8, 32, dtype=torch.bfloat16)[:, :, ::2], offsets,
                             None, torch.zeros(4, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="offsets"):
        pkg.GroupedGemm.like(A, B, offsets.long(), None, torch.zeros(4, 16, dtype=torch.bfloat16))
    W = torch.zeros(1, 16, 32, dtype=torch.uint8)
    X, D = torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros(1, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="scales"):
        pkg.W4Gemm.like(X, W, torch.zeros(1, 16, 3, dtype=torch.bfloat16), None, None, D, 32)


def test_pack_w4_puts_the_even_k_low():
    q = torch.tensor([[1, 2, 15, 0]])
    assert pkg.pack_w4(q).tolist() == [[0x21, 0x0F]]


def test_planned_tensors_are_compared():
    p = experts._Planned("x", torch.zeros(4, 1, 8))
    # the stride of a dimension of one does not matter
    p.pointer(torch.zeros(4, 1, 8).as_strided((4, 1, 8), (8, 99, 1)))
    with pytest.raises(ValueError, match="x: planned"):
        p.pointer(torch.zeros(4, 1, 9))
    with pytest.raises(ValueError, match="x: planned"):
        p.pointer(torch.zeros(4, 1, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="x: planned"):
        p.pointer(torch.zeros(4, 1, 16)[:, :, ::2])
