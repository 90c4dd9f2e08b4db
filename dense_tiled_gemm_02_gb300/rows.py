"""Operators on rows held in 8 bits, for torch tensors.

* ``RmsNorm``: a residual's addition and the root-mean-square norm of each row,
  out in the rows' type or as scaled rows of 8 bits; and the gradients.
* ``Rows8``: rows to 8 bits and back: block rows (a power of two for every 32
  values, what training keeps for its backward pass) and scaled rows (one fp32
  scale a row, what the 8-bit product reads).
* ``Rows8Grad``: weight gradients from block rows, dense or grouped by expert.
* ``I8Gemm``: scaled rows times weights of 8-bit integers with a scale for each
  output, dense or grouped by expert.

Handles, plans, streams and errors are those of ``experts.py``;
``include/gemm.h`` states the contracts.
"""
from __future__ import annotations

import torch

import dense_tiled_gemm_02_gb300 as _gemm

from .experts import (_new_zeros, _on_one_device, _Op, _plan_of, _Planned, _row_stride,
                      _stack_stride, _type)

BLOCK = 32  # values that share a power of two
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (none without CUDA)


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _int8_rows(t: torch.Tensor, shape, what: str) -> int:
    """Leading dimension of int8 rows of this shape."""
    if tuple(t.shape) != tuple(shape) or t.dtype != torch.int8:
        raise ValueError(f"{what} must be int8 {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return _row_stride(t, what)


def _packed(t: torch.Tensor, shape, dtype, what: str) -> None:
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)} strides {t.stride()}")


def _check_offsets(offsets, E: int) -> None:
    if offsets is None:
        if E != 1:
            raise ValueError("offsets are needed for more than one expert")
    else:
        _packed(offsets, (E + 1,), torch.int32, "offsets")


def _given(plan, t, what: str):
    """The pointer of an optional operand, which must be there as planned."""
    if (plan is None) != (t is None):
        raise ValueError(f"planned {'without' if plan is None else 'with'} {what}")
    return None if t is None else plan.pointer(t)


# The methods that enqueue write out what _Op._call does: handing it the pointers
# costs a fifteenth of the smallest calls.


class RmsNorm(_Op):
    """h = x + residual, y = h * rstd * weight with rstd = (mean h^2 + eps)^-1/2."""

    @classmethod
    def like(cls, x, weight, y, scales=None, residual=None, h=None, eps: float = 1e-6) -> "RmsNorm":
        """Plan for rows like x (T x H).  y is of x's type, or int8 with `scales`
        (T fp32); `residual` and `h` (the sum, of x's type) go together."""
        T, H = x.shape
        i8 = y.dtype == torch.int8
        if tuple(weight.shape) != (H,) or not weight.is_contiguous():
            raise ValueError(f"weight must be {H} contiguous values, got {tuple(weight.shape)}")
        if weight.dtype not in (x.dtype, torch.float32):
            raise ValueError(f"weight is {weight.dtype}: neither x's {x.dtype} nor float32")
        if tuple(y.shape) != (T, H) or y.dtype not in (x.dtype, torch.int8):
            raise ValueError(f"y must be {(T, H)} {x.dtype} or int8, got {tuple(y.shape)} {y.dtype}")
        if i8 != (scales is not None):
            raise ValueError("scales go with an int8 y")
        if (residual is None) != (h is None):
            raise ValueError("residual and h go together")
        for name, t in (("residual", residual), ("h", h)):
            if t is not None and (t.shape != x.shape or t.dtype != x.dtype):
                raise ValueError(f"{name} must have x's shape and type")
        if scales is not None:
            _packed(scales, (T,), torch.float32, "scales")
        if not 0 <= eps < float("inf"):
            raise ValueError(f"eps must be finite and not negative, got {eps}")
        _on_one_device(x.device, weight=weight, y=y, scales=scales, residual=residual, h=h)
        desc = _gemm.NormDesc(
            T, H, _type(x), _type(weight), _gemm.GEMM_I8 if i8 else _type(y),
            int(residual is not None), eps, _row_stride(x, "x"),
            0 if residual is None else _row_stride(residual, "residual"),
            0 if h is None else _row_stride(h, "h"), _row_stride(y, "y"))
        op = cls("gemm_norm_create", desc, x.device)
        op._x, op._weight, op._y = _Planned("x", x), _Planned("weight", weight), _Planned("y", y)
        op._residual = None if residual is None else _Planned("residual", residual)
        op._h = None if h is None else _Planned("h", h)
        op._scales = None if scales is None else _Planned("scales", scales)
        op._rstd = _plan_of("rstd", (T,), torch.float32, x)
        op._dweight = _plan_of("dweight", (H,), torch.float32, x)
        op._h8 = _plan_of("h", (T, H), torch.int8, x)
        op._exponents = _plan_of("exponents", (T, _blocks(H)), torch.uint8, x)
        return op

    def run(self, x, weight, y, scales=None, residual=None, h=None, rstd=None, stream=None) -> None:
        """Enqueue the norm; rstd (T fp32), if given, is what `backward` needs."""
        stream = _current(self._index) if stream is None else getattr(stream, "cuda_stream", stream)
        rc = self._lib.gemm_norm_run(
            self.handle, self._x.pointer(x), _given(self._residual, residual, "residual"),
            self._weight.pointer(weight), _given(self._h, h, "h"), self._y.pointer(y),
            _given(self._scales, scales, "scales"),
            None if rstd is None else self._rstd.pointer(rstd), stream)
        if rc != _gemm.GEMM_OK:
            raise _gemm.GemmError(rc, "gemm_norm_run")

    def backward(self, dy, h, weight, rstd, dx, dweight=None, dresidual=None, exponents=None,
                 stream=None) -> None:
        """Enqueue dx (of x and residual) and dweight (H fp32) from dy and what
        comes to h by the residual, dresidual.  h: the forward pass's (x without
        a residual), or with `exponents` its block rows (see Rows8), packed."""
        if self._scales is not None:
            raise ValueError("planned for an int8 y, which has no gradient")
        rows = (self._h8 if exponents is not None else self._x if self._h is None else self._h)
        stream = _current(self._index) if stream is None else getattr(stream, "cuda_stream", stream)
        rc = self._lib.gemm_norm_backward(
            self.handle, self._y.pointer(dy), rows.pointer(h),
            None if exponents is None else self._exponents.pointer(exponents),
            self._weight.pointer(weight), self._rstd.pointer(rstd),
            None if dresidual is None else
            (self._x if self._h is None else self._h).pointer(dresidual),
            self._x.pointer(dx), None if dweight is None else self._dweight.pointer(dweight), stream)
        if rc != _gemm.GEMM_OK:
            raise _gemm.GemmError(rc, "gemm_norm_backward")


class Rows8(_Op):
    """Rows to 8 bits and back."""

    @classmethod
    def like(cls, X, q, scales) -> "Rows8":
        """Plan for rows X (T x H) and their integers q (int8).  scales uint8 (T,
        ceil(H / 32)): block rows, the exponents of a power of two for every 32
        values (127 for 1); scales fp32 (T): scaled rows."""
        T, H = X.shape
        ldq = _int8_rows(q, (T, H), "q")
        block = BLOCK if scales.dtype == torch.uint8 else 0
        if block:
            _packed(scales, (T, _blocks(H)), torch.uint8, "scales")
        else:
            _packed(scales, (T,), torch.float32, "scales")
        _on_one_device(X.device, q=q, scales=scales)
        op = cls("gemm_rows8_create", _gemm.Rows8Desc(T, H, _type(X), block, _row_stride(X, "X"), ldq),
                 X.device)
        op._X, op._q, op._scales = _Planned("X", X), _Planned("q", q), _Planned("scales", scales)
        return op

    @staticmethod
    def empty(X, block: bool = True):
        """Fresh (q, scales) for rows like X: block rows, or scaled rows."""
        T, H = X.shape
        q = torch.empty((T, H), dtype=torch.int8, device=X.device)
        if block:
            return q, torch.empty((T, _blocks(H)), dtype=torch.uint8, device=X.device)
        return q, torch.empty(T, dtype=torch.float32, device=X.device)

    def pack(self, X, q, scales, stream=None) -> None:
        """Enqueue q and scales from X."""
        stream = _current(self._index) if stream is None else getattr(stream, "cuda_stream", stream)
        rc = self._lib.gemm_rows8_pack(self.handle, self._X.pointer(X), self._q.pointer(q),
                                       self._scales.pointer(scales), stream)
        if rc != _gemm.GEMM_OK:
            raise _gemm.GemmError(rc, "gemm_rows8_pack")

    def unpack(self, q, scales, X, stream=None) -> None:
        """Enqueue X from q and scales."""
        stream = _current(self._index) if stream is None else getattr(stream, "cuda_stream", stream)
        rc = self._lib.gemm_rows8_unpack(self.handle, self._q.pointer(q),
                                         self._scales.pointer(scales), self._X.pointer(X), stream)
        if rc != _gemm.GEMM_OK:
            raise _gemm.GemmError(rc, "gemm_rows8_unpack")


class Rows8Grad(_Op):
    """Weight gradients from block rows: D_e = A_e^T B_e (+ C_e)."""

    @classmethod
    def like(cls, q, exponents, B, offsets, C, D) -> "Rows8Grad":
        """Plan for A (R x K) as block rows q and exponents, B (R x N) of a
        16-bit type and D (E, K, N); offsets None for E = 1."""
        R, K = q.shape
        ldq = _int8_rows(q, (R, K), "q")
        _packed(exponents, (R, _blocks(K)), torch.uint8, "exponents")
        if (B.dim() != 2 or B.shape[0] != R or D.dim() != 3 or
                tuple(D.shape[1:]) != (K, B.shape[1])):
            raise ValueError(f"q {tuple(q.shape)} and B {tuple(B.shape)} do not give D "
                             f"{tuple(D.shape)}")
        E, N = D.shape[0], B.shape[1]
        _check_offsets(offsets, E)
        if C is not None and (C.shape != D.shape or C.dtype != D.dtype):
            raise ValueError("C must have D's shape and type")
        _on_one_device(q.device, exponents=exponents, B=B, offsets=offsets, C=C, D=D)
        desc = _gemm.Rows8GradDesc(
            E, R, K, N, _type(B), 0 if C is None else _type(C), _type(D), ldq, _row_stride(B, "B"),
            0 if C is None else _stack_stride(C, "C"), _stack_stride(D, "D"))
        op = cls("gemm_rows8_grad_create", desc, q.device)
        op._q, op._exponents = _Planned("q", q), _Planned("exponents", exponents)
        op._B, op._D = _Planned("B", B), _Planned("D", D)
        op._offsets = None if offsets is None else _Planned("offsets", offsets)
        op._C = None if C is None else _Planned("C", C)
        return op

    def run(self, q, exponents, B, offsets, C, D, stream=None) -> None:
        """Enqueue the gradients of all experts (C None: nothing is added)."""
        if C is not None and self._C is None:
            raise ValueError("planned without C")
        self._call("gemm_rows8_grad_run", stream, self._q.pointer(q),
                   self._exponents.pointer(exponents), self._B.pointer(B),
                   _given(self._offsets, offsets, "offsets"),
                   None if C is None else self._C.pointer(C), self._D.pointer(D))


class I8Gemm(_Op):
    """Scaled rows times weights of 8-bit integers."""

    @classmethod
    def like(cls, X, x_scales, W, w_scales, offsets, D) -> "I8Gemm":
        """Plan D[r, n] = x_scales[r] w_scales[e, n] sum_k X[r, k] W[e, n, k]: X
        (R, K) and W (E, N, K) int8, scales fp32; offsets (E + 1) group the
        rows, None for E = 1."""
        R, K = X.shape
        if W.dim() != 3 or W.shape[2] != K or W.dtype != torch.int8:
            raise ValueError(f"W must be int8 (E, N, {K}), got {W.dtype} {tuple(W.shape)}")
        E, N = W.shape[:2]
        ldx = _int8_rows(X, (R, K), "X")
        _packed(x_scales, (R,), torch.float32, "x_scales")
        _packed(w_scales, (E, N), torch.float32, "w_scales")
        if tuple(D.shape) != (R, N):
            raise ValueError(f"D must be {(R, N)}, got {tuple(D.shape)}")
        _check_offsets(offsets, E)
        _on_one_device(X.device, x_scales=x_scales, W=W, w_scales=w_scales, offsets=offsets, D=D)
        desc = _gemm.I8Desc(E, R, K, N, _type(D), ldx, _stack_stride(W, "W"), _row_stride(D, "D"))
        op = cls("gemm_i8_create", desc, X.device)
        op._X, op._W, op._D = _Planned("X", X), _Planned("W", W), _Planned("D", D)
        op._x_scales, op._w_scales = _Planned("x_scales", x_scales), _Planned("w_scales", w_scales)
        op._offsets = None if offsets is None else _Planned("offsets", offsets)
        return op

    def run(self, X, x_scales, W, w_scales, offsets, D, stream=None) -> None:
        """Enqueue the products."""
        stream = _current(self._index) if stream is None else getattr(stream, "cuda_stream", stream)
        rc = self._lib.gemm_i8_run(
            self.handle, self._X.pointer(X), self._x_scales.pointer(x_scales), self._W.pointer(W),
            self._w_scales.pointer(w_scales), _given(self._offsets, offsets, "offsets"),
            self._D.pointer(D), stream)
        if rc != _gemm.GEMM_OK:
            raise _gemm.GemmError(rc, "gemm_i8_run")


def i8_matmul(X, x_scales, W, w_scales, offsets=None, out_dtype=torch.bfloat16, D=None,
              stream=None):
    """D = (X * x_scales) @ (W * w_scales)^T (plans a fresh handle each call; a
    new D and `stream` as in grouped_matmul)."""
    if D is None:
        D = _new_zeros((X.shape[0], W.shape[1]), out_dtype, X.device, stream)
    g = I8Gemm.like(X, x_scales, W, w_scales, offsets, D)
    try:
        g.run(X, x_scales, W, w_scales, offsets, D, stream)
    finally:
        g.close()
    return D
