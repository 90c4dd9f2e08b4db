"""Operators of mixture-of-experts layers and of 4-bit weights, for torch tensors.

* ``Route``: the k largest logits of each token, their softmax gates, and the
  order of the chosen (token, choice) slots sorted by expert; and the
  gradient of the logits.
* ``Permute``: rows of tokens into that order, the gated sum back, and the
  gradients of both.
* ``GroupedGemm``: one matrix product per expert over ragged groups of rows;
  its B's other layout gives the input gradient, its three-dimensional D the
  weight gradient.
* ``W4Gemm``: rows times 4-bit weights with a scale (and zero point) per group
  of K, dense or grouped by expert.

Each class wraps a handle of the C ABI (``include/gemm.h`` states the
contracts), planned for the shapes, types and strides of example tensors by
``like``; the calls only enqueue on the current stream, or the one given.
Tensors that differ from the planned ones raise ``ValueError`` before anything
is launched.
"""
from __future__ import annotations

import ctypes

import torch

import dense_tiled_gemm_02_gb300 as _gemm


def _type(t: torch.Tensor) -> int:
    codes = {torch.float16: _gemm.GEMM_F16, torch.bfloat16: _gemm.GEMM_BF16,
             torch.float32: _gemm.GEMM_F32}
    if t.dtype not in codes:
        raise ValueError(f"element type {t.dtype} is not float16, bfloat16 or float32")
    return codes[t.dtype]


def _row_stride(t: torch.Tensor, what: str) -> int:
    """Leading dimension of a row-major matrix (rows contiguous)."""
    rows, cols = t.shape
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1 or rows > 1 and s0 < cols:
        raise ValueError(f"{what} with strides {t.stride()} is not row-major")
    return s0 if rows > 1 and s0 >= cols else max(cols, 1)


def _stack_stride(t: torch.Tensor, what: str) -> int:
    """Leading dimension of E row-major matrices stored one after another."""
    E, rows, cols = t.shape
    if t.numel() == 0:
        return max(cols, 1)
    se, s0, s1 = t.stride()
    ld = s0 if rows > 1 else (se if E > 1 else max(cols, 1))
    if cols > 1 and s1 != 1 or ld < cols or E > 1 and se != rows * ld:
        raise ValueError(f"{what} with strides {t.stride()} is not a stack of row-major matrices")
    return max(ld, 1)


def _on_one_device(device: torch.device, **operands) -> None:
    """Refuse operands elsewhere: their pointers would go to the kernels."""
    for name, t in operands.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


class _Planned:
    """What a tensor argument must look like: shape, dtype and (for
    dimensions longer than one) strides."""
    __slots__ = ("name", "shape", "dtype", "stride", "device", "index", "packed")

    def __init__(self, name: str, t: torch.Tensor, device=None):
        self.name, self.shape, self.dtype, self.stride = name, t.shape, t.dtype, t.stride()
        self.device = device or t.device
        self.index, self.packed = self.device.index, t.is_contiguous()

    def pointer(self, t: torch.Tensor) -> int:
        # The usual case first, by the cheapest calls: this runs for every
        # operand of every call, and half of a decode step's calls is this.
        if (t.shape == self.shape and t.dtype is self.dtype and t.get_device() == self.index and
                (t.is_contiguous() if self.packed else t.stride() == self.stride)):
            return t.data_ptr()
        if (t.shape != self.shape or t.dtype is not self.dtype or t.device != self.device or
                any(n > 1 and a != b for n, a, b in zip(t.shape, t.stride(), self.stride))):
            raise ValueError(f"{self.name}: planned for {tuple(self.shape)} {self.dtype} strides "
                             f"{self.stride} on {self.device}, got {tuple(t.shape)} {t.dtype} "
                             f"strides {t.stride()} on {t.device}")
        return t.data_ptr()


def _plan_of(name: str, shape, dtype, like: torch.Tensor) -> _Planned:
    """The plan of a packed tensor of this shape on like's device."""
    return _Planned(name, torch.empty(shape, dtype=dtype, device="meta"), like.device)


class _Op:
    """A handle of the C ABI."""

    def __init__(self, create: str, desc, device: torch.device):
        if device.type != "cuda":
            raise ValueError(f"operands on {device}: a CUDA device is needed")
        self._lib = _gemm.load()
        self.desc, self.device, self._index = desc, device, device.index
        self.handle = None
        h = ctypes.c_void_p()
        with torch.cuda.device(device):
            rc = getattr(self._lib, create)(ctypes.byref(h), ctypes.byref(desc))
        if rc != _gemm.GEMM_OK:
            raise _gemm.GemmError(rc, create)
        self.handle = h.value

    def _call(self, name: str, stream, *pointers) -> None:
        # the raw handle: making a Stream object costs 2 us, a third of the
        # smallest calls
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(self._index)
        else:
            stream = getattr(stream, "cuda_stream", stream)
        rc = getattr(self._lib, name)(self.handle, *pointers, stream)
        if rc != _gemm.GEMM_OK:
            raise _gemm.GemmError(rc, name)

    def status(self, stream=None) -> int:
        """Synchronise the stream; return and clear the device status."""
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        return self._lib.gemm_op_status(self.handle, getattr(stream, "cuda_stream", stream))

    def plan(self) -> str:
        buf = ctypes.create_string_buffer(256)
        self._lib.gemm_op_plan_string(self.handle, buf, len(buf))
        return buf.value.decode()

    def workspace_bytes(self) -> int:
        return self._lib.gemm_op_workspace_bytes(self.handle)

    def debug_set(self, flags: int, timeout_ns: int = 0) -> int:
        return self._lib.gemm_op_debug_set(self.handle, flags, timeout_ns)

    def close(self) -> None:
        if self.handle is not None:
            self._lib.gemm_op_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Route(_Op):
    """Top-k routing of T tokens over E experts."""

    @classmethod
    def like(cls, logits: torch.Tensor, k: int, normalize: bool = True) -> "Route":
        T, E = logits.shape
        ld = _row_stride(logits, "logits")
        op = cls("gemm_route_create",
                 _gemm.RouteDesc(T, E, k, _type(logits), int(normalize), ld), logits.device)
        i32 = torch.int32
        op._logits = _Planned("logits", logits)
        op._experts = _plan_of("experts", (T, k), i32, logits)
        op._gates = _plan_of("gates", (T, k), torch.float32, logits)
        op._offsets = _plan_of("offsets", (E + 1,), i32, logits)
        op._row_slot = _plan_of("row_slot", (T * k,), i32, logits)
        op._slot_row = _plan_of("slot_row", (T, k), i32, logits)
        return op

    def outputs(self):
        """Fresh (experts, gates, offsets, row_slot, slot_row)."""
        return tuple(torch.empty(p.shape, dtype=p.dtype, device=self.device)
                     for p in (self._experts, self._gates, self._offsets, self._row_slot,
                               self._slot_row))

    def run(self, logits, experts, gates, offsets, row_slot, slot_row, stream=None) -> None:
        """Enqueue the routing of these logits into the five outputs."""
        self._call("gemm_route_run", stream, self._logits.pointer(logits),
                   self._experts.pointer(experts), self._gates.pointer(gates),
                   self._offsets.pointer(offsets), self._row_slot.pointer(row_slot),
                   self._slot_row.pointer(slot_row))

    def backward(self, logits, experts, gates, dgates, dlogits, stream=None) -> None:
        """Enqueue dlogits from the gradient of the gates."""
        self._call("gemm_route_backward", stream, self._logits.pointer(logits),
                   self._experts.pointer(experts), self._gates.pointer(gates),
                   self._gates.pointer(dgates), self._logits.pointer(dlogits))


class Permute(_Op):
    """Rows of T tokens to T * k rows sorted by expert, and back."""

    @classmethod
    def like(cls, X: torch.Tensor, slot_row: torch.Tensor) -> "Permute":
        """Plan for tokens like X (T x H) and a routing like slot_row (T x k);
        the sorted arrays are packed (T * k) x H."""
        T, H = X.shape
        if slot_row.dim() != 2 or slot_row.shape[0] != T:
            raise ValueError(f"slot_row {tuple(slot_row.shape)} does not have {T} rows")
        k = slot_row.shape[1]
        op = cls("gemm_permute_create",
                 _gemm.PermuteDesc(T, H, k, _type(X), _row_stride(X, "X"), max(H, 1)), X.device)
        op._tokens = _Planned("tokens", X)
        op._rows = _plan_of("rows", (T * k, H), X.dtype, X)
        op._row_slot = _plan_of("row_slot", (T * k,), torch.int32, X)
        op._slot_row = _plan_of("slot_row", (T, k), torch.int32, X)
        op._gates = _plan_of("gates", (T, k), torch.float32, X)
        return op

    def gather(self, X, row_slot, slot_row, Xs, stream=None) -> None:
        """Enqueue Xs[slot_row[t, j]] = X[t]; rows without a slot are zeroed."""
        self._call("gemm_permute_gather", stream, self._tokens.pointer(X),
                   self._row_slot.pointer(row_slot), self._slot_row.pointer(slot_row),
                   self._rows.pointer(Xs))

    def combine(self, Ys, slot_row, gates, Y, stream=None) -> None:
        """Enqueue Y[t] = sum_j gates[t, j] Ys[slot_row[t, j]] (gates None: 1,
        which is gather's gradient)."""
        self._call("gemm_permute_combine", stream, self._rows.pointer(Ys),
                   self._slot_row.pointer(slot_row),
                   None if gates is None else self._gates.pointer(gates), self._tokens.pointer(Y))

    def combine_backward(self, dY, Ys, row_slot, slot_row, gates, dYs, dgates,
                         stream=None) -> None:
        """Enqueue dYs[slot_row[t, j]] = gates[t, j] dY[t] and dgates[t, j] =
        <dY[t], Ys[slot_row[t, j]]>."""
        self._call("gemm_permute_combine_backward", stream, self._tokens.pointer(dY),
                   self._rows.pointer(Ys), self._row_slot.pointer(row_slot),
                   self._slot_row.pointer(slot_row), self._gates.pointer(gates),
                   self._rows.pointer(dYs), self._gates.pointer(dgates))


class GroupedGemm(_Op):
    """One matrix product per expert over ragged groups of rows."""

    @classmethod
    def like(cls, A, B, offsets, C, D) -> "GroupedGemm":
        """Plan D[r] = A[r] B_e (+ C[r]) for a B of shape (E, K, N), each matrix
        row- or column-major, or, when D is (E, K, N), the weight gradient
        D_e = A_e^T B_e (+ C_e)."""
        E = offsets.shape[0] - 1
        R, K = A.shape
        grad = D.dim() == 3
        if grad:
            if B.dim() != 2 or B.shape[0] != R or tuple(D.shape) != (E, K, B.shape[1]):
                raise ValueError(f"A {tuple(A.shape)}, B {tuple(B.shape)} and {E} experts do not "
                                 f"give D {tuple(D.shape)}")
            N = B.shape[1]
            layout, ldb = _gemm.GEMM_ROW_MAJOR, _row_stride(B, "B")
            ld_of = _stack_stride
        else:
            if B.dim() != 3 or tuple(B.shape[:2]) != (E, K) or tuple(D.shape) != (R, B.shape[2]):
                raise ValueError(f"A {tuple(A.shape)}, B {tuple(B.shape)} and {E} experts do not "
                                 f"give D {tuple(D.shape)}")
            N = B.shape[2]
            # a single column lies along K where it can: its rows of one
            # element would have to follow each other over all experts
            if B.stride(2) == 1 and N > 1 or N <= 1 and B.stride(1) != 1:
                layout, ldb = _gemm.GEMM_ROW_MAJOR, _stack_stride(B, "B")
            else:
                layout, ldb = _gemm.GEMM_COL_MAJOR, _stack_stride(B.transpose(1, 2), "B")
            ld_of = _row_stride
        if A.dtype != B.dtype:
            raise ValueError(f"A is {A.dtype} and B is {B.dtype}")
        if C is not None and (C.shape != D.shape or C.dtype != D.dtype):
            raise ValueError("C must have D's shape and type")
        if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
            raise ValueError("offsets must be E + 1 contiguous int32 values")
        _on_one_device(A.device, B=B, offsets=offsets, C=C, D=D)
        desc = _gemm.GroupedDesc(
            1 if grad else 0, E, R, K, N, _type(A), 0 if C is None else _type(C), _type(D), layout,
            _row_stride(A, "A"), ldb, 0 if C is None else ld_of(C, "C"), ld_of(D, "D"))
        op = cls("gemm_grouped_create", desc, A.device)
        op._A, op._B, op._D = _Planned("A", A), _Planned("B", B), _Planned("D", D)
        op._offsets = _Planned("offsets", offsets)
        op._C = None if C is None else _Planned("C", C)
        return op

    def run(self, A, B, offsets, C, D, stream=None) -> None:
        """Enqueue the products of all experts (C None: nothing is added)."""
        if C is not None and self._C is None:
            raise ValueError("planned without C")
        self._call("gemm_grouped_run", stream, self._A.pointer(A), self._B.pointer(B),
                   self._offsets.pointer(offsets), None if C is None else self._C.pointer(C),
                   self._D.pointer(D))


class W4Gemm(_Op):
    """Rows times 4-bit weights with group scales."""

    @classmethod
    def like(cls, X, W, scales, zeros, offsets, D, group: int) -> "W4Gemm":
        """Plan D = X w^T, w = (q - zeros) * scales: W (E, N, K / 2) uint8 (see
        pack_w4), scales and zeros (E, N, ceil(K / group)), zeros None for 8;
        offsets (E + 1) group the rows, None for E = 1."""
        R, K = X.shape
        if group < 1:
            raise ValueError(f"group must be a multiple of 32, got {group}")
        E, N = W.shape[:2]
        G = -(-K // group)
        if tuple(W.shape) != (E, N, K // 2) or W.dtype != torch.uint8 or not W.is_contiguous():
            raise ValueError(f"W must be packed uint8 (E, N, {K // 2}), got {tuple(W.shape)}")
        for name, t in (("scales", scales), ("zeros", zeros)):
            if t is not None and (tuple(t.shape) != (E, N, G) or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {(E, N, G)}, got {tuple(t.shape)}")
        if zeros is not None and zeros.dtype != torch.uint8:
            raise ValueError("zeros must be uint8")
        if tuple(D.shape) != (R, N):
            raise ValueError(f"D must be {(R, N)}, got {tuple(D.shape)}")
        if offsets is None:
            if E != 1:
                raise ValueError("offsets are needed for more than one expert")
        elif (tuple(offsets.shape) != (E + 1,) or offsets.dtype != torch.int32 or
              not offsets.is_contiguous()):
            raise ValueError("offsets must be E + 1 contiguous int32 values")
        _on_one_device(X.device, W=W, scales=scales, zeros=zeros, offsets=offsets, D=D)
        desc = _gemm.W4Desc(E, group, int(zeros is not None), R, K, N, _type(X), _type(scales),
                            _type(D), _row_stride(X, "X"), _row_stride(D, "D"))
        op = cls("gemm_w4_create", desc, X.device)
        op._X, op._W, op._D = _Planned("X", X), _Planned("W", W), _Planned("D", D)
        op._scales = _Planned("scales", scales)
        op._zeros = None if zeros is None else _Planned("zeros", zeros)
        op._offsets = None if offsets is None else _Planned("offsets", offsets)
        return op

    def run(self, X, W, scales, zeros, offsets, D, stream=None) -> None:
        """Enqueue D[r, n] = sum_k X[r, k] (q - zero) scale."""
        for name, plan, t in (("zeros", self._zeros, zeros), ("offsets", self._offsets, offsets)):
            if (plan is None) != (t is None):
                raise ValueError(f"planned {'without' if plan is None else 'with'} {name}")
        self._call("gemm_w4_run", stream, self._X.pointer(X), self._W.pointer(W),
                   self._scales.pointer(scales),
                   None if zeros is None else self._zeros.pointer(zeros),
                   None if offsets is None else self._offsets.pointer(offsets),
                   self._D.pointer(D))


def pack_w4(q: torch.Tensor) -> torch.Tensor:
    """4-bit values (..., K), K even, as W4Gemm reads them: (..., K / 2) uint8,
    the even k in the low half.  Other values than 0..15 are refused (which
    waits for the device)."""
    if q.shape[-1] % 2:
        raise ValueError(f"K = {q.shape[-1]} is odd")
    if q.numel():
        low, high = torch.aminmax(q)
        if not (low >= 0 and high <= 15):  # NaN is not either
            raise ValueError(f"4-bit values are 0..15, not {low.item()}..{high.item()}")
    q = q.to(torch.uint8)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous()


def _new_zeros(shape, dtype, device, stream) -> torch.Tensor:
    """Zeros that a call on `stream` may write."""
    D = torch.zeros(shape, dtype=dtype, device=device)
    _gemm._after_current(stream, D)
    return D


def grouped_matmul(A, B, offsets, C=None, out_dtype=None, D=None, stream=None):
    """D[r] = A[r] @ B[e] (+ C[r]) for the rows r of each expert e (plans a
    fresh handle each call).  A new D's rows of no expert are zero, and a
    `stream` waits for the current one before it writes them."""
    if D is None:
        D = _new_zeros((A.shape[0], B.shape[2]), out_dtype or A.dtype, A.device, stream)
    g = GroupedGemm.like(A, B, offsets, C, D)
    try:
        g.run(A, B, offsets, C, D, stream)
    finally:
        g.close()
    return D


def w4_matmul(X, W, scales, zeros=None, offsets=None, group: int = 128, out_dtype=None, D=None,
              stream=None):
    """D = X @ ((q - zeros) * scales)^T (plans a fresh handle each call; a new
    D and `stream` as in grouped_matmul)."""
    if D is None:
        D = _new_zeros((X.shape[0], W.shape[1]), out_dtype or X.dtype, X.device, stream)
    g = W4Gemm.like(X, W, scales, zeros, offsets, D, group)
    try:
        g.run(X, W, scales, zeros, offsets, D, stream)
    finally:
        g.close()
    return D
