"""GB300 (sm_103a) tiled GEMM, D = A*B + C, behind a C ABI.

This package is a thin ctypes binding over ``libgb300gemm.so`` (built from
``csrc/`` by ``build.py``).  It only marshals arguments: every step of the
computation runs in the library's CUDA kernels.  If the library is missing
or cannot be loaded, importing the binding's entry points raises; there is
no CPU fallback.

Low-level names mirror ``include/gemm.h``: ``gemm_create``, ``gemm_run``,
``gemm_get_status``, ``gemm_destroy``, ``gemm_strerror``,
``gemm_plan_string``, ``gemm_workspace_bytes``, ``gemm_raster_tile``,
``gemm_debug_set``, ``gemm_timing_enable``, ``gemm_timing_read``,
``gemm_host_io_enable``, ``gemm_run_host_batch``, ``gemm_pair_schedule``,
``gemm_cta_schedule``, ``gemm_decode_ring``, ``gemm_run_splitk_noalloc``,
``gemm_noalloc_status``, ``gemm_run_mx``, ``gemm_trace_set``.
``Gemm`` wraps a handle for torch tensors.  The operators of
mixture-of-experts layers and of 4-bit weights (``Route``, ``Permute``,
``GroupedGemm``, ``W4Gemm``) are in ``experts.py``.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

GEMM_F16, GEMM_BF16, GEMM_F32, GEMM_I8, GEMM_I32 = 1, 2, 3, 4, 5
GEMM_E4M3, GEMM_E5M2 = 6, 7  # OCP OFP8 8-bit float operands
GEMM_MXE4M3, GEMM_MXE5M2 = 8, 9  # the same with E8M0 scales per 32-element K block
GEMM_ROW_MAJOR, GEMM_COL_MAJOR = 0, 1
GEMM_OK = 0
GEMM_ERR_INVALID_ARG = -1
GEMM_ERR_UNSUPPORTED = -2
GEMM_ERR_MISALIGNED = -3
GEMM_ERR_CUDA = -4
GEMM_ERR_DEVICE_TIMEOUT = -5
GEMM_ERR_ALLOC_FAILED = -6
GEMM_ERR_NO_DEVICE = -7
GEMM_DEBUG_SKIP_FIRST_FILL = 1
GEMM_DEBUG_SKIP_ONE_FILL = 2

EXPORTED = ["gemm_create", "gemm_run", "gemm_get_status", "gemm_destroy", "gemm_strerror",
            "gemm_plan_string", "gemm_workspace_bytes", "gemm_raster_tile", "gemm_debug_set",
            "gemm_run_splitk_noalloc", "gemm_noalloc_status", "gemm_timing_enable", "gemm_timing_read",
            "gemm_host_io_enable", "gemm_run_host_batch", "gemm_pair_schedule",
            "gemm_cta_schedule", "gemm_decode_ring", "gemm_run_mx", "gemm_trace_set",
            "gemm_op_status", "gemm_op_destroy", "gemm_op_workspace_bytes", "gemm_op_plan_string",
            "gemm_op_debug_set", "gemm_route_create", "gemm_route_run", "gemm_route_backward",
            "gemm_permute_create", "gemm_permute_gather", "gemm_permute_combine",
            "gemm_permute_combine_backward", "gemm_grouped_create", "gemm_grouped_run",
            "gemm_w4_create", "gemm_w4_run"]
GEMM_TRACE_EVENTS = 32
GEMM_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


class GemmDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("ab_type", ctypes.c_int), ("c_type", ctypes.c_int), ("d_type", ctypes.c_int),
                ("layout_a", ctypes.c_int), ("layout_b", ctypes.c_int),
                ("layout_c", ctypes.c_int), ("layout_d", ctypes.c_int),
                ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldc", ctypes.c_int64),
                ("ldd", ctypes.c_int64)]


class RouteDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("type", ctypes.c_int), ("normalize", ctypes.c_int32), ("ld", ctypes.c_int64)]


class PermuteDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("k", ctypes.c_int32),
                ("type", ctypes.c_int), ("ld_tokens", ctypes.c_int64),
                ("ld_rows", ctypes.c_int64)]


class GroupedDesc(ctypes.Structure):
    _fields_ = [("form", ctypes.c_int), ("E", ctypes.c_int32), ("R", ctypes.c_int64),
                ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("ab_type", ctypes.c_int),
                ("c_type", ctypes.c_int), ("d_type", ctypes.c_int), ("layout_b", ctypes.c_int),
                ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldc", ctypes.c_int64),
                ("ldd", ctypes.c_int64)]


class W4Desc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("group", ctypes.c_int32), ("has_zeros", ctypes.c_int32),
                ("R", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64),
                ("x_type", ctypes.c_int), ("scale_type", ctypes.c_int), ("d_type", ctypes.c_int),
                ("ldx", ctypes.c_int64), ("ldd", ctypes.c_int64)]


class GemmError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {gemm_strerror(code)} ({code})")
        self.code = code


_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_needed: bool = True) -> ctypes.CDLL:
    """Load the CUDA library (building it first if asked); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_needed:
        _build.build()
    if not os.path.exists(_build.LIB):
        raise RuntimeError(f"CUDA library not built: {_build.LIB}")
    lib = ctypes.CDLL(_build.LIB)
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.gemm_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(GemmDesc)]
    lib.gemm_create.restype = ci
    lib.gemm_run.argtypes = [vp, vp, vp, vp, vp, vp]
    lib.gemm_run.restype = ci
    lib.gemm_run_mx.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
    lib.gemm_run_mx.restype = ci
    lib.gemm_get_status.argtypes = [vp, vp]
    lib.gemm_get_status.restype = ci
    lib.gemm_destroy.argtypes = [vp]
    lib.gemm_destroy.restype = ci
    lib.gemm_strerror.argtypes = [ci]
    lib.gemm_strerror.restype = ctypes.c_char_p
    lib.gemm_plan_string.argtypes = [vp, ctypes.c_char_p, ctypes.c_size_t]
    lib.gemm_plan_string.restype = ci
    lib.gemm_workspace_bytes.argtypes = [vp]
    lib.gemm_workspace_bytes.restype = i64
    lib.gemm_raster_tile.argtypes = [i64, i64, i64, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    lib.gemm_raster_tile.restype = ci
    lib.gemm_debug_set.argtypes = [vp, ci, ctypes.c_uint64]
    lib.gemm_debug_set.restype = ci
    lib.gemm_trace_set.argtypes = [vp, vp]
    lib.gemm_trace_set.restype = ci
    lib.gemm_run_splitk_noalloc.argtypes = [ctypes.POINTER(GemmDesc), ci, vp, vp, vp, vp, vp]
    lib.gemm_run_splitk_noalloc.restype = ci
    lib.gemm_noalloc_status.argtypes = [vp]
    lib.gemm_noalloc_status.restype = ci
    lib.gemm_pair_schedule.argtypes = [i64, i64, i64, ci, ci, ci, ci, ci, ci, ctypes.POINTER(i64)]
    lib.gemm_pair_schedule.restype = ci
    lib.gemm_cta_schedule.argtypes = [i64, i64, i64, ci, ci, ci, ci, ci, ci, ctypes.POINTER(i64)]
    lib.gemm_cta_schedule.restype = ci
    lib.gemm_timing_enable.argtypes = [vp, ci]
    lib.gemm_timing_enable.restype = ci
    lib.gemm_timing_read.argtypes = [vp, ctypes.POINTER(ctypes.c_float), ci]
    lib.gemm_timing_read.restype = ci
    lib.gemm_decode_ring.argtypes = [ci, i64, ci, ctypes.POINTER(ci), ctypes.POINTER(i64)]
    lib.gemm_decode_ring.restype = ci
    lib.gemm_host_io_enable.argtypes = [vp]
    lib.gemm_host_io_enable.restype = ci
    lib.gemm_run_host_batch.argtypes = [vp, ci, ctypes.POINTER(vp), ctypes.POINTER(vp),
                                        ctypes.POINTER(vp), ctypes.POINTER(vp), vp]
    lib.gemm_run_host_batch.restype = ci
    for name, desc in (("gemm_route_create", RouteDesc), ("gemm_permute_create", PermuteDesc),
                       ("gemm_grouped_create", GroupedDesc), ("gemm_w4_create", W4Desc)):
        getattr(lib, name).argtypes = [ctypes.POINTER(vp), ctypes.POINTER(desc)]
    for name, pointers in (("gemm_route_run", 6), ("gemm_route_backward", 5),
                           ("gemm_permute_gather", 4), ("gemm_permute_combine", 4),
                           ("gemm_permute_combine_backward", 7), ("gemm_grouped_run", 5),
                           ("gemm_w4_run", 6)):
        # handle, operands, stream
        getattr(lib, name).argtypes = [vp] * (pointers + 2)
        getattr(lib, name).restype = ci
    lib.gemm_op_status.argtypes = [vp, vp]
    lib.gemm_op_destroy.argtypes = [vp]
    lib.gemm_op_workspace_bytes.argtypes = [vp]
    lib.gemm_op_workspace_bytes.restype = i64
    lib.gemm_op_plan_string.argtypes = [vp, ctypes.c_char_p, ctypes.c_size_t]
    lib.gemm_op_debug_set.argtypes = [vp, ci, ctypes.c_uint64]
    _lib = lib
    return lib


# ---------------------------------------------------------------- the C ABI, by name
def gemm_create(desc: GemmDesc) -> tuple[int, int | None]:
    h = ctypes.c_void_p()
    rc = load().gemm_create(ctypes.byref(h), ctypes.byref(desc))
    return rc, (h.value if rc == GEMM_OK else None)


def gemm_run(h: int, A: int, B: int, C: int | None, D: int, stream: int | None) -> int:
    return load().gemm_run(h, A, B, C, D, stream)


def gemm_run_mx(h: int, A: int, SA: int, B: int, SB: int, C: int | None, D: int,
                stream: int | None) -> int:
    return load().gemm_run_mx(h, A, SA, B, SB, C, D, stream)


def gemm_get_status(h: int, stream: int | None) -> int:
    return load().gemm_get_status(h, stream)


def gemm_destroy(h: int | None) -> int:
    return load().gemm_destroy(h)


def gemm_strerror(code: int) -> str:
    return load().gemm_strerror(code).decode()


def gemm_plan_string(h: int) -> str:
    buf = ctypes.create_string_buffer(1024)
    load().gemm_plan_string(h, buf, len(buf))
    return buf.value.decode()


def gemm_workspace_bytes(h: int) -> int:
    return load().gemm_workspace_bytes(h)


def gemm_raster_tile(t: int, num_pid_m: int, num_pid_n: int, group_m: int):
    pm, pn = ctypes.c_int64(), ctypes.c_int64()
    rc = load().gemm_raster_tile(t, num_pid_m, num_pid_n, group_m, ctypes.byref(pm),
                                 ctypes.byref(pn))
    return rc, pm.value, pn.value


def gemm_debug_set(h: int, flags: int, timeout_ns: int = 0) -> int:
    return load().gemm_debug_set(h, flags, timeout_ns)


def gemm_trace_set(h: int, dev_buf: int | None) -> int:
    return load().gemm_trace_set(h, dev_buf)


def gemm_pair_schedule(tiles_m: int, tiles_n: int, group_m: int, num_kb: int, ksub: int,
                       clusters: int, stream_k: int, cid: int) -> list[tuple]:
    """All units of cluster cid: (tile_row, tile_col, kb0, kb1, shared, part, slot).
    stream_k: 0 round-robin, 1 equal stream-K runs, 2 the kernel's default
    (chained runs where they apply)."""
    lib = load()
    n = lib.gemm_pair_schedule(tiles_m, tiles_n, group_m, num_kb, ksub, clusters, int(stream_k),
                               cid, 0, None)
    if n < 0:
        raise GemmError(n, "gemm_pair_schedule")
    out = (ctypes.c_int64 * 7)()
    units = []
    for i in range(n):
        rc = lib.gemm_pair_schedule(tiles_m, tiles_n, group_m, num_kb, ksub, clusters,
                                    int(stream_k), cid, i, out)
        if rc < 0:
            raise GemmError(rc, "gemm_pair_schedule")
        units.append(tuple(out))
    return units


def gemm_cta_schedule(tiles_m: int, tiles_n: int, group_m: int, num_kb: int, splits: int,
                      grid: int, stream_k: bool, cta: int) -> list[tuple]:
    """All units of CTA `cta` of the single-CTA kernel: (tile, tile_row, tile_col,
    kb0, kb1, pieces, piece, slot written, slot read for this piece)."""
    lib = load()
    n = lib.gemm_cta_schedule(tiles_m, tiles_n, group_m, num_kb, splits, grid, int(stream_k),
                              cta, 0, None)
    if n < 0:
        raise GemmError(n, "gemm_cta_schedule")
    out = (ctypes.c_int64 * 9)()
    units = []
    for i in range(n):
        rc = lib.gemm_cta_schedule(tiles_m, tiles_n, group_m, num_kb, splits, grid,
                                   int(stream_k), cta, i, out)
        if rc < 0:
            raise GemmError(rc, "gemm_cta_schedule")
        units.append(tuple(out))
    return units


def gemm_decode_ring(M: int, K: int, cpb: int) -> tuple[int, int, int]:
    """(stages, columns per stage, shared-memory bytes) of the decode kernel's
    bulk-copy ring; stages < 0 is an error code."""
    cps, smem = ctypes.c_int(), ctypes.c_int64()
    rc = load().gemm_decode_ring(M, K, cpb, ctypes.byref(cps), ctypes.byref(smem))
    return rc, cps.value, smem.value


def gemm_timing_enable(h: int, n: int) -> int:
    return load().gemm_timing_enable(h, n)


def gemm_timing_read(h: int, n: int) -> tuple[int, list[float]]:
    buf = (ctypes.c_float * max(n, 1))()
    rc = load().gemm_timing_read(h, buf, n)
    return rc, [buf[i] for i in range(max(rc, 0))]


def gemm_host_io_enable(h: int) -> int:
    return load().gemm_host_io_enable(h)


def gemm_run_host_batch(h: int, A: list, B: list, C: list | None, D: list,
                        stream: int | None) -> int:
    """D[i] = A[i]*B[i] + C[i] for lists of host addresses (C None or entries None: C = 0)."""
    n = len(A)
    arr = ctypes.c_void_p * max(n, 1)
    c_arr = None if C is None else arr(*C)
    return load().gemm_run_host_batch(h, n, arr(*A), arr(*B), c_arr, arr(*D), stream)


def gemm_run_splitk_noalloc(desc: GemmDesc, splits: int, A: int, B: int, C: int | None, D: int,
                            stream: int | None) -> int:
    """Split-K GEMM for callers that cannot allocate device memory (scratch is a
    static device array; see include/gemm.h)."""
    return load().gemm_run_splitk_noalloc(ctypes.byref(desc), splits, A, B, C, D, stream)


def gemm_noalloc_status(stream: int | None) -> int:
    """Status word left by the latest no-allocation call on the current device."""
    return load().gemm_noalloc_status(stream)


# ---------------------------------------------------------------- torch convenience
def _torch_type(dtype) -> int:
    import torch
    return {torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16, torch.float32: GEMM_F32,
            torch.int8: GEMM_I8, torch.int32: GEMM_I32, torch.float8_e4m3fn: GEMM_E4M3,
            torch.float8_e5m2: GEMM_E5M2}[dtype]


def layout_of(t) -> tuple[int, int]:
    """(layout, ld) of a 2-D tensor that is row- or column-major strided."""
    rows, cols = t.shape
    s0, s1 = t.stride()
    if s1 == 1 and (s0 >= max(cols, 1) or rows <= 1):
        return GEMM_ROW_MAJOR, max(s0, cols, 1)
    if s0 == 1 and (s1 >= max(rows, 1) or cols <= 1):
        return GEMM_COL_MAJOR, max(s1, rows, 1)
    raise ValueError(f"operand with strides {t.stride()} is neither row- nor column-major")


class Gemm:
    """A planned GEMM for fixed shapes, types and layouts."""

    def __init__(self, desc: GemmDesc):
        rc, h = gemm_create(desc)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_create")
        self.desc = desc
        self.handle = h

    @classmethod
    def like(cls, A, B, C, D, mx: bool = False) -> "Gemm":
        """Plan for the shapes, dtypes and strides of these tensors (mx: 8-bit
        float operands with block scales, run with run_mx)."""
        M, K = A.shape
        K2, N = B.shape
        assert K == K2 and tuple(D.shape) == (M, N)
        la, lda = layout_of(A)
        lb, ldb = layout_of(B)
        ld_, ldd = layout_of(D)
        if C is not None:
            assert tuple(C.shape) == (M, N)
            lc, ldc = layout_of(C)
            ct = _torch_type(C.dtype)
        else:
            lc, ldc, ct = GEMM_ROW_MAJOR, 0, 0
        ab = _torch_type(A.dtype)
        if mx:
            ab = {GEMM_E4M3: GEMM_MXE4M3, GEMM_E5M2: GEMM_MXE5M2}[ab]
        desc = GemmDesc(M, N, K, ab, ct, _torch_type(D.dtype), la, lb, lc, ld_,
                        lda, ldb, ldc, ldd)
        return cls(desc)

    def run(self, A, B, C, D, stream=None) -> None:
        """Enqueue D = A*B + C on stream (torch.cuda.Stream or raw handle)."""
        if stream is None:
            import torch
            stream = torch.cuda.current_stream()
        s = getattr(stream, "cuda_stream", stream)
        rc = gemm_run(self.handle, A.data_ptr(), B.data_ptr(),
                      None if C is None else C.data_ptr(), D.data_ptr(), s)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_run")

    def run_mx(self, A, SA, B, SB, C, D, stream=None) -> None:
        """Enqueue D = (A*SA)(B*SB) + C for a block-scaled handle (SA: M x ceil(K/32)
        and SB: N x ceil(K/32) uint8 E8M0 exponents on the device)."""
        if stream is None:
            import torch
            stream = torch.cuda.current_stream()
        s = getattr(stream, "cuda_stream", stream)
        rc = gemm_run_mx(self.handle, A.data_ptr(), SA.data_ptr(), B.data_ptr(), SB.data_ptr(),
                         None if C is None else C.data_ptr(), D.data_ptr(), s)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_run_mx")

    def run_ptrs(self, A: int, B: int, C: int | None, D: int, stream: int | None) -> None:
        rc = gemm_run(self.handle, A, B, C, D, stream)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_run")

    def host_io_enable(self) -> None:
        """Allocate the device copies and streams that run_host_batch uses."""
        rc = gemm_host_io_enable(self.handle)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_host_io_enable")

    def run_host_batch(self, As, Bs, Cs, Ds, stream=None) -> None:
        """Enqueue Ds[i] = As[i]*Bs[i] + Cs[i] for host (ideally pinned) tensors,
        each in the storage order of the description; copies overlap the GEMMs."""
        if stream is None:
            import torch
            stream = torch.cuda.current_stream()
        s = getattr(stream, "cuda_stream", stream)
        for t in list(As) + list(Bs) + list(Ds) + [c for c in (Cs or []) if c is not None]:
            if t.is_cuda:
                raise ValueError("run_host_batch takes host tensors")
        rc = gemm_run_host_batch(self.handle, [a.data_ptr() for a in As],
                                 [b.data_ptr() for b in Bs],
                                 None if Cs is None else
                                 [None if c is None else c.data_ptr() for c in Cs],
                                 [d.data_ptr() for d in Ds], s)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_run_host_batch")

    def status(self, stream=None) -> int:
        s = getattr(stream, "cuda_stream", stream)
        return gemm_get_status(self.handle, s)

    def plan(self) -> str:
        return gemm_plan_string(self.handle)

    def timing_enable(self, n: int) -> None:
        """Time the tensor-core kernel of the next n runs with CUDA events."""
        rc = gemm_timing_enable(self.handle, n)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_timing_enable")

    def timing_read(self, n: int) -> list[float]:
        """Kernel durations (ms) of the runs recorded since timing_enable."""
        rc, ms = gemm_timing_read(self.handle, n)
        if rc < 0:
            raise GemmError(rc, "gemm_timing_read")
        return ms

    def workspace_bytes(self) -> int:
        return gemm_workspace_bytes(self.handle)

    def close(self) -> None:
        if self.handle is not None:
            gemm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _after_current(stream, new) -> None:
    """Let `stream` (a torch stream, a raw handle, or None: the current one)
    wait for what the current stream has enqueued before it writes the tensor
    `new`, just made there: its filling, and the last use of its memory."""
    import torch
    if stream is None or not new.is_cuda:
        return
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), new.device)
    stream.wait_stream(torch.cuda.current_stream(new.device))


def matmul_add(A, B, C=None, out_dtype=None, D=None, stream=None):
    """D = A @ B + C through the library (plans a fresh handle each call).
    Without a D, a given `stream` waits for the current one: the new D's memory
    may still be in use there."""
    import torch
    if D is None:
        dt = out_dtype or (torch.int32 if A.dtype == torch.int8 else A.dtype)
        D = torch.empty((A.shape[0], B.shape[1]), dtype=dt, device=A.device)
        _after_current(stream, D)
    g = Gemm.like(A, B, C, D)
    try:
        g.run(A, B, C, D, stream)
    finally:
        g.close()
    return D


_EXPERTS = ("GroupedGemm", "Permute", "Route", "W4Gemm", "grouped_matmul", "pack_w4", "w4_matmul")


def __getattr__(name):
    # experts.py needs torch at import; this module does not
    if name in _EXPERTS:
        from . import experts
        return getattr(experts, name)
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
