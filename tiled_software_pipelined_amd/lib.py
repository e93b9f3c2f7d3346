"""Python binding of libtgemm (argument marshalling only).

Every step of the product runs in the HIP kernels of ``libtgemm.so``; this
module checks tensor arguments, caches plans and calls the C ABI of
``include/tgemm.h`` with raw device pointers and torch's current stream.
There is no CPU fallback: if the library is missing, importing this module
raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtgemm.so")

# dtype codes of the C ABI
F32, BF16, I8 = 0, 1, 2
F16 = 3  # an input of quantize_fp8 and orthogonalize; no plan's type
DTYPE_NAMES = {F32: "f32", BF16: "bf16", I8: "i8"}

OK = 0
ERRORS = {-1: "TGEMM_E_ARG", -2: "TGEMM_E_NULL", -3: "TGEMM_E_ALIGN", -4: "TGEMM_E_ARCH",
          -5: "TGEMM_E_VARIANT", -6: "TGEMM_E_HIP"}

# variant field values (include/tgemm.h)
KERNEL_AUTO, KERNEL_NAIVE, KERNEL_TILED = 0, 1, 2
LOADER_VGPR, LOADER_DIRECT = 1, 2
LDS_PLAIN, LDS_XOR, LDS_XOR_POISON = 1, 2, 3
ACCESS_WIDE, ACCESS_NARROW = 1, 2
FRAG_REUSE, FRAG_PER_MMA, FRAG_SLICE = 1, 2, 3
STORE_VECTOR, STORE_SCALAR = 1, 2
COPY_BURST, COPY_SPREAD, COPY_LATE = 1, 2, 3
C_STORES_AUTO, C_STORES_STREAM, C_STORES_PLAIN = 0, 1, 2
READ_B32, READ_B64, READ_B128, READ_TR, READ_KVEC = 1, 2, 3, 4, 5
LANES_BLOCKS, LANES_QUARTERS, LANES_ZORDER, LANES_ZQUARTERS = 1, 2, 3, 4
ORDER_ROW_MAJOR = -1


class Variant(ctypes.Structure):
    """Mirror of ``tgemm_variant``; zero fields mean "default"."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "kernel", "tile_m", "tile_n", "tile_k", "stages", "loader", "lds_layout", "access", "frag",
        "wg_group", "waves_m", "waves_n", "store", "copy_sched", "frag_read", "lane_map")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}

    def __repr__(self):
        return "Variant(%s)" % ", ".join("%s=%d" % kv for kv in self.as_dict().items() if kv[1])


class PlanInfo(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldc", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("variant", Variant), ("grid", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("lds_bytes", ctypes.c_int32),
                ("loads_per_stage", ctypes.c_int32), ("a_guarded", ctypes.c_int32),
                ("b_guarded", ctypes.c_int32), ("name", ctypes.c_char * 96), ("n_main", ctypes.c_int64),
                ("rem_name", ctypes.c_char * 96), ("packed_name", ctypes.c_char * 96),
                ("waves_per_simd", ctypes.c_int32)]


EXPORTS = ("gemm_plan", "gemm_plan_variant", "gemm_run", "gemm_destroy", "tgemm_last_error",
           "gemm_plan_get_info", "gemm_variant_count", "gemm_variant_get", "tgemm_version",
           "tgemm_lds_read_probe", "tgemm_mfma_rate_probe", "gemm_workspace_bytes", "gemm_run_ws",
           "gemm_kernel_occupancy", "gemm_clock_slots", "gemm_run_clocked", "gemm_run_noalloc",
           "tgemm_set_c_store_policy", "tgemm_fp8_quantize", "tgemm_fp8_gemm", "tgemm_fp8_gemm_kernel",
           "tgemm_fp8_linear_bytes", "tgemm_fp8_linear_forward", "tgemm_fp8_linear_backward",
           "tgemm_orthogonalize_workspace_bytes", "tgemm_orthogonalize", "tgemm_ffn_bytes", "tgemm_ffn_forward",
           "tgemm_ffn_backward", "tgemm_xent_bytes", "tgemm_xent_forward", "tgemm_xent_backward",
           "tgemm_clip_workspace_bytes", "tgemm_clip")


def _load():
    # Load torch first: its HIP runtime (libamdhip64, SONAME libamdhip64.so.7)
    # is then the one libtgemm binds to, so device memory, streams and the
    # kernel launches all belong to one runtime in this process.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError("libtgemm.so is not built (%s); run "
                          "`python -m tiled_software_pipelined_amd.build`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    lib.gemm_plan.argtypes = [i64, i64, i64, i32, i64, i64, i64]
    lib.gemm_plan.restype = vp
    lib.gemm_plan_variant.argtypes = [i64, i64, i64, i32, i64, i64, i64, ctypes.POINTER(Variant)]
    lib.gemm_plan_variant.restype = vp
    lib.gemm_run.argtypes = [vp, vp, vp, vp, vp]
    lib.gemm_run.restype = ctypes.c_int
    lib.gemm_destroy.argtypes = [vp]
    lib.gemm_destroy.restype = None
    lib.tgemm_last_error.argtypes = []
    lib.tgemm_last_error.restype = ctypes.c_char_p
    lib.gemm_plan_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
    lib.gemm_kernel_occupancy.argtypes = [vp, i32, ctypes.POINTER(i32)]
    lib.gemm_kernel_occupancy.restype = ctypes.c_int
    lib.gemm_clock_slots.argtypes = [vp]
    lib.gemm_clock_slots.restype = i64
    lib.gemm_run_clocked.argtypes = [vp, vp, vp, vp, vp, i64, vp]
    lib.gemm_run_clocked.restype = ctypes.c_int
    lib.gemm_plan_get_info.restype = ctypes.c_int
    lib.gemm_variant_count.argtypes = [i32]
    lib.gemm_variant_count.restype = ctypes.c_int
    lib.gemm_variant_get.argtypes = [i32, i32, ctypes.POINTER(Variant)]
    lib.gemm_variant_get.restype = ctypes.c_int
    lib.tgemm_version.argtypes = []
    lib.tgemm_version.restype = ctypes.c_char_p
    lib.tgemm_lds_read_probe.argtypes = [i32, i32, i32, i32, vp, vp]
    lib.tgemm_lds_read_probe.restype = ctypes.c_int
    lib.gemm_workspace_bytes.argtypes = [vp, vp, vp]
    lib.gemm_workspace_bytes.restype = i64
    lib.gemm_run_ws.argtypes = [vp, vp, vp, vp, vp, i64, vp]
    lib.gemm_run_ws.restype = ctypes.c_int
    lib.gemm_run_noalloc.argtypes = [vp, vp, vp, vp, vp]
    lib.gemm_run_noalloc.restype = ctypes.c_int
    lib.tgemm_mfma_rate_probe.argtypes = [i32, i32, i32, vp, vp, vp, vp]
    lib.tgemm_mfma_rate_probe.restype = ctypes.c_int
    lib.tgemm_set_c_store_policy.argtypes = [i32]
    lib.tgemm_set_c_store_policy.restype = ctypes.c_int
    lib.tgemm_fp8_quantize.argtypes = [i64, i64, i32, vp, i64, i32, i32, vp, i64, vp, i64, vp, i64, vp, i64, vp]
    lib.tgemm_fp8_quantize.restype = ctypes.c_int
    lib.tgemm_fp8_gemm.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, i32, vp, i64, vp, i64, vp, i64, vp]
    lib.tgemm_fp8_gemm.restype = ctypes.c_int
    lib.tgemm_fp8_gemm_kernel.argtypes = [i64, i64, i64, i64, i64, i32]
    lib.tgemm_fp8_gemm_kernel.restype = ctypes.c_char_p
    lib.tgemm_fp8_linear_bytes.argtypes = [i64, i64, i64, i32, ctypes.POINTER(i64)]
    lib.tgemm_fp8_linear_bytes.restype = ctypes.c_int
    lib.tgemm_fp8_linear_forward.argtypes = [i64, i64, i64, i32, vp, i64, i32, vp, i64, vp, i64, i32, vp, vp, vp]
    lib.tgemm_fp8_linear_forward.restype = ctypes.c_int
    lib.tgemm_fp8_linear_backward.argtypes = [i64, i64, i64, i32, vp, i64, i32, i32, vp, vp, i64, vp, i64, vp, vp]
    lib.tgemm_fp8_linear_backward.restype = ctypes.c_int
    f64 = ctypes.c_double
    lib.tgemm_orthogonalize_workspace_bytes.argtypes = [i64, i64, i64]
    lib.tgemm_orthogonalize_workspace_bytes.restype = i64
    lib.tgemm_orthogonalize.argtypes = [i64, i64, i64, i32, vp, i64, i64, vp, i64, i64, i32, ctypes.POINTER(f64), f64, vp,
                                        i64, vp]
    lib.tgemm_orthogonalize.restype = ctypes.c_int
    four = [i64, i64, i64, i64]
    lib.tgemm_ffn_bytes.argtypes = four + [i32, ctypes.POINTER(i64)]
    lib.tgemm_ffn_bytes.restype = ctypes.c_int
    lib.tgemm_ffn_forward.argtypes = four + [i32, i32] + [vp, i64] * 5 + [i32, vp, vp, vp]
    lib.tgemm_ffn_forward.restype = ctypes.c_int
    lib.tgemm_ffn_backward.argtypes = four + [i32, i32] + [vp, i64] * 5 + [i32, vp] + [vp, i64] * 4 + [vp, vp]
    lib.tgemm_ffn_backward.restype = ctypes.c_int
    lib.tgemm_xent_bytes.argtypes = [i64, i64, i64, i32, ctypes.POINTER(i64)]
    lib.tgemm_xent_bytes.restype = ctypes.c_int
    lib.tgemm_xent_forward.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, vp, i64, i32, i32, vp, vp, vp, vp]
    lib.tgemm_xent_forward.restype = ctypes.c_int
    lib.tgemm_xent_backward.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, vp, i32, vp, vp, i32, vp, i64, vp, i64, vp, vp]
    lib.tgemm_xent_backward.restype = ctypes.c_int
    lib.tgemm_clip_workspace_bytes.argtypes = [i64, vp]
    lib.tgemm_clip_workspace_bytes.restype = i64
    lib.tgemm_clip.argtypes = [i64, vp, vp, vp, vp, f64, f64, vp, vp, i64, vp]
    lib.tgemm_clip.restype = ctypes.c_int
    return lib


_lib = _load()


class TgemmError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("%s: %s" % (ERRORS.get(code, code), msg))
        self.code = code


def last_error() -> str:
    return _lib.tgemm_last_error().decode()


def set_c_store_policy(policy: int) -> int:
    """tgemm_set_c_store_policy: C_STORES_AUTO / _STREAM / _PLAIN for every
    later run in this process; returns the previous policy."""
    rc = _lib.tgemm_set_c_store_policy(int(policy))
    if rc < 0:
        raise TgemmError(rc, last_error())
    return rc


def version() -> str:
    return _lib.tgemm_version().decode()


LDS_PROBE_KINDS = ("ds_read_b32", "ds_read_b64", "ds_read_b128", "ds_read_b64_tr_b16")
LDS_PROBE_PATTERNS = ("linear", "swizzled")
LDS_PROBE_THREADS = 256


def lds_read_probe(kind: int, pattern: int, reps: int, out):
    """Launch the LDS read-path probe on the current stream: one workgroup
    per 256 entries of ``out`` (a uint32-compatible int32 GPU tensor)."""
    import torch
    if not out.is_cuda or out.dtype != torch.int32 or out.numel() % LDS_PROBE_THREADS or not out.is_contiguous():
        raise ValueError("out must be a contiguous int32 GPU tensor of 256 * workgroups entries")
    wgs = out.numel() // LDS_PROBE_THREADS
    stream = torch.cuda.current_stream(out.device).cuda_stream
    with torch.cuda.device(out.device):
        rc = _lib.tgemm_lds_read_probe(kind, pattern, reps, wgs, out.data_ptr(), stream)
    if rc != OK:
        raise TgemmError(rc, "tgemm_lds_read_probe(kind=%d, pattern=%d, reps=%d, workgroups=%d)" % (
            kind, pattern, reps, wgs))
    return out


# kinds of tgemm_mfma_rate_probe: the bare bf16 / int8 matrix instruction, the
# fp32 FMA, and the bf16 matrix stream of the default GEMM kernel with its LDS
# fragment reads, then also its direct global->LDS copies
RATE_PROBE_KINDS = ("bf16", "i8", "f32", "bf16_lds", "bf16_lds_dma")
RATE_PROBE_THREADS = 256
RATE_PROBE_OPS_PER_INST = {"bf16": 2 * 32 * 32 * 16, "i8": 2 * 32 * 32 * 32, "f32": 2 * 64,
                           "bf16_lds": 2 * 32 * 32 * 16, "bf16_lds_dma": 2 * 32 * 32 * 16}


def mfma_rate_probe(kind: int, reps: int, operands, out, clocks):
    """Launch the matrix-core rate probe on the current stream.

    operands: contiguous GPU tensor of workgroups * 256 * 8 16-byte entries
    (any dtype; its bytes are the operand registers), out: int32 GPU tensor
    of workgroups * 256 entries, clocks: int64 GPU tensor of 2 * workgroups
    entries (shader-clock and real-time ticks per workgroup)."""
    import torch
    if not out.is_cuda or out.dtype != torch.int32 or out.numel() % RATE_PROBE_THREADS or not out.is_contiguous():
        raise ValueError("out must be a contiguous int32 GPU tensor of 256 * workgroups entries")
    wgs = out.numel() // RATE_PROBE_THREADS
    if (not operands.is_cuda or not operands.is_contiguous()
            or operands.numel() * operands.element_size() != wgs * RATE_PROBE_THREADS * 8 * 16):
        raise ValueError("operands must be a contiguous GPU tensor of workgroups * 256 * 8 * 16 bytes")
    if not clocks.is_cuda or clocks.dtype != torch.int64 or clocks.numel() != 2 * wgs or not clocks.is_contiguous():
        raise ValueError("clocks must be a contiguous int64 GPU tensor of 2 * workgroups entries")
    stream = torch.cuda.current_stream(out.device).cuda_stream
    with torch.cuda.device(out.device):
        rc = _lib.tgemm_mfma_rate_probe(kind, reps, wgs, operands.data_ptr(), out.data_ptr(), clocks.data_ptr(),
                                        stream)
    if rc != OK:
        raise TgemmError(rc, "tgemm_mfma_rate_probe(kind=%d, reps=%d, workgroups=%d)" % (kind, reps, wgs))
    return out, clocks


def variants(dtype: int):
    """The variants compiled into the library for a dtype code."""
    out = []
    for i in range(_lib.gemm_variant_count(dtype)):
        v = Variant()
        if _lib.gemm_variant_get(dtype, i, ctypes.byref(v)) != OK:
            raise TgemmError(-1, last_error())
        out.append(v)
    return out


class Plan:
    """A ``tgemm_plan`` (host metadata only; never touches the GPU)."""

    def __init__(self, M, N, K, dtype, lda=None, ldb=None, ldc=None, variant: Variant | None = None):
        lda = K if lda is None else lda
        ldb = N if ldb is None else ldb
        ldc = N if ldc is None else ldc
        self.M, self.N, self.K, self.dtype = int(M), int(N), int(K), int(dtype)
        self.lda, self.ldb, self.ldc = int(lda), int(ldb), int(ldc)
        if variant is None:
            h = _lib.gemm_plan(M, N, K, dtype, lda, ldb, ldc)
        else:
            h = _lib.gemm_plan_variant(M, N, K, dtype, lda, ldb, ldc, ctypes.byref(variant))
        if not h:
            raise TgemmError(-1, last_error())
        self._h = h

    def info(self) -> PlanInfo:
        info = PlanInfo()
        rc = _lib.gemm_plan_get_info(self._h, ctypes.byref(info))
        if rc != OK:
            raise TgemmError(rc, last_error())
        return info

    @property
    def name(self) -> str:
        return self.info().name.decode()

    def kernel_for(self, A: int, B: int, workspace: bool = True) -> str:
        """Name of the main kernel that runs for operands at these addresses:
        the repacked plan's when the binding would use a workspace."""
        info = self.info()
        if workspace and self.workspace_bytes(A, B) > 0:
            return info.packed_name.decode()
        return info.name.decode()

    def occupancy(self, packed: bool = False) -> int:
        """Workgroups of the main kernel (packed: the repacked plan's) that one
        compute unit holds at once, from the HIP runtime's calculator (GPU only)."""
        n = ctypes.c_int32(0)
        rc = _lib.gemm_kernel_occupancy(self._h, 1 if packed else 0, ctypes.byref(n))
        if rc != OK:
            raise TgemmError(rc, last_error())
        return int(n.value)

    def clock_slots(self) -> int:
        """Values of the clock buffer gemm_run_clocked needs (0: nothing to clock)."""
        return int(_lib.gemm_clock_slots(self._h))

    def run_clocked_ptr(self, A: int, B: int, C: int, clocks: int, clocks_len: int, stream: int = 0) -> None:
        """gemm_run_clocked on raw device pointers."""
        rc = _lib.gemm_run_clocked(self._h, ctypes.c_void_p(A), ctypes.c_void_p(B), ctypes.c_void_p(C),
                                   ctypes.c_void_p(clocks), clocks_len, ctypes.c_void_p(stream))
        if rc != OK:
            raise TgemmError(rc, last_error())

    def run_ptr(self, A: int, B: int, C: int, stream: int = 0) -> None:
        """Enqueue on raw device pointers (the caller keeps the buffers alive)."""
        rc = _lib.gemm_run(self._h, ctypes.c_void_p(A), ctypes.c_void_p(B), ctypes.c_void_p(C),
                           ctypes.c_void_p(stream))
        if rc != OK:
            raise TgemmError(rc, last_error())

    def workspace_bytes(self, A: int, B: int) -> int:
        """Workspace bytes gemm_run_ws uses to repack misaligned operands at these
        addresses (0 where the plan's kernel reads them in place)."""
        return int(_lib.gemm_workspace_bytes(self._h, ctypes.c_void_p(A), ctypes.c_void_p(B)))

    def run_ws_ptr(self, A: int, B: int, C: int, ws: int, ws_bytes: int, stream: int = 0) -> None:
        """gemm_run_ws on raw device pointers (the caller keeps the buffers alive)."""
        rc = _lib.gemm_run_ws(self._h, ctypes.c_void_p(A), ctypes.c_void_p(B), ctypes.c_void_p(C),
                              ctypes.c_void_p(ws), ws_bytes, ctypes.c_void_p(stream))
        if rc != OK:
            raise TgemmError(rc, last_error())

    def run_noalloc_ptr(self, A: int, B: int, C: int, stream: int = 0) -> None:
        """gemm_run_noalloc on raw device pointers: repacks misaligned operands
        into the library's fixed device array (no allocation)."""
        rc = _lib.gemm_run_noalloc(self._h, ctypes.c_void_p(A), ctypes.c_void_p(B), ctypes.c_void_p(C),
                                   ctypes.c_void_p(stream))
        if rc != OK:
            raise TgemmError(rc, last_error())

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:  # module globals are gone at interpreter exit
            _lib.gemm_destroy(h)
            self._h = None


_cache: dict = {}
_cache_lock = threading.Lock()


def _torch_dtype_code(t):
    import torch
    m = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8}
    if t.dtype not in m:
        raise TypeError("unsupported dtype %s (float32, bfloat16, int8)" % t.dtype)
    return m[t.dtype]


def _ld(t, name):
    """Leading dimension (row stride in elements) of a row-major 2-D tensor.

    Rows must not overlap: a row stride below the row length (a broadcast or
    otherwise aliased view) would make the kernels read past the rows the
    tensor's storage holds, so it is rejected."""
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must be row-major with unit column stride" % name)
    if t.shape[0] > 1 and t.shape[1] > 0 and t.stride(0) < t.shape[1]:
        raise ValueError("%s has overlapping rows (row stride %d < %d columns); pass a contiguous copy"
                         % (name, t.stride(0), t.shape[1]))
    return max(int(t.stride(0)), int(t.shape[1]), 1) if t.shape[0] > 1 else max(int(t.shape[1]), 1)


CLOCK_VALUES = 6  # TGEMM_CLOCK_VALUES: values per workgroup written by gemm_run_clocked
NOALLOC_MAX_BYTES = 64 << 20  # TGEMM_NOALLOC_MAX_BYTES: the fixed workspace of gemm_run_noalloc


def clock_ghz(clocks) -> float:
    """Mean shader clock (GHz) of clocked runs: a host array of CLOCK_VALUES
    values per workgroup as gemm_run_clocked writes them (any number of runs
    stacked); shader ticks over 100 MHz real-time ticks from start to end,
    summed over workgroups."""
    import numpy as np
    c = np.asarray(clocks, dtype=np.uint64).reshape(-1, CLOCK_VALUES).astype(np.float64)
    shader = float((c[:, 4] - c[:, 0]).sum())
    real = float((c[:, 5] - c[:, 1]).sum())
    if real <= 0:
        raise ValueError("no real-time ticks recorded")
    return shader / real * 0.1


def clock_split_us(clocks):
    """Per workgroup of clocked runs: (K-loop microseconds, C write-back
    microseconds) from the real-time ticks (100 MHz), as two arrays."""
    import numpy as np
    c = np.asarray(clocks, dtype=np.uint64).reshape(-1, CLOCK_VALUES).astype(np.int64)
    return (c[:, 3] - c[:, 1]) * 0.01, (c[:, 5] - c[:, 3]) * 0.01


def plan_for(M, N, K, dtype, lda, ldb, ldc, variant: Variant | None = None) -> Plan:
    key = (M, N, K, dtype, lda, ldb, ldc, None if variant is None else tuple(variant.as_dict().items()))
    with _cache_lock:
        p = _cache.get(key)
        if p is None:
            p = Plan(M, N, K, dtype, lda, ldb, ldc, variant)
            _cache[key] = p
    return p


def gemm(A, B, out=None, variant: Variant | None = None, workspace: bool = True):
    """C = A @ B on the current CUDA/HIP stream.

    A: (M, K), B: (K, N) torch tensors on the GPU, both float32, both bfloat16
    or both int8, row-major (row stride may exceed the row length).  Returns
    C (M, N): float32 for float32/bfloat16 inputs, int32 for int8 inputs.
    ``out`` may be a preallocated row-major C (its row stride is used as ldc).
    Operands whose rows are not 16-byte aligned are read in place by the
    matrix-core kernels.  With ``workspace`` (default plans only), where the
    plan's kernel needs aligned rows (fp32) they are repacked into a device
    buffer taken from torch's allocator on the current stream (gemm_run_ws);
    otherwise a kernel that reads such rows in place runs (gemm_run).
    """
    import torch
    if not (A.is_cuda and B.is_cuda):
        raise ValueError("A and B must be GPU tensors")
    if A.device != B.device:
        raise ValueError("A and B must be on the same device (%s, %s)" % (A.device, B.device))
    if A.dtype != B.dtype:
        raise TypeError("A and B must have the same dtype")
    code = _torch_dtype_code(A)
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, K2))
    out_dtype = torch.int32 if code == I8 else torch.float32
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    elif out.dtype != out_dtype or tuple(out.shape) != (M, N) or out.device != A.device:
        raise ValueError("out must be a %s tensor of shape (%d, %d) on %s" % (out_dtype, M, N, A.device))
    lda, ldb, ldc = _ld(A, "A"), _ld(B, "B"), _ld(out, "out")
    p = plan_for(M, N, K, code, lda, ldb, ldc, variant)
    stream = torch.cuda.current_stream(A.device).cuda_stream
    with torch.cuda.device(A.device):
        need = p.workspace_bytes(A.data_ptr(), B.data_ptr()) if workspace and variant is None else 0
        if need > 0:
            # stream-ordered: the block returns to torch's pool for this
            # stream when `ws` is dropped, after the work queued here
            ws = torch.empty(need + 256, dtype=torch.uint8, device=A.device)
            base = (ws.data_ptr() + 255) // 256 * 256
            p.run_ws_ptr(A.data_ptr(), B.data_ptr(), out.data_ptr(), base, need, stream)
        else:
            p.run_ptr(A.data_ptr(), B.data_ptr(), out.data_ptr(), stream)
    return out


# ---- 8-bit floating point products with block scales --------------------------

import torch  # noqa: E402  (_load has imported it)
from torch.autograd import forward_ad  # noqa: E402

FP8_BLOCK = 128  # elements of a row that share a scale
E4M3, E5M2 = 0, 1
BLOCKS = {"row": 0, "square": 1}
KEEP_X, KEEP_W, KEEP_POWERS = 1, 2, 8
_FP8_CODES = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}
_REAL_CODES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}

# Small calls are bound by their way here: the raw handle of the current
# stream costs 0.1 us where torch.cuda.current_stream makes an object in 2 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(device, fn, *args):
    """fn(*args, current stream of device), on that device; raises on an error code."""
    index = device.index
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != OK:
        raise TgemmError(rc, last_error())


def _fp8_code(dtype):
    code = _FP8_CODES.get(dtype)
    if code is None:
        raise TypeError("unsupported 8-bit type %s (float8_e4m3fn, float8_e5m2)" % dtype)
    return code


def _real_code(t, name):
    code = _REAL_CODES.get(t.dtype)
    if code is None:
        raise TypeError("%s has unsupported dtype %s (float32, bfloat16, float16)" % (name, t.dtype))
    return code


def _image(rows, cols, dtype, device):
    """An empty quantised operand: values, their row stride, scales, theirs.
    Rows start where a product reads them fastest: long ones on 128-byte lines
    (4096x4096 with K = 4099: 73 us back to back, 54 so), short ones and those of
    the scales on 16-byte boundaries."""
    ldq = -(-cols // 128) * 128 if cols >= 1024 else -(-cols // 16) * 16
    lds = -(-rows // 16) * 16
    q = torch.empty((rows, ldq), dtype=dtype, device=device)
    s = torch.empty((-(-cols // FP8_BLOCK), lds), dtype=torch.float8_e8m0fnu, device=device)
    return q if ldq == cols else q[:, :cols], ldq, s if lds == rows else s[:, :rows], lds


def quantize_fp8(X, dtype=torch.float8_e4m3fn, block="row", transpose=False):
    """(Q, S), the 8-bit image of X with a power-of-two scale for each 128
    elements of a row; with ``transpose`` (Q, S, Qt, St), also that of X
    transposed.

    X: (rows, cols) float32, bfloat16 or float16 on the GPU, row-major (row
    stride may exceed the row length).  Q: (rows, cols) of ``dtype``
    (float8_e4m3fn or float8_e5m2); S: (ceil(cols / 128), rows)
    float8_e8m0fnu; X[r, c] is near Q[r, c] * S[c // 128, r].  Both are views of
    padded rows where a product reads those faster.  With block
    "square" one scale serves each 128 x 128 block of X, and Qt is Q
    transposed (weights, whose two images then hold the same values); with
    "row" each image's scales follow its own rows.  A scale is the least power
    of two (at least 2^-127) that keeps its block's finite values within the
    type's range.  NaN stays NaN, and an infinity becomes the type's infinity
    or NaN.  Runs on the current stream.  Not differentiable: the images carry no
    gradient of an X that requires one (:func:`linear_fp8` does).
    """
    fmt = _fp8_code(dtype)
    if block not in BLOCKS:
        raise ValueError("block must be \"row\" or \"square\", got %r" % (block,))
    if not X.is_cuda:
        raise ValueError("X must be a GPU tensor")
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    code, device = _real_code(X, "X"), X.device
    rows, cols = X.shape
    ldx = cols if X.is_contiguous() else _ld(X, "X")
    q, ldq, s, lds = _image(rows, cols, dtype, device)
    if not transpose:
        _call(device, _lib.tgemm_fp8_quantize, rows, cols, code, X.data_ptr(), ldx, fmt, BLOCKS[block], q.data_ptr(), ldq,
              s.data_ptr(), lds, None, 0, None, 0)
        return q, s
    qt, ldqt, st, ldst = _image(cols, rows, dtype, device)
    _call(device, _lib.tgemm_fp8_quantize, rows, cols, code, X.data_ptr(), ldx, fmt, BLOCKS[block], q.data_ptr(), ldq,
          s.data_ptr(), lds, qt.data_ptr(), ldqt, st.data_ptr(), ldst)
    return q, s, qt, st


def _scales(s, rows, cols, device, name):
    """Row stride of a scale table (ceil(cols / 128), rows) that a product may read."""
    if s.dtype is not torch.float8_e8m0fnu and s.dtype is not torch.uint8:
        raise TypeError("%s must be float8_e8m0fnu (or its bytes as uint8), got %s" % (name, s.dtype))
    blocks = -(-cols // FP8_BLOCK)
    if tuple(s.shape) != (blocks, rows) or s.device != device:
        raise ValueError("%s must be of shape (%d, %d) on %s, got %s on %s" % (
            name, blocks, rows, device, tuple(s.shape), s.device))
    if rows % 4 == 0 and s.is_contiguous() and s.data_ptr() % 4 == 0:
        return rows
    if blocks == 0 or rows == 0:
        return -(-max(rows, 1) // 4) * 4
    if rows > 1 and s.stride(1) != 1:
        raise ValueError("%s must have unit stride along its rows" % name)
    ld = s.stride(0) if blocks > 1 else -(-rows // 4) * 4
    if ld < rows or ld % 4 or s.data_ptr() % 4:
        raise ValueError("%s needs rows on 4-byte boundaries (row stride %d for %d rows): quantize_fp8 lays them out so"
                         % (name, ld, rows))
    # the product reads whole 4-byte words of the last row
    end = s.storage_offset() + (blocks - 1) * ld + -(-rows // 4) * 4
    if end > s.untyped_storage().nbytes():
        raise ValueError("%s must be readable up to %d rows (a multiple of 4): quantize_fp8 lays tables out so"
                         % (name, -(-rows // 4) * 4))
    return ld


def gemm_fp8(A, SA, B, SB, out=None):
    """C = A @ B^T of two quantised operands, on the current stream.

    A: (M, K), B: (N, K), float8_e4m3fn or float8_e5m2 each, row-major (row
    stride may exceed the row length, rows may start at any byte), with their
    scale tables SA (ceil(K / 128), M) and SB (ceil(K / 128), N) as
    :func:`quantize_fp8` returns them.  Returns C (M, N) bfloat16, rounded
    once from the matrix cores' float sums; ``out`` may be a preallocated
    row-major C.  Not differentiable: C carries no gradient.
    """
    device = A.device
    if not (A.is_cuda and B.is_cuda):
        raise ValueError("A and B must be GPU tensors")
    if device != B.device:
        raise ValueError("A and B must be on the same device (%s, %s)" % (device, B.device))
    fa, fb = _fp8_code(A.dtype), _fp8_code(B.dtype)
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    (M, K), (N, K2) = A.shape, B.shape
    lda = K if A.is_contiguous() else _ld(A, "A")
    ldb = K2 if B.is_contiguous() else _ld(B, "B")
    if K != K2:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, K2))
    ldsa, ldsb = _scales(SA, M, K, device, "SA"), _scales(SB, N, K, device, "SB")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=device)
        ldc = N
    elif out.dtype != torch.bfloat16 or tuple(out.shape) != (M, N) or out.device != device:
        raise ValueError("out must be a bfloat16 tensor of shape (%d, %d) on %s" % (M, N, device))
    else:
        ldc = _ld(out, "out")
    _call(device, _lib.tgemm_fp8_gemm, M, N, K, fa, A.data_ptr(), lda, SA.data_ptr(), ldsa, fb, B.data_ptr(), ldb,
          SB.data_ptr(), ldsb, out.data_ptr(), ldc)
    return out


def gemm_fp8_kernel(M, N, K, lda=None, ldb=None, piece=0) -> str:
    """Name of the kernel :func:`gemm_fp8` launches first for these sizes, or
    (piece 1) for the columns or rows it splits off; "" where there is none."""
    return _lib.tgemm_fp8_gemm_kernel(M, N, K, K if lda is None else lda, K if ldb is None else ldb, piece).decode()


def _rows(t):
    """t as a row-major matrix whose rows do not overlap: itself, or a copy."""
    ok = (t.shape[1] <= 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1])
    return t if ok else t.contiguous()


@functools.lru_cache(maxsize=512)
def _linear_bytes(M, N, K, keep):
    """Bytes of (saved, forward's scratch, backward's scratch), at least one each."""
    n = (ctypes.c_int64 * 3)()
    rc = _lib.tgemm_fp8_linear_bytes(M, N, K, keep, n)
    if rc != OK:
        raise TgemmError(rc, last_error())
    return tuple(max(v, 1) for v in n)


def _linear_forward(x, w, keep):
    """y of shape (..., N) in x's dtype, and the buffer for the backward pass.
    (torch's allocator gives stream-ordered blocks on 512-byte boundaries: a
    scratch that is dropped here is reused after the work queued on it.)"""
    device, K, N = x.device, x.shape[-1], w.shape[0]
    M = math.prod(x.shape[:-1])
    x2, w2 = _rows(x.reshape(M, K)), _rows(w)
    sizes = _linear_bytes(M, N, K, keep)
    # kept for the backward pass: one byte an element of x and of w
    saved = torch.empty(sizes[0], dtype=torch.uint8, device=device)
    scratch = torch.empty(sizes[1], dtype=torch.uint8, device=device)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=device)
    _call(device, _lib.tgemm_fp8_linear_forward, M, N, K, _real_code(x, "x"), x2.data_ptr(), _ld(x2, "x"),
          _real_code(w, "w"), w2.data_ptr(), _ld(w2, "w"), y.data_ptr(), N, keep, saved.data_ptr(), scratch.data_ptr())
    y = y.reshape(x.shape[:-1] + (N,)) if x.dim() != 2 else y
    return y if x.dtype == torch.bfloat16 else y.to(x.dtype), saved


class _LinearFp8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, grad_dtype):
        keep = (KEEP_X if ctx.needs_input_grad[0] else 0) | (KEEP_W if ctx.needs_input_grad[1] else 0)
        y, saved = _linear_forward(x, w, keep)
        ctx.save_for_backward(saved)
        ctx.args = math.prod(x.shape[:-1]), w.shape[0], x.shape[-1], keep, grad_dtype, x.shape, x.dtype, w.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        (saved,) = ctx.saved_tensors
        M, N, K, keep, grad_dtype, x_shape, x_dtype, w_dtype = ctx.args
        device = gy.device
        g = _rows(gy.reshape(M, N))  # a broadcast gradient (of a sum, say) has no rows of its own
        scratch = torch.empty(_linear_bytes(M, N, K, keep)[2], dtype=torch.uint8, device=device)
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=device) if keep & KEEP_X else None
        dw = torch.empty((N, K), dtype=torch.bfloat16, device=device) if keep & KEEP_W else None
        _call(device, _lib.tgemm_fp8_linear_backward, M, N, K, _real_code(g, "gradient"), g.data_ptr(), _ld(g, "gradient"),
              _fp8_code(grad_dtype), keep, saved.data_ptr(), None if dx is None else dx.data_ptr(), K,
              None if dw is None else dw.data_ptr(), K, scratch.data_ptr())
        if dx is not None:
            dx = dx.reshape(x_shape).to(x_dtype)
        return dx, None if dw is None else dw.to(w_dtype), None


def linear_fp8(x, w, grad_dtype=torch.float8_e4m3fn):
    """y = x @ w^T with x and w quantised to float8_e4m3fn, differentiable.

    x: (..., K), w: (N, K), each float32, bfloat16 or float16.  x is
    quantised with a scale for each 128 elements of a row, w for each 128 x
    128 block; y has x's dtype (the product itself is rounded to bfloat16).
    The backward pass quantises the gradient of y to ``grad_dtype``
    (float8_e4m3fn or float8_e5m2), along its rows for x's gradient and along
    its columns for w's, and takes both products from the 8-bit images kept by
    the forward pass: dx = g w, dw = g^T x.  Rounding is passed straight
    through.  Gradients are rounded to bfloat16 like y and have their inputs'
    dtypes; second derivatives and forward-mode ones are refused.  A weight that does not change between calls is better quantised
    once (:func:`quantize_fp8`, then :func:`gemm_fp8`).  To capture a training
    step into a graph, capture torch.autograd.grad, or make sure that no eager
    graph of the same leaves is alive: torch's nodes that accumulate into
    ``.grad`` stay on the stream of the first one.
    """
    _fp8_code(grad_dtype)
    if not (x.is_cuda and w.is_cuda) or x.device != w.device:
        raise ValueError("x and w must be on one GPU (%s, %s)" % (x.device, w.device))
    if x.dim() < 1 or w.dim() != 2 or x.shape[-1] != w.shape[1]:
        raise ValueError("x %s and w %s do not make x @ w^T" % (tuple(x.shape), tuple(w.shape)))
    # straight to the kernels where nothing can want a derivative: a dual tensor
    # of torch.autograd.forward_ad has a tangent and no requires_grad, and the
    # autograd function refuses it (it has no forward-mode rule)
    if forward_ad._current_level < 0 and not (torch.is_grad_enabled() and (x.requires_grad or w.requires_grad)):
        return _linear_forward(x, w, 0)[0]
    return _LinearFp8.apply(x, w, grad_dtype)


# ---- orthogonalised update ------------------------------------------------------

ORTHOGONALIZE_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _matrices(t):
    """(batch, rows, cols), row stride and batch stride of a tensor whose last
    two axes are row-major matrices that do not overlap and whose leading axes
    step evenly; None otherwise."""
    rows, cols = t.shape[-2:]
    batch = math.prod(t.shape[:-2])
    if t.numel() == 0:
        return (batch, rows, cols), max(cols, 1), rows * max(cols, 1)
    if cols > 1 and t.stride(-1) != 1 or rows > 1 and t.stride(-2) < cols:
        return None
    ld = t.stride(-2) if rows > 1 else cols
    step, span = None, 1  # stride of one matrix, matrices counted so far
    for n, s in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != step * span:
            return None
        span *= n
    if step is None:
        step = (rows - 1) * ld + cols
    elif step < (rows - 1) * ld + cols:
        return None
    return (batch, rows, cols), ld, step


def _newton_schulz(steps, coefficients):
    """The number of steps and their coefficients as the library takes them:
    three doubles for each of 1 to 64 steps (a 32-bit count reads no others)."""
    if not 1 <= steps <= 64 or steps != int(steps):
        raise TgemmError(-1, "steps=%s (1 .. 64)" % (steps,))
    steps, flat = int(steps), list(coefficients)
    if len(flat) == 3 and not hasattr(flat[0], "__len__"):
        flat = flat * steps
    elif len(flat) != steps or any(len(c) != 3 for c in flat):
        raise ValueError("coefficients must be (a, b, c) or one such triple for each of the %d steps" % steps)
    else:
        flat = [v for c in flat for v in c]
    return steps, (ctypes.c_double * (3 * steps))(*map(float, flat))


def orthogonalize(G, steps=5, coefficients=ORTHOGONALIZE_COEFFICIENTS, eps=1e-7, out=None):
    """The orthogonalised update of the Muon optimiser: G with its singular
    values brought near one by ``steps`` (1 to 64) Newton-Schulz steps.

    G: (..., rows, cols) float32, bfloat16 or float16 on the GPU, each matrix
    by itself.  X = G / (|G| + eps) (Frobenius norm), then for each step
    X <- a X + (b A + c A^2) X with A = X X^T (on the shorter side).
    ``coefficients``: (a, b, c), or one such triple for each step; refused
    where they would let singular values leave the range the kernels hold
    (3.5).  Returns bfloat16 of G's shape, rounded once; ``out`` may be a
    preallocated bfloat16 tensor of evenly spaced row-major matrices (G itself
    included).  The workspace comes from torch's allocator on the current
    stream.  Not differentiable: the result carries no gradient of G.
    """
    if not G.is_cuda:
        raise ValueError("G must be a GPU tensor")
    code = _real_code(G, "G")
    if G.dim() < 2:
        raise ValueError("G must have at least 2 dimensions")
    steps, coef = _newton_schulz(steps, coefficients)
    if out is None:
        out = torch.empty(G.shape, dtype=torch.bfloat16, device=G.device)
    elif out.dtype != torch.bfloat16 or out.shape != G.shape or out.device != G.device:
        raise ValueError("out must be a bfloat16 tensor of shape %s on %s" % (tuple(G.shape), G.device))
    place = _matrices(out)
    if place is None:
        raise ValueError("out must hold evenly spaced row-major matrices (shape %s, strides %s)" % (
            tuple(out.shape), out.stride()))
    if _matrices(G) is None:
        G = G.contiguous()
    (batch, rows, cols), ldg, stride_g = _matrices(G)
    _, ldo, stride_o = place
    need = _lib.tgemm_orthogonalize_workspace_bytes(batch, rows, cols)
    if need < 0:
        raise ValueError("G of shape %s is out of range (2^20 rows and columns, 2^16 matrices)" % (tuple(G.shape),))
    # stream-ordered: the block returns to torch's pool for this stream when
    # `ws` is dropped, after the work queued here; the pool's blocks start on
    # 512-byte boundaries
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=G.device)
    _call(G.device, _lib.tgemm_orthogonalize, batch, rows, cols, code, G.data_ptr(), ldg, stride_g, out.data_ptr(), ldo,
          stride_o, steps, coef, float(eps), ws.data_ptr(), need)
    return out


# ---- products of a training step with fused ends --------------------------------

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}
FFN_X, FFN_GATE, FFN_UP, FFN_DOWN = 1, 2, 4, 8
MOST_STRIDE = 1 << 22  # elements from a row to the next
_HALF_CODES = {torch.bfloat16: BF16, torch.float16: F16}


def _half_code(tensors, names):
    """The type code of tensors that are all bfloat16 or all float16 on one GPU."""
    first = tensors[0]
    dtype, device = first.dtype, first.device
    code = _HALF_CODES.get(dtype)
    if code is None:
        raise TypeError("%s has unsupported dtype %s (bfloat16, float16)" % (names[0], dtype))
    for t, name in zip(tensors, names):
        if t.dtype is not dtype:
            raise TypeError("%s must have %s's dtype %s, got %s" % (name, names[0], dtype, t.dtype))
        if t.device != device or not t.is_cuda:
            raise ValueError("%s must be on one GPU (%s, got %s)" % (" and ".join(names), device, t.device))
    return code


def _read(t):
    """(row-major matrix that the kernels may read, its row stride): t, or a copy."""
    if t.is_contiguous() and t.shape[1] <= MOST_STRIDE:
        return t, t.shape[1]
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and not t.shape[1] <= t.stride(0) <= MOST_STRIDE:
        t = t.contiguous()
        return t, t.shape[1]
    return t, t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _wants_derivative(tensors):
    """Whether a call may be differentiated (a dual tensor of forward-mode
    differentiation counts: the autograd functions refuse it)."""
    return forward_ad._current_level >= 0 or torch.is_grad_enabled() and any(t.requires_grad for t in tensors)


@functools.lru_cache(maxsize=512)
def _ffn_bytes(M, K, F, N, keep):
    n = (ctypes.c_int64 * 3)()
    rc = _lib.tgemm_ffn_bytes(M, K, F, N, keep, n)
    if rc != OK:
        raise TgemmError(rc, last_error())
    return tuple(max(v, 1) for v in n)


def _ffn_call(x, w_gate, w_up, w_down):
    """Sizes (M, K, F, N), and the operands with their row strides."""
    K, (N, F) = x.shape[-1], w_down.shape
    M = x.numel() // K if K else math.prod(x.shape[:-1])
    return (M, K, F, N), (*_read(x if x.dim() == 2 else x.reshape(M, K)), *_read(w_gate), *_read(w_up), *_read(w_down))


def _pointers(operands):
    """The tensors of (tensor, stride, tensor, stride, ..) as their addresses."""
    return [v if type(v) is int else v.data_ptr() for v in operands]


def _ffn_forward(x, sizes, operands, code, act, keep):
    """y of shape (..., N), and the buffer for the backward pass (None where keep is 0)."""
    device, N = x.device, sizes[3]
    room = _ffn_bytes(*sizes, keep)
    saved = torch.empty(room[0], dtype=torch.uint8, device=device) if keep else None
    scratch = torch.empty(room[1], dtype=torch.uint8, device=device)
    y = torch.empty(x.shape[:-1] + (N,), dtype=x.dtype, device=device)
    _call(device, _lib.tgemm_ffn_forward, *sizes, code, act, *_pointers(operands), y.data_ptr(), N, keep,
          saved.data_ptr() if keep else None, scratch.data_ptr())
    return y, saved


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, code, act):
        needs = ctx.needs_input_grad
        keep = needs[0] * FFN_X + needs[1] * FFN_GATE + needs[2] * FFN_UP + needs[3] * FFN_DOWN
        sizes, operands = _ffn_call(x, w_gate, w_up, w_down)
        y, saved = _ffn_forward(x, sizes, operands, code, act, keep)
        ctx.save_for_backward(x, w_gate, w_up, w_down, saved)
        ctx.args = sizes, code, act, keep
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        *inputs, saved = ctx.saved_tensors
        sizes, code, act, keep = ctx.args
        M, K, F, N = sizes
        device = gy.device
        _, operands = _ffn_call(*inputs)
        g, ldy = _read(gy if gy.dim() == 2 else gy.reshape(M, N))
        scratch = torch.empty(_ffn_bytes(M, K, F, N, keep)[2], dtype=torch.uint8, device=device)
        grads = [torch.empty_like(t, memory_format=torch.contiguous_format) if keep >> i & 1 else None for i, t in enumerate(inputs)]
        dx, dg, du, dd = [None if t is None else t.data_ptr() for t in grads]
        _call(device, _lib.tgemm_ffn_backward, M, K, F, N, code, act, *_pointers(operands), g.data_ptr(), ldy, keep,
              saved.data_ptr(), dx, K, dg, K, du, K, dd, F, scratch.data_ptr())
        return (*grads, None, None)


def gated_ffn(x, w_gate, w_up, w_down, activation="silu"):
    """The gated feed-forward block, y = (act(x @ w_gate^T) * (x @ w_up^T)) @ w_down^T,
    differentiable.

    x: (..., K), w_gate and w_up: (F, K), w_down: (N, F), all bfloat16 or all
    float16; rows may be apart (parts of one (2 F, K) tensor serve as w_gate and
    w_up).  ``activation``: "silu", "gelu", "gelu_tanh" or "relu".  Returns
    (..., N) of x's dtype.  Sums are float; the inner values are rounded to
    x's dtype (so are both projections' gradients), y and each gradient once.  The two
    projections, the activation and their product are one kernel; up to 16 tokens
    without gradients take kernels that read each weight once.  For the backward pass
    both projections are kept in 24 bits, six bytes for each token and inner unit (two
    where w_down's gradient alone is wanted); it computes only the gradients that are
    asked for; second derivatives and forward-mode ones are refused.  To capture a
    training step into a graph, see :func:`linear_fp8`.
    """
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError("activation must be one of %s, got %r" % (", ".join(map(repr, ACTIVATIONS)), activation))
    tensors = (x, w_gate, w_up, w_down)
    code = _half_code(tensors, ("x", "w_gate", "w_up", "w_down"))
    if x.dim() < 1 or w_gate.dim() != 2 or w_down.dim() != 2 or w_up.shape != w_gate.shape or \
            x.shape[-1] != w_gate.shape[1] or w_down.shape[1] != w_gate.shape[0]:
        raise ValueError("x %s, w_gate %s, w_up %s and w_down %s do not make a feed-forward block" % tuple(
            tuple(t.shape) for t in tensors))
    if not _wants_derivative(tensors):
        return _ffn_forward(x, *_ffn_call(*tensors), code, act, 0)[0]
    return _GatedFfn.apply(x, w_gate, w_up, w_down, code, act)


# Keeping the powers of the logits spares a product of 2 K operations an element
# and costs two passes of two bytes.  Training step in us, made again and kept,
# every token counting:
#   4096x32000x256   453  482      1000x50257x768    415   372
#   4096x32000x512   649  607      8192x128256x4096 28045 21903
#   4096x32000x1024 1058  912      256x32000x2048    209   182
POWERS_LEAST = 512


@functools.lru_cache(maxsize=512)
def _xent_bytes(M, V, K, keep):
    n = (ctypes.c_int64 * 3)()
    rc = _lib.tgemm_xent_bytes(M, V, K, keep, n)
    if rc != OK:
        raise TgemmError(rc, last_error())
    return tuple(max(v, 1) for v in n)


def _xent_forward(x, w, target, ignore, reduction, code, keep):
    """The loss, and what the backward pass reads of the rows."""
    device, (V, K) = x.device, w.shape
    M = target.numel()
    (x2, ldx), (w2, ldw), t = _read(x.reshape(M, K)), _read(w), target.contiguous()
    loss = torch.empty(() if reduction else target.shape, dtype=torch.float32, device=device)
    sizes = _xent_bytes(M, V, K, keep)
    saved, scratch = (torch.empty(n, dtype=torch.uint8, device=device) for n in sizes[:2])
    _call(device, _lib.tgemm_xent_forward, M, V, K, code, x2.data_ptr(), ldx, w2.data_ptr(), ldw, t.data_ptr(), ignore, reduction,
          keep, loss.data_ptr(), saved.data_ptr(), scratch.data_ptr())
    return loss, saved


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, target, ignore, reduction, code, powers):
        loss, saved = _xent_forward(x, w, target, ignore, reduction, code, powers)
        ctx.save_for_backward(x, w, target, saved)
        ctx.args = reduction, code, powers
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gloss):
        x, w, target, saved = ctx.saved_tensors
        reduction, code, powers = ctx.args
        device, (V, K) = x.device, w.shape
        M = target.numel()
        keep = (KEEP_X if ctx.needs_input_grad[0] else 0) | (KEEP_W if ctx.needs_input_grad[1] else 0) | powers
        (x2, ldx), (w2, ldw), t, g = _read(x.reshape(M, K)), _read(w), target.contiguous(), gloss.contiguous()
        scratch = torch.empty(_xent_bytes(M, V, K, keep)[2], dtype=torch.uint8, device=device)
        dx = torch.empty(x.shape, dtype=x.dtype, device=device) if keep & KEEP_X else None
        dw = torch.empty(w.shape, dtype=w.dtype, device=device) if keep & KEEP_W else None
        _call(device, _lib.tgemm_xent_backward, M, V, K, code, x2.data_ptr(), ldx, w2.data_ptr(), ldw, t.data_ptr(), reduction,
              g.data_ptr(), saved.data_ptr(), keep, None if dx is None else dx.data_ptr(), K,
              None if dw is None else dw.data_ptr(), K, scratch.data_ptr())
        return dx, dw, None, None, None, None, None


def linear_cross_entropy(x, w, target, ignore_index=-100, reduction="mean", keep_bytes=4 * 2 ** 30):
    """Softmax cross entropy of the logits x @ w^T, without a tensor of them (but see
    ``keep_bytes``), differentiable: logsumexp(x @ w^T) - (x @ w^T)[target] of each
    token.

    x: (..., K), w: (V, K), both bfloat16 or both float16; target: int64 of
    x.shape[:-1].  Tokens whose target is ``ignore_index`` do not count, whatever
    they hold, and cost nothing (the products leave them out); any other target
    outside 0 .. V - 1 makes the loss NaN.
    ``reduction``: "mean" over the tokens that count (NaN where none does),
    "sum", or "none" (a loss for each token, zero where it does not count).
    Returns float32; the loss's logits and softmax are float throughout.

    The backward pass goes by pieces of the vocabulary (scratch: about 512 MB at
    most, or 16 KB a token where that is more, and dx's float sums where there are
    several pieces).  With gradients wanted and K of at least 512, the forward pass
    keeps each logit's power of e, relative to a maximum of its row and rounded to
    10 bits (float16: 12), where all of them take at most ``keep_bytes`` (2 V bytes a
    token, whether it counts or not: as much as logits of 16 bits; 0: never); otherwise
    the backward pass makes the logits again, which takes up to 1.3 times as long for
    the step.  It rounds the logits' gradients to x's dtype, scaled by a factor that the
    results do not keep, so that small probabilities hold in float16 too.  Gradients
    have their inputs' dtypes;
    second derivatives and forward-mode ones are refused.  To capture a training
    step into a graph, see :func:`linear_fp8`.
    """
    how = REDUCTIONS.get(reduction)
    if how is None:
        raise ValueError("reduction must be one of %s, got %r" % (", ".join(map(repr, REDUCTIONS)), reduction))
    code = _half_code((x, w), ("x", "w"))
    if x.dim() < 1 or w.dim() != 2 or x.shape[-1] != w.shape[1]:
        raise ValueError("x %s and w %s do not make x @ w^T" % (tuple(x.shape), tuple(w.shape)))
    if target.dtype != torch.int64:
        raise TypeError("target must be int64, got %s" % target.dtype)
    if target.shape != x.shape[:-1] or target.device != x.device:
        raise ValueError("target must be of shape %s on %s, got %s on %s" % (
            tuple(x.shape[:-1]), x.device, tuple(target.shape), target.device))
    if not -2 ** 63 <= ignore_index < 2 ** 63 or ignore_index != int(ignore_index):
        raise ValueError("ignore_index must be an int64, got %r" % (ignore_index,))
    if not keep_bytes >= 0:
        raise ValueError("keep_bytes must not be negative, got %r" % (keep_bytes,))
    if not _wants_derivative((x, w)):
        return _xent_forward(x, w, target, int(ignore_index), how, code, 0)[0]
    V, K = w.shape
    powers = KEEP_POWERS if K >= POWERS_LEAST and V <= 2 ** 28 and 2 * target.numel() * ((V + 63) // 64 * 64) <= keep_bytes else 0
    return _LinearCrossEntropy.apply(x, w, target, int(ignore_index), how, code, powers)


def _dense(t):
    """Whether t's elements fill a block of memory, each once."""
    if t.is_contiguous():
        return True
    span = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != span:
            return False
        span *= size
    return True


def clip_grad_norm(grads, max_norm, eps=1e-6, out=None):
    """Scale tensors so that their norm, taken as one vector, is at most
    ``max_norm``; returns the norm that they had (a float32 scalar on the GPU).

    grads: one or more float32, bfloat16 or float16 tensors on one GPU, of any
    shapes, dense (their elements fill a block of memory in any order of axes),
    none of them twice and no two with elements in common.  Each is multiplied by min(1, max_norm / (norm + eps)) in
    place, or into the tensor of ``out`` at its place (same shape, dtype and
    strides; it may be the same tensor, and shares no element with another).  Squares are summed in 64 bits; the
    product is rounded once.  A norm that is infinite makes the factor zero (and
    infinities NaN), a NaN makes everything NaN, as does a quotient that has no
    value (``max_norm`` infinite as well; 0 / 0).  Nothing waits for the GPU.  Not
    differentiable.
    """
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    max_norm, eps = float(max_norm), float(eps)
    if not max_norm >= 0 or not eps >= 0:
        raise ValueError("max_norm and eps must not be negative or NaN, got %r and %r" % (max_norm, eps))
    out = grads if out is None else list(out)
    if len(out) != len(grads):
        raise ValueError("out must hold a tensor for each of the %d of grads, got %d" % (len(grads), len(out)))
    n, device = len(grads), grads[0].device
    if not grads[0].is_cuda:
        raise ValueError("grads must be GPU tensors")
    index = device.index
    codes, counts, ins = [], [], []
    for t in grads:
        code = _REAL_CODES.get(t.dtype)
        if code is None:
            raise TypeError("grads has unsupported dtype %s (float32, bfloat16, float16)" % t.dtype)
        if t.get_device() != index:
            raise ValueError("grads must be on one GPU (%s, %s)" % (device, t.device))
        if not t.is_contiguous() and not _dense(t):
            raise ValueError("grads must be dense (shape %s, strides %s)" % (tuple(t.shape), t.stride()))
        codes.append(code)
        counts.append(t.numel())
        ins.append(t.data_ptr())
    outs = ins
    if out is not grads:
        outs = []
        for t, o in zip(grads, out):
            if o.dtype is not t.dtype or o.get_device() != index or o.shape != t.shape or not (
                    o.is_contiguous() and t.is_contiguous()) and o.stride() != t.stride():
                raise ValueError("out must match grads: %s %s %s with strides %s, got %s %s %s with strides %s" % (
                    t.dtype, tuple(t.shape), device, t.stride(), o.dtype, tuple(o.shape), o.device, o.stride()))
            outs.append(o.data_ptr())
    for pointers in (ins,) if outs is ins else (ins, outs):
        if len(set(pointers)) != n:  # empty tensors may share an address
            used = [p for p, c in zip(pointers, counts) if c]
            if len(set(used)) != len(used):
                raise ValueError("a tensor is given twice")
    if outs is not ins and outs != ins:
        known = {p for p, c in zip(ins, counts) if c}
        if any(q != p and q in known for p, q, c in zip(ins, outs, counts) if c):
            raise ValueError("a tensor of out is another one of grads")
    i64s = ctypes.c_int64 * n
    sizes = i64s(*counts)
    need = _lib.tgemm_clip_workspace_bytes(n, sizes)
    if need < 0:
        raise ValueError("grads hold more elements than 2^40")
    pointers = ctypes.c_void_p * n
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    norm = torch.empty((), dtype=torch.float32, device=device)
    _call(device, _lib.tgemm_clip, n, pointers(*ins), pointers(*outs), sizes, (ctypes.c_int32 * n)(*codes), max_norm, eps,
          norm.data_ptr(), ws.data_ptr(), need)
    try:
        torch.autograd.graph.increment_version(out)
    except RuntimeError:  # inference tensors have no version
        torch.autograd.graph.increment_version([t for t in out if not t.is_inference()])
    return norm
