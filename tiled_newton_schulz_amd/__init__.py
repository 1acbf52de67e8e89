"""Python binding of libhimuon (MI355X tiled Newton-Schulz).

Argument marshalling only: every function here forwards to the C entry point
of the same name in include/himuon.h, taking torch tensors for device memory
and torch's current stream.  All arithmetic runs in the library's HIP kernels;
importing this module fails if the library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Iterable, NamedTuple, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhimuon.so")

BF16 = 0
FP32 = 1
BF16_PRECISE = 2   # bf16 storage, fp32 arithmetic throughout
I32, I64 = 0, 1      # element types of id arrays
MAX_STEPS = 16
MAX_ENTRIES = 1024   # teacher entries of a row (himuon_distill)
MAX_TOP = 64         # alternatives of a row (himuon_token_logprobs)
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}   # of a gated block
MAX_NORM_COLS = 32768
ADAMW_BLOCK = 256    # elements that share a scale in 8-bit states

STATUS = {0: "HIMUON_OK", 1: "HIMUON_ERR_INVALID_ARGUMENT", 2: "HIMUON_ERR_UNSUPPORTED",
          3: "HIMUON_ERR_LAYOUT", 4: "HIMUON_ERR_OVERLAP", 5: "HIMUON_ERR_WORKSPACE", 6: "HIMUON_ERR_HIP"}
NOALLOC_SCRATCH_BYTES = 128 << 20
EXPORTS = ["himuon_plan", "himuon_workspace_size", "himuon_tiled_ns", "himuon_tiled_ns_noalloc",
           "himuon_tiled_ns_schedule",
           "himuon_muon_step", "himuon_gram_ns", "himuon_gram_ns_workspace", "himuon_pair_stats",
           "himuon_pair_stats_workspace", "himuon_grouped_mm", "himuon_grouped_wgrad",
           "himuon_grouped_wgrad_workspace", "himuon_grouped_gated_mm", "himuon_grouped_gated_mm_grad",
           "himuon_layer_norm", "himuon_layer_norm_grad", "himuon_layer_norm_grad_workspace", "himuon_adamw_step",
           "himuon_distill",
           "himuon_distill_workspace", "himuon_distill_grad", "himuon_token_logprobs",
           "himuon_token_logprobs_workspace", "himuon_token_logprobs_grad", "himuon_status_string",
           "himuon_last_hip_error", "himuon_version"]


class himuon_matrix_t(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64)]


class himuon_adamw_state_t(ctypes.Structure):
    _fields_ = [("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class himuon_plan_info_t(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_int64), ("resident_launches", ctypes.c_int64),
                ("chunks", ctypes.c_int64), ("launches", ctypes.c_int64),
                ("kernel_tile", ctypes.c_int64), ("workspace_full", ctypes.c_size_t),
                ("workspace_min", ctypes.c_size_t), ("tail_tiles", ctypes.c_int64)]


class HimuonError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = STATUS.get(code, str(code))
        if code == 6:
            msg += f" (hipError {lib.himuon_last_hip_error()})"
        super().__init__(f"{where}: {msg}")


def _load():
    # torch first: it brings its own HIP runtime (same soname as the system
    # one), and the library must bind to that instance, the one that owns the
    # device memory and streams it is handed.  Loaded the other way round, the
    # process would hold two HIP runtimes and the library's would see no device.
    import torch  # noqa: F401

    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python tiled_newton_schulz_amd/build.py` "
                          "(or __graft_entry__.build()) first")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    L.himuon_plan.argtypes = [P(himuon_matrix_t), ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                              ctypes.c_int, ctypes.c_size_t, P(himuon_plan_info_t)]
    L.himuon_plan.restype = ctypes.c_int
    L.himuon_workspace_size.argtypes = [P(himuon_matrix_t), ctypes.c_int32, ctypes.c_int32, ctypes.c_int,
                                        P(ctypes.c_size_t), P(ctypes.c_size_t)]
    L.himuon_workspace_size.restype = ctypes.c_int
    L.himuon_tiled_ns.argtypes = [P(himuon_matrix_t), ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                  P(ctypes.c_float), ctypes.c_int, ctypes.c_float, ctypes.c_void_p,
                                  ctypes.c_size_t, ctypes.c_void_p]
    L.himuon_tiled_ns.restype = ctypes.c_int
    L.himuon_tiled_ns_noalloc.argtypes = [P(himuon_matrix_t), ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                          P(ctypes.c_float), ctypes.c_int, ctypes.c_float, ctypes.c_void_p]
    L.himuon_tiled_ns_noalloc.restype = ctypes.c_int
    L.himuon_tiled_ns_schedule.argtypes = [P(himuon_matrix_t), ctypes.c_int32, P(ctypes.c_int32), ctypes.c_int32,
                                           P(ctypes.c_float), ctypes.c_int, ctypes.c_float, ctypes.c_void_p,
                                           ctypes.c_size_t, ctypes.c_void_p]
    L.himuon_tiled_ns_schedule.restype = ctypes.c_int
    L.himuon_muon_step.argtypes = [P(himuon_matrix_t), P(himuon_matrix_t), P(himuon_matrix_t), ctypes.c_int32,
                                   ctypes.c_int32, ctypes.c_int32, P(ctypes.c_float), ctypes.c_float,
                                   ctypes.c_float, ctypes.c_int, ctypes.c_float, ctypes.c_void_p,
                                   ctypes.c_size_t, ctypes.c_void_p]
    L.himuon_muon_step.restype = ctypes.c_int
    L.himuon_gram_ns.argtypes = [P(himuon_matrix_t), ctypes.c_int32, ctypes.c_int32, P(ctypes.c_float),
                                 ctypes.c_int32, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t,
                                 ctypes.c_void_p]
    L.himuon_gram_ns.restype = ctypes.c_int
    L.himuon_gram_ns_workspace.argtypes = [P(himuon_matrix_t), ctypes.c_int32, ctypes.c_int,
                                           P(ctypes.c_size_t), P(ctypes.c_size_t)]
    L.himuon_gram_ns_workspace.restype = ctypes.c_int
    L.himuon_pair_stats.argtypes = [P(himuon_matrix_t), P(himuon_matrix_t), ctypes.c_int32, ctypes.c_int,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    L.himuon_pair_stats.restype = ctypes.c_int
    L.himuon_pair_stats_workspace.argtypes = [P(himuon_matrix_t), ctypes.c_int32, P(ctypes.c_size_t)]
    L.himuon_pair_stats_workspace.restype = ctypes.c_int
    M, V, I, F, Z = P(himuon_matrix_t), ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    E, D, A = ctypes.c_int, ctypes.c_double, P(himuon_adamw_state_t)
    for name, args in {
            "himuon_grouped_mm": [M, M, I, I, V, M, E, V],
            "himuon_grouped_wgrad": [M, M, V, M, I, E, V, Z, V],
            "himuon_grouped_wgrad_workspace": [M, M, I, E, P(Z)],
            "himuon_grouped_gated_mm": [M, M, I, I, V, M, M, E, E, V],
            "himuon_grouped_gated_mm_grad": [M, M, I, I, V, M, M, M, E, E, V],
            "himuon_layer_norm": [M, V, V, F, M, V, E, V],
            "himuon_layer_norm_grad": [M, V, V, M, M, V, V, E, V, Z, V],
            "himuon_layer_norm_grad_workspace": [M, E, P(Z)],
            "himuon_adamw_step": [M, M, A, I, I, D, D, D, D, D, ctypes.c_int64, V, E, E, V],
            "himuon_distill": [M, V, E, M, F, I, V, V, V, M, E, V, Z, V],
            "himuon_distill_workspace": [M, E, I, P(Z)],
            "himuon_distill_grad": [M, V, E, M, F, I, V, V, M, E, V],
            "himuon_token_logprobs": [M, V, E, F, I, V, V, V, V, V, E, V, Z, V],
            "himuon_token_logprobs_workspace": [M, I, E, P(Z)],
            "himuon_token_logprobs_grad": [M, V, E, F, V, V, V, V, M, E, V]}.items():
        getattr(L, name).argtypes = args
        getattr(L, name).restype = E
    L.himuon_status_string.argtypes = [ctypes.c_int]
    L.himuon_status_string.restype = ctypes.c_char_p
    L.himuon_last_hip_error.argtypes = []
    L.himuon_last_hip_error.restype = ctypes.c_int32
    L.himuon_version.argtypes = []
    L.himuon_version.restype = ctypes.c_int32
    return L


lib = _load()


# ---- marshalling helpers -------------------------------------------------
def _dtype_code(t, precise: bool = False) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16_PRECISE if precise else BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")


def descriptor(t) -> himuon_matrix_t:
    """Descriptor of a 2-D tensor.  Row-major views pass as they are; a
    transposed view (unit stride along dim 0) is passed as its row-major
    transpose, which is exact because the tiled map commutes with transposition
    under the (0, 0)-anchored tiling."""
    if t.dim() != 2:
        raise ValueError("matrices must be 2-D")
    H, W = t.shape
    s0, s1 = t.stride()
    if s1 == 1 or W == 1:
        return himuon_matrix_t(t.data_ptr(), H, W, s0 if H > 1 else max(W, 1))
    if s0 == 1 or H == 1:
        return himuon_matrix_t(t.data_ptr(), W, H, s1 if W > 1 else max(H, 1))
    raise ValueError("matrix must have unit stride along one dimension")


def shape_descriptor(rows: int, cols: int, ld: int | None = None, ptr: int = 1 << 20) -> himuon_matrix_t:
    """Descriptor with a placeholder address, for planning queries only."""
    return himuon_matrix_t(ptr, rows, cols, cols if ld is None else ld)


def _descs(ts) -> ctypes.Array:
    arr = (himuon_matrix_t * max(len(ts), 1))()
    for i, t in enumerate(ts):
        arr[i] = t if isinstance(t, himuon_matrix_t) else descriptor(t)
    return arr


def coeff_array(abc, K: int):
    """(a, b, c) per step as a float array of 3K entries.  `abc` is one triple
    (used for every step), a flat list of 3K numbers, or K triples."""
    if K == 0:
        return (ctypes.c_float * 3)()
    flat = []
    items = list(abc)
    if len(items) == 3 and not hasattr(items[0], "__len__"):
        flat = [float(x) for x in items] * K
    elif items and hasattr(items[0], "__len__"):
        for tri in items:
            flat.extend(float(x) for x in tri)
    else:
        flat = [float(x) for x in items]
    if len(flat) != 3 * K:
        raise ValueError("need one (a, b, c) triple per step")
    return (ctypes.c_float * (3 * K))(*flat)


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(code: int, where: str):
    if code != 0:
        raise HimuonError(code, where)


# ---- entry points ----------------------------------------------------------
def himuon_plan(mats: Sequence, T: int, K: int, dtype: int, workspace_bytes: int = 0) -> dict:
    d = _descs(mats)
    info = himuon_plan_info_t()
    _check(lib.himuon_plan(d, len(mats), T, K, dtype, workspace_bytes, ctypes.byref(info)), "himuon_plan")
    return {f: getattr(info, f) for f, _ in himuon_plan_info_t._fields_}


def himuon_workspace_size(mats: Sequence, T: int, dtype: int | None = None) -> tuple[int, int]:
    if dtype is None:
        dtype = _dtype_code(mats[0])
    d = _descs(mats)
    full, mn = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.himuon_workspace_size(d, len(mats), T, dtype, ctypes.byref(full), ctypes.byref(mn)),
           "himuon_workspace_size")
    return full.value, mn.value


def _in_memory(workspace, nbytes, device):
    """nbytes, if the workspace has as many from its first element on, on the device."""
    if workspace.device != device:
        raise ValueError("workspace must be on the matrices' GPU")
    if nbytes > workspace.untyped_storage().nbytes() - workspace.storage_offset() * workspace.element_size():
        raise ValueError("workspace is smaller than its stated size")
    return nbytes


def _workspace(mats, T, dtype, workspace, workspace_bytes, device):
    import torch
    if workspace is not None:
        nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
        return workspace, workspace.data_ptr(), _in_memory(workspace, nbytes, device)
    full, mn = himuon_workspace_size(mats, T, dtype)
    if full == 0:
        return None, None, 0
    cap = full if workspace_bytes is None else max(min(full, workspace_bytes), 0)
    buf = torch.empty(max(cap, 1), dtype=torch.uint8, device=device)
    return buf, buf.data_ptr(), cap


def himuon_tiled_ns(mats: Sequence, T: int, K: int, abc=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                    workspace=None, workspace_bytes: int | None = None, stream=None, precise: bool = False):
    """Tiled Newton-Schulz in place on a list of 2-D bf16 or fp32 CUDA tensors.

    workspace: optional uint8 device tensor; if omitted the binding allocates
    one through torch (capped at workspace_bytes when given).  precise: bf16
    data with fp32 arithmetic throughout (HIMUON_BF16_PRECISE)."""
    if len(mats) == 0:
        return
    dtype = _dtype_code(mats[0], precise)
    d = _descs(mats)
    ws, ptr, nbytes = _workspace(mats, T, dtype, workspace, workspace_bytes, mats[0].device)
    code = lib.himuon_tiled_ns(d, len(mats), T, K, coeff_array(abc, K), dtype, eps,
                               ctypes.c_void_p(ptr), nbytes, _stream_handle(stream))
    _check(code, "himuon_tiled_ns")
    return ws


def himuon_tiled_ns_noalloc(mats: Sequence, T: int, K: int, abc=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                            stream=None):
    """Tiled Newton-Schulz in place, with no device allocation: the step path
    runs through the library's own 128 MiB scratch on the device.  Calls that
    overlap in time on one device race on that scratch."""
    if len(mats) == 0:
        return
    dtype = _dtype_code(mats[0])
    d = _descs(mats)
    code = lib.himuon_tiled_ns_noalloc(d, len(mats), T, K, coeff_array(abc, K), dtype, eps,
                                       _stream_handle(stream))
    _check(code, "himuon_tiled_ns_noalloc")


def himuon_tiled_ns_schedule(mats: Sequence, Ts: Sequence[int], abc=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                             workspace=None, workspace_bytes: int | None = None, stream=None, precise: bool = False):
    """len(Ts) Newton-Schulz steps in place, step k on the Ts[k] x Ts[k] tiles
    (non-increasing, nested sizes; one normalisation, on the first size)."""
    if len(mats) == 0:
        return
    dtype = _dtype_code(mats[0], precise)
    d = _descs(mats)
    K = len(Ts)
    ts = (ctypes.c_int32 * max(1, K))(*[int(t) for t in Ts])
    if workspace is None:
        # the largest need of any pass, capped
        need = max(himuon_workspace_size(mats, int(t), dtype)[0] for t in set(Ts)) if K else 0
        if need:
            import torch
            need = need if workspace_bytes is None else max(min(need, workspace_bytes), 0)
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=mats[0].device)
            workspace_bytes = need
    ptr = workspace.data_ptr() if workspace is not None else None
    nbytes = 0 if workspace is None else (workspace.numel() if workspace_bytes is None else workspace_bytes)
    if workspace is not None:
        _in_memory(workspace, nbytes, mats[0].device)
    code = lib.himuon_tiled_ns_schedule(d, len(mats), ts, K, coeff_array(abc, K), dtype, eps,
                                        ctypes.c_void_p(ptr), nbytes, _stream_handle(stream))
    _check(code, "himuon_tiled_ns_schedule")
    return workspace


def himuon_muon_step(W: Sequence, M: Sequence, G: Sequence, T: int, K: int, abc=(3.4445, -4.7750, 2.0315),
                     mu: float = 0.95, eta: float = 0.02, eps: float = 1e-7, workspace=None,
                     workspace_bytes: int | None = None, stream=None, precise: bool = False):
    """Fused Muon step M <- mu M + G, W <- W - eta tiledNS(M), in place."""
    n = len(M)
    if not (len(W) == len(G) == n):
        raise ValueError("W, M, G must have equal length")
    if n == 0:
        return
    dtype = _dtype_code(M[0], precise)
    dW, dM, dG = _descs(W), _descs(M), _descs(G)
    ws, ptr, nbytes = _workspace(M, T, dtype, workspace, workspace_bytes, M[0].device)
    code = lib.himuon_muon_step(dW, dM, dG, n, T, K, coeff_array(abc, K), mu, eta, dtype, eps,
                                ctypes.c_void_p(ptr), nbytes, _stream_handle(stream))
    _check(code, "himuon_muon_step")
    return ws


def himuon_gram_ns_workspace(mats: Sequence, dtype: int | None = None) -> tuple[int, int]:
    """(full, min) workspace bytes of himuon_gram_ns for these matrices."""
    if dtype is None:
        dtype = _dtype_code(mats[0])
    d = _descs(mats)
    full, mn = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.himuon_gram_ns_workspace(d, len(mats), dtype, ctypes.byref(full), ctypes.byref(mn)),
           "himuon_gram_ns_workspace")
    return full.value, mn.value


def himuon_gram_ns(mats: Sequence, K: int, abc=(3.4445, -4.7750, 2.0315), restart: int = 2, eps: float = 1e-7,
                   workspace=None, workspace_bytes: int | None = None, stream=None, precise: bool = False):
    """Full-matrix Newton-Schulz of each matrix, in place, through its Gram
    matrix with a restart before step restart + 1 (0: none)."""
    if len(mats) == 0:
        return
    dtype = _dtype_code(mats[0], precise)
    d = _descs(mats)
    if workspace is None:
        full = himuon_gram_ns_workspace(mats, dtype)[0]
        cap = full if workspace_bytes is None else max(min(full, workspace_bytes), 0)
        if cap:
            import torch
            workspace = torch.empty(cap, dtype=torch.uint8, device=mats[0].device)
        workspace_bytes = cap
    else:
        if workspace_bytes is None:
            workspace_bytes = workspace.numel() * workspace.element_size()
        _in_memory(workspace, workspace_bytes, mats[0].device)
    ptr = workspace.data_ptr() if workspace is not None else None
    code = lib.himuon_gram_ns(d, len(mats), K, coeff_array(abc, K), restart, dtype, eps,
                              ctypes.c_void_p(ptr), workspace_bytes, _stream_handle(stream))
    _check(code, "himuon_gram_ns")
    return workspace


def himuon_pair_stats_workspace(a: Sequence) -> int:
    """Workspace bytes himuon_pair_stats needs for pairs shaped like `a`."""
    d = _descs(a)
    nbytes = ctypes.c_size_t(0)
    _check(lib.himuon_pair_stats_workspace(d, len(a), ctypes.byref(nbytes)), "himuon_pair_stats_workspace")
    return nbytes.value


def _row_major(t) -> bool:
    return t.stride(1) == 1 or t.shape[1] == 1


def himuon_pair_stats(a: Sequence, b: Sequence, out=None, workspace=None, stream=None):
    """(n, 3) float64 device tensor: sum a*b, sum a*a, sum b*b for each pair.

    a[i] and b[i] are equal-shaped bf16 or fp32 tensors with the same memory
    orientation (both row-major, or both transposed views); `out` and
    `workspace` are optional device tensors (float64 of 3n elements, uint8)."""
    import torch
    n = len(a)
    if len(b) != n:
        raise ValueError("a and b must have equal length")
    if n == 0:
        return torch.empty((0, 3), dtype=torch.float64)
    dtype = _dtype_code(a[0])
    for x, y in zip(a, b):
        if x.shape != y.shape:
            raise ValueError("pairs must have equal shapes")
        if _row_major(x) != _row_major(y):
            raise ValueError("both matrices of a pair must have the same orientation")
    da, db = _descs(a), _descs(b)
    dev = a[0].device
    if out is None:
        out = torch.empty((n, 3), dtype=torch.float64, device=dev)
    if workspace is None:
        workspace = torch.empty(max(himuon_pair_stats_workspace(a), 8), dtype=torch.uint8, device=dev)
    nbytes = _in_memory(workspace, workspace.numel() * workspace.element_size(), dev)
    code = lib.himuon_pair_stats(da, db, n, dtype, ctypes.c_void_p(out.data_ptr()),
                                 ctypes.c_void_p(workspace.data_ptr()), nbytes, _stream_handle(stream))
    _check(code, "himuon_pair_stats")
    return out


# ---- the experts' products -------------------------------------------------------
class Matrices:
    """Descriptors of the weight matrices of a layer's experts, made once and
    used for any number of calls.  It keeps the tensors, whose values may change
    but not their place: one that was given other memory (t.data = ..., set_, a
    storage resized) makes the next call raise ValueError."""

    is_cuda = True   # checked when they are made

    def __init__(self, array, n, shape, transposed, dtype, device, tensors):
        self.array, self.n, self.shape, self.transposed = array, n, shape, transposed
        self.dtype, self.device, self.tensors = dtype, device, tensors
        self.places = self._places()

    def _places(self):
        if isinstance(self.tensors, list):
            return [t.data_ptr() for t in self.tensors]
        return self.tensors.data_ptr()

    def in_place(self):
        """Itself, if the tensors are still where they were described."""
        if self._places() != self.places:
            raise ValueError("matrices were described before their tensors got other memory: describe them again")
        return self

    def __len__(self):
        return self.n


def _stacked(base: int, n: int, step: int, rows: int, cols: int, ld: int):
    """Descriptors of n equal matrices, `step` bytes apart."""
    import numpy as np
    a = np.empty((n, 4), dtype=np.int64)
    a[:, 0] = base + step * np.arange(n, dtype=np.int64)
    a[:, 1:] = rows, cols, ld
    return (himuon_matrix_t * n).from_buffer(a)


def matrices(w) -> Matrices:
    """Descriptors of equal-shaped matrices: a list of 2-D tensors or one 3-D
    tensor (one matrix per leading index), bf16 or fp32 on one GPU, all
    row-major or all transposed views of row-major matrices."""
    import torch
    if isinstance(w, Matrices):
        return w.in_place()
    if isinstance(w, torch.Tensor):
        if w.dim() != 3:
            raise ValueError("stacked matrices must be a 3-D tensor")
        n, K, N = w.shape
        if n == 0 or K == 0 or N == 0:
            raise ValueError("matrices must not be empty")
        _need_gpu(w)
        st, s0, s1 = w.stride()
        es = w.element_size()
        if s1 == 1 or N == 1:
            arr, tr = _stacked(w.data_ptr(), n, st * es, K, N, max(s0, N) if K == 1 else s0), False
        elif s0 == 1 or K == 1:
            arr, tr = _stacked(w.data_ptr(), n, st * es, N, K, s1), True
        else:
            raise ValueError("matrices must have unit stride along one dimension")
        return Matrices(arr, n, (K, N), tr, w.dtype, w.device, w)
    w = list(w)
    if not w:
        raise ValueError("need at least one matrix")
    first = w[0]
    row_major = all(t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] == 1) for t in w)
    transposed = not row_major and all(t.dim() == 2 and (t.stride(0) == 1 or t.shape[0] == 1) for t in w)
    if not row_major and not transposed:
        raise ValueError("matrices must be 2-D, all row-major or all transposed views")
    for t in w:
        if t.shape != first.shape or t.dtype != first.dtype or t.device != first.device:
            raise ValueError("matrices must agree in shape, dtype and device")
        if t.numel() == 0:
            raise ValueError("matrices must not be empty")
    _need_gpu(first)
    arr = (himuon_matrix_t * len(w))(*[_rows(t.t() if transposed else t) for t in w])
    return Matrices(arr, len(w), tuple(first.shape), transposed, first.dtype, first.device, w)


def _need_gpu(*ts):
    """All on one GPU (a host pointer would fault there)."""
    dev = ts[0].device
    for t in ts:
        if not t.is_cuda or t.device != dev:
            raise ValueError("tensors must be on one GPU")


def _rows(t) -> himuon_matrix_t:
    """Descriptor of a row-major 2-D tensor (it may have no rows)."""
    if t.dim() != 2:
        raise ValueError("matrices must be 2-D")
    H, W = t.shape
    s0, s1 = t.stride()
    if W == 0:
        raise ValueError("rows must not be empty")
    if s1 != 1 and W != 1:
        raise ValueError("rows must have unit stride")
    return himuon_matrix_t(t.data_ptr() if H else None, H, W, s0 if H > 1 else max(W, 1))


class _placed:
    """The device and stream of a call, set for the tensors allocated in it, so
    that their memory belongs to the stream that uses it; yields the stream's
    handle.  Where both are the current ones nothing is set (setting them costs
    more host time than the rest of a small call)."""
    __slots__ = ("device", "stream", "set")

    def __init__(self, device, stream):
        self.device, self.stream, self.set = device, stream, None

    def __enter__(self):
        import torch
        index = self.device.index
        if self.stream is None and index == torch.cuda.current_device():
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # a tenth of current_stream()'s time
            return ctypes.c_void_p(raw(index) if raw else torch.cuda.current_stream(index).cuda_stream)
        self.set = contextlib.ExitStack()
        self.set.enter_context(torch.cuda.device(self.device))
        stream = self.stream
        if stream is None:
            stream = torch.cuda.current_stream()
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=self.device)
            self.set.enter_context(torch.cuda.stream(stream))
        return ctypes.c_void_p(stream.cuda_stream)

    def __exit__(self, *exc):
        if self.set is not None:
            self.set.close()
        return False


def _ends(ends, n, device):
    import torch
    if ends.dtype != torch.int32:
        raise TypeError("ends must be int32")
    if ends.dim() != 1 or ends.shape[0] != n or not ends.is_contiguous() or ends.device != device:
        raise ValueError("ends must be a contiguous vector with one entry per expert, on the operands' GPU")
    return ctypes.c_void_p(ends.data_ptr())


def himuon_grouped_mm(x, w, ends, out=None, stream=None):
    """y[r] = x[r] @ w[e] for the rows r of expert e, ends[e-1] <= r < ends[e].

    x: (M, K), rows sorted by expert.  w: the experts' (K, N) weights as
    matrices() takes them, or its result; transposed views give the product
    with the stored matrices' transposes (the input gradient of a layer is
    himuon_grouped_mm(dy, w.transpose(1, 2), ends)).  ends: int32, on the GPU.
    Rows past ends[-1] become zero.  out: optional (M, N) tensor."""
    import torch
    w = matrices(w)
    K, N = w.shape
    _need_gpu(x, w, ends) if out is None else _need_gpu(x, w, ends, out)
    if x.dtype != w.dtype or (out is not None and out.dtype != x.dtype):
        raise TypeError("x, w and out must have one dtype")
    with _placed(x.device, stream) as s:
        if out is None:
            out = torch.empty((x.shape[0], N), dtype=x.dtype, device=x.device)
        dx, dy = _rows(x), _rows(out)
        _check(lib.himuon_grouped_mm(ctypes.byref(dx), w.array, w.n, int(w.transposed), _ends(ends, w.n, x.device),
                                     ctypes.byref(dy), _dtype_code(x), s), "himuon_grouped_mm")
    return out


def himuon_grouped_wgrad_workspace(x, dy, n: int) -> int:
    """Workspace bytes himuon_grouped_wgrad needs for operands like x and dy and
    n experts."""
    need = ctypes.c_size_t(0)
    a, b = _rows(x), _rows(dy)
    _check(lib.himuon_grouped_wgrad_workspace(ctypes.byref(a), ctypes.byref(b), n, _dtype_code(x), ctypes.byref(need)),
           "himuon_grouped_wgrad_workspace")
    return need.value


def himuon_grouped_wgrad(x, dy, ends, out=None, workspace=None, stream=None):
    """The weight gradients x_e^T dy_e of every expert, (n, K, N) or the given
    `out` (as matrices() takes them; transposed views are written as stored).
    Zero for an expert without rows."""
    import torch
    _need_gpu(x, dy, ends)
    if x.dtype != dy.dtype:
        raise TypeError("x and dy must have one dtype")
    n = ends.shape[0]
    with _placed(x.device, stream) as s:
        if out is None:
            out = torch.empty((n, x.shape[1], dy.shape[1]), dtype=x.dtype, device=x.device)
        g = matrices(out)
        if g.dtype != x.dtype or g.device != x.device:
            raise TypeError("out must have the operands' dtype and device")
        if g.n != n or g.shape != (x.shape[1], dy.shape[1]):
            raise ValueError("out must hold one (K, N) matrix per expert")
        a, b = (_rows(dy), _rows(x)) if g.transposed else (_rows(x), _rows(dy))
        code = _dtype_code(x)
        keep, wp, wb = _scratch(lib.himuon_grouped_wgrad_workspace, "himuon_grouped_wgrad_workspace", workspace,
                                x.device, ctypes.byref(a), ctypes.byref(b), n, code)
        _check(lib.himuon_grouped_wgrad(ctypes.byref(a), ctypes.byref(b), _ends(ends, n, x.device), g.array, n, code,
                                        wp, wb, s), "himuon_grouped_wgrad")
    return out


class Gated(NamedTuple):
    h: object
    pre: object = None


class GatedGrad(NamedTuple):
    grad: object
    h: object = None


def _activation(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def _filled(t, rows, cols, like, what):
    """t, or a new tensor, of the given shape, with the type and place of `like`, and
    its descriptor."""
    if t is None:
        t = like.new_empty((rows, cols))
        return t, himuon_matrix_t(t.data_ptr(), rows, cols, cols)
    if t.dtype != like.dtype:
        raise TypeError(f"{what} must have the operands' dtype")
    if t.shape != (rows, cols) or t.device != like.device:
        raise ValueError(f"{what} must be of shape {(rows, cols)}, on the operands' GPU")
    return t, _rows(t)


def himuon_grouped_gated_mm(x, w, ends, act: str = "silu", keep=False, out=None, stream=None) -> Gated:
    """The gated experts' block up to its down product: with [g | u] = x[r] @ w[e]
    for the rows r of expert e, h = act(g) * u, in one kernel.

    x: (M, K), rows sorted by expert.  w: the experts' (K, 2 N) weights as
    matrices() takes them, the gate's projection in the first N columns.  ends: as
    for himuon_grouped_mm.  act: silu, gelu, gelu_tanh or relu.  keep: also
    [g | u] (M, 2 N), for the gradient: True, or the tensor to write.  out:
    optional (M, N) tensor.  Returns (h, pre)."""
    w = matrices(w)
    K, N2 = w.shape
    _need_gpu(x, w, ends)
    if x.dtype != w.dtype:
        raise TypeError("x and w must have one dtype")
    if N2 % 2:
        raise ValueError("w must hold as many gate as up columns")
    code = _activation(act)
    with _placed(x.device, stream) as s:
        M = x.shape[0]
        h, dh = _filled(out, M, N2 // 2, x, "out")
        pre = dp = None
        if keep is not False and keep is not None:
            pre, dp = _filled(None if keep is True else keep, M, N2, x, "keep")
        dx = _rows(x)
        _check(lib.himuon_grouped_gated_mm(ctypes.byref(dx), w.array, w.n, int(w.transposed), _ends(ends, w.n, x.device),
                                           ctypes.byref(dh), None if dp is None else ctypes.byref(dp), code,
                                           _dtype_code(x), s), "himuon_grouped_gated_mm")
    return Gated(h, pre)


def himuon_grouped_gated_mm_grad(dy, w, ends, pre, act: str = "silu", hidden=False, out=None, stream=None) -> GatedGrad:
    """Back through the block's down product y = h @ w[e] and its gate in one
    kernel: from dy (M, K) and the forward pass's pre = [g | u] (M, 2 N) the
    gradient of pre.

    w: the down product's (N, K) weights as matrices() takes them.  hidden: also h
    again (M, N), for the gradient of w: True, or the tensor to write.  out: the
    tensor to write, which may be pre itself.  Returns (grad, h).  The block's other
    gradients are himuon_grouped_mm(grad, w_in.transpose(1, 2), ends),
    himuon_grouped_wgrad(x, grad, ends) and himuon_grouped_wgrad(h, dy, ends)."""
    w = matrices(w)
    N, K = w.shape
    _need_gpu(dy, w, ends, pre)
    if dy.dtype != w.dtype or pre.dtype != dy.dtype:
        raise TypeError("dy, w and pre must have one dtype")
    code = _activation(act)
    with _placed(dy.device, stream) as s:
        M = dy.shape[0]
        grad, dg = _filled(out, M, 2 * N, dy, "out")
        h = dh = None
        if hidden is not False and hidden is not None:
            h, dh = _filled(None if hidden is True else hidden, M, N, dy, "hidden")
        dd, dp = _rows(dy), _rows(pre)
        _check(lib.himuon_grouped_gated_mm_grad(ctypes.byref(dd), w.array, w.n, int(w.transposed),
                                                _ends(ends, w.n, dy.device), ctypes.byref(dp), ctypes.byref(dg),
                                                None if dh is None else ctypes.byref(dh), code, _dtype_code(dy), s),
               "himuon_grouped_gated_mm_grad")
    return GatedGrad(grad, h)


# ---- layer normalisation -----------------------------------------------------------
class Normed(NamedTuple):
    y: object
    stats: object = None


class NormGrad(NamedTuple):
    dx: object = None
    dweight: object = None
    dbias: object = None


def _columns(t, x, what):
    if t is None:
        return None
    if t.dtype != x.dtype:
        raise TypeError(f"{what} must have the rows' dtype")
    if t.shape != (x.shape[1],) or not t.is_contiguous() or t.device != x.device:
        raise ValueError(f"{what} must be contiguous with one entry per column, on the rows' GPU")
    return t.data_ptr()


def himuon_layer_norm(x, weight=None, bias=None, eps: float = 1e-5, stats: bool = True, out=None,
                      stream=None) -> Normed:
    """Layer normalisation of the rows of x (N, D): (x - mean) / sqrt(var + eps) *
    weight + bias.  weight, bias: (D,) of x's type, or None.  out: the tensor to
    write, which may be x.  Returns (y, stats), stats (N, 2) float32, mean and 1 /
    sqrt(var + eps), for himuon_layer_norm_grad (None with stats=False)."""
    import torch
    _need_gpu(x)
    dx = _rows(x)
    with _placed(x.device, stream) as s:
        y, dy = _filled(out, dx.rows, dx.cols, x, "out")
        st = torch.empty((dx.rows, 2), dtype=torch.float32, device=x.device) if stats else None
        _check(lib.himuon_layer_norm(ctypes.byref(dx), _columns(weight, x, "weight"), _columns(bias, x, "bias"), eps,
                                     ctypes.byref(dy), None if st is None else st.data_ptr(), _dtype_code(x), s),
               "himuon_layer_norm")
    return Normed(y, st)


def himuon_layer_norm_grad_workspace(x) -> int:
    """Workspace bytes himuon_layer_norm_grad needs for rows like x."""
    need = ctypes.c_size_t(0)
    dx = _rows(x)
    _check(lib.himuon_layer_norm_grad_workspace(ctypes.byref(dx), _dtype_code(x), ctypes.byref(need)),
           "himuon_layer_norm_grad_workspace")
    return need.value


def himuon_layer_norm_grad(x, weight, stats, dy, dx=True, dweight=True, dbias=True, workspace=None,
                           stream=None) -> NormGrad:
    """Gradients of himuon_layer_norm's x, weight and bias from dy (N, D) and the
    stats of the forward call.  dx, dweight, dbias: True, the tensor to write (dx may
    be dy or x), or False.  Returns (dx, dweight, dbias)."""
    import torch
    _need_gpu(x, stats, dy)
    if dy.dtype != x.dtype:
        raise TypeError("x and dy must have one dtype")
    N, D = x.shape
    sp = _vector(stats, N, "stats", x.device, 2)
    wanted = lambda t: t is not None and t is not False
    with _placed(x.device, stream) as s:
        gx, c = _filled(None if dx is True else dx, N, D, x, "dx") if wanted(dx) else (None, None)
        vec = lambda t: x.new_empty(D) if t is True else t
        gw, gb = vec(dweight) if wanted(dweight) else None, vec(dbias) if wanted(dbias) else None
        a, b = _rows(x), _rows(dy)
        code = _dtype_code(x)
        keep, wp, wb = None, None, 0
        if gw is not None or gb is not None:
            keep, wp, wb = _scratch(lib.himuon_layer_norm_grad_workspace, "himuon_layer_norm_grad_workspace", workspace,
                                    x.device, ctypes.byref(a), code)
        _check(lib.himuon_layer_norm_grad(ctypes.byref(a), _columns(weight, x, "weight"), sp, ctypes.byref(b),
                                          None if c is None else ctypes.byref(c), _columns(gw, x, "dweight"),
                                          _columns(gb, x, "dbias"), code, wp, wb, s), "himuon_layer_norm_grad")
    return NormGrad(gx, gw, gb)


# ---- AdamW -------------------------------------------------------------------------
class Tensors:
    """Descriptors of tensors of any shapes, made once and used for any number of
    calls.  It keeps the tensors, whose values may change but not their place (see
    Matrices)."""

    def __init__(self, array, tensors, dtype, device, shapes):
        self.array, self.tensors, self.dtype, self.device = array, tensors, dtype, device
        self.shapes, self.key = shapes, repr(shapes).encode()   # (bytes compare at once)
        self.places = self._places()

    def _places(self):
        import torch
        return list(map(torch.Tensor.data_ptr, self.tensors))

    def in_place(self):
        """Itself, if the tensors are still where they were described."""
        if self._places() != self.places:
            raise ValueError("tensors were described before they got other memory: describe them again")
        return self

    def __len__(self):
        return len(self.tensors)


def tensors(ts) -> Tensors:
    """Descriptors of bf16 or fp32 tensors of one type on one GPU: contiguous ones
    of any shape, or 2-D ones with unit stride along the rows."""
    if isinstance(ts, Tensors):
        return ts.in_place()
    ts = list(ts)
    arr = (himuon_matrix_t * max(len(ts), 1))()
    if not ts:
        return Tensors(arr, ts, None, None, [])
    first = ts[0]
    if not first.is_cuda:
        raise ValueError("tensors must be on one GPU")
    dtype, device = first.dtype, first.device
    _dtype_code(first)
    for i, t in enumerate(ts):
        if t.dtype != dtype:
            raise TypeError("tensors must have one dtype")
        if t.device != device:
            raise ValueError("tensors must be on one GPU")
        n = t.numel()
        if n == 0:
            raise ValueError("tensors must not be empty")
        if t.is_contiguous():
            cols = t.shape[-1] if t.dim() else 1
            arr[i] = himuon_matrix_t(t.data_ptr(), n // cols, cols, cols)
        elif t.dim() <= 2:
            arr[i] = _rows(t if t.dim() == 2 else t.unsqueeze(0))
        else:
            raise ValueError("tensors must be contiguous, or 2-D with unit stride along the rows")
    return Tensors(arr, ts, dtype, device, [tuple(t.shape) for t in ts])


class AdamWState:
    """States of an AdamW step for given tensors, zero at first.  m and v are flat,
    each tensor's part beginning at a multiple of ADAMW_BLOCK elements (`starts`):
    float32 (bits=32), or float8_e4m3fn codes of m and of sqrt(v) with one float32
    scale for each block, m_scale and v_scale (bits=8)."""

    def __init__(self, like: Tensors, bits: int):
        import numpy as np
        import torch
        if bits not in (8, 32):
            raise ValueError("bits must be 8 or 32")
        self.bits, self.shapes, self.key, self.device = bits, like.shapes, like.key, like.device
        n = len(like)
        sizes = np.array([like.array[i].rows * like.array[i].cols for i in range(n)], dtype=np.int64)
        blocks = -(-sizes // ADAMW_BLOCK)
        firsts = np.concatenate([[0], np.cumsum(blocks)]).astype(np.int64)
        self.starts = (firsts[:-1] * ADAMW_BLOCK).tolist()
        total = int(firsts[-1])
        dtype = torch.float32 if bits == 32 else torch.float8_e4m3fn
        flat = lambda: torch.zeros(total * ADAMW_BLOCK, dtype=torch.float32 if bits == 32 else torch.uint8,
                                   device=like.device).view(dtype)
        self.m, self.v = flat(), flat()
        self.m_scale = self.v_scale = None
        if bits == 8:
            self.m_scale, self.v_scale = (torch.zeros(total, dtype=torch.float32, device=like.device) for _ in range(2))
        es = self.m.element_size()
        a = np.zeros((max(n, 1), 4), dtype=np.int64)
        if n:
            a[:, 0] = self.m.data_ptr() + firsts[:-1] * (ADAMW_BLOCK * es)
            a[:, 1] = self.v.data_ptr() + firsts[:-1] * (ADAMW_BLOCK * es)
            if bits == 8:
                a[:, 2] = self.m_scale.data_ptr() + firsts[:-1] * 4
                a[:, 3] = self.v_scale.data_ptr() + firsts[:-1] * 4
        self.array = (himuon_adamw_state_t * max(n, 1)).from_buffer(a)
        self.places = self._places()

    def _places(self):
        return [t.data_ptr() for t in (self.m, self.v, self.m_scale, self.v_scale) if t is not None]

    def in_place(self):
        """Itself, if its tensors are still where they were made (load saved states
        with copy_)."""
        if self._places() != self.places:
            raise ValueError("states got other memory: copy into them instead")
        return self


def adamw_state(like, bits: int = 32) -> AdamWState:
    """New (zero) states for tensors as himuon_adamw_step takes them."""
    import torch
    like = tensors(like)
    if like.device is None:
        return AdamWState(like, bits)
    with torch.cuda.device(like.device):
        return AdamWState(like, bits)


def himuon_adamw_step(w, g, state: AdamWState, lr: float, step: int, betas=(0.9, 0.999), eps: float = 1e-8,
                      weight_decay: float = 0.0, grad_scale=None, stream=None):
    """One AdamW step on all tensors of w at once, in place, from gradients g and
    the states adamw_state(w) made.  w, g: lists of tensors (bf16 or fp32, each list
    of one type, which may differ), or what tensors() made of them once (a list is
    described anew in each call: 1 us of the host's time a tensor).  step: 1 in the
    first step.  grad_scale: float32 tensor of one element on the GPU that the
    gradients are multiplied by.  A captured call repeats its lr and step, and so 8-bit
    states' random bits: slow averages may not move in its replays, so such steps are
    to be called, not replayed."""
    import torch
    w, g = tensors(w), tensors(g)
    state.in_place()
    if w.key != g.key or w.key != state.key:
        raise ValueError("weights, gradients and states must agree in number and shapes")
    if len(w) == 0:
        return
    if g.device != w.device or state.device != w.device:
        raise ValueError("tensors must be on one GPU")
    sp = None
    if grad_scale is not None:
        if grad_scale.dtype != torch.float32:
            raise TypeError("grad_scale must be float32")
        if grad_scale.numel() != 1 or grad_scale.device != w.device:
            raise ValueError("grad_scale must be one element, on the tensors' GPU")
        sp = ctypes.c_void_p(grad_scale.data_ptr())
    with _placed(w.device, stream) as s:
        _check(lib.himuon_adamw_step(w.array, g.array, state.array, len(w), state.bits, lr, betas[0], betas[1], eps,
                                     weight_decay, step, sp, _dtype_code(w), _dtype_code(g), s), "himuon_adamw_step")


# ---- losses over logits ------------------------------------------------------------
class Distilled(NamedTuple):
    loss: object
    lse: object
    grad: object = None


class TokenLogprobs(NamedTuple):
    logp: object
    entropy: object
    lse: object
    top_idx: object = None
    top_logp: object = None


def _vector(t, n, what, device, width=0):
    import torch
    if t is None:
        return None
    if t.dtype != torch.float32:
        raise TypeError(f"{what} must be float32")
    if t.shape != ((n, width) if width else (n,)) or not t.is_contiguous() or t.device != device:
        entry = f"{width} entries" if width else "one entry"
        raise ValueError(f"{what} must be contiguous with {entry} per row, on the rows' GPU")
    return ctypes.c_void_p(t.data_ptr())


def _ids(t, shape, what, device):
    import torch
    if t is None:
        return None, 1
    if t.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{what} must be int32 or int64")
    if t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what} must be contiguous, of shape {tuple(shape)}, on the logits' GPU")
    return ctypes.c_void_p(t.data_ptr()), int(t.dtype == torch.int64)


def _scratch(size_fn, where, workspace, device, *args):
    """(tensor kept alive, pointer, bytes) of a call's workspace."""
    import torch
    if workspace is None:
        need = ctypes.c_size_t(0)
        _check(size_fn(*args, ctypes.byref(need)), where)
        if need.value == 0:
            return None, None, 0
        workspace = torch.empty(need.value, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        # (an expanded tensor has less memory than elements)
        raise ValueError("workspace must be contiguous, on the operands' GPU")
    return workspace, ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()


def _teacher(z, idx, t):
    import torch
    if t.dtype != torch.float32:
        raise TypeError("teacher values must be float32")
    if t.dim() != 2 or t.shape[0] != z.shape[0]:
        raise ValueError("teacher values must have one row per row of logits")
    _need_gpu(z, idx, t)
    return (_rows(t), *_ids(idx, t.shape, "idx", z.device))


def _grad_out(z, out):
    import torch
    if out is None:
        out = torch.empty(z.shape, dtype=z.dtype, device=z.device)
    elif out.dtype != z.dtype or out.shape != z.shape or out.device != z.device:
        raise ValueError("the gradient must have the logits' dtype, shape and device")
    return out, _rows(out)


def himuon_distill_workspace(z, grad: bool = False) -> int:
    """Workspace bytes himuon_distill needs for logits like z."""
    need = ctypes.c_size_t(0)
    dz = _rows(z)
    _check(lib.himuon_distill_workspace(ctypes.byref(dz), _dtype_code(z), int(grad), ctypes.byref(need)),
           "himuon_distill_workspace")
    return need.value


def himuon_distill(z, idx, t, temperature: float = 1.0, normalize: bool = True, weight=None, grad=False,
                   workspace=None, stream=None) -> Distilled:
    """Loss of each row of student logits z (N, V) against a teacher's top
    entries: ids idx (N, k) and values t (N, k, float32); absent entries have an
    id outside [0, V).  normalize: the teacher's probabilities are the softmax
    of t / temperature over the row's entries, else exp(t).  grad: also the
    gradient of sum(loss) in the same call: True, or the tensor to write (z
    itself is allowed).  Returns (loss, lse, grad); lse is (N, 2), log sum exp of
    z / temperature and what its rounding to fp32 lost."""
    import torch
    T, ip, i64 = _teacher(z, idx, t)
    dev = z.device
    with _placed(dev, stream) as s:
        N = z.shape[0]
        loss = torch.empty(N, dtype=torch.float32, device=dev)
        lse = torch.empty((N, 2), dtype=torch.float32, device=dev)
        dz = _rows(z)
        g = dg = None
        if grad is not False and grad is not None:
            g, dg = _grad_out(z, None if grad is True else grad)
        keep, wp, wb = _scratch(lib.himuon_distill_workspace, "himuon_distill_workspace", workspace, dev,
                                ctypes.byref(dz), _dtype_code(z), int(g is not None))
        _check(lib.himuon_distill(ctypes.byref(dz), ip, i64, ctypes.byref(T), temperature, int(normalize),
                                  _vector(weight, N, "weight", dev), ctypes.c_void_p(loss.data_ptr()),
                                  ctypes.c_void_p(lse.data_ptr()), ctypes.byref(dg) if g is not None else None,
                                  _dtype_code(z), wp, wb, s), "himuon_distill")
    return Distilled(loss, lse, g)


def himuon_distill_grad(z, idx, t, lse, g, temperature: float = 1.0, normalize: bool = True, out=None, stream=None):
    """The gradient of the logits alone, from the lse of a himuon_distill call
    and the gradients g (N,) of the unweighted row losses."""
    T, ip, i64 = _teacher(z, idx, t)
    dev = z.device
    N = z.shape[0]
    with _placed(dev, stream) as s:
        out, do = _grad_out(z, out)
        dz = _rows(z)
        _check(lib.himuon_distill_grad(ctypes.byref(dz), ip, i64, ctypes.byref(T), temperature, int(normalize),
                                       _vector(lse, N, "lse", dev, 2), _vector(g, N, "g", dev), ctypes.byref(do),
                                       _dtype_code(z), s), "himuon_distill_grad")
    return out


def himuon_token_logprobs_workspace(z, top: int = 0) -> int:
    """Workspace bytes himuon_token_logprobs needs for logits like z."""
    need = ctypes.c_size_t(0)
    dz = _rows(z)
    _check(lib.himuon_token_logprobs_workspace(ctypes.byref(dz), top, _dtype_code(z), ctypes.byref(need)),
           "himuon_token_logprobs_workspace")
    return need.value


def himuon_token_logprobs(z, tokens=None, top: int = 0, temperature: float = 1.0, workspace=None,
                          stream=None) -> TokenLogprobs:
    """Log probabilities of the given tokens (N,) under softmax(z / temperature)
    of logits z (N, V), with each row's entropy, lse and, for top > 0, its top
    alternatives (ids int32, best first, and their log probabilities).  A token
    outside [0, V) skips its row.  Without tokens logp is None."""
    import torch
    if tokens is None:
        _need_gpu(z)
    else:
        _need_gpu(z, tokens)
    dev = z.device
    N = z.shape[0]
    tp, i64 = _ids(tokens, (N,), "tokens", dev)
    with _placed(dev, stream) as s:
        vec = lambda: torch.empty(N, dtype=torch.float32, device=dev)
        logp, entropy = vec() if tokens is not None else None, vec()
        lse = torch.empty((N, 2), dtype=torch.float32, device=dev)
        ti = torch.empty((N, top), dtype=torch.int32, device=dev) if top > 0 else None
        tl = torch.empty((N, top), dtype=torch.float32, device=dev) if top > 0 else None
        ptr = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())
        dz = _rows(z)
        keep, wp, wb = _scratch(lib.himuon_token_logprobs_workspace, "himuon_token_logprobs_workspace", workspace, dev,
                                ctypes.byref(dz), top, _dtype_code(z))
        _check(lib.himuon_token_logprobs(ctypes.byref(dz), tp, i64, temperature, top, ptr(logp), ptr(entropy),
                                         ptr(lse), ptr(ti), ptr(tl), _dtype_code(z), wp, wb, s),
               "himuon_token_logprobs")
    return TokenLogprobs(logp, entropy, lse, ti, tl)


def himuon_token_logprobs_grad(z, tokens, lse, entropy, g_logp=None, g_entropy=None, temperature: float = 1.0,
                               out=None, stream=None):
    """The gradient of the logits through logp and entropy, from the lse and
    entropy of a himuon_token_logprobs call and the gradients (N,) of each."""
    if tokens is None:
        _need_gpu(z)
    else:
        _need_gpu(z, tokens)
    dev = z.device
    N = z.shape[0]
    tp, i64 = _ids(tokens, (N,), "tokens", dev)
    with _placed(dev, stream) as s:
        out, do = _grad_out(z, out)
        dz = _rows(z)
        _check(lib.himuon_token_logprobs_grad(ctypes.byref(dz), tp, i64, temperature, _vector(lse, N, "lse", dev, 2),
                                              _vector(entropy, N, "entropy", dev),
                                              _vector(g_logp, N, "g_logp", dev),
                                              _vector(g_entropy, N, "g_entropy", dev), ctypes.byref(do),
                                              _dtype_code(z), s), "himuon_token_logprobs_grad")
    return out


def himuon_status_string(code: int) -> str:
    return lib.himuon_status_string(code).decode()


def himuon_last_hip_error() -> int:
    return lib.himuon_last_hip_error()


def himuon_version() -> int:
    return lib.himuon_version()
