"""W12 for GB300: Python binding of the C-ABI library libw12.so.

W12 is the lossless 12-bit BF16 weight format of "SpecPilot" (arXiv
2611.02501), section 4.1.  Every step of encode, decode, verify and GEMM runs
in the library's CUDA kernels; this module only marshals arguments (torch
tensors -> device pointers, the current CUDA stream) and allocates device
memory through torch.  There is no CPU fallback: if the library cannot be
loaded, every call raises.

Entry points (same names as the C ABI in include/w12.h):
    w12_encode(W)                      -> W12Tensor
    w12_decode(t, out=None)            -> torch.bfloat16 [N,K]
    w12_verify_roundtrip(W, t)         -> (status, n_mismatch)
    w12_gemm(A, t, Y=None, ...)        -> torch.bfloat16 [M,N]
    w12_gemm_workspace_bytes(M, N, K)  -> int
    w12_rmsnorm(x, weight, ...)        -> dict of y / h / q8 / scale
    w12_rope_append(q, k, pos, ...)    -> (q, k), and keys and values into a paged cache
    w12_tree_attn(q, k, v, cache, ...) -> torch.bfloat16 [n, heads, dim]
    w12_tree_accept(logits, token, parent, ...) -> dict of count / nodes / next
    w12_gdn_scan(S, q, k, v, alpha, beta, ...)  -> (outputs, states)
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libw12.so")

W12_OK = 0
W12_ERR_INVALID = -1
W12_ERR_ALIGN = -2
W12_ERR_CAPACITY = -3
W12_ERR_CUDA = -4
W12_ERR_MISMATCH = -5
W12_ERR_TIMEOUT = -6
W12_ERR_CORRUPT = -7
W12_ERR_UNSUPPORTED = -8

W12_PATH_AUTO, W12_PATH_MMA, W12_PATH_TC = 0, 1, 2
W12_GEMM_OVERLAP_PREVIOUS = 1
W12_GEMM_NESTED8 = 2  # multiply by the nested 8-bit view (hi plane only)
W12_GEMM_SILU_MUL = 4  # fused gate/up epilogue: Y[m, 8s+i] = silu(row 16s+i) * (row 16s+8+i)
W12_GEMM_TEST_STALL = 1 << 30  # tests only: one bounded wait runs out
W12_LIST_MAX = 64  # GEMMs per launch of w12_gemm_list

# Every symbol include/w12.h declares.
EXPORTS = (
    "w12_rows_padded", "w12_cols_padded", "w12_hi_bytes", "w12_lo_bytes", "w12_groups",
    "w12_esc_ptr_len", "w12_encode", "w12_encode_test_stall",
    "w12_decode", "w12_verify_workspace_bytes", "w12_verify_roundtrip",
    "w12_gemm_workspace_bytes", "w12_gemm", "w12_gemm_noalloc", "w12_gemm_noalloc_status",
    "w12_gemm_workspace_status", "w12_gemm_list_workspace_bytes", "w12_gemm_list",
    "w12_tree_workspace_bytes", "w12_tree_select",
    "w12_gdn_workspace_bytes", "w12_gdn_tree", "w12_gdn_status",
    "w12_rmsnorm", "w12_rope_append",
    "w12_tree_attn_workspace_bytes", "w12_tree_attn", "w12_tree_attn_status",
    "w12_tree_accept", "w12_gdn_scan_workspace_bytes", "w12_gdn_scan",
    "w12_status_string", "w12_version",
)

# Size of the scratch array built into the library for w12_gemm_noalloc.
W12_NOALLOC_SCRATCH_BYTES = 4 << 20


class W12Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class _Tensor(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("hi", ctypes.c_void_p), ("lo", ctypes.c_void_p), ("base", ctypes.c_void_p),
        ("esc_ptr", ctypes.c_void_p), ("esc", ctypes.c_void_p),
        ("esc_cap", ctypes.c_int64), ("n_esc", ctypes.c_int64),
    ]


class GemmItem(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("lda", ctypes.c_int64), ("w", ctypes.POINTER(_Tensor)),
                ("Y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("M", ctypes.c_int64),
                ("after", ctypes.c_int32), ("flags", ctypes.c_int32)]


class GemmOpts(ctypes.Structure):
    _fields_ = [("max_ctas", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("path", ctypes.c_int32), ("flags", ctypes.c_int32)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_tokens", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


# w12_rope_args and w12_attn_args, packed in one step (native alignment): a
# ctypes structure set field by field took longer than the launches.
_rope_args = struct.Struct("@PPP qqq PP qq q iii ii P q i P P PP f P P")
_attn_args = struct.Struct("@PPP qqq P q qq i P q i PPP ff iii 4x")
_accept_args = struct.Struct("@P qqq i PPPPP qq P f PP q P qq P i PPP q")
_scan_args = struct.Struct("@PP PPP qqq PP P q i PPP q i qq iiii P")


_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load libw12.so (raises if it is missing: there is no fallback)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libw12.so not built ({p}); run __graft_entry__.build() or "
                               "python lossless_bit_weight_02_gb300/_build.py")
        lib = ctypes.CDLL(p)
        i64, vp, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
        st = ctypes.c_int
        sig = {
            "w12_rows_padded": (i64, [i64]),
            "w12_cols_padded": (i64, [i64]),
            "w12_hi_bytes": (i64, [i64, i64]),
            "w12_lo_bytes": (i64, [i64, i64]),
            "w12_groups": (i64, [i64]),
            "w12_esc_ptr_len": (i64, [i64, i64]),
            "w12_encode": (st, [vp, i64, ctypes.POINTER(_Tensor), vp]),
            "w12_encode_test_stall": (None, [ctypes.c_int]),
            "w12_decode": (st, [ctypes.POINTER(_Tensor), vp, i64, vp]),
            "w12_verify_workspace_bytes": (sz, []),
            "w12_verify_roundtrip": (st, [vp, i64, ctypes.POINTER(_Tensor), ctypes.POINTER(i64), vp, sz, vp]),
            "w12_gemm_workspace_bytes": (sz, [i64, i64, i64, ctypes.POINTER(GemmOpts)]),
            "w12_gemm": (st, [vp, i64, ctypes.POINTER(_Tensor), vp, i64, i64, vp, sz,
                              ctypes.POINTER(GemmOpts), vp]),
            "w12_gemm_noalloc": (st, [vp, i64, ctypes.POINTER(_Tensor), vp, i64, i64,
                                      ctypes.POINTER(GemmOpts), vp]),
            "w12_gemm_noalloc_status": (st, [vp]),
            "w12_gemm_workspace_status": (st, [vp, sz, vp]),
            "w12_gemm_list_workspace_bytes": (sz, [ctypes.POINTER(GemmItem), ctypes.c_int32,
                                                   ctypes.POINTER(GemmOpts)]),
            "w12_gemm_list": (st, [ctypes.POINTER(GemmItem), ctypes.c_int32, vp, sz, ctypes.POINTER(GemmOpts), vp]),
            "w12_tree_workspace_bytes": (sz, [ctypes.c_int32, ctypes.c_int32]),
            "w12_tree_select": (st, [vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                     ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "w12_gdn_workspace_bytes": (sz, [i64, i64, i64, ctypes.c_int32]),
            "w12_gdn_tree": (st, [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp, sz,
                                  ctypes.c_int32, vp]),
            "w12_gdn_status": (st, [vp, sz, vp]),
            "w12_rmsnorm": (st, [vp, i64, vp, i64, vp, ctypes.c_float, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                 vp]),
            "w12_rope_append": (st, [ctypes.c_char_p, vp]),
            "w12_tree_attn_workspace_bytes": (sz, [i64, i64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]),
            "w12_tree_attn": (st, [ctypes.c_char_p, vp, vp, sz, vp]),
            "w12_tree_attn_status": (st, [vp, sz, vp]),
            "w12_tree_accept": (st, [ctypes.c_char_p, vp]),
            "w12_gdn_scan_workspace_bytes": (sz, [i64, i64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]),
            "w12_gdn_scan": (st, [ctypes.c_char_p, vp, sz, vp]),
            "w12_status_string": (ctypes.c_char_p, [st]),
            "w12_version": (ctypes.c_int32, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    try:
        return load().w12_status_string(status).decode()
    except Exception:
        return f"status {status}"


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None) -> ctypes.c_void_p:
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _raw_stream is not None:  # the current stream's handle without building a Stream object
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(status: int, what: str):
    if status != W12_OK:
        raise W12Error(status, what)


def _need_cuda(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _out_cols(t: "W12Tensor", flags: int) -> int:
    return t.N // 2 if flags & W12_GEMM_SILU_MUL else t.N


def _check_gemm_operands(A: torch.Tensor, t: "W12Tensor", Y: torch.Tensor | None, flags: int = 0):
    """The C side trusts lda / ldy and writes M rows of N outputs, so the
    shapes, strides and devices are checked here, before any pointer is
    passed: A is [M, K] and Y is [M, N] ([M, N/2] with W12_GEMM_SILU_MUL),
    both with unit column stride, on the device that holds the W12 tensor,
    which must be the current device (the library launches on the current
    device)."""
    if flags & W12_GEMM_SILU_MUL and t.N % 16:
        raise ValueError(f"W12_GEMM_SILU_MUL needs N a multiple of 16, got {t.N}")
    _need_cuda(A, "A", torch.bfloat16)
    if A.dim() != 2 or A.shape[1] != t.K or (A.shape[0] > 0 and t.K > 0 and A.stride(1) != 1):
        raise ValueError(f"A must be [M, {t.K}] with unit column stride, got {tuple(A.shape)} "
                         f"strides {A.stride()}")
    dev = t.hi.device
    if A.device != dev:
        raise ValueError(f"A is on {A.device}, the W12 tensor on {dev}")
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"the W12 tensor is on {dev} but the current device is cuda:{torch.cuda.current_device()}")
    if Y is not None:
        _need_cuda(Y, "Y", torch.bfloat16)
        cols = _out_cols(t, flags)
        if Y.dim() != 2 or tuple(Y.shape) != (A.shape[0], cols) or (Y.numel() > 0 and Y.stride(1) != 1):
            raise ValueError(f"Y must be [{A.shape[0]}, {cols}] with unit column stride, got {tuple(Y.shape)} "
                             f"strides {Y.stride()}")
        if Y.device != dev:
            raise ValueError(f"Y is on {Y.device}, the W12 tensor on {dev}")


@dataclass
class W12Tensor:
    """A W12 tensor in device memory (all arrays are torch CUDA tensors)."""
    N: int
    K: int
    hi: torch.Tensor       # uint8 [Np*Kp]
    lo: torch.Tensor       # uint8 [Np*Kp/2]
    base: torch.Tensor     # uint8 [N]
    esc_ptr: torch.Tensor  # int32 [Np/16 * groups(K) + 1]
    esc: torch.Tensor      # int32 [esc_cap] (bit pattern of key<<16 | BF16 bits)
    n_esc: int

    @property
    def esc_cap(self) -> int:
        return self.esc.numel()

    def struct(self) -> _Tensor:
        """The C view of the tensor, cached while the same array objects and
        shape are in place (n_esc is refreshed on every call); arrays must not
        be re-pointed in place (Tensor.set_)."""
        c = self.__dict__.get("_cview")
        if (c is None or c[0] is not self.hi or c[1] is not self.lo or c[2] is not self.base
                or c[3] is not self.esc_ptr or c[4] is not self.esc or c[5] != (self.N, self.K)):
            s = _Tensor(self.N, self.K, self.hi.data_ptr(), self.lo.data_ptr(), self.base.data_ptr(),
                        self.esc_ptr.data_ptr(), self.esc.data_ptr(), self.esc_cap, self.n_esc)
            c = (self.hi, self.lo, self.base, self.esc_ptr, self.esc, (self.N, self.K), s)
            self.__dict__["_cview"] = c
        s = c[6]
        s.n_esc = self.n_esc
        return s

    def nbytes(self) -> int:
        """Bytes the tensor stores (all of which the GEMM reads): both
        planes, bases, group offsets and escape entries."""
        return self.hi.numel() + self.lo.numel() + self.N + 4 * self.esc_ptr.numel() + 4 * self.n_esc

    def bits_per_weight(self) -> float:
        return 8.0 * self.nbytes() / max(1, self.N * self.K)

    def rows(self, n0: int, n1: int) -> "W12Tensor":
        """Rows [n0, n1) as a W12 tensor of their own (n0 a multiple of 16):
        plane tiles, bases and the stripes' escape entries are sliced, the
        group offsets rebased (a fresh device tensor)."""
        assert 0 <= n0 <= n1 <= self.N and n0 % 16 == 0
        KT = cols_padded(self.K) // 64
        G = groups(self.K)
        t0, t1 = n0 // 16, (n1 + 15) // 16
        ptr = self.esc_ptr[t0 * G:t1 * G + 1]
        e0 = int(ptr[0].item())
        e1 = int(ptr[-1].item())
        return W12Tensor(n1 - n0, self.K, self.hi[t0 * KT * 1024:t1 * KT * 1024],
                         self.lo[t0 * KT * 512:t1 * KT * 512], self.base[n0:n1], (ptr - e0).contiguous(),
                         self.esc[e0:e1], e1 - e0)


def rows_padded(N: int) -> int:
    return int(load().w12_rows_padded(N))


def groups(K: int) -> int:
    return int(load().w12_groups(K))


def cols_padded(K: int) -> int:
    return int(load().w12_cols_padded(K))


_array_sizes: dict = {}


def _sizes_of(N: int, K: int):
    """(hi bytes, lo bytes, esc_ptr entries) from the library's size queries,
    kept per shape."""
    key = (N, K)
    v = _array_sizes.get(key)
    if v is None:
        lib = load()
        v = (int(lib.w12_hi_bytes(N, K)), int(lib.w12_lo_bytes(N, K)), int(lib.w12_esc_ptr_len(N, K)))
        _array_sizes[key] = v
    return v


def empty_tensor(N: int, K: int, esc_cap: int, device) -> W12Tensor:
    """An uninitialised W12 tensor: one device allocation, the five arrays
    carved out of it at 256-byte aligned offsets."""
    hb, lb, pl = _sizes_of(N, K)
    a = lambda x: (x + 255) & ~255
    o_lo = a(hb)
    o_base = o_lo + a(lb)
    o_ptr = o_base + a(N)
    o_esc = o_ptr + a(4 * pl)
    buf = torch.empty(max(1, o_esc + 4 * esc_cap), dtype=torch.uint8, device=device)
    return W12Tensor(N, K, buf[:hb], buf[o_lo:o_lo + lb], buf[o_base:o_base + N],
                     buf[o_ptr:o_ptr + 4 * pl].view(torch.int32), buf[o_esc:o_esc + 4 * esc_cap].view(torch.int32), 0)


def w12_encode(W: torch.Tensor, esc_cap: int | None = None, stream=None, out: W12Tensor | None = None) -> W12Tensor:
    """BF16 [N,K] (CUDA) -> W12Tensor.  Grows the escape arrays if needed.
    With `out` (a W12Tensor of the same N, K, e.g. from empty_tensor), encodes
    into its buffers instead of allocating; its escape array keeps its
    capacity (entries past n_esc are unused), and a tensor needing more
    escapes than it holds raises W12Error(W12_ERR_CAPACITY)."""
    _need_cuda(W, "W", torch.bfloat16)
    assert W.dim() == 2 and W.stride(1) == 1
    N, K = W.shape
    lib = load()
    if out is not None:
        if (out.N, out.K) != (N, K):
            raise ValueError(f"out is {out.N}x{out.K}, W is {N}x{K}")
        s = out.struct()
        st = lib.w12_encode(ctypes.c_void_p(W.data_ptr()), W.stride(0), ctypes.byref(s), _stream(stream))
        out.n_esc = s.n_esc
        _check(st, "w12_encode")
        return out
    if esc_cap is None:
        esc_cap = max(1024, (N * K) // 256)
    for _ in range(2):
        t = empty_tensor(N, K, esc_cap, W.device)
        s = t.struct()
        st = lib.w12_encode(ctypes.c_void_p(W.data_ptr()), W.stride(0), ctypes.byref(s), _stream(stream))
        t.n_esc = s.n_esc
        if st == W12_ERR_CAPACITY:
            esc_cap = s.n_esc
            continue
        _check(st, "w12_encode")
        t.esc = t.esc[:t.n_esc]
        return t
    raise W12Error(W12_ERR_CAPACITY, "w12_encode")


def w12_decode(t: W12Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty(t.N, t.K, dtype=torch.bfloat16, device=t.hi.device)
    _need_cuda(out, "out", torch.bfloat16)
    s = t.struct()
    _check(load().w12_decode(ctypes.byref(s), ctypes.c_void_p(out.data_ptr()), out.stride(0) if t.K else t.K,
                             _stream(stream)), "w12_decode")
    return out


_ws_cache: dict = {}


def verify_workspace(device) -> torch.Tensor:
    key = ("verify", torch.device(device))
    if key not in _ws_cache:
        _ws_cache[key] = torch.zeros(int(load().w12_verify_workspace_bytes()), dtype=torch.uint8, device=device)
    return _ws_cache[key]


def w12_verify_roundtrip(W: torch.Tensor, t: W12Tensor, workspace: torch.Tensor | None = None, stream=None):
    """Bitwise load-time check.  Returns (status, n_mismatch); status is
    W12_OK, W12_ERR_MISMATCH or W12_ERR_CORRUPT (other errors raise)."""
    _need_cuda(W, "W", torch.bfloat16)
    ws = workspace if workspace is not None else verify_workspace(W.device)
    s = t.struct()
    nm = ctypes.c_int64(0)
    st = load().w12_verify_roundtrip(ctypes.c_void_p(W.data_ptr()), W.stride(0) if t.K else t.K, ctypes.byref(s),
                                     ctypes.byref(nm), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                     _stream(stream))
    if st not in (W12_OK, W12_ERR_MISMATCH, W12_ERR_CORRUPT):
        _check(st, "w12_verify_roundtrip")
    return st, nm.value


def make_opts(max_ctas=0, split_k=0, path=W12_PATH_AUTO, flags=0) -> GemmOpts:
    return GemmOpts(max_ctas, split_k, path, flags)


def w12_gemm_workspace_bytes(M: int, N: int, K: int, opts: GemmOpts | None = None) -> int:
    o = opts if opts is not None else make_opts()
    return int(load().w12_gemm_workspace_bytes(M, N, K, ctypes.byref(o)))


class Workspace:
    """A zero-filled device workspace that grows on demand (torch-allocated)."""

    def __init__(self, device, nbytes: int = 0):
        self.device = torch.device(device)
        self.buf = torch.zeros(max(256, nbytes), dtype=torch.uint8, device=self.device)

    def ensure(self, nbytes: int) -> torch.Tensor:
        if self.buf.numel() < nbytes:
            self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        return self.buf


def default_workspace(device) -> Workspace:
    key = ("gemm", torch.device(device))
    if key not in _ws_cache:
        _ws_cache[key] = Workspace(device)
    return _ws_cache[key]


def w12_gemm(A: torch.Tensor, t: W12Tensor, Y: torch.Tensor | None = None, workspace: Workspace | None = None,
             opts: GemmOpts | None = None, stream=None) -> torch.Tensor:
    """Y[M,N] = A[M,K] * W^T with W in W12 (BF16 out, FP32 accumulation)."""
    o = opts if opts is not None else make_opts()
    _check_gemm_operands(A, t, Y, o.flags)
    M = A.shape[0]
    if Y is None:
        Y = torch.empty(M, _out_cols(t, o.flags), dtype=torch.bfloat16, device=A.device)
    need = w12_gemm_workspace_bytes(M, t.N, t.K, o)
    ws = (workspace or default_workspace(A.device)).ensure(max(need, 256))
    s = t.struct()
    _check(load().w12_gemm(ctypes.c_void_p(A.data_ptr()), A.stride(0), ctypes.byref(s),
                           ctypes.c_void_p(Y.data_ptr()), Y.stride(0), M, ctypes.c_void_p(ws.data_ptr()),
                           ws.numel(), ctypes.byref(o), _stream(stream)), "w12_gemm")
    return Y


class GemmCall:
    """w12_gemm with every argument marshalled once (for launch loops and
    benchmarks): calling the object only invokes the C entry point."""

    def __init__(self, A: torch.Tensor, t: W12Tensor, Y: torch.Tensor, workspace: Workspace,
                 opts: GemmOpts | None = None, stream=None):
        self._opts = opts if opts is not None else make_opts()
        _check_gemm_operands(A, t, Y, self._opts.flags)
        need = w12_gemm_workspace_bytes(A.shape[0], t.N, t.K, self._opts)
        ws = workspace.ensure(max(need, 256))
        self._keep = (A, t, Y, ws)  # the buffer itself: a later ensure() may replace it
        self._struct = t.struct()
        self._fn = load().w12_gemm
        self._args = (ctypes.c_void_p(A.data_ptr()), A.stride(0), ctypes.byref(self._struct),
                      ctypes.c_void_p(Y.data_ptr()), Y.stride(0), A.shape[0], ctypes.c_void_p(ws.data_ptr()),
                      ws.numel(), ctypes.byref(self._opts), _stream(stream))

    def __call__(self):
        st = self._fn(*self._args)
        if st != W12_OK:
            raise W12Error(st, "w12_gemm")


class GemmListCall:
    """w12_gemm_list with every argument marshalled once: calling the object
    only invokes the C entry point.  entries: a sequence of (A, t, Y, after,
    flags) with A [M, K] and Y [M, N] (or [M, N/2] with W12_GEMM_SILU_MUL)
    CUDA bfloat16 tensors, t a W12Tensor, after -1 or the index of an earlier
    entry whose output this entry's A depends on."""

    def __init__(self, entries, workspace: Workspace, opts: GemmOpts | None = None, stream=None):
        self._opts = opts if opts is not None else make_opts()
        n = len(entries)
        self._structs = []
        items = (GemmItem * max(1, n))()
        for i, (A, t, Y, after, flags) in enumerate(entries):
            _check_gemm_operands(A, t, Y, flags)
            if not -1 <= after < i:
                raise ValueError(f"entry {i}: after must be -1 or an earlier entry, got {after}")
            st = t.struct()
            self._structs.append(st)
            items[i] = GemmItem(A.data_ptr(), A.stride(0), ctypes.pointer(st), Y.data_ptr(), Y.stride(0),
                                A.shape[0], after, flags)
        self._items = items
        need = int(load().w12_gemm_list_workspace_bytes(items, n, ctypes.byref(self._opts)))
        if n and need == 0:
            raise W12Error(W12_ERR_INVALID, "w12_gemm_list_workspace_bytes")
        ws = workspace.ensure(max(need, 256))
        self._keep = (entries, ws)
        self._fn = load().w12_gemm_list
        self._args = (items, n, ctypes.c_void_p(ws.data_ptr()), ws.numel(), ctypes.byref(self._opts),
                      _stream(stream))

    def __call__(self):
        st = self._fn(*self._args)
        if st != W12_OK:
            raise W12Error(st, "w12_gemm_list")


def w12_gemm_list(entries, workspace: Workspace | None = None, opts: GemmOpts | None = None, stream=None):
    """Several small-M GEMMs in one persistent launch (w12_gemm_list); see
    GemmListCall.  Returns the outputs."""
    ws = workspace or default_workspace(entries[0][0].device if entries else "cuda")
    GemmListCall(entries, ws, opts, stream)()
    return [e[2] for e in entries]


def w12_gemm_noalloc(A: torch.Tensor, t: W12Tensor, Y: torch.Tensor, opts: GemmOpts | None = None,
                     stream=None) -> torch.Tensor:
    """w12_gemm without a workspace: the library's built-in scratch array is
    used (for callers that cannot allocate device memory).  Y must be given."""
    if Y is None:
        raise ValueError("w12_gemm_noalloc needs the output Y")
    o = opts if opts is not None else make_opts()
    _check_gemm_operands(A, t, Y, o.flags)
    s = t.struct()
    _check(load().w12_gemm_noalloc(ctypes.c_void_p(A.data_ptr()), A.stride(0), ctypes.byref(s),
                                   ctypes.c_void_p(Y.data_ptr()), Y.stride(0), A.shape[0], ctypes.byref(o),
                                   _stream(stream)), "w12_gemm_noalloc")
    return Y


W12_TREE_MAX_DEPTH = 16
W12_TREE_MAX_CANDIDATES = 16
W12_TREE_MAX_BUDGET = 256
W12_GDN_PATH = 0
W12_GDN_WY = 1
W12_GDN_MAX_DEPTH = 16
W12_GDN_MAX_NODES = 1024
W12_GDN_MAX_REQUESTS = 65536


class TreeCall:
    """w12_tree_select with its outputs and workspace allocated and every
    argument marshalled once: calling the object only invokes the C entry
    point.  lp: CUDA float32 [R, D, C] log-probabilities (read at each call).
    Outputs (device): req, depth, path (int64 holding the uint64 bits), score,
    parent ([budget] when shared, else [R, budget]) and count ([1] or [R])."""

    def __init__(self, lp: torch.Tensor, budget: int, shared: bool, stream=None):
        if not (lp.is_cuda and lp.dtype == torch.float32 and lp.dim() == 3 and lp.is_contiguous()):
            raise ValueError("lp must be a contiguous CUDA float32 [R, D, C] tensor")
        R, D, C = lp.shape
        n = budget if shared else R * budget
        dev = lp.device
        self.out = {"req": torch.empty(n, dtype=torch.int32, device=dev),
                    "depth": torch.empty(n, dtype=torch.int32, device=dev),
                    "path": torch.empty(n, dtype=torch.int64, device=dev),
                    "score": torch.empty(n, dtype=torch.float32, device=dev),
                    "parent": torch.empty(n, dtype=torch.int32, device=dev),
                    "count": torch.empty(1 if shared else R, dtype=torch.int32, device=dev)}
        need = int(load().w12_tree_workspace_bytes(R, budget))
        self._ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        self._keep = lp
        self._fn = load().w12_tree_select
        self._args = (ctypes.c_void_p(lp.data_ptr()), R, D, C, budget, 1 if shared else 0,
                      *(ctypes.c_void_p(self.out[k].data_ptr())
                        for k in ("req", "depth", "path", "score", "parent", "count")),
                      ctypes.c_void_p(self._ws.data_ptr()), self._ws.numel(), _stream(stream))
        if not shared:
            for k in ("req", "depth", "path", "score", "parent"):
                self.out[k] = self.out[k].view(R, budget)

    def __call__(self) -> dict:
        _check(self._fn(*self._args), "w12_tree_select")
        return self.out


def w12_tree_select(lp: torch.Tensor, budget: int, shared: bool, stream=None) -> dict:
    """Best-first draft-tree node selection (w12_tree_select); see TreeCall."""
    return TreeCall(lp, budget, shared, stream)()


class GdnCall:
    """w12_gdn_tree with its output and workspace allocated and every argument
    marshalled once: calling the object only invokes the C entry point.
    S0: CUDA float32 [R, H, D, D]; q, k, v: CUDA bfloat16 [n, H, D]; alpha,
    beta: CUDA float32 [n, H]; parent: CUDA int32 [n]; req: CUDA int32 [n] or
    None.  mode: W12_GDN_PATH or W12_GDN_WY.  Output `out`: float32 [n, H, D]."""

    def __init__(self, S0, q, k, v, alpha, beta, parent, req=None, mode=None, stream=None):
        mode = W12_GDN_WY if mode is None else mode
        if not (S0.is_cuda and S0.dtype == torch.float32 and S0.dim() == 4 and S0.is_contiguous()):
            raise ValueError("S0 must be a contiguous CUDA float32 [R, H, D, D] tensor")
        R, H, D, D2 = S0.shape
        if D2 != D:
            raise ValueError("S0 must be square per head")
        n = q.shape[0]
        for name, x, shape, dt in (("q", q, (n, H, D), torch.bfloat16), ("k", k, (n, H, D), torch.bfloat16),
                                   ("v", v, (n, H, D), torch.bfloat16), ("alpha", alpha, (n, H), torch.float32),
                                   ("beta", beta, (n, H), torch.float32), ("parent", parent, (n,), torch.int32)):
            if not (x.is_cuda and x.dtype == dt and tuple(x.shape) == shape and x.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor of shape {shape}")
        if req is not None and not (req.is_cuda and req.dtype == torch.int32 and tuple(req.shape) == (n,)
                                    and req.is_contiguous()):
            raise ValueError("req must be a contiguous CUDA int32 [n] tensor or None")
        self.out = torch.empty(n, H, D, dtype=torch.float32, device=q.device)
        need = int(load().w12_gdn_workspace_bytes(n, H, D, mode))
        if need == 0:
            raise W12Error(W12_ERR_INVALID, "w12_gdn_workspace_bytes")
        self._ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        self._keep = (S0, q, k, v, alpha, beta, parent, req)
        self._fn = load().w12_gdn_tree
        ptr = lambda x: ctypes.c_void_p(x.data_ptr() if x is not None else None)  # noqa: E731
        self._args = (ptr(S0), ptr(q), ptr(k), ptr(v), ptr(alpha), ptr(beta), ptr(parent), ptr(req),
                      n, H, R, D, ptr(self.out), ptr(self._ws), self._ws.numel(), mode, _stream(stream))
        self._stream = stream

    def __call__(self) -> torch.Tensor:
        _check(self._fn(*self._args), "w12_gdn_tree")
        return self.out

    def status(self) -> int:
        """The device-side tree check of the last call (synchronous)."""
        return load().w12_gdn_status(ctypes.c_void_p(self._ws.data_ptr()), self._ws.numel(), _stream(self._stream))


def w12_gdn_tree(S0, q, k, v, alpha, beta, parent, req=None, mode=None, stream=None) -> torch.Tensor:
    """Gated-delta-rule outputs of draft-tree nodes (w12_gdn_tree); see GdnCall."""
    return GdnCall(S0, q, k, v, alpha, beta, parent, req, mode, stream)()


W12_NORM_MAX_K = 65536
W12_ROPE_MAX_AXES = 4
W12_ATTN_MAX_NODES = 65536
W12_ATTN_MAX_REQUESTS = 4096
W12_ATTN_REUSE_PLAN = 1  # the tree, lengths and pages are those of the last call on the workspace
W12_ATTN_TEST_STALL = 4  # tests only: a bounded wait runs out


def _rows(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """The row stride (elements) of a tensor of this shape whose rows (first
    dimension) are contiguous inside and may lie any distance apart, but not
    over one another (a broadcast has a row stride of 0)."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    st = t.stride()
    width = 1
    for d in range(len(st) - 1, 0, -1):
        if st[d] != width and shape[d] > 1 and t.numel():
            raise ValueError(f"{name}: rows must be contiguous, got strides {st}")
        width *= shape[d]
    if shape[0] < 2:
        return width
    if st[0] < width:
        raise ValueError(f"{name}: rows of {width} must not overlap, got strides {st}; pass a contiguous copy")
    return st[0]


def _vector(t: torch.Tensor, name: str, n: int, dtype, device) -> int:
    """The address of a contiguous [n] tensor."""
    if t.dtype is not dtype or t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [{n}] tensor on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _current_device_of(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev = t.device
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {dev} but the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _stream_of(dev: torch.device) -> int:
    """The handle of the device's current stream."""
    return _raw_stream(dev.index) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def w12_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                out8: bool = False, h_out: torch.Tensor | None = None, y_out: torch.Tensor | None = None,
                stream=None) -> dict:
    """h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight (w12_rmsnorm).
    x, residual: CUDA bfloat16 [M, K], rows any distance apart; weight: bfloat16
    [K].  Returns {"y": bfloat16 [M, K]}, or with out8 {"q8": float8_e4m3fn
    [M, K], "scale": float32 [M, ceil(K / 128)]} (value = q8 * scale of its 128
    columns; for a GEMM that reads such codes, w12_gemm reads bfloat16), and
    with a residual also "h": bfloat16 [M, K].  h_out / y_out:
    write there instead (h_out may be x or residual, y_out may be x)."""
    if stream is not None:  # as if called under that stream: the outputs are allocated there
        with torch.cuda.stream(stream):
            return w12_rmsnorm(x, weight, eps, residual, out8, h_out, y_out)
    bf = torch.bfloat16
    dev = _current_device_of(x, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x must be [M, K], got {tuple(shape)}")
    M, K = shape
    ldx = _rows(x, "x", shape, bf, dev)
    wp = _vector(weight, "weight", K, bf, dev)
    out = {}
    rp = hp = yp = qp = sp = None
    ldr = ldh = ldy = ldq = lds = 0
    if residual is not None:
        ldr = _rows(residual, "residual", shape, bf, dev)
        rp = residual.data_ptr()
    if h_out is not None:
        ldh = _rows(h_out, "h_out", shape, bf, dev)
    elif residual is not None:
        h_out = torch.empty(shape, dtype=bf, device=dev)
        ldh = K
    if h_out is not None:
        hp = h_out.data_ptr()
        out["h"] = h_out
    if out8:
        if y_out is not None:
            raise ValueError("y_out is for the bfloat16 output")
        q8 = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
        lds = (K + 127) // 128
        scale = torch.empty((M, lds), dtype=torch.float32, device=dev)
        qp, ldq, sp = q8.data_ptr(), K, scale.data_ptr()
        out["q8"], out["scale"] = q8, scale
    else:
        if y_out is not None:
            ldy = _rows(y_out, "y_out", shape, bf, dev)
        else:
            y_out = torch.empty(shape, dtype=bf, device=dev)
            ldy = K
        yp = y_out.data_ptr()
        out["y"] = y_out
    st = (_lib or load()).w12_rmsnorm(x.data_ptr(), ldx, rp, ldr, wp, eps, M, K, hp, ldh, yp, ldy, qp, ldq, sp, lds,
                                      _stream_of(dev))
    if st:
        raise W12Error(st, "w12_rmsnorm")
    return out


class KvCache:
    """A paged cache of keys and values: k and v CUDA bfloat16 [pages,
    page_tokens, heads, dim] of the same strides, unit stride in dim; a
    head-major cache [pages, heads, page_tokens, dim] is passed as its
    permuted view."""

    __slots__ = ("k", "v", "device", "page_tokens", "heads", "dim", "_c", "_at", "_sizes")

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        bf = torch.bfloat16
        shape, st = k.shape, k.stride()
        if not (k.is_cuda and k.dtype is bf and v.dtype is bf and len(shape) == 4 and v.shape == shape
                and v.stride() == st and v.device == k.device):
            raise ValueError("k and v must be CUDA bfloat16 [pages, page_tokens, heads, dim] tensors of equal strides")
        pages, page, heads, dim = shape
        if st[3] != 1 and dim > 1:
            raise ValueError(f"the cache must have unit stride in dim, got strides {st}")
        self.k, self.v, self.device = k, v, k.device
        self.page_tokens, self.heads, self.dim = page, heads, dim
        self._c = _Cache(k.data_ptr(), v.data_ptr(), pages, page, heads, dim, st[0], st[1], st[2])
        self._at = ctypes.addressof(self._c)
        self._sizes = (*shape, *st)


def w12_rope_append(q, k, pos, inv_freq, axis=None, interleaved=False, q_norm=None, k_norm=None, eps=1e-6, v=None,
                    cache: KvCache | None = None, slots=None, q_out=None, k_out=None, stream=None):
    """Rotary positions on q and k, and the write of k and v into a paged
    cache (w12_rope_append).  q: CUDA bfloat16 [n, q_heads, dim] (or None), k,
    v: [n, heads, dim]; rows may lie any distance apart, so views of the QKV GEMM's
    output work.  pos: int32 [n] or [axes, n]; inv_freq: float32 [rot / 2];
    axis: the axis of every frequency (a sequence or bytes), None: axis 0.
    inv_freq None: no rotation (a plain append).  q_norm / k_norm: bfloat16
    [dim], per-head RMS norm before the rotation.  cache and slots (int64 [n],
    -1: skip): rotated k and v go there.  Returns (q, k): new tensors, or q_out
    / k_out (which may be the inputs); k is None where the keys go to the cache
    and no k_out is given."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return w12_rope_append(q, k, pos, inv_freq, axis, interleaved, q_norm, k_norm, eps, v, cache, slots, q_out,
                                   k_out)
    bf = torch.bfloat16
    ref = q if q is not None else k
    if ref is None or ref.dim() != 3:
        raise ValueError("q and k must be [n, heads, dim]")
    dev = _current_device_of(ref, "q" if q is not None else "k")
    n, _, dim = ref.shape
    qp = kp = vp = qo = ko = pp = ap = fp = qn = kn = cp = sp = None
    ldq = ldk = ldv = ldqo = ldko = ld_pos = 0
    Hq = Hkv = rot = n_axes = 0
    if q is not None:
        shape = q.shape
        ldq = _rows(q, "q", shape, bf, dev)
        qp, Hq = q.data_ptr(), shape[1]
        if q_out is None:
            q_out = torch.empty(shape, dtype=bf, device=dev)
            ldqo = Hq * dim
        else:
            ldqo = _rows(q_out, "q_out", shape, bf, dev)
        qo = q_out.data_ptr()
    if k is not None:
        shape = k.shape
        if len(shape) != 3 or shape[0] != n or shape[2] != dim:
            raise ValueError(f"k must be [{n}, heads, {dim}], got {tuple(shape)}")
        ldk = _rows(k, "k", shape, bf, dev)
        kp, Hkv = k.data_ptr(), shape[1]
        if k_out is not None:
            ldko = _rows(k_out, "k_out", shape, bf, dev)
        elif slots is None:
            k_out = torch.empty(shape, dtype=bf, device=dev)
            ldko = Hkv * dim
        if k_out is not None:
            ko = k_out.data_ptr()
    if (slots is None) != (cache is None):
        raise ValueError("cache and slots go together")
    if slots is not None:
        if k is None or v is None:
            raise ValueError("appending needs k and v")
        ldv = _rows(v, "v", k.shape, bf, dev)
        vp = v.data_ptr()
        sp = _vector(slots, "slots", n, torch.int64, dev)
        if cache.device != dev:
            raise ValueError(f"the cache must be on {dev}")
        cp = cache._at
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rot / 2]")
        half = inv_freq.shape[0]
        fp = _vector(inv_freq, "inv_freq", half, torch.float32, dev)
        d = pos.dim()
        if not (pos.dtype is torch.int32 and d in (1, 2) and pos.shape[-1] == n and pos.device == dev
                and (n < 2 or pos.stride(-1) == 1)):
            raise ValueError(f"pos must be an int32 [{n}] or [axes, {n}] tensor on {dev}")
        rot, pp = 2 * half, pos.data_ptr()
        n_axes = pos.shape[0] if d == 2 else 1
        ld_pos = pos.stride(0) if n_axes > 1 else n
        if axis is not None:
            if len(axis) != half:
                raise ValueError(f"axis must name one axis for each of the {half} frequencies")
            axis = ctypes.create_string_buffer(bytes(axis), half)
            ap = ctypes.addressof(axis)
    if q_norm is not None:
        qn = _vector(q_norm, "q_norm", dim, bf, dev)
    if k_norm is not None:
        kn = _vector(k_norm, "k_norm", dim, bf, dev)
    args = _rope_args.pack(qp or 0, kp or 0, vp or 0, ldq, ldk, ldv, qo or 0, ko or 0, ldqo, ldko, n, Hq, Hkv, dim, rot,
                           1 if interleaved else 0, pp or 0, ld_pos, n_axes, ap or 0, fp or 0, qn or 0, kn or 0, eps,
                           cp or 0, sp or 0)
    st = (_lib or load()).w12_rope_append(args, _stream_of(dev))
    if st:
        raise W12Error(st, "w12_rope_append")
    return q_out, k_out


def w12_kv_append(k, v, cache: KvCache, slots, stream=None):
    """Write keys and values (already rotated) into the cache's slots: a
    step's accepted nodes (w12_rope_append without a rotation)."""
    w12_rope_append(None, k, None, None, v=v, cache=cache, slots=slots, stream=stream)


def _capturing(dev: torch.device) -> bool:
    return dev.type == "cuda" and torch.cuda.is_current_stream_capturing()


class AttnWorkspace:
    """The workspace of w12_tree_attn (zero-filled, grown on demand).  It also
    holds the analysis of the last tree, so the layers of one verify step share
    one workspace and every layer after the first passes reuse_plan=True.  (Not
    with replays between them of a graph that plans in the same workspace.)

    A call that is captured in a CUDA graph needs a workspace that already has
    its size (make the call once before, with the same workspace): zeros made
    during a capture are filled in by that graph's replays only.  Buffers that
    were outgrown stay with the workspace, because a graph may hold their
    addresses; sizes are powers of two, so they add up to less than the last."""

    def __init__(self, device):
        self.device = torch.device(device)
        self.buf = self._zeros(256)
        self._outgrown = []
        self._plan = None  # what the plan in buf was made from (w12_tree_attn)
        self._plan_captured = False  # it is made when a graph is replayed
        # A call is several launches that hand one another results through buf: another thread's must not come
        # between them (the library is called without the interpreter's lock).
        self._lock = threading.Lock()

    def _zeros(self, nbytes: int) -> torch.Tensor:
        if _capturing(self.device):
            raise RuntimeError("the attention workspace cannot be made or grown while the stream is captured: make the "
                               "call once before the capture, with a workspace of its own, and capture it with that one")
        return torch.zeros(nbytes, dtype=torch.uint8, device=self.device)

    def ensure(self, nbytes: int) -> torch.Tensor:
        if self.buf.numel() < nbytes:
            buf = self._zeros(1 << (nbytes - 1).bit_length())
            self._outgrown.append(self.buf)
            self.buf, self._plan = buf, None
        return self.buf

    def status(self, stream=None) -> int:
        """W12_OK, W12_ERR_INVALID (the last tree, a length or a page broke a
        rule: NaN outputs) or W12_ERR_TIMEOUT (synchronous)."""
        return load().w12_tree_attn_status(ctypes.c_void_p(self.buf.data_ptr()), self.buf.numel(), _stream(stream))


def default_attn_workspace(device) -> AttnWorkspace:
    """One workspace per device, current stream and host thread: calls that
    share one must not overlap, and another thread's tree between two layers
    would take the place of their plan."""
    device = torch.device(device)
    key = ("attn", device.index, _stream_of(device), threading.get_ident())
    ws = _ws_cache.get(key)
    if ws is None:
        ws = _ws_cache[key] = AttnWorkspace(device)
    return ws


_attn_bytes: dict = {}


def _attn_workspace_bytes(n: int, R: int, Hq: int, heads: int, dim: int) -> int:
    key = (n, R, Hq, heads, dim)
    need = _attn_bytes.get(key)
    if need is None:
        need = int(load().w12_tree_attn_workspace_bytes(n, R, Hq, heads, dim))
        if need == 0:
            raise W12Error(W12_ERR_INVALID, "w12_tree_attn_workspace_bytes")
        if len(_attn_bytes) > 4096:
            _attn_bytes.clear()
        _attn_bytes[key] = need
    return need


def w12_tree_attn(q, k, v, cache: KvCache, block_table, ctx_len, parent=None, req=None, scale: float = 0.0,
                  softcap: float = 0.0, window: int = 0, out=None, workspace: AttnWorkspace | None = None,
                  reuse_plan: bool = False, max_ctas: int = 0, stream=None) -> torch.Tensor:
    """Attention of draft-tree nodes over a paged cache (w12_tree_attn).
    q: CUDA bfloat16 [n, q_heads, dim]; k, v: the nodes' own [n, heads, dim];
    rows may lie any distance apart.  block_table: int32 [R, width]; ctx_len: int32
    [R]; parent, req: int32 [n] or None (no parents: plain decode; no req:
    request 0).  Returns bfloat16 [n, q_heads, dim].  reuse_plan: the tree, the
    lengths and the pages hold what they held in the last call on this
    workspace (not looked at), and their sizes, the heads, the window and the
    cache's sizes and strides are the same (ValueError where they are not)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return w12_tree_attn(q, k, v, cache, block_table, ctx_len, parent, req, scale, softcap, window, out,
                                 workspace, reuse_plan, max_ctas)
    bf, i32 = torch.bfloat16, torch.int32
    dev = _current_device_of(q, "q")
    shape = q.shape
    if len(shape) != 3 or block_table.dim() != 2:
        raise ValueError("q must be [n, q_heads, dim] and block_table [R, width]")
    n, Hq, dim = shape
    heads = cache.heads
    if dim != cache.dim or Hq % heads or cache.device != dev:
        raise ValueError(f"q has {Hq} heads of {dim} on {dev}, the cache {heads} of {cache.dim} on {cache.device}")
    R, width = block_table.shape
    kv = (n, heads, dim)
    if out is None:
        out = torch.empty(shape, dtype=bf, device=dev)
        ldo = Hq * dim
    else:
        ldo = _rows(out, "out", shape, bf, dev)
    args = _attn_args.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _rows(q, "q", shape, bf, dev), _rows(k, "k", kv, bf, dev),
        _rows(v, "v", kv, bf, dev), out.data_ptr(), ldo, n, R, Hq, block_table.data_ptr(),
        _rows(block_table, "block_table", (R, width), i32, dev), width, _vector(ctx_len, "ctx_len", R, i32, dev),
        _vector(parent, "parent", n, i32, dev) if parent is not None else 0,
        _vector(req, "req", n, i32, dev) if req is not None else 0, scale, softcap, window, max_ctas,
        W12_ATTN_REUSE_PLAN if reuse_plan else 0)
    need = _attn_workspace_bytes(n, R, Hq, heads, dim)
    ws = workspace if workspace is not None else default_attn_workspace(dev)
    if ws.buf.device != dev:
        raise ValueError(f"the workspace is on {ws.buf.device}, the tensors on {dev}")
    # With a plan made for other sizes the kernels would go by node numbers and offsets that are not this call's.
    plan = (n, R, Hq, width, window, cache._sizes)
    with ws._lock:
        if not reuse_plan:
            ws._plan, ws._plan_captured = None, _capturing(dev)
        elif ws._plan != plan or (ws._plan_captured and not _capturing(dev)):
            raise ValueError("reuse_plan: the last call on this workspace had another number of nodes or requests, other "
                             "heads, another window or cache, or was captured and has not run")
        buf = ws.ensure(need)
        st = (_lib or load()).w12_tree_attn(args, cache._at, buf.data_ptr(), buf.numel(), _stream_of(dev))
        if st:
            raise W12Error(st, "w12_tree_attn")
        ws._plan = plan
    return out


W12_ACCEPT_TEST_STALL = 65536  # tests only, with max_depth: a bounded wait runs out


def w12_tree_accept(logits, token, parent, req=None, temperature=1.0, uniform=None, noise=None, draft=None,
                    draft_row=None, row=None, root_row=None, max_depth: int = 16, stream=None) -> dict:
    """Which drafted nodes are accepted, and the token after them
    (w12_tree_accept).  logits: CUDA bfloat16 or float32 [rows, V], rows any
    distance apart; token, parent, req: int32 [n] (req None: request 0); row:
    int32 [n], the row of every node (None: its index); root_row: int32 [R], the
    row of every request's last accepted token (None: the rows from n on, which
    then are as many as the requests).  temperature: a number or float32 [R];
    uniform: float32 [n]; noise: float32 [R, V], exponential (both may be None
    where temperature is the number 0).  draft: float32 [draft_rows, V]
    probabilities with draft_row: int32 [n], None where the tokens were not
    drawn.  Returns {"count": int32 [R], "nodes": int32 [R, max_depth], "next":
    int32 [R]}; count -1: the request broke a rule."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return w12_tree_accept(logits, token, parent, req, temperature, uniform, noise, draft, draft_row, row,
                                   root_row, max_depth)
    i32, f32 = torch.int32, torch.float32
    dev = _current_device_of(logits, "logits")
    shape = logits.shape
    if len(shape) != 2 or logits.dtype not in (torch.bfloat16, f32):
        raise ValueError(f"logits must be a bfloat16 or float32 [rows, V] tensor, got {logits.dtype} {tuple(shape)}")
    m, V = shape
    n = token.shape[0] if token.dim() == 1 else -1
    R = root_row.shape[0] if root_row is not None else m - n
    if n < 0 or R < 1:
        raise ValueError(f"token must be [n], and logits have a row for every request behind the {n} nodes' (or root_row)")
    width = max_depth & ~W12_ACCEPT_TEST_STALL
    if not 1 <= width <= 256:
        raise ValueError(f"max_depth must be in 1 .. 256, got {max_depth}")
    vec = lambda t, name, size, dt: _vector(t, name, size, dt, dev) if t is not None else 0  # noqa: E731
    by_request = isinstance(temperature, torch.Tensor)
    drawn = by_request or temperature != 0
    if drawn and (noise is None or (uniform is None and n > 0)):
        raise ValueError("uniform and noise are needed unless temperature is the number 0")
    if (draft is None) != (draft_row is None):
        raise ValueError("draft and draft_row go together")
    if draft is not None and (draft.dim() != 2 or draft.shape[1] != V):
        raise ValueError(f"draft must be [draft_rows, {V}], got {tuple(draft.shape)}")
    ldl = _rows(logits, "logits", shape, logits.dtype, dev)
    ldn = _rows(noise, "noise", (R, V), f32, dev) if noise is not None else 0
    ldd = _rows(draft, "draft", draft.shape, f32, dev) if draft is not None else 0
    nodes = torch.empty((R, width), dtype=i32, device=dev)
    count, after = nodes.new_empty(R), nodes.new_empty(R)
    args = _accept_args.pack(
        logits.data_ptr(), ldl, m, V, logits.dtype is f32, vec(token, "token", n, i32), vec(parent, "parent", n, i32),
        vec(req, "req", n, i32), vec(row, "row", n, i32), vec(root_row, "root_row", R, i32), n, R,
        vec(temperature, "temperature", R, f32) if by_request else 0, 0.0 if by_request else temperature,
        vec(uniform, "uniform", n, f32), noise.data_ptr() if noise is not None else 0, ldn,
        draft.data_ptr() if draft is not None else 0, ldd, draft.shape[0] if draft is not None else 0,
        vec(draft_row, "draft_row", n, i32), max_depth, count.data_ptr(), nodes.data_ptr(),
        after.data_ptr(), width)
    st = (_lib or load()).w12_tree_accept(args, _stream_of(dev))
    if st:
        raise W12Error(st, "w12_tree_accept")
    return {"count": count, "nodes": nodes, "next": after}


W12_GDN_AUTO = 2
W12_GDN_TEST_STALL = 64  # tests only, with W12_GDN_WY: a bounded wait runs out


_scan_bytes: dict = {}


def _scan_workspace_bytes(n: int, R: int, H: int, D: int, mode: int) -> int:
    key = (n, R, H, D, mode)
    need = _scan_bytes.get(key)
    if need is None:
        need = int(load().w12_gdn_scan_workspace_bytes(n, R, H, D, mode))
        if len(_scan_bytes) > 4096:
            _scan_bytes.clear()
        _scan_bytes[key] = need
    return need


def w12_gdn_scan(S, q, k, v, alpha, beta, start=None, rows=None, count=None, S_out=None, out=None, out32: bool = False,
                 mode: int = W12_GDN_AUTO, status=None, stream=None):
    """The gated delta rule over sequences (w12_gdn_scan).  S: CUDA float32 [R,
    H, D, D], the states before; q, k: bfloat16 [n, key_heads, D] (q None: the
    states only), v: [n, H, D], rows any distance apart; alpha, beta: float32
    [n, H].  The sequences: start, int32 [R + 1], rows start[r] .. start[r + 1]
    - 1; or rows, int32 [R, width], with count, int32 [R] (such as
    w12_tree_accept's nodes and count); neither: one sequence of all rows.
    S_out: where the states after go (None: S itself).  out: bfloat16 or float32
    [n, H, D], written at the sequences' rows (None: a new one, float32 with
    out32), apart from q, k and v (other columns of one buffer are).  mode: W12_GDN_AUTO
    (one of the others for the whole call, by n / R), W12_GDN_PATH or W12_GDN_WY.  status: int32 [1],
    which gets 1 where a sequence broke a rule (it is left out then) or a wait
    gave up (what it was for is NaN then), else 0.
    Returns (out, S_out)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return w12_gdn_scan(S, q, k, v, alpha, beta, start, rows, count, S_out, out, out32, mode, status)
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    dev = _current_device_of(S, "S")
    if S.dim() != 4 or S.dtype is not f32 or not S.is_contiguous() or S.shape[2] != S.shape[3]:
        raise ValueError(f"S must be a contiguous float32 [R, H, D, D] tensor, got {S.dtype} {tuple(S.shape)}")
    R, H, D, _ = S.shape
    if S_out is None:
        S_out = S
    elif S_out.shape != S.shape or S_out.dtype is not f32 or S_out.device != dev or not S_out.is_contiguous():
        raise ValueError(f"S_out must be a contiguous float32 {tuple(S.shape)} tensor on {dev}")
    if v.dim() != 3 or k.dim() != 3:
        raise ValueError("k and v must be [n, heads, D]")
    n, Hk = v.shape[0], k.shape[1]
    kv = (n, Hk, D)
    if (rows is None) != (count is None) or (rows is not None and start is not None):
        raise ValueError("the sequences are given by start, or by rows and count")
    width = ld_rows = 0
    if rows is not None:
        if rows.dim() != 2:
            raise ValueError(f"rows must be [{R}, width], got {tuple(rows.shape)}")
        width = rows.shape[1]
        ld_rows = _rows(rows, "rows", (R, width), i32, dev)
    elif start is None:
        if R != 1:
            raise ValueError("several requests need start, or rows and count")
    op = qp = ldq = ldo = 0
    if q is None:
        if out is not None:
            raise ValueError("there are no outputs without q")
    else:
        qp, ldq = q.data_ptr(), _rows(q, "q", kv, bf, dev)
        if out is None:
            out = torch.empty(n, H, D, dtype=f32 if out32 else bf, device=dev)
        elif out.dtype not in (bf, f32):
            raise ValueError(f"out must be bfloat16 or float32, got {out.dtype}")
        op, ldo = out.data_ptr(), _rows(out, "out", (n, H, D), out.dtype, dev)
    for name, t in (("alpha", alpha), ("beta", beta)):
        if t.shape != (n, H) or t.dtype is not f32 or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 [{n}, {H}] tensor on {dev}")
    args = _scan_args.pack(
        S.data_ptr(), S_out.data_ptr(), qp, k.data_ptr(), v.data_ptr(), ldq, _rows(k, "k", kv, bf, dev),
        _rows(v, "v", (n, H, D), bf, dev), alpha.data_ptr(), beta.data_ptr(), op, ldo, out is not None and out.dtype is f32,
        _vector(start, "start", R + 1, i32, dev) if start is not None else 0, rows.data_ptr() if rows is not None else 0,
        _vector(count, "count", R, i32, dev) if count is not None else 0, ld_rows, width, n, R, H, Hk, D, mode,
        _vector(status, "status", 1, i32, dev) if status is not None else 0)
    need = _scan_workspace_bytes(n, R, H, D, mode & ~W12_GDN_TEST_STALL if rows is None else W12_GDN_PATH)
    # the allocator's own order of a stream's calls keeps those that overlap apart; a captured call's belongs to its graph
    buf = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    st = (_lib or load()).w12_gdn_scan(args, buf.data_ptr() if need else 0, need, _stream_of(dev))
    if st:
        raise W12Error(st, "w12_gdn_scan")
    return out, S_out


def w12_gemm_noalloc_status(stream=None) -> int:
    """W12_ERR_TIMEOUT if a bounded wait of the last w12_gemm_noalloc call on
    the current device gave up (read and cleared; synchronous), else W12_OK."""
    return load().w12_gemm_noalloc_status(_stream(stream))


def w12_gemm_workspace_status(workspace: Workspace, stream=None) -> int:
    return load().w12_gemm_workspace_status(ctypes.c_void_p(workspace.buf.data_ptr()), workspace.buf.numel(),
                                            _stream(stream))
