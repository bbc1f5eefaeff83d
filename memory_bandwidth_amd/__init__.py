"""Thin Python binding of libq4gemv.so (the MI355X int4 decode-GEMV library).

Every function has the name of the C entry point it calls and only marshals
arguments: it checks dtypes, shapes, contiguity and device, passes raw device
pointers and torch's current HIP stream, and raises Q4Error on a non-zero
status.  (The 8-bit calls do so in C++, by the module _bind_i8.)  All arithmetic
runs in the library's HIP kernels; there is no other implementation here.
Importing this module without the built library works (so CPU-only tooling can
inspect it), but every call then raises; without _bind_i8 the 8-bit ones do.

Storage format (see include/q4gemv.h): x float32 [M, K]; wq uint8 [N, K/2]
(two codes per byte, low nibble = even k); scales float16 or uint16 [N, K/g]
(binary16 bits); zeros uint8 [N, ceil(K/g / 2)] (low nibble = even group).
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4gemv.so")

Q4_OK, Q4_EINVAL, Q4_ENULL, Q4_EALIGN, Q4_EDEVICE, Q4_ELAUNCH = 0, -1, -2, -3, -4, -5

# Exported C symbols, in the order include/q4gemv.h, include/q4blocks.h and
# include/q4scan.h declare them.
EXPORTS = ("gemv_q4", "gemv_q4_ws", "gemv_q4_workspace_size", "gemv_q4_static", "gemv_q4_swiglu", "gemv_f32", "dequant_q4", "read_reduce",
           "read_reduce_passes", "copy_vec4", "write_fill",
           "gemv_q4_geometry", "gemv_q4_path", "q4_strerror", "q4_abi_version",
           "gemv_q4_set_geometry", "gemv_q4_clear_geometry",
           "block_geometry", "gemv_block", "dequant_block", "gemv_block_set_config",
           "gemv_block_config", "scan2", "scan2_set_config", "scan2_config")

# Exported C symbols, in the order include/q4i8.h declares them.
EXPORTS_I8 = ("quant_i8", "gemm_i8", "gemm_i8_swiglu", "gemm_i8_grouped", "gemm_i8_grouped_swiglu",
              "gemm_i8_geometry")

# Exported C symbols, in the order include/q4f8.h declares them.
EXPORTS_F8 = ("quant_f8", "quant_f8_block", "gemm_f8", "gemm_f8_swiglu", "gemm_f8_swiglu_backward",
              "gemm_f8_geometry")

# Element types of include/q4i8.h.
I8_F32, I8_F16, I8_BF16 = 0, 1, 2
I8_TYPES = {torch.float32: I8_F32, torch.float16: I8_F16, torch.bfloat16: I8_BF16}

# Block formats of include/q4blocks.h.
BLK_Q4_0, BLK_Q8_0, BLK_Q4_K, BLK_Q5_K, BLK_Q6_K = 1, 2, 3, 4, 5
BLOCK_FORMATS = {"q4_0": BLK_Q4_0, "q8_0": BLK_Q8_0, "q4_k": BLK_Q4_K, "q5_k": BLK_Q5_K,
                 "q6_k": BLK_Q6_K}

Q4_PATH_FMA, Q4_PATH_INTEGER = 0, 1

_lib = None


class Q4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {strerror(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"HIP library {LIB_PATH} is not built; run "
                           "`python -m memory_bandwidth_amd.build` first")
    L = ctypes.CDLL(LIB_PATH)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.gemv_q4.argtypes = [P, P, P, P, P, I, I, I, I, P]
    L.gemv_q4_ws.argtypes = [P, P, P, P, P, I, I, I, I, P, Z, P]
    L.gemv_q4_workspace_size.argtypes = [I, I, I, I, ctypes.POINTER(Z)]
    L.gemv_q4_static.argtypes = [P, P, P, P, P, I, I, I, I, P]
    L.gemv_q4_swiglu.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, P]
    L.gemv_f32.argtypes = [P, P, P, I, I, I, P]
    L.dequant_q4.argtypes = [P, P, P, P, P, I, I, I, P]
    L.read_reduce.argtypes = [P, Z, P, I, P]
    L.read_reduce_passes.argtypes = [P, Z, I, P, I, P]
    L.copy_vec4.argtypes = [P, P, Z, I, I, P]
    L.write_fill.argtypes = [P, Z, ctypes.c_float, I, P]
    IP = ctypes.POINTER(ctypes.c_int)
    L.gemv_q4_geometry.argtypes = [I, I, I, I, IP, IP, IP, IP, IP, IP]
    L.gemv_q4_path.argtypes = [I, I, I, I]
    L.gemv_q4_set_geometry.argtypes = [I, I, I, I, I, I, I]
    L.gemv_q4_clear_geometry.argtypes = []
    L.block_geometry.argtypes = [I, IP, IP]
    L.gemv_block.argtypes = [I, P, P, P, I, I, I, P]
    L.dequant_block.argtypes = [I, P, P, I, I, P]
    L.gemv_block_set_config.argtypes = [I, I, I, I]
    L.gemv_block_config.argtypes = [I, IP, IP, IP]
    L.scan2.argtypes = [P, P, P, I, I, I, P]
    L.scan2_set_config.argtypes = [I, I, I, I]
    L.scan2_config.argtypes = [IP, IP, IP, IP]
    L.quant_i8.argtypes = [P, I, P, P, I, I, P]
    L.gemm_i8.argtypes = [P, P, P, P, P, P, I, I, I, I, P]
    L.gemm_i8_swiglu.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P]
    L.gemm_i8_grouped.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P]
    L.gemm_i8_grouped_swiglu.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, P]
    L.gemm_i8_geometry.argtypes = [I, I, I, I, I, IP, IP, IP, IP]
    Q = ctypes.c_int64
    L.quant_f8.argtypes = [P, I, P, P, Q, Q, I, I, P]
    L.quant_f8_block.argtypes = [P, I, P, P, P, P, I, I, P]
    L.gemm_f8.argtypes = [P, P, Q, Q, I, P, P, P, P, I, I, I, I, P]
    L.gemm_f8_swiglu.argtypes = [P, P, Q, Q, I, P, P, P, P, P, I, I, I, I, P]
    L.gemm_f8_swiglu_backward.argtypes = [P, I, P, P, Q, Q, I, P, P, P, P, P, I, I, I, I, P]
    L.gemm_f8_geometry.argtypes = [I, I, I, I, I, IP, IP, IP, IP]
    for f in EXPORTS_I8 + EXPORTS_F8:
        getattr(L, f).restype = ctypes.c_int
    L.q4_strerror.argtypes = [I]
    L.q4_strerror.restype = ctypes.c_char_p
    L.q4_abi_version.argtypes = []
    for f in ("gemv_q4", "gemv_q4_ws", "gemv_q4_workspace_size", "gemv_q4_static", "gemv_q4_swiglu", "gemv_f32", "dequant_q4", "read_reduce",
              "read_reduce_passes", "copy_vec4", "write_fill", "gemv_q4_geometry", "gemv_q4_path", "q4_abi_version",
              "gemv_q4_set_geometry", "gemv_q4_clear_geometry", "block_geometry", "gemv_block",
              "dequant_block", "gemv_block_set_config", "gemv_block_config", "scan2",
              "scan2_set_config", "scan2_config"):
        getattr(L, f).restype = ctypes.c_int
    _lib = L
    return L


def strerror(status: int) -> str:
    return lib().q4_strerror(status).decode()


def _check(fn: str, status: int) -> None:
    if status != Q4_OK:
        raise Q4Error(fn, status)


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(dev: torch.device) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _need(t: torch.Tensor, name: str, dtypes, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _q4_operands(x: torch.Tensor, wq: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                 group_size: int, N: int | None = None):
    """Checks one int4 matrix against x; returns (M, N, K, g)."""
    _need(x, "x", (torch.float32,))
    dev = x.device
    _need(wq, "wq", (torch.uint8,), dev)
    _need(scales, "scales", (torch.float16, torch.uint16, torch.int16), dev)
    _need(zeros, "zeros", (torch.uint8,), dev)
    if x.dim() != 2 or wq.dim() != 2:
        raise ValueError("x must be [M, K] and wq [N, K/2]")
    M, K = x.shape
    n = wq.shape[0]
    g = int(group_size)
    G = K // g if g else 0
    if (wq.shape[1] * 2 != K or tuple(scales.shape) != (n, G) or tuple(zeros.shape) != (n, (G + 1) // 2)
            or (N is not None and n != N)):
        raise ValueError(f"shape mismatch: x{tuple(x.shape)} wq{tuple(wq.shape)} "
                         f"scales{tuple(scales.shape)} zeros{tuple(zeros.shape)} g={g}")
    return M, n, K, g


def _out(out: torch.Tensor | None, M: int, N: int, dev: torch.device) -> torch.Tensor:
    if out is None:
        return torch.empty((M, N), dtype=torch.float32, device=dev)
    _need(out, "out", (torch.float32,), dev)
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [M, N]")
    return out


def gemv_q4_workspace_size(M: int, N: int, K: int, group_size: int) -> int:
    """Workspace bytes with which gemv_q4_ws may split K over workgroups (0: none needed)."""
    n = ctypes.c_size_t()
    _check("gemv_q4_workspace_size", lib().gemv_q4_workspace_size(M, N, K, group_size, ctypes.byref(n)))
    return n.value


def gemv_q4(x: torch.Tensor, wq: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
            group_size: int, out: torch.Tensor | None = None,
            workspace: torch.Tensor | bool | None = None) -> torch.Tensor:
    """y[M, N] = x[M, K] . dequant(W_q[N, K])^T on the current stream.

    workspace: None takes one from torch's allocator when the shape can use
    it (gemv_q4_ws); a uint8 tensor on x's device is used as given; False
    calls gemv_q4 without one."""
    M, N, K, g = _q4_operands(x, wq, scales, zeros, group_size)
    out = _out(out, M, N, x.device)
    if workspace is False:
        _check("gemv_q4", lib().gemv_q4(_ptr(x), _ptr(wq), _ptr(scales), _ptr(zeros), _ptr(out),
                                        M, N, K, g, _stream(x.device)))
        return out
    if workspace is None or workspace is True:
        n = gemv_q4_workspace_size(M, N, K, g)
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device) if n else None
    else:
        _need(workspace, "workspace", (torch.uint8,), x.device)
    wp, wn = (_ptr(workspace), workspace.numel()) if workspace is not None else (None, 0)
    _check("gemv_q4_ws", lib().gemv_q4_ws(_ptr(x), _ptr(wq), _ptr(scales), _ptr(zeros), _ptr(out),
                                          M, N, K, g, wp, wn, _stream(x.device)))
    return out


def gemv_q4_swiglu(x: torch.Tensor, gate: tuple, up: tuple, group_size: int,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """y = silu(x . Wg^T) * (x . Wu^T); gate and up are (wq, scales, zeros)."""
    M, N, K, g = _q4_operands(x, *gate, group_size)
    _q4_operands(x, *up, group_size, N=N)
    out = _out(out, M, N, x.device)
    (wg, sg, zg), (wu, su, zu) = gate, up
    _check("gemv_q4_swiglu", lib().gemv_q4_swiglu(
        _ptr(x), _ptr(wg), _ptr(sg), _ptr(zg), _ptr(wu), _ptr(su), _ptr(zu), _ptr(out),
        M, N, K, g, _stream(x.device)))
    return out


def gemv_f32(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Dense control: y[M, N] = x[M, K] . w[N, K]^T on the current stream."""
    _need(x, "x", (torch.float32,))
    dev = x.device
    _need(w, "w", (torch.float32,), dev)
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [M, K] and w [N, K]")
    M, K = x.shape
    N = w.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), dev)
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N]")
    _check("gemv_f32", lib().gemv_f32(_ptr(x), _ptr(w), _ptr(out), M, N, K, _stream(dev)))
    return out


def dequant_q4(wq: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, group_size: int,
               want_weights: bool = True, want_codes: bool = True):
    """Returns (W float32 [N, K] or None, codes uint8 [N, K] or None)."""
    _need(wq, "wq", (torch.uint8,))
    dev = wq.device
    _need(scales, "scales", (torch.float16, torch.uint16, torch.int16), dev)
    _need(zeros, "zeros", (torch.uint8,), dev)
    N, K = wq.shape[0], wq.shape[1] * 2
    g = int(group_size)
    G = K // g if g else 0
    if tuple(scales.shape) != (N, G) or tuple(zeros.shape) != (N, (G + 1) // 2):
        raise ValueError("scales/zeros shape mismatch")
    w = torch.empty((N, K), dtype=torch.float32, device=dev) if want_weights else None
    c = torch.empty((N, K), dtype=torch.uint8, device=dev) if want_codes else None
    _check("dequant_q4", lib().dequant_q4(_ptr(wq), _ptr(scales), _ptr(zeros), _ptr(w), _ptr(c),
                                          N, K, g, _stream(dev)))
    return w, c


def _partials(buf: torch.Tensor, n_partials: int, partials: torch.Tensor | None) -> torch.Tensor:
    _need(buf, "buf", (torch.float32,))
    if partials is None:
        return torch.empty(n_partials, dtype=torch.float32, device=buf.device)
    _need(partials, "partials", (torch.float32,), buf.device)
    if partials.numel() < n_partials:
        raise ValueError("partials too small")
    return partials


def read_reduce(buf: torch.Tensor, n_partials: int, partials: torch.Tensor | None = None) -> torch.Tensor:
    """Launches the streaming read probe (non-temporal loads); returns the
    per-workgroup partial sums (add them for the total)."""
    partials = _partials(buf, n_partials, partials)
    _check("read_reduce", lib().read_reduce(_ptr(buf), buf.numel(), _ptr(partials), n_partials,
                                            _stream(buf.device)))
    return partials


def read_reduce_passes(buf: torch.Tensor, n_partials: int, passes: int,
                       partials: torch.Tensor | None = None) -> torch.Tensor:
    """The read probe walking buf `passes` times with plain loads (so that a
    buffer that fits a cache is re-read from it); per-workgroup partial sums."""
    partials = _partials(buf, n_partials, partials)
    _check("read_reduce_passes", lib().read_reduce_passes(
        _ptr(buf), buf.numel(), passes, _ptr(partials), n_partials, _stream(buf.device)))
    return partials


def copy_vec4(src: torch.Tensor, dst: torch.Tensor | None = None, passes: int = 1,
              n_blocks: int = 0) -> torch.Tensor:
    """Copies src into dst (a new tensor if None) with the copy probe."""
    _need(src, "src", (torch.float32,))
    if dst is None:
        dst = torch.empty_like(src)
    else:
        _need(dst, "dst", (torch.float32,), src.device)
        if dst.numel() != src.numel():
            raise ValueError("dst and src differ in size")
    _check("copy_vec4", lib().copy_vec4(_ptr(src), _ptr(dst), src.numel(), passes, n_blocks,
                                        _stream(src.device)))
    return dst


def write_fill(buf: torch.Tensor, value: float, n_blocks: int = 0) -> torch.Tensor:
    """Fills buf with value using the write probe."""
    _need(buf, "buf", (torch.float32,))
    _check("write_fill", lib().write_fill(_ptr(buf), buf.numel(), float(value), n_blocks,
                                          _stream(buf.device)))
    return buf


def gemv_q4_geometry(M: int, N: int, K: int, group_size: int) -> dict:
    """Launch geometry gemv_q4 picks for a shape (host-only, needs no GPU)."""
    vals = [ctypes.c_int() for _ in range(6)]
    _check("gemv_q4_geometry", lib().gemv_q4_geometry(M, N, K, group_size,
                                                      *[ctypes.byref(v) for v in vals]))
    keys = ("grid", "block", "rows_per_wave", "lanes_per_row", "ksplit", "segments")
    return {k: v.value for k, v in zip(keys, vals)}


def gemv_q4_path(M: int, N: int, K: int, group_size: int) -> int:
    """Q4_PATH_FMA or Q4_PATH_INTEGER: the arithmetic path gemv_q4 takes (host-only)."""
    r = lib().gemv_q4_path(M, N, K, group_size)
    if r < 0:
        raise Q4Error("gemv_q4_path", r)
    return r


def abi_version() -> int:
    return lib().q4_abi_version()


def gemv_q4_set_geometry(M: int, N: int, K: int, group_size: int, path: int, waves: int = 0,
                         ksplit: int = 0) -> None:
    """Fix gemv_q4's geometry for one exact shape (host-only); raises Q4Error
    when the kernels cannot run that combination."""
    _check("gemv_q4_set_geometry", lib().gemv_q4_set_geometry(M, N, K, group_size, path, waves, ksplit))


def gemv_q4_clear_geometry() -> None:
    """Forget every geometry fixed by gemv_q4_set_geometry."""
    _check("gemv_q4_clear_geometry", lib().gemv_q4_clear_geometry())


# ---------------------------------------------------------------- block formats

def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        if fmt not in BLOCK_FORMATS:
            raise ValueError(f"unknown block format {fmt!r}")
        return BLOCK_FORMATS[fmt]
    return int(fmt)


def block_geometry(fmt) -> tuple[int, int]:
    """(elements, bytes) of one block of the format (host-only)."""
    e, b = ctypes.c_int(), ctypes.c_int()
    _check("block_geometry", lib().block_geometry(_fmt(fmt), ctypes.byref(e), ctypes.byref(b)))
    return e.value, b.value


def _block_matrix(fmt, w: torch.Tensor, K: int, dev=None) -> tuple[int, int]:
    _need(w, "w", (torch.uint8,), dev)
    e, b = block_geometry(fmt)
    if w.dim() != 2 or K % e or w.shape[1] != K // e * b:
        raise ValueError(f"w must be [N, K / {e} * {b}] bytes for K = {K}, got {tuple(w.shape)}")
    return w.shape[0], K // e * b


def gemv_block(fmt, x: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """y[1, N] = x[1, K] . W^T for a block-format matrix w uint8 [N, row_bytes]."""
    _need(x, "x", (torch.float32,))
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    N, _ = _block_matrix(fmt, w, K, x.device)
    out = _out(out, M, N, x.device)
    _check("gemv_block", lib().gemv_block(_fmt(fmt), _ptr(x), _ptr(w), _ptr(out), M, N, K,
                                          _stream(x.device)))
    return out


def dequant_block(fmt, w: torch.Tensor, K: int) -> torch.Tensor:
    """W float32 [N, K], bit-exact, from a block-format matrix."""
    N, _ = _block_matrix(fmt, w, K)
    out = torch.empty((N, K), dtype=torch.float32, device=w.device)
    _check("dequant_block", lib().dequant_block(_fmt(fmt), _ptr(w), _ptr(out), N, K,
                                                _stream(w.device)))
    return out


def gemv_block_set_config(fmt, rows_per_lane: int = 0, waves_per_group: int = 0,
                          groups_per_cu: int = 0) -> None:
    """Row slots per lane (1, 2, 4), wavefronts per workgroup (4, 8) and
    workgroups per CU (0 = one per row block) of gemv_block for one format;
    all zero restores the default (host-only)."""
    _check("gemv_block_set_config", lib().gemv_block_set_config(_fmt(fmt), rows_per_lane,
                                                                waves_per_group, groups_per_cu))


def gemv_block_config(fmt) -> tuple[int, int, int]:
    v = [ctypes.c_int() for _ in range(3)]
    _check("gemv_block_config", lib().gemv_block_config(_fmt(fmt), *[ctypes.byref(t) for t in v]))
    return tuple(t.value for t in v)


# ---------------------------------------------------------------- 2-bit scan

def scan2(codes: torch.Tensor, lut: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """scores[V, Q] = sum_d lut[q, d, code(v, d)] for codes uint32 (or int32)
    [V, D/16] and lut float32 [Q, D, 4]."""
    _need(codes, "codes", (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,))
    dev = codes.device
    _need(lut, "lut", (torch.float32,), dev)
    if codes.dim() != 2 or lut.dim() != 3 or lut.shape[2] != 4 or lut.shape[1] != 16 * codes.shape[1]:
        raise ValueError(f"codes must be [V, D/16] and lut [Q, D, 4]: got {tuple(codes.shape)}, "
                         f"{tuple(lut.shape)}")
    V, Q, D = codes.shape[0], lut.shape[0], lut.shape[1]
    out = _out(out, V, Q, dev)
    _check("scan2", lib().scan2(_ptr(codes), _ptr(lut), _ptr(out), V, D, Q, _stream(dev)))
    return out


def scan2_set_config(lut_in_lds: int = 0, vectors_per_thread: int = 0,
                     threads_per_group: int = 0, threads_per_vector: int = 0) -> None:
    """The scan's knobs: table in LDS (1) or memory (0), vectors per thread
    (1, 2), threads per workgroup (64, 256, 1024), threads per vector (1, 2,
    4, 8; an upper bound); all zero restores the default (host-only)."""
    _check("scan2_set_config", lib().scan2_set_config(lut_in_lds, vectors_per_thread,
                                                      threads_per_group, threads_per_vector))


def scan2_config() -> tuple[int, int, int, int]:
    v = [ctypes.c_int() for _ in range(4)]
    _check("scan2_config", lib().scan2_config(*[ctypes.byref(t) for t in v]))
    return tuple(t.value for t in v)


# ---------------------------------------------------------------- 8-bit activations and weights
#
# A call of these at one row takes longer on the host than on the GPU, so they
# go through a module in C++ (csrc/bind_i8.cpp) that tests the arguments,
# allocates and calls.  It returns None where an argument is not what it must
# be; the checks here then run one by one, to raise what is wrong.

_bind = None


def _load_bind():
    """The module, given the library's entry points; raises if either has not been
    built, or the module for another torch."""
    global _bind
    L = lib()
    try:
        from . import _bind_i8
    except ImportError as e:
        raise RuntimeError("the module _bind_i8 is not built for this Python; run "
                           "`python -m memory_bandwidth_amd.build` first") from e
    if _bind_i8.torch != torch.__version__:
        raise RuntimeError(f"the module _bind_i8 is built for torch {_bind_i8.torch}, this is {torch.__version__}; "
                           "run `python -m memory_bandwidth_amd.build` again")
    _bind_i8.init(getattr(torch._C, "_cuda_getCurrentRawStream", None),
                  *(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in EXPORTS_I8[:5]))
    _bind_i8.init_f8(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in EXPORTS_F8[:5]))
    _bind = _bind_i8
    return _bind


def _i8_check(tensors: dict) -> None:
    """Raises for the first tensor of the wrong type, place or layout, then for
    the first of the wrong shape.  tensors: name -> (tensor, dtypes, shape), None
    in a shape where any size will do."""
    dev = None
    for name, (t, dtypes, _) in tensors.items():
        _need(t, name, dtypes, dev)
        dev = t.device
    for name, (t, _, shape) in tensors.items():
        if t.dim() != len(shape) or any(s is not None and s != n for s, n in zip(shape, t.shape)):
            want = ", ".join("*" if s is None else str(s) for s in shape)
            raise ValueError(f"{name} must be [{want}], got {list(t.shape)}")


_I8, _F32, _I32 = torch.int8, torch.float32, torch.int32
_X_TYPES = tuple(I8_TYPES)


def _size(t, d: int):
    """t.shape[d], None where t has none such: for messages only."""
    return t.shape[d] if isinstance(t, torch.Tensor) and -t.dim() <= d < t.dim() else None


def _i8_check_product(a, a_scales, w, w_scales, bias, offsets, grouped, out, dtype) -> None:
    if dtype not in I8_TYPES:
        raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    E = (None if _size(offsets, 0) is None else _size(offsets, 0) - 1,) if grouped else ()
    M, N, K = _size(a, 0), _size(w, -2), _size(a, 1)
    tensors = {"a": (a, (_I8,), (None, None)), "a_scales": (a_scales, (_F32,), (M,))}
    if grouped:
        tensors["offsets"] = (offsets, (_I32,), (None,))
    tensors["w"] = (w, (_I8,), (*E, N, K))
    tensors["w_scales"] = (w_scales, (_F32,), (*E, N))
    if bias is not None:
        tensors["bias"] = (bias, (_F32,), (N,))
    if out is not None:
        tensors["out"] = (out, (dtype,), (M, N))
    _i8_check(tensors)


def _i8_refuse_product(*args) -> None:
    _i8_check_product(*args)
    raise ValueError("unsupported arguments")


def _i8_refuse_pair(a, a_scales, gate, up, offsets, grouped, out, dtype) -> None:
    for w, w_scales in (gate, up):
        if not isinstance(w, torch.Tensor) or not isinstance(w_scales, torch.Tensor):
            raise TypeError("gate and up must each be (weights, scales), two torch.Tensors")
    if gate[0].shape != up[0].shape:
        raise ValueError(f"gate and up must have one shape, got {list(gate[0].shape)} and {list(up[0].shape)}")
    for w, w_scales in (gate, up):
        _i8_check_product(a, a_scales, w, w_scales, None, offsets, grouped, out, dtype)
    raise ValueError("unsupported arguments")


def quant_i8(x: torch.Tensor, out: tuple | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes int8 [M, K], scales float32 [M]) of x [M, K], float32, float16 or
    bfloat16: scales[m] = max|x[m]| / 127 and codes = x / scales to the nearest
    integer.  K is a multiple of 16, M below 2^22.  A row with an Inf or a NaN
    gets the scale NaN and zero codes."""
    codes, scales = (None, None) if out is None else out
    got = (_bind or _load_bind()).quant(x, codes, scales)
    if type(got) is tuple:
        return got
    if got is None:
        _need(x, "x", _X_TYPES)
        if x.dim() != 2:
            raise ValueError(f"x must be [M, K], got {list(x.shape)}")
        tensors = {"x": (x, _X_TYPES, (None, None))}
        if out is not None:
            tensors.update(codes=(codes, (_I8,), x.shape), scales=(scales, (_F32,), x.shape[:1]))
        _i8_check(tensors)
        raise ValueError("unsupported arguments")
    raise Q4Error("quant_i8", got)


def gemm_i8(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
            bias: torch.Tensor | None = None, dtype=torch.float32,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """y[M, N] = (a[M, K] . w[N, K]^T) * a_scales[M] * w_scales[N] (+ bias[N]), the sums exact.

    a and w int8, scales and bias float32; y is of `dtype` (float32, float16
    or bfloat16).  K is a multiple of 16."""
    y = (_bind or _load_bind()).gemm(a, a_scales, w, w_scales, bias, None, dtype, out)
    if y is None:
        _i8_refuse_product(a, a_scales, w, w_scales, bias, None, False, out, dtype)
    if type(y) is int:
        raise Q4Error("gemm_i8", y)
    return y


def gemm_i8_swiglu(a: torch.Tensor, a_scales: torch.Tensor, gate: tuple, up: tuple,
                   dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """y = silu(g) * u with g, u the gemm_i8 of a with gate and up, each (w, w_scales)."""
    (wg, sg), (wu, su) = gate, up
    y = (_bind or _load_bind()).swiglu(a, a_scales, wg, sg, wu, su, None, dtype, out)
    if y is None:
        _i8_refuse_pair(a, a_scales, gate, up, None, False, out, dtype)
    if type(y) is int:
        raise Q4Error("gemm_i8_swiglu", y)
    return y


def gemm_i8_grouped(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                    offsets: torch.Tensor, dtype=torch.float32,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """The gemm_i8 of rows offsets[e] .. offsets[e + 1] of a with matrix e of w
    [E, N, K], w_scales [E, N].  offsets is int32 [E + 1] on the GPU, and is
    read there.  Rows outside every group are not written."""
    y = None if offsets is None else \
        (_bind or _load_bind()).gemm(a, a_scales, w, w_scales, None, offsets, dtype, out)
    if y is None:
        _i8_refuse_product(a, a_scales, w, w_scales, None, offsets, True, out, dtype)
    if type(y) is int:
        raise Q4Error("gemm_i8_grouped", y)
    return y


def gemm_i8_grouped_swiglu(a: torch.Tensor, a_scales: torch.Tensor, gate: tuple, up: tuple,
                           offsets: torch.Tensor, dtype=torch.float32,
                           out: torch.Tensor | None = None) -> torch.Tensor:
    """gemm_i8_swiglu of rows offsets[e] .. offsets[e + 1] with matrices e of gate and up."""
    (wg, sg), (wu, su) = gate, up
    y = None if offsets is None else \
        (_bind or _load_bind()).swiglu(a, a_scales, wg, sg, wu, su, offsets, dtype, out)
    if y is None:
        _i8_refuse_pair(a, a_scales, gate, up, offsets, True, out, dtype)
    if type(y) is int:
        raise Q4Error("gemm_i8_grouped_swiglu", y)
    return y


def gemm_i8_geometry(matrices: int, M: int, N: int, K: int, groups: int = 0) -> dict:
    """Launch geometry of the products for a shape (host-only, needs no GPU):
    matrices is 2 for the SwiGLU forms, groups 0 for a product without groups.
    grid is the workgroups of all launches, the tile that of the first."""
    vals = [ctypes.c_int() for _ in range(4)]
    _check("gemm_i8_geometry", lib().gemm_i8_geometry(matrices, M, groups, N, K, *[ctypes.byref(v) for v in vals]))
    return dict(zip(("tile_rows", "tile_cols", "grid", "block"), (v.value for v in vals)))


# ---------------------------------------------------------------- 8-bit floating point
#
# Codes are torch.float8_e4m3fn; a scale stands for 128 values of a row, or for a
# block of 128 x 128.  autograd does not see these calls: their results never
# require grad, whatever the arguments do, and a training step makes the calls of
# its backward pass itself, or from a torch.autograd.Function of its own.

_F8 = torch.float8_e4m3fn


def _blocks(n):
    return None if n is None else -(-n // 128)


def _f8_check(tensors: dict, strided: str) -> None:
    """_i8_check, where the tensor named `strided` may have any strides."""
    t, dtypes, shape = tensors.get(strided, (None, None, None))
    if isinstance(t, torch.Tensor) and t.layout == torch.strided:
        tensors[strided] = (t.new_empty(t.shape), dtypes, shape)
    _i8_check(tensors)


def _f8_check_product(a, a_scales, w, w_scales, bias, dtype, out, width=1, dh=None) -> None:
    if dtype not in I8_TYPES:
        raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    M, N, K = _size(a, 0), _size(w, 0), _size(a, 1)
    rows = _blocks(M) if _size(a_scales, 0) == _blocks(M) else M
    tensors = {"a": (a, (_F8,), (None, None)), "a_scales": (a_scales, (_F32,), (rows, _blocks(K))),
               "w": (w, (_F8,), (N, K)), "w_scales": (w_scales, (_F32,), (_blocks(N), _blocks(K)))}
    if bias is not None:
        tensors["bias"] = (bias, (_F32,), (N,))
    if dh is not None:
        tensors["dh"] = (dh[0], _X_TYPES, (M, N))
    if out is not None:
        tensors["out"] = (out, (dtype,), (M, None if N is None else width * N))
    _f8_check(tensors, "a_scales")


def _f8_refuse_product(*args) -> None:
    _f8_check_product(*args)
    raise ValueError("unsupported arguments")


def _f8_refuse_pair(a, a_scales, gate, up, dtype, out, width=1, dh=None) -> None:
    for w, w_scales in (gate, up):
        if not isinstance(w, torch.Tensor) or not isinstance(w_scales, torch.Tensor):
            raise TypeError("gate and up must each be (weights, scales), two torch.Tensors")
    if gate[0].shape != up[0].shape:
        raise ValueError(f"gate and up must have one shape, got {list(gate[0].shape)} and {list(up[0].shape)}")
    for w, w_scales in (gate, up):
        _f8_check_product(a, a_scales, w, w_scales, None, dtype, out, width, dh)
    raise ValueError("unsupported arguments")


def _f8_refuse_input(x, given: dict, rows: bool) -> None:
    _need(x, "x", _X_TYPES)
    if x.dim() != 2:
        raise ValueError(f"x must be [rows, columns], got {list(x.shape)}")
    _f8_check({"x": (x, _X_TYPES, (None, None)), **given}, "scales" if rows else "")
    raise ValueError("unsupported arguments")


def quant_f8(x: torch.Tensor, out: tuple | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes float8_e4m3fn [M, K], scales float32 [M, ceil(K / 128)]) of x [M, K], float32,
    float16 or bfloat16: a scale is the largest magnitude of its 128 values / 448, a
    code the e4m3 value nearest to x / scale.  K is a multiple of 16, M below
    2^22.  A block with an Inf or a NaN gets the scale NaN and zero codes.

    New scales lie block by block (their .t() is contiguous), as the products read
    them best; scales given with out may have any strides, of up to 2^20 from row to
    row and 2^31 from block to block, that give each of them a place of its own.

    The results do not require grad, also where x does: no gradient passes through."""
    codes, scales = (None, None) if out is None else out
    got = (_bind or _load_bind()).quant_f8(x, codes, scales)
    if type(got) is tuple:
        return got
    if got is None:
        shape = (_size(x, 0), _size(x, 1))
        _f8_refuse_input(x, {} if out is None else {
            "codes": (codes, (_F8,), shape), "scales": (scales, (_F32,), (shape[0], _blocks(shape[1])))}, True)
    raise Q4Error("quant_f8", got)


def quant_f8_block(x: torch.Tensor, layout: str = "rows", out: tuple | None = None) -> tuple:
    """x [R, C] (float32, float16 or bfloat16, C a multiple of 16, R below 2^22) to
    codes with a scale for each 128 x 128 block, by quant_f8's rule.  By layout:

      "rows"     (codes [R, C], scales [ceil(R / 128), ceil(C / 128)])
      "columns"  (codes [C, R16], scales [ceil(C / 128), ceil(R / 128)]) of the transpose, R16 = R
                 rounded up to a multiple of 16 and the codes behind R zero
      "both"     all four, from one pass

    The codes of a value are the same in both.  No gradient passes through, as in quant_f8."""
    if layout not in ("rows", "columns", "both"):
        raise ValueError(f"layout must be 'rows', 'columns' or 'both', got {layout!r}")
    as_is, turned = layout != "columns", layout != "rows"
    names = ("codes", "scales") * as_is + ("codes_t", "scales_t") * turned
    if out is not None and len(out) != len(names):
        raise ValueError(f"out must be ({', '.join(names)})")
    given = dict(zip(names, out)) if out is not None else {}
    got = (_bind or _load_bind()).quant_block_f8(
        x, as_is, turned, *(given.get(n) for n in ("codes", "scales", "codes_t", "scales_t")))
    if type(got) is tuple:
        return got
    if got is None:
        R, C = _size(x, 0) or 0, _size(x, 1) or 0
        shapes = {"codes": (R, C), "scales": (_blocks(R), _blocks(C)), "codes_t": (C, -(-R // 16) * 16),
                  "scales_t": (_blocks(C), _blocks(R))}
        _f8_refuse_input(x, {n: (t, (_F8,) if n.startswith("codes") else (_F32,), shapes[n])
                             for n, t in given.items()}, False)
    raise Q4Error("quant_f8_block", got)


def gemm_f8(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
            bias: torch.Tensor | None = None, dtype=torch.float32,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """y[M, N] = dequant(a)[M, K] . dequant(w)[N, K]^T (+ bias[N]).

    a and w float8_e4m3fn; a_scales float32 [M, ceil(K / 128)], of any strides up to
    2^20 from row to row and 2^31 from block to block, or one for each block of 128
    rows too, [ceil(M / 128), ceil(K / 128)]; w_scales float32
    [ceil(N / 128), ceil(K / 128)]; bias float32.  y is of `dtype`
    (float32, float16 or bfloat16), and dtype chooses how exact the sums are.  K is
    a multiple of 16.

    float32: products are exact and their sums of fp32's accuracy.  float16 and
    bfloat16: the matrix cores' 8-bit products, twice as fast, which lose of every
    eight consecutive k up to 7 * 2^-13 of the largest product: some 2^-16 of the
    result for normally distributed values, more than float16's own rounding
    where one product is far above its neighbours, and any part of a result whose
    products cancel.  Ask for float32 there.

    y does not require grad, whatever a, the scales or bias do: the gradients are
    products of their own (see gemm_f8_swiglu_backward)."""
    y = (_bind or _load_bind()).gemm_f8(a, a_scales, w, w_scales, bias, dtype, out)
    if y is None:
        _f8_refuse_product(a, a_scales, w, w_scales, bias, dtype, out)
    if type(y) is int:
        raise Q4Error("gemm_f8", y)
    return y


def gemm_f8_swiglu(a: torch.Tensor, a_scales: torch.Tensor, gate: tuple, up: tuple,
                   dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """y = silu(g) * u with g, u the gemm_f8 of a with gate and up, each (w, w_scales), as
    exact as gemm_f8's of that dtype; neither is stored.  y does not require grad:
    gemm_f8_swiglu_backward has the gradients of g and u."""
    (wg, sg), (wu, su) = gate, up
    y = (_bind or _load_bind()).swiglu_f8(a, a_scales, wg, sg, wu, su, dtype, out)
    if y is None:
        _f8_refuse_pair(a, a_scales, gate, up, dtype, out)
    if type(y) is int:
        raise Q4Error("gemm_f8_swiglu", y)
    return y


def gemm_f8_swiglu_backward(dh: torch.Tensor, a: torch.Tensor, a_scales: torch.Tensor, gate: tuple, up: tuple,
                            dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradients of gemm_f8_swiglu's g and u, side by side: d [M, 2 N] for dh [M, N],
    the gradient of y (float32, float16 or bfloat16).

    g and u are computed again, as exact as gemm_f8's of that dtype.  The gradient of
    the activations is d . [Wg; Wu] and that of [Wg; Wu] is d^T . x, both gemm_f8 of d's
    codes: of quant_f8(d) with the weights' quant_f8_block(.., "columns"), and of
    quant_f8_block(d, "columns") with quant_f8_block(x, "columns")."""
    (wg, sg), (wu, su) = gate, up
    d = None if dh is None else \
        (_bind or _load_bind()).swiglu_backward_f8(dh, a, a_scales, wg, sg, wu, su, dtype, out)
    if d is None:
        _f8_refuse_pair(a, a_scales, gate, up, dtype, out, 2, (dh,))
    if type(d) is int:
        raise Q4Error("gemm_f8_swiglu_backward", d)
    return d


def gemm_f8_geometry(matrices: int, M: int, N: int, K: int, dtype=torch.float32) -> dict:
    """Launch geometry of the products for a shape and output type (host-only, needs no
    GPU): matrices is 2 for the gated forms.  grid is the workgroups of all
    launches, the tile that of the first."""
    if dtype not in I8_TYPES:
        raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    vals = [ctypes.c_int() for _ in range(4)]
    _check("gemm_f8_geometry", lib().gemm_f8_geometry(matrices, I8_TYPES[dtype], M, N, K, *[ctypes.byref(v) for v in vals]))
    return dict(zip(("tile_rows", "tile_cols", "grid", "block"), (v.value for v in vals)))
