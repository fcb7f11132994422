"""Python binding of libsgpt (the C ABI declared in include/sgpt.h).

Argument marshalling only: every function here checks tensor dtypes, devices
and shapes, passes raw device pointers and the current CUDA stream to the
C entry point of the same name, and turns a non-OK status into SgptError.
All arithmetic of the solver runs in the library's CUDA kernels; PyTorch only
provides device memory and streams. There is no fallback: if the library is
missing, every call raises.
"""

from __future__ import annotations

import ctypes
import os
import warnings
from dataclasses import dataclass, field

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsgpt.so")

SGPT_OK = 0
STATUS_NAMES = {
    0: "OK", 1: "INVALID_ARG", 2: "NOT_PD", 3: "NONFINITE", 4: "TIMEOUT",
    5: "CUDA", 6: "UNSUPPORTED", 7: "BAD_MASK", 8: "WORKSPACE",
}
PATTERN_UNSTRUCTURED = 0
PATTERN_NM = 1

EXPORTS = (
    "sgpt_status_string", "sgpt_abi_version", "sgpt_kernel_launches", "sgpt_set_wait_limit",
    "sgpt_workspace_bytes",
    "sgpt_info_clear", "sgpt_sync_status", "sgpt_hessian_zero",
    "sgpt_hessian_accumulate", "sgpt_hessian_compute", "sgpt_factor", "sgpt_prune", "sgpt_prune_noalloc", "sgpt_pack24",
    "sgpt_pack_nm", "sgpt_pack_nm_meta_words", "sgpt_quant_grid", "sgpt_recon_error", "sgpt_prune_layer",
    "sgpt_mlp_block_workspace_bytes", "sgpt_prune_mlp_block", "sgpt_linear_bf16", "sgpt_to_bf16",
    "sgpt_sparse24_linear", "sgpt_sparse24_meta_tiles_bytes", "sgpt_sparse24_tile_meta",
    "sgpt_quant_codes", "sgpt_quant_tokens", "sgpt_quant_tokens_silu", "sgpt_linear_i8", "sgpt_attention",
    "sgpt_attn_block_workspace_bytes", "sgpt_prune_attn_block",
)
DRIVER_SEQUENTIAL = 0
DRIVER_PARALLEL = 1


class SgptError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{where}: SGPT_{'ERR_' if status else ''}{self.name} ({status})")


class _Params(ctypes.Structure):
    _fields_ = [("pattern", ctypes.c_int), ("n", ctypes.c_int), ("m", ctypes.c_int),
                ("sparsity", ctypes.c_float), ("blocksize", ctypes.c_int),
                ("damp", ctypes.c_float), ("forced", ctypes.c_int),
                ("qbits", ctypes.c_int), ("qgrid", ctypes.c_void_p)]


@dataclass(frozen=True)
class Params:
    """Sparsity pattern and solver knobs (mirrors sgpt_params)."""
    pattern: str = "2:4"        # "N:M" (e.g. "2:4", "16:64") or "unstructured:<fraction>"
    blocksize: int = 128
    damp: float = 0.01
    forced: bool = False
    qbits: int = 0              # >0: quantize the kept weights to 2**qbits levels per row
    qgrid: object = field(default=None, compare=False)   # [d_out, 2] fp32 CUDA tensor or None

    @property
    def is_nm(self) -> bool:
        return not self.pattern.startswith("unstructured")

    @property
    def nm(self) -> tuple[int, int]:
        """(N, M) of an N:M pattern."""
        n, m = (int(x) for x in self.pattern.split(":"))
        return n, m

    @property
    def sparsity(self) -> float:
        return 0.0 if self.is_nm else float(self.pattern.split(":")[1])

    def to_c(self) -> _Params:
        grid = None
        if self.qgrid is not None:
            _dev(self.qgrid, torch.float32, "qgrid")
            grid = self.qgrid.data_ptr()
        if self.is_nm:
            n, m = (int(x) for x in self.pattern.split(":"))
            return _Params(PATTERN_NM, n, m, 0.0, self.blocksize, self.damp, int(self.forced),
                           int(self.qbits), grid)
        return _Params(PATTERN_UNSTRUCTURED, 0, 0, self.sparsity, self.blocksize, self.damp,
                       int(self.forced), int(self.qbits), grid)


class _MlpBlock(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("W_gate", "W_up", "W_down", "mask_gate", "mask_up", "mask_down")]


class _AttnBlock(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("W_q", "W_k", "W_v", "W_o", "mask_q", "mask_k", "mask_v", "mask_o")]


_lib = None
_marshal = None         # the extension module that marshals the hot calls' arguments


def lib() -> ctypes.CDLL:
    """Load libsgpt.so once; raise loudly if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m post_pruning_b200.build` (needs nvcc)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    pp = ctypes.POINTER(_Params)
    sig = {
        "sgpt_status_string": (ctypes.c_char_p, [i32]),
        "sgpt_abi_version": (i32, []),
        "sgpt_kernel_launches": (ctypes.c_uint64, []),
        "sgpt_set_wait_limit": (i64, [i64]),
        "sgpt_workspace_bytes": (sz, [i32, i32, i64, pp]),
        "sgpt_info_clear": (i32, [vp, vp]),
        "sgpt_sync_status": (i32, [vp, vp]),
        "sgpt_hessian_zero": (i32, [vp, i32, vp]),
        "sgpt_hessian_accumulate": (i32, [vp, vp, i64, i32, vp, sz, vp, vp]),
        "sgpt_hessian_compute": (i32, [vp, vp, i64, i32, vp, sz, vp, vp]),
        "sgpt_factor": (i32, [vp, i64, i32, ctypes.c_float, vp, vp, sz, vp, vp]),
        "sgpt_prune": (i32, [vp, i32, i32, i32, vp, pp, vp, vp, vp, sz, vp, vp]),
        "sgpt_prune_noalloc": (i32, [vp, i32, i32, i32, vp, pp, vp, vp, vp, vp]),
        "sgpt_pack24": (i32, [vp, i32, i32, i32, vp, vp, vp, vp, vp]),
        "sgpt_pack_nm": (i32, [vp, i32, i32, i32, vp, i32, i32, vp, vp, vp, vp]),
        "sgpt_pack_nm_meta_words": (i32, [i32, i32, i32]),
        "sgpt_quant_grid": (i32, [vp, i32, i32, i32, i32, vp, vp]),
        "sgpt_mlp_block_workspace_bytes": (sz, [i32, i32, i64]),
        "sgpt_prune_mlp_block": (i32, [ctypes.POINTER(_MlpBlock), i32, i32, vp, i64, i32, pp, vp, vp, vp, sz,
                                       vp, vp]),
        "sgpt_linear_bf16": (i32, [vp, vp, i64, i32, i32, vp, vp, vp]),
        "sgpt_to_bf16": (i32, [vp, i32, i32, i32, vp, vp, vp]),
        "sgpt_sparse24_linear": (i32, [vp, vp, i32, i32, vp, i64, vp, vp, vp]),
        "sgpt_sparse24_meta_tiles_bytes": (sz, [i32, i32]),
        "sgpt_sparse24_tile_meta": (i32, [vp, i32, i32, vp, vp]),
        "sgpt_quant_codes": (i32, [vp, i32, i32, i32, vp, i32, vp, vp, vp]),
        "sgpt_quant_tokens": (i32, [vp, i64, i32, i64, vp, vp, vp, vp, vp]),
        "sgpt_quant_tokens_silu": (i32, [vp, vp, i64, i32, i64, i64, vp, vp, vp, vp, vp]),
        "sgpt_linear_i8": (i32, [vp, vp, vp, i64, vp, vp, i32, i32, i32, vp, i32, vp, vp]),
        "sgpt_attention": (i32, [vp, i64, vp, i64, vp, i64, vp, i32, i64, i32, i32, i32, ctypes.c_float, vp, i64,
                                 vp, vp]),
        "sgpt_attn_block_workspace_bytes": (sz, [i32, i32, i32, i32, i64]),
        "sgpt_prune_attn_block": (i32, [ctypes.POINTER(_AttnBlock), i32, i32, i32, i32, ctypes.c_float, vp, i64, vp,
                                        i32, i32, pp, vp, vp, vp, sz, vp, vp]),
        "sgpt_recon_error": (i32, [vp, vp, i32, i32, i32, vp, vp, vp, sz, vp]),
        "sgpt_prune_layer": (i32, [vp, i32, i32, i32, vp, i64, vp, vp, pp, vp, vp, vp, vp,
                                   vp, sz, vp, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    global _marshal
    _lib, _marshal = L, _load_marshal(L)
    return L


def _load_marshal(L):
    """The extension module, built with the library; None where there is none
    for this torch (the Python functions then make every call)."""
    try:
        from . import _marshal as m
    except ImportError as e:
        why = str(e)
    else:
        built = getattr(m, "torch_version", None)
        if built == torch.__version__:
            m.bind(*(ctypes.cast(getattr(L, "sgpt_" + name), ctypes.c_void_p).value for name in
                     ("quant_tokens", "quant_tokens_silu", "linear_i8", "attention")))
            return m
        why = f"it was built for torch {built}"
    warnings.warn("post_pruning_b200._marshal is not used, calls take 5-9 us more of host time "
                  f"(python -m post_pruning_b200.build builds it): {why}", RuntimeWarning, stacklevel=3)
    return None


# ------------------------------------------------------------------ helpers

def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, dtype, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _one_device(*tensors: torch.Tensor) -> int:
    """The index of the CUDA device of `tensors`, which must be one."""
    try:
        dev = tensors[0].get_device()                  # -1 on the CPU
        for t in tensors:
            if t.get_device() != dev:
                raise ValueError("all tensors must be on one device")
    except AttributeError:
        raise TypeError("all operands must be CUDA tensors") from None
    if dev < 0:
        raise TypeError("all operands must be CUDA tensors")
    return dev


def _one_word(dev_info: torch.Tensor):
    """dev_info: an int32 tensor whose first word the kernels read and write."""
    if dev_info.dtype is not torch.int32:
        raise TypeError("dev_info must be int32")
    if dev_info.numel() < 1:
        raise ValueError("dev_info must have one word")


# the handle of a device's current stream, without the Stream object that
# torch.cuda.current_stream() builds (3 us of a call that takes 6)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _enqueue(entry: str, dev: int, stream, *args):
    """Calls a C entry whose last argument is the stream, with the tensors'
    device current."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _enqueue(entry, dev, stream, *args)
    status = getattr(_lib or lib(), entry)(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if status != SGPT_OK:
        raise SgptError(status, entry)


def _rowmajor(t: torch.Tensor, name: str) -> int:
    """Leading dimension of a 2-D tensor with unit column stride."""
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    return t.stride(0)


def _row_stride(t: torch.Tensor, name: str) -> int:
    """_rowmajor, where the stride of a single row (which no access uses) does
    not matter."""
    ld = _rowmajor(t, name)
    return ld if t.shape[0] > 1 else t.shape[1]


def _check(status: int, where: str):
    if status != SGPT_OK:
        raise SgptError(status, where)


def kernel_launches() -> int:
    """Kernels libsgpt has enqueued since it was loaded."""
    return int(lib().sgpt_kernel_launches())


def set_wait_limit(cycles: int) -> int:
    """Cycles a device-side wait polls before it records TIMEOUT (<= 0: the
    default). Returns the previous value. For testing failure paths."""
    return int(lib().sgpt_set_wait_limit(int(cycles)))


def workspace_bytes(d_out: int, d_in: int, n_tok: int = 0, params: Params | None = None) -> int:
    p = (params or Params()).to_c()
    return int(lib().sgpt_workspace_bytes(d_out, d_in, n_tok, ctypes.byref(p)))


def workspace(d_out: int, d_in: int, n_tok: int = 0, params: Params | None = None,
              device="cuda") -> torch.Tensor:
    """A byte tensor large enough for every call at these sizes."""
    return torch.empty(workspace_bytes(d_out, d_in, n_tok, params), dtype=torch.uint8, device=device)


def new_info(device="cuda") -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


# ------------------------------------------------------------- entry points

def info_clear(dev_info: torch.Tensor, stream=None):
    _check(lib().sgpt_info_clear(_ptr(dev_info), _stream(stream)), "sgpt_info_clear")


def sync_status(dev_info: torch.Tensor, stream=None) -> int:
    """Blocking; returns the status code (0 = OK) without raising."""
    return int(lib().sgpt_sync_status(_ptr(dev_info), _stream(stream)))


def raise_on_info(dev_info: torch.Tensor, stream=None, where="device"):
    _check(sync_status(dev_info, stream), where)


def hessian_zero(H: torch.Tensor, stream=None):
    _dev(H, torch.float32, "H")
    _check(lib().sgpt_hessian_zero(_ptr(H), H.shape[0], _stream(stream)), "sgpt_hessian_zero")


def hessian_accumulate(H: torch.Tensor, X: torch.Tensor, ws: torch.Tensor, dev_info: torch.Tensor,
                       stream=None):
    _dev(H, torch.float32, "H")
    _dev(X, torch.bfloat16, "X")
    d = H.shape[0]
    if H.shape != (d, d) or not H.is_contiguous() or X.dim() != 2 or X.shape[1] != d or not X.is_contiguous():
        raise ValueError("H must be [d, d] and X [n, d], both contiguous")
    _check(lib().sgpt_hessian_accumulate(_ptr(H), _ptr(X), X.shape[0], d, _ptr(ws), ws.numel(),
                                         _ptr(dev_info), _stream(stream)), "sgpt_hessian_accumulate")


def hessian_compute(H: torch.Tensor, X: torch.Tensor, ws: torch.Tensor, dev_info: torch.Tensor, stream=None):
    """H = X^T X (sgpt_hessian_compute): like hessian_zero + hessian_accumulate
    without reading H."""
    _dev(H, torch.float32, "H")
    _dev(X, torch.bfloat16, "X")
    d = H.shape[0]
    if H.shape != (d, d) or not H.is_contiguous() or X.dim() != 2 or X.shape[1] != d or not X.is_contiguous():
        raise ValueError("H must be [d, d] and X [n, d], both contiguous")
    _check(lib().sgpt_hessian_compute(_ptr(H), _ptr(X), X.shape[0], d, _ptr(ws), ws.numel(),
                                      _ptr(dev_info), _stream(stream)), "sgpt_hessian_compute")


def factor(H: torch.Tensor, n_total: int, damp: float, U: torch.Tensor, ws: torch.Tensor,
           dev_info: torch.Tensor, stream=None):
    _dev(H, torch.float32, "H")
    _dev(U, torch.float32, "U")
    d = H.shape[0]
    if H.shape != (d, d) or U.shape != (d, d) or not H.is_contiguous() or not U.is_contiguous():
        raise ValueError("H and U must be contiguous [d, d]")
    _check(lib().sgpt_factor(_ptr(H), n_total, d, damp, _ptr(U), _ptr(ws), ws.numel(), _ptr(dev_info),
                             _stream(stream)), "sgpt_factor")


def prune(W: torch.Tensor, U: torch.Tensor, params: Params, mask: torch.Tensor, ws: torch.Tensor,
          dev_info: torch.Tensor, row_loss: torch.Tensor | None = None, stream=None):
    _dev(W, torch.float32, "W")
    _dev(U, torch.float32, "U")
    _dev(mask, torch.int32, "mask")
    ldw = _rowmajor(W, "W")
    r, d = W.shape
    if mask.shape != (r, d // 32) or not mask.is_contiguous():
        raise ValueError("mask must be contiguous int32 [d_out, d_in/32]")
    if row_loss is not None:
        _dev(row_loss, torch.float32, "row_loss")
    p = params.to_c()
    _check(lib().sgpt_prune(_ptr(W), r, d, ldw, _ptr(U), ctypes.byref(p), _ptr(mask), _ptr(row_loss),
                            _ptr(ws), ws.numel(), _ptr(dev_info), _stream(stream)), "sgpt_prune")


NOALLOC_MAX_ROWS = 8192


def prune_noalloc(W: torch.Tensor, U: torch.Tensor, params: Params, mask: torch.Tensor,
                  dev_info: torch.Tensor, row_loss: torch.Tensor | None = None, stream=None):
    """sgpt_prune without a workspace, for callers that cannot allocate device
    memory where they call it: the scratch is a fixed array inside the library
    (d_out <= NOALLOC_MAX_ROWS). Calls that overlap on the GPU race on it."""
    _dev(W, torch.float32, "W")
    _dev(U, torch.float32, "U")
    _dev(mask, torch.int32, "mask")
    ldw = _rowmajor(W, "W")
    r, d = W.shape
    if mask.shape != (r, d // 32) or not mask.is_contiguous():
        raise ValueError("mask must be contiguous int32 [d_out, d_in/32]")
    if row_loss is not None:
        _dev(row_loss, torch.float32, "row_loss")
    p = params.to_c()
    _check(lib().sgpt_prune_noalloc(_ptr(W), r, d, ldw, _ptr(U), ctypes.byref(p), _ptr(mask),
                                    _ptr(row_loss), _ptr(dev_info), _stream(stream)),
           "sgpt_prune_noalloc")


def pack24(W: torch.Tensor, mask: torch.Tensor, values: torch.Tensor, meta: torch.Tensor,
           dev_info: torch.Tensor, stream=None):
    _dev(W, torch.float32, "W")
    _dev(values, torch.float32, "values")
    _dev(mask, torch.int32, "mask")
    _dev(meta, torch.int32, "meta")
    ldw = _rowmajor(W, "W")
    r, d = W.shape
    if values.shape != (r, d // 2) or meta.shape != (r, d // 32):
        raise ValueError("values must be [d_out, d_in/2] and meta [d_out, d_in/32]")
    _check(lib().sgpt_pack24(_ptr(W), r, d, ldw, _ptr(mask), _ptr(values), _ptr(meta), _ptr(dev_info),
                             _stream(stream)), "sgpt_pack24")


def quant_grid(W: torch.Tensor, qbits: int, grid: torch.Tensor, stream=None):
    """Per-row quantization grid of the dense W (sgpt_quant_grid): grid
    [d_out, 2] fp32 = (scale, zero point)."""
    _dev(W, torch.float32, "W")
    _dev(grid, torch.float32, "grid")
    ldw = _rowmajor(W, "W")
    r, d = W.shape
    if grid.shape != (r, 2) or not grid.is_contiguous():
        raise ValueError("grid must be contiguous [d_out, 2]")
    _check(lib().sgpt_quant_grid(_ptr(W), r, d, ldw, qbits, _ptr(grid), _stream(stream)), "sgpt_quant_grid")


def to_bf16(W: torch.Tensor, Wb: torch.Tensor, dev_info: torch.Tensor, stream=None):
    """Wb = W rounded to bf16 (sgpt_to_bf16)."""
    _dev(W, torch.float32, "W")
    _dev(Wb, torch.bfloat16, "Wb")
    ldw = _rowmajor(W, "W")
    if Wb.shape != W.shape or not Wb.is_contiguous():
        raise ValueError("Wb must be contiguous with W's shape")
    _check(lib().sgpt_to_bf16(_ptr(W), W.shape[0], W.shape[1], ldw, _ptr(Wb), _ptr(dev_info), _stream(stream)),
           "sgpt_to_bf16")


def linear_bf16(X: torch.Tensor, Wb: torch.Tensor, Y: torch.Tensor, dev_info: torch.Tensor, stream=None):
    """Y = X Wb^T on the tensor cores (sgpt_linear_bf16): X [n, d_in] and Wb
    [d_out, d_in] bf16, Y [n, d_out] fp32."""
    _dev(X, torch.bfloat16, "X")
    _dev(Wb, torch.bfloat16, "Wb")
    _dev(Y, torch.float32, "Y")
    n, d_in = X.shape
    d_out = Wb.shape[0]
    if Wb.shape[1] != d_in or Y.shape != (n, d_out) or not (X.is_contiguous() and Wb.is_contiguous()
                                                             and Y.is_contiguous()):
        raise ValueError("X [n, d_in], Wb [d_out, d_in], Y [n, d_out], all contiguous")
    _check(lib().sgpt_linear_bf16(_ptr(X), _ptr(Wb), n, d_in, d_out, _ptr(Y), _ptr(dev_info), _stream(stream)),
           "sgpt_linear_bf16")


def sparse24_meta_tiles(meta: torch.Tensor, d_in: int, out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """sgpt_pack24's metadata words meta [d_out, d_in/32] int32 re-arranged
    for sparse24_linear (sgpt_sparse24_tile_meta); done once per weight
    matrix. Returns (or fills) an int32 buffer of
    sgpt_sparse24_meta_tiles_bytes(d_out, d_in) bytes."""
    _dev(meta, torch.int32, "meta")
    d_out = meta.shape[0]
    if meta.shape != (d_out, d_in // 32) or not meta.is_contiguous():
        raise ValueError("meta [d_out, d_in/32], contiguous")
    nbytes = lib().sgpt_sparse24_meta_tiles_bytes(d_out, d_in)
    if nbytes == 0:
        raise ValueError(f"unsupported sizes d_out={d_out} d_in={d_in}")
    if out is None:
        out = torch.empty(nbytes // 4, dtype=torch.int32, device=meta.device)
    _dev(out, torch.int32, "out")
    if out.numel() * 4 < nbytes or not out.is_contiguous():
        raise ValueError(f"out needs {nbytes} contiguous bytes")
    _check(lib().sgpt_sparse24_tile_meta(_ptr(meta), d_out, d_in, _ptr(out), _stream(stream)),
           "sgpt_sparse24_tile_meta")
    return out


def sparse24_linear(values: torch.Tensor, meta_tiles: torch.Tensor, X: torch.Tensor, Y: torch.Tensor,
                    dev_info: torch.Tensor, stream=None):
    """Y = X W^T from W's packed 2:4 form on the sparse tensor cores
    (sgpt_sparse24_linear): values [d_out, d_in/2] bf16, meta_tiles from
    sparse24_meta_tiles, X [n, d_in] bf16, Y [n, d_out] fp32."""
    _dev(values, torch.bfloat16, "values")
    _dev(meta_tiles, torch.int32, "meta_tiles")
    _dev(X, torch.bfloat16, "X")
    _dev(Y, torch.float32, "Y")
    d_out, half = values.shape
    n, d_in = X.shape
    if half * 2 != d_in or Y.shape != (n, d_out):
        raise ValueError("values [d_out, d_in/2], X [n, d_in], Y [n, d_out]")
    if meta_tiles.numel() * 4 < lib().sgpt_sparse24_meta_tiles_bytes(d_out, d_in):
        raise ValueError("meta_tiles too small for these sizes")
    if not (values.is_contiguous() and meta_tiles.is_contiguous() and X.is_contiguous() and Y.is_contiguous()):
        raise ValueError("all operands must be contiguous")
    _check(lib().sgpt_sparse24_linear(_ptr(values), _ptr(meta_tiles), d_out, d_in, _ptr(X), n, _ptr(Y),
                                      _ptr(dev_info), _stream(stream)), "sgpt_sparse24_linear")


def quant_codes(W: torch.Tensor, grid: torch.Tensor, codes: torch.Tensor, dev_info: torch.Tensor, qbits: int = 8,
                stream=None):
    """8-bit codes of W on its rows' grid (sgpt_quant_codes), once per weight
    matrix: W [d_out, d_in] fp32, grid [d_out, 2] fp32 (quant_grid's, or the
    qgrid of the sweep), codes [d_out, d_in] int8."""
    _dev(W, torch.float32, "W")
    _dev(grid, torch.float32, "grid")
    _dev(codes, torch.int8, "codes")
    ldw = _rowmajor(W, "W")
    r, d = W.shape
    if grid.shape != (r, 2) or codes.shape != (r, d) or not grid.is_contiguous() or not codes.is_contiguous():
        raise ValueError("grid must be contiguous [d_out, 2] and codes contiguous [d_out, d_in]")
    dev = _one_device(W, grid, codes, dev_info)
    _one_word(dev_info)
    _enqueue("sgpt_quant_codes", dev, stream, _ptr(W), r, d, ldw, _ptr(grid), qbits,
             _ptr(codes), _ptr(dev_info))


# The calls below are made once per token and layer, and checking their
# arguments here takes longer than launching them. So the extension module
# (csrc/marshal.cpp) is asked first: it makes the same checks and the call,
# and answers the status, or -1 where the arguments are not plainly valid (or
# on another device than the current one); then they are checked again here,
# to raise what is wrong with them or to make the call.

def _token_codes(n: int, d: int, Xq: torch.Tensor, scale: torch.Tensor, sums: torch.Tensor):
    """Xq [n, d] int8, scale [n] fp32, sums [n] int32, contiguous."""
    if not (Xq.dtype is torch.int8 and scale.dtype is torch.float32 and sums.dtype is torch.int32):
        raise TypeError("Xq must be int8, scale float32 and sums int32")
    if not (Xq.shape == (n, d) and scale.shape == (n,) and sums.shape == (n,) and Xq.is_contiguous()
            and scale.is_contiguous() and sums.is_contiguous()):
        raise ValueError("Xq must be [n, d], scale and sums [n], all contiguous")


def quant_tokens(X: torch.Tensor, Xq: torch.Tensor, scale: torch.Tensor, sums: torch.Tensor,
                 dev_info: torch.Tensor, stream=None):
    """X [n, d] bf16 to 8 bits with a scale per token (sgpt_quant_tokens):
    Xq [n, d] int8, scale [n] fp32, sums [n] int32 (the codes' row sums)."""
    if stream is None and _marshal is not None:
        status = _marshal.quant_tokens(X, Xq, scale, sums, dev_info)
        if status == SGPT_OK:
            return
        if status > 0:
            raise SgptError(status, "sgpt_quant_tokens")
    dev = _one_device(X, Xq, scale, sums, dev_info)
    _one_word(dev_info)
    if X.dtype is not torch.bfloat16:
        raise TypeError("X must be bfloat16")
    ldx = _row_stride(X, "X")
    n, d = X.shape
    _token_codes(n, d, Xq, scale, sums)
    _enqueue("sgpt_quant_tokens", dev, stream, X.data_ptr(), n, d, ldx, Xq.data_ptr(), scale.data_ptr(),
             sums.data_ptr(), dev_info.data_ptr())


def quant_tokens_silu(G: torch.Tensor, U: torch.Tensor, Xq: torch.Tensor, scale: torch.Tensor, sums: torch.Tensor,
                      dev_info: torch.Tensor, stream=None):
    """quant_tokens of silu(G) * U, an MLP's gated activation, without
    rounding it to bf16 in between (sgpt_quant_tokens_silu)."""
    if stream is None and _marshal is not None:
        status = _marshal.quant_tokens_silu(G, U, Xq, scale, sums, dev_info)
        if status == SGPT_OK:
            return
        if status > 0:
            raise SgptError(status, "sgpt_quant_tokens_silu")
    dev = _one_device(G, U, Xq, scale, sums, dev_info)
    _one_word(dev_info)
    if not (G.dtype is torch.bfloat16 and U.dtype is torch.bfloat16):
        raise TypeError("G and U must be bfloat16")
    ldg, ldu = _row_stride(G, "G"), _row_stride(U, "U")
    n, d = G.shape
    if U.shape != (n, d):
        raise ValueError("G and U must have the same shape")
    _token_codes(n, d, Xq, scale, sums)
    _enqueue("sgpt_quant_tokens_silu", dev, stream, G.data_ptr(), U.data_ptr(), n, d, ldg, ldu, Xq.data_ptr(),
             scale.data_ptr(), sums.data_ptr(), dev_info.data_ptr())


def linear_i8(Xq: torch.Tensor, scale: torch.Tensor, sums: torch.Tensor, codes: torch.Tensor, grid: torch.Tensor,
              Y: torch.Tensor, dev_info: torch.Tensor, qbits: int = 8, stream=None):
    """Y = X W^T in 8-bit integers (sgpt_linear_i8): Xq, scale, sums from
    quant_tokens, codes [d_out, d_in] int8 from quant_codes with its grid and
    qbits, Y [n, d_out] fp32 or bf16."""
    if stream is None and _marshal is not None:
        status = _marshal.linear_i8(Xq, scale, sums, codes, grid, Y, dev_info, qbits)
        if status == SGPT_OK:
            return
        if status > 0:
            raise SgptError(status, "sgpt_linear_i8")
    dev = _one_device(Xq, scale, sums, codes, grid, Y, dev_info)
    _one_word(dev_info)
    y_bf16 = Y.dtype is torch.bfloat16
    if not (codes.dtype is torch.int8 and grid.dtype is torch.float32 and (y_bf16 or Y.dtype is torch.float32)):
        raise TypeError("codes must be int8, grid float32 and Y float32 or bfloat16")
    if Xq.dim() != 2 or codes.dim() != 2:
        raise ValueError("Xq must be [n, d_in] and codes [d_out, d_in]")
    n, d_in = Xq.shape
    d_out = codes.shape[0]
    _token_codes(n, d_in, Xq, scale, sums)
    if not (codes.shape[1] == d_in and grid.shape == (d_out, 2) and Y.shape == (n, d_out) and codes.is_contiguous()
            and grid.is_contiguous() and Y.is_contiguous()):
        raise ValueError("codes must be [d_out, d_in], grid [d_out, 2] and Y [n, d_out], all contiguous")
    _enqueue("sgpt_linear_i8", dev, stream, Xq.data_ptr(), scale.data_ptr(), sums.data_ptr(), n, codes.data_ptr(),
             grid.data_ptr(), qbits, d_in, d_out, Y.data_ptr(), y_bf16, dev_info.data_ptr())


def _heads_stride(t: torch.Tensor, name: str) -> int:
    """Row stride of a bf16 [rows, heads, width] with consecutive heads."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if len(shape) != 3 or stride[2] != 1 or (stride[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"{name} must be [rows, heads, width] with consecutive heads")
    return stride[0] if shape[0] > 1 else shape[1] * shape[2]


def attention(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, offsets: torch.Tensor, O: torch.Tensor,
              dev_info: torch.Tensor, scale: float | None = None, stream=None):
    """Causal attention over packed prompts (sgpt_attention): Q, O [n_tok,
    heads, width], K, V [n_tok, kv_heads, width] bf16 (width 64 or 128; rows
    may be strided, e.g. parts of one q/k/v buffer), offsets [n_seq + 1] int32
    on the device: sequence s has the rows offsets[s]:offsets[s + 1]. scale:
    width ** -0.5 when None."""
    if stream is None and _marshal is not None:
        status = _marshal.attention(Q, K, V, offsets, O, dev_info, scale)
        if status == SGPT_OK:
            return
        if status > 0:
            raise SgptError(status, "sgpt_attention")
    dev = _one_device(Q, K, V, offsets, O, dev_info)
    _one_word(dev_info)
    ldq, ldk, ldv, ldo = _heads_stride(Q, "Q"), _heads_stride(K, "K"), _heads_stride(V, "V"), _heads_stride(O, "O")
    n, heads, width = shape = Q.shape
    kv_heads = K.shape[1]
    if not (O.shape == shape and K.shape == (n, kv_heads, width) and V.shape == K.shape):
        raise ValueError("Q and O must be [n_tok, heads, width], K and V [n_tok, kv_heads, width]")
    if offsets.dtype is not torch.int32:
        raise TypeError("offsets must be int32")
    if offsets.dim() != 1 or offsets.shape[0] < 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be contiguous [n_seq + 1]")
    _enqueue("sgpt_attention", dev, stream, Q.data_ptr(), ldq, K.data_ptr(), ldk, V.data_ptr(), ldv, offsets.data_ptr(),
             offsets.shape[0] - 1, n, heads, kv_heads, width, width ** -0.5 if scale is None else scale, O.data_ptr(),
             ldo, dev_info.data_ptr())


def mlp_block_workspace(hidden: int, inter: int, n_tok: int, device="cuda") -> torch.Tensor:
    b = int(lib().sgpt_mlp_block_workspace_bytes(hidden, inter, n_tok))
    if b == 0:
        raise ValueError("unsupported block sizes")
    return torch.empty(b, dtype=torch.uint8, device=device)


def prune_mlp_block(W_gate: torch.Tensor, W_up: torch.Tensor, W_down: torch.Tensor, masks, X: torch.Tensor,
                    params: Params, X_next: torch.Tensor, ws: torch.Tensor, dev_info: torch.Tensor,
                    mode: int = DRIVER_SEQUENTIAL, Z: torch.Tensor | None = None, stream=None):
    """One synthetic MLP block pruned layer by layer (sgpt_prune_mlp_block).
    masks: (gate, up, down) int32 mask-bit tensors."""
    for t, name in ((W_gate, "W_gate"), (W_up, "W_up"), (W_down, "W_down")):
        _dev(t, torch.float32, name)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _dev(X, torch.bfloat16, "X")
    _dev(X_next, torch.bfloat16, "X_next")
    inter, hidden = W_gate.shape
    if W_up.shape != (inter, hidden) or W_down.shape != (hidden, inter):
        raise ValueError("W_gate, W_up [inter, hidden] and W_down [hidden, inter]")
    n = X.shape[0]
    if X.shape != (n, hidden) or X_next.shape != (n, hidden):
        raise ValueError("X and X_next must be [n_tok, hidden]")
    if Z is not None:
        _dev(Z, torch.bfloat16, "Z")
        if Z.shape != (n, inter) or not Z.is_contiguous():
            raise ValueError("Z must be contiguous [n_tok, inter]")
    mg, mu, md = masks
    for m_, shape in ((mg, (inter, hidden // 32)), (mu, (inter, hidden // 32)), (md, (hidden, inter // 32))):
        _dev(m_, torch.int32, "mask")
        if m_.shape != shape or not m_.is_contiguous():
            raise ValueError(f"mask must be contiguous {shape}")
    blk = _MlpBlock(_ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(mg), _ptr(mu), _ptr(md))
    p = params.to_c()
    _check(lib().sgpt_prune_mlp_block(ctypes.byref(blk), hidden, inter, _ptr(X), n, mode, ctypes.byref(p),
                                      _ptr(X_next), _ptr(Z), _ptr(ws), ws.numel(), _ptr(dev_info),
                                      _stream(stream)), "sgpt_prune_mlp_block")


def attn_block_workspace(hidden: int, heads: int, kv_heads: int, width: int, n_tok: int,
                         device="cuda") -> torch.Tensor:
    b = int(lib().sgpt_attn_block_workspace_bytes(hidden, heads, kv_heads, width, n_tok))
    if b == 0:
        raise ValueError("unsupported block sizes")
    return torch.empty(b, dtype=torch.uint8, device=device)


def prune_attn_block(W_q: torch.Tensor, W_k: torch.Tensor, W_v: torch.Tensor, W_o: torch.Tensor, masks,
                     X: torch.Tensor, offsets: torch.Tensor, width: int, params: Params, X_next: torch.Tensor,
                     ws: torch.Tensor, dev_info: torch.Tensor, mode: int = DRIVER_SEQUENTIAL,
                     A: torch.Tensor | None = None, scale: float | None = None, stream=None):
    """The attention part of a decoder block pruned layer by layer over packed
    prompts (sgpt_prune_attn_block). W_q [heads * width, hidden], W_k, W_v
    [kv_heads * width, hidden], W_o [hidden, heads * width] fp32; masks:
    (q, k, v, o) int32 mask-bit tensors; offsets [n_seq + 1] int32; A [n_tok,
    heads * width] bf16 receives o's input. scale: width ** -0.5 when None."""
    dq, hidden = W_q.shape
    dk = W_k.shape[0]
    n = X.shape[0]
    if width < 1 or dq % width or dk % width:
        raise ValueError("the rows of W_q, W_k and W_v are whole heads of `width`")
    dev = _one_device(W_q, W_k, W_v, W_o, *masks, X, offsets, X_next, ws, dev_info, *(() if A is None else (A,)))
    _one_word(dev_info)
    for t, name, shape in ((W_q, "W_q", (dq, hidden)), (W_k, "W_k", (dk, hidden)), (W_v, "W_v", (dk, hidden)),
                           (W_o, "W_o", (hidden, dq))):
        _dev(t, torch.float32, name)
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {shape}")
    for t, shape in zip(masks, ((dq, hidden // 32), (dk, hidden // 32), (dk, hidden // 32), (hidden, dq // 32)),
                        strict=True):
        _dev(t, torch.int32, "mask")
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"mask must be contiguous {shape}")
    for t, name, shape in ((X, "X", (n, hidden)), (X_next, "X_next", (n, hidden)), (A, "A", (n, dq))):
        if t is None:
            continue
        _dev(t, torch.bfloat16, name)
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {shape}")
    _dev(offsets, torch.int32, "offsets")
    if offsets.dim() != 1 or offsets.shape[0] < 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be contiguous [n_seq + 1]")
    blk = _AttnBlock(*(_ptr(t) for t in (W_q, W_k, W_v, W_o, *masks)))
    p = params.to_c()
    _enqueue("sgpt_prune_attn_block", dev, stream, ctypes.byref(blk), hidden, dq // width, dk // width, width,
             width ** -0.5 if scale is None else scale, _ptr(X), n, _ptr(offsets), offsets.shape[0] - 1, mode,
             ctypes.byref(p), _ptr(X_next), _ptr(A), _ptr(ws), ws.numel(), _ptr(dev_info))


def pack_nm_meta_words(d_in: int, n: int, m: int) -> int:
    """uint32 metadata words per row of an N:M pack (-1 if unsupported)."""
    return int(lib().sgpt_pack_nm_meta_words(d_in, n, m))


def pack_nm(W: torch.Tensor, mask: torch.Tensor, n: int, m: int, values: torch.Tensor, meta: torch.Tensor,
            dev_info: torch.Tensor, stream=None):
    """N:M packing (sgpt_pack_nm): values [d_out, d_in*n/m] fp32, meta
    [d_out, pack_nm_meta_words(d_in, n, m)] int32."""
    _dev(W, torch.float32, "W")
    _dev(values, torch.float32, "values")
    _dev(mask, torch.int32, "mask")
    _dev(meta, torch.int32, "meta")
    ldw = _rowmajor(W, "W")
    r, d = W.shape
    words = pack_nm_meta_words(d, n, m)
    if words < 0:
        raise ValueError(f"unsupported N:M {n}:{m} for d_in {d}")
    if values.shape != (r, d * n // m) or meta.shape != (r, words) or not values.is_contiguous() \
            or not meta.is_contiguous():
        raise ValueError(f"values must be [d_out, {d * n // m}] and meta [d_out, {words}], contiguous")
    _check(lib().sgpt_pack_nm(_ptr(W), r, d, ldw, _ptr(mask), n, m, _ptr(values), _ptr(meta), _ptr(dev_info),
                              _stream(stream)), "sgpt_pack_nm")


def recon_error(W0: torch.Tensor, W: torch.Tensor, H: torch.Tensor, num_den: torch.Tensor,
                ws: torch.Tensor | None = None, stream=None):
    """num_den (float64 [2], device) = (tr(dW H dW^T), tr(W0 H W0^T)).
    ws: a workspace for these sizes (one is allocated when None)."""
    _dev(W0, torch.float32, "W0")
    _dev(W, torch.float32, "W")
    _dev(H, torch.float32, "H")
    _dev(num_den, torch.float64, "num_den")
    ldw = _rowmajor(W, "W")
    if _rowmajor(W0, "W0") != ldw or W0.shape != W.shape:
        raise ValueError("W0 and W must share shape and leading dimension")
    r, d = W.shape
    if ws is None:
        ws = workspace(r, d, device=W.device)
    _check(lib().sgpt_recon_error(_ptr(W0), _ptr(W), r, d, ldw, _ptr(H), _ptr(num_den), _ptr(ws), ws.numel(),
                                  _stream(stream)), "sgpt_recon_error")


def prune_layer(W: torch.Tensor, H: torch.Tensor, U: torch.Tensor, params: Params,
                mask: torch.Tensor, ws: torch.Tensor, dev_info: torch.Tensor,
                X: torch.Tensor | None = None, n_tok: int | None = None,
                values: torch.Tensor | None = None, meta: torch.Tensor | None = None,
                row_loss: torch.Tensor | None = None, stream=None):
    """One layer end to end (sgpt_prune_layer); X None means H holds X^T X."""
    _dev(W, torch.float32, "W")
    _dev(H, torch.float32, "H")
    _dev(U, torch.float32, "U")
    _dev(mask, torch.int32, "mask")
    ldw = _rowmajor(W, "W")
    r, d = W.shape
    if X is not None:
        _dev(X, torch.bfloat16, "X")
        if X.dim() != 2 or X.shape[1] != d or not X.is_contiguous():
            raise ValueError("X must be contiguous [n, d_in]")
        n_tok = X.shape[0]
    if n_tok is None:
        raise ValueError("n_tok is required when H is given")
    p = params.to_c()
    _check(lib().sgpt_prune_layer(_ptr(W), r, d, ldw, _ptr(X), n_tok, _ptr(H), _ptr(U), ctypes.byref(p),
                                  _ptr(mask), _ptr(values), _ptr(meta), _ptr(row_loss), _ptr(ws),
                                  ws.numel(), _ptr(dev_info), _stream(stream)), "sgpt_prune_layer")


# --------------------------------------------------------------- conveniences

@dataclass
class LayerBuffers:
    """Device buffers for pruning one layer shape (allocated once, reused)."""
    d_out: int
    d_in: int
    n_tok: int
    H: torch.Tensor
    U: torch.Tensor
    mask: torch.Tensor
    values: torch.Tensor
    meta: torch.Tensor
    row_loss: torch.Tensor
    ws: torch.Tensor
    info: torch.Tensor

    @classmethod
    def sharing(cls, other: "LayerBuffers", d_out: int, device="cuda", nm=(2, 4)) -> "LayerBuffers":
        """Buffers for another weight matrix that reads the same input: it
        shares H and U (factor once, sweep each matrix) and has its own
        outputs and workspace."""
        mine = cls.allocate(d_out, other.d_in, 0, device, with_hu=False, nm=nm)
        mine.H, mine.U, mine.n_tok = other.H, other.U, other.n_tok
        return mine

    @classmethod
    def allocate(cls, d_out: int, d_in: int, n_tok: int, device="cuda", with_hu: bool = True,
                 nm=(2, 4)) -> "LayerBuffers":
        """nm: the (N, M) the packed outputs are sized for."""
        f32 = dict(dtype=torch.float32, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        hu = (d_in, d_in) if with_hu else (0, 0)
        n, m = nm
        words = max(pack_nm_meta_words(d_in, n, m), 0)
        return cls(d_out, d_in, n_tok,
                   H=torch.empty(hu, **f32), U=torch.empty(hu, **f32),
                   mask=torch.empty((d_out, d_in // 32), **i32),
                   values=torch.empty((d_out, d_in * n // m), **f32),
                   meta=torch.empty((d_out, words), **i32),
                   row_loss=torch.empty(d_out, **f32),
                   ws=workspace(d_out, d_in, n_tok, device=device),
                   info=new_info(device))

    def packs(self, params: Params) -> bool:
        """Whether the packed outputs are sized for this pattern."""
        if not params.is_nm:
            return False
        n, m = params.nm
        return self.values.shape[1] == self.d_in * n // m and \
            self.meta.shape[1] == pack_nm_meta_words(self.d_in, n, m)

    def run(self, W: torch.Tensor, X: torch.Tensor | None, params: Params, stream=None):
        pack = self.packs(params)
        prune_layer(W, self.H, self.U, params, self.mask, self.ws, self.info, X=X,
                    n_tok=self.n_tok, values=self.values if pack else None,
                    meta=self.meta if pack else None, row_loss=self.row_loss, stream=stream)


class LayerGraphs:
    """The four phases of one layer prune captured as CUDA graphs.

    hessian (H = X^T X), factor, prune (row loss cleared + sweep) and,
    for 2:4, pack. Replaying them in order does exactly what
    LayerBuffers.run does, with the launch overhead of one graph per phase.
    Capture reads no data: buffers are bound by address, so W and X must
    stay where they were at capture time. Replay on the current stream with
    replay(), or phase by phase through .graphs.
    """

    PHASES = ("hessian", "factor", "prune", "pack")

    def __init__(self, bufs: LayerBuffers, W: torch.Tensor, X: torch.Tensor | None, params: Params,
                 phases=PHASES):
        self.bufs, self.W, self.X, self.params = bufs, W, X, params
        self.phases = tuple(ph for ph in phases if not (ph == "pack" and not bufs.packs(params)))
        # one eager pass first: per-process kernel attributes are set outside capture
        self._eager()
        torch.cuda.synchronize()
        self.graphs = {}
        self.kernels = {}        # libsgpt kernels captured in each graph
        for name in self.phases:
            g = torch.cuda.CUDAGraph()
            before = kernel_launches()
            with torch.cuda.graph(g):
                self._phase(name)
            self.kernels[name] = kernel_launches() - before
            self.graphs[name] = g

    def _phase(self, name: str):
        b, p = self.bufs, self.params
        if name == "hessian":
            info_clear(b.info)
            hessian_compute(b.H, self.X, b.ws, b.info)
        elif name == "factor":
            factor(b.H, b.n_tok, p.damp, b.U, b.ws, b.info)
        elif name == "prune":
            b.row_loss.zero_()
            prune(self.W, b.U, p, b.mask, b.ws, b.info, row_loss=b.row_loss)
        elif name == "pack":
            pack_nm(self.W, b.mask, *p.nm, b.values, b.meta, b.info)

    def _eager(self):
        for name in self.phases:
            self._phase(name)

    def replay(self):
        for g in self.graphs.values():
            g.replay()


class HostPruner:
    """End-to-end pruning from host memory through the public API.

    Owns the device buffers of one layer shape and pinned host outputs.
    run() copies W and X from (pinned) host memory to the device, prunes the
    layer from X with sgpt_prune_layer, copies the pruned weights, the mask
    and (for the N:M pattern it was sized for, 2:4 by default) the packed
    values and metadata back to the host, and checks the device status. All
    copies are enqueued on the current stream.
    """

    def __init__(self, d_out: int, d_in: int, n_tok: int, device="cuda", nm=(2, 4)):
        self.bufs = LayerBuffers.allocate(d_out, d_in, n_tok, device, nm=nm)
        self.W = torch.empty((d_out, d_in), dtype=torch.float32, device=device)
        self.X = torch.empty((n_tok, d_in), dtype=torch.bfloat16, device=device)
        pin = dict(pin_memory=True)
        self.W_out = torch.empty((d_out, d_in), dtype=torch.float32, **pin)
        self.mask_out = torch.empty((d_out, d_in // 32), dtype=torch.int32, **pin)
        self.values_out = torch.empty(self.bufs.values.shape, dtype=torch.float32, **pin)
        self.meta_out = torch.empty(self.bufs.meta.shape, dtype=torch.int32, **pin)

    def h2d_bytes(self) -> int:
        return self.W.numel() * 4 + self.X.numel() * 2

    def d2h_bytes(self, params: Params) -> int:
        b = self.W_out.numel() * 4 + self.mask_out.numel() * 4
        if self.bufs.packs(params):
            b += self.values_out.numel() * 4 + self.meta_out.numel() * 4
        return b

    def enqueue(self, W_host: torch.Tensor, X_host: torch.Tensor | None, params: Params, stream=None,
                X_device: torch.Tensor | None = None):
        """Copies and pruning, all asynchronous. X_host None reuses the X on
        the device from the previous call; X_device prunes from an X already
        on the device (for example another pruner's, when several layers read
        the same input)."""
        self.W.copy_(W_host, non_blocking=True)
        if X_device is None and X_host is not None:
            self.X.copy_(X_host, non_blocking=True)
        self.bufs.run(self.W, self.X if X_device is None else X_device, params, stream=stream)
        self.W_out.copy_(self.W, non_blocking=True)
        self.mask_out.copy_(self.bufs.mask, non_blocking=True)
        if self.bufs.packs(params):
            self.values_out.copy_(self.bufs.values, non_blocking=True)
            self.meta_out.copy_(self.bufs.meta, non_blocking=True)

    def run(self, W_host: torch.Tensor, X_host: torch.Tensor, params: Params, stream=None):
        self.enqueue(W_host, X_host, params, stream)
        raise_on_info(self.bufs.info, stream, "HostPruner.run")
        if self.bufs.packs(params):
            return self.W_out, self.mask_out, self.values_out, self.meta_out
        return self.W_out, self.mask_out, None, None
