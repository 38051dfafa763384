"""block_scaled_fp4_04_amd -- NVFP4 / MXFP4 block-scaled 4-bit quantization and
the quantized linear-layer GEMMs it feeds, on AMD Instinct MI355X (gfx950).

This module is a thin binding over the C ABI of ``libfp4blk.so`` (declared in
``include/fp4blk.h``): it checks tensors, hands device pointers and torch's
current stream to the library, and maps status codes to exceptions.  Every step
of the computation runs in the library's HIP kernels; there is no fallback.  If
the library is not built, importing the functions raises.

Formats ("NVFP4", newton.com.tw wiki, section "Technical principle"; edge-FP4
article, eefocus.com, section "FP4 as the next core standard"):

* NVFP4: E2M1 codes, two per byte (even column in the low nibble), one E4M3
  scale byte per 16 elements, one FP32 scale per tensor (or per row for
  dynamically quantized activations): 4.5 bits per value.
* MXFP4: E2M1 codes, one E8M0 byte per 32 elements: 4.25 bits per value.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libfp4blk.so")

FP4_F32, FP4_BF16 = 0, 1
PER_TENSOR, PER_ROW = 0, 1
MX_OCP_FLOOR, MX_CEIL = 0, 1

_EXPORTS = {
    # name: (restype, argtypes)
}


class Fp4Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


_lib = None


def _declare(L):
    p, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    f32 = ctypes.c_float
    sig = {
        "fp4_status_str": (ctypes.c_char_p, [i32]),
        "fp4blk_version": (i32, []),
        "fp4blk_check_device": (i32, []),
        "fp4blk_read_ceiling": (i32, [p, sz, i32, p, p]),
        "nvfp4_quantize_workspace": (sz, [i64, i64, i32]),
        "nvfp4_quantize": (i32, [p, i32, i64, i64, i64, p, p, p, i32, p, sz, p, p]),
        "nvfp4_dequantize": (i32, [p, p, p, i32, i64, i64, p, i32, i64, p]),
        "gemm_w4a16": (i32, [p, i64, i64, i64, p, p, p, i64, p, i32, i64, p]),
        "nvfp4_pack_decode": (i32, [p, p, i64, i64, p, p, p]),
        "gemm_w4a16_decode": (i32, [p, i64, i64, i64, p, p, p, i64, p, i32, i64, p]),
        "gemm_w4a4_workspace": (sz, [i64, i64, i32]),
        "gemm_w4a4_workspace_offsets": (None, [i64, i64, p, p, p]),
        "gemm_w4a4": (i32, [p, i64, i64, i64, i32, p, p, p, i64, p, i32, i64, p, sz, p]),
        "gemm_nvfp4_w4a4_prequant": (i32, [p, p, p, i32, i64, i64, p, p, p, i64, p, i32, i64, p]),
        "gemm_w4a4_seg": (i32, [p, i64, i64, i64, i32, p, p, p, i64, p, i32, i64, p, sz, p]),
        "gemm_w4a4_noalloc": (i32, [p, i64, i64, i64, i32, p, p, p, i64, p, i32, i64, p]),
        "gemm_nvfp4_w4a4_prequant_seg": (i32, [p, p, p, i32, i64, i64, p, p, p, i64, p, i32, i64, p]),
        "mxfp4_quantize": (i32, [p, i32, i64, i64, i64, p, p, i32, p, p]),
        "mxfp4_dequantize": (i32, [p, p, i64, i64, p, i32, i64, p]),
        "mxfp4_gemm_w4a4_workspace": (sz, [i64, i64]),
        "mxfp4_gemm_w4a4_a_segment_major": (i32, [i64, i64, i64]),
        "mxfp4_gemm_w4a4": (i32, [p, i64, i64, i64, i32, p, p, i64, p, i32, i64, p, sz, p]),
        "mxfp4_gemm_prequant": (i32, [p, p, i64, i64, p, p, i64, p, i32, i64, p]),
        "mxfp4_gemm_w4a4_seg_workspace": (sz, [i64, i64]),
        "mxfp4_gemm_w4a4_seg": (i32, [p, i64, i64, i64, i32, p, p, i64, p, i32, i64, p, sz, p]),
        "mxfp4_gemm_prequant_seg": (i32, [p, p, i64, i64, p, p, i64, p, i32, i64, p]),
        "mxfp4_gemm_w4a16": (i32, [p, i64, i64, i64, p, p, i64, p, i32, i64, p]),
        "mxfp4_pack_decode": (i32, [p, p, i64, i64, p, p, p]),
        "mxfp4_gemm_w4a16_decode": (i32, [p, i64, i64, i64, p, p, i64, p, i32, i64, p]),
        "mxfp8_quantize": (i32, [p, i32, i64, i64, i64, p, p, i32, p, p]),
        "mxfp4_gemm_w4a8_workspace": (sz, [i64, i64]),
        "mxfp4_gemm_w4a8": (i32, [p, i64, i64, i64, i32, p, p, i64, p, i32, i64, p, sz, p]),
        "mxfp4_gemm_w4a8_prequant": (i32, [p, p, i64, i64, p, p, i64, p, i32, i64, p]),
        "mxfp4_gemm_w4a8_seg": (i32, [p, i64, i64, i64, i32, p, p, i64, p, i32, i64, p, sz, p]),
        "mxfp4_gemm_w4a8_prequant_seg": (i32, [p, p, i64, i64, p, p, i64, p, i32, i64, p]),
        "nvfp4_grouped_gemm_w4a16": (i32, [p, i64, i64, i64, p, p, i64, i64, p, p, p, i64, p, i32, i64, p]),
        "mxfp4_grouped_gemm_w4a16": (i32, [p, i64, i64, i64, p, p, i64, i64, p, p, i64, p, i32, i64, p]),
        "nvfp4_grouped_gemm_w4a4_workspace": (sz, [i64, i64]),
        "nvfp4_grouped_gemm_w4a4": (i32, [p, i64, i64, i64, p, p, i64, i64, p, p, p, i64, p, i32, i64, p, sz,
                                          p]),
        "nvfp4_grouped_gemm_w4a4_prequant": (i32, [p, p, p, i64, i64, p, p, i64, i64, p, p, p, i64, p, i32,
                                                   i64, p]),
        "kv_cache_append": (i32, [p, p, p, i32, i64, i64, i64, i64, i64, p, i32, p, p]),
        "kv_cache_read": (i32, [p, p, i64, i64, i64, p, i64, p, p, i32, i64, i64, i64, i64, p]),
        "attn_decode_paged_workspace": (sz, [i64, i64, p, i64]),
        "attn_decode_paged": (i32, [p, i64, i64, i64, i64, p, p, i64, i64, p, f32, i64, p, i32, i64, i64, p, p, sz,
                                    p]),
        "attn_prefill": (i32, [p, i64, i64, i64, i64, p, p, i64, i64, i64, i64, i64, i64, i64, p, p, i64, f32, i32,
                               i64, p, i32, i64, i64, p, p, sz, p]),
        "attn_prefill_workspace": (sz, [i64, i64, i64, i64, i64, i64]),
        "qk_norm_rope": (i32, [p, p, i32, i64, i64, i64, i64, i64, i64, i64, i64, p, p, i64, i64, f32, p, p, i64, i32, p,
                               p, i32, i64, i64, i64, i64, p]),
        "qk_norm_rope_append": (i32, [p, p, p, p, i32, i64, i64, i64, i64, i64, i64, i64, i64, p, p, i64, i64, f32, p, p,
                                      i64, i32, p, i32, p, p, i32, i64, i64, p]),
        "kv_pages_extend_workspace": (sz, [i64, i64]),
        "kv_pages_extend": (i32, [p, p, i64, i64, i64, p, p, i64, p, p, p, p, p, p, p, sz, p]),
        "kv_pages_collect_workspace": (sz, [i64, i64, i64]),
        "kv_pages_collect": (i32, [p, p, i64, i64, i64, p, p, sz, p]),
        "kv_pages_reorder": (i32, [p, i64, i64, i64, i64, p, p, i64, p, i64, p, p]),
        "kv_cache_copy": (i32, [p, p, i64, p]),
        "beam_select_workspace": (sz, [i64, i64, i64, i64, i32]),
        "beam_select": (i32, [p, i32, i64, i64, i64, i64, p, p, i64, i64, p, p, p, p, sz, p]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return sig


def lib():
    """The loaded libfp4blk (ctypes handle).  Raises if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
                "(hipcc, gfx950); there is no fallback path")
        # torch first: the library links against torch's HIP runtime, which must
        # be the single HIP runtime in this process
        L = ctypes.CDLL(LIB_PATH)
        _EXPORTS.update(_declare(L))
        _lib = L
    return _lib


def exported_names():
    lib()
    return sorted(_EXPORTS)


def status_str(s: int) -> str:
    return lib().fp4_status_str(int(s)).decode()


def _check(s: int):
    if s != 0:
        raise Fp4Error(s, status_str(s))


_recording = None  # list of (function, arguments) while prepare() records
_recording_keep = []  # the tensors behind the recorded pointers


def _run(fn, *args):
    """Every library call goes through here: made at once, or recorded by prepare()."""
    if _recording is not None:
        _recording.append((fn, args))
        return
    _check(fn(*args))


class Prepared:
    """Library calls recorded by prepare(), replayed with the same pointers, sizes and
    stream.  It holds the tensors the calls use, so their memory stays valid."""

    def __init__(self, calls, keep):
        self._calls = calls
        self._keep = keep

    def __call__(self, *_ignored):
        for fn, args in self._calls:
            s = fn(*args)
            if s != 0:
                raise Fp4Error(s, status_str(s))


def prepare(thunk, *keep) -> Prepared:
    """Runs `thunk` (one or more calls of this module) with every argument check made
    and the library calls recorded instead of launched, and returns a callable that
    launches exactly those calls again: the same device pointers, sizes and stream,
    without the Python-side checks and allocation.  For tight loops (decode steps,
    benchmarks) where the checks would cost more than a short kernel.  The callable
    holds every tensor whose memory the calls use (and what the thunk returns), so
    that memory stays valid; the tensors' contents may change between calls."""
    global _recording, _recording_keep
    if _recording is not None:
        raise RuntimeError("prepare() calls do not nest")
    _recording, _recording_keep = [], []
    try:
        result = thunk()
        calls, held = _recording, _recording_keep
    finally:
        _recording, _recording_keep = None, []
    return Prepared(calls, (result, keep, held))


def _stream() -> int:
    """The current device's current stream (its handle, without a Stream object around it).  Calls come
    here with device tensors in hand, so the device runtime is up."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t):
    if t is not None and _recording is not None:
        _recording_keep.append(t)  # prepare(): the replayed calls keep using this memory
    return None if t is None else t.data_ptr()


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return FP4_F32
    if t.dtype == torch.bfloat16:
        return FP4_BF16
    raise TypeError(f"expected float32 or bfloat16, got {t.dtype}")


def _out_dt(dtype) -> int:
    if dtype == torch.float32:
        return FP4_F32
    if dtype == torch.bfloat16:
        return FP4_BF16
    raise TypeError(f"outputs are float32 or bfloat16, got {dtype}")


def _need_cuda(*ts):
    """Every tensor given is a device tensor, and all are on one device: its index."""
    first = None
    for t in ts:
        if t is None:
            continue
        d = t.get_device()  # -1 for a host tensor
        if d < 0:
            raise ValueError("libfp4blk takes device tensors")
        if first is None:
            first = d
        elif d != first:
            raise ValueError(f"tensors on several devices: {sorted({str(x.device) for x in ts if x is not None})}")
    return first


# Argument checks.  The C ABI receives bare pointers and sizes, so it cannot see a
# tensor that is smaller than the sizes passed with it; these checks run before
# anything is handed to the library (shapes and dtypes first, then devices).

def _shape(t: torch.Tensor, shape, what: str):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _u8(t: torch.Tensor, shape, what: str):
    """A packed byte array: uint8, the given shape, contiguous (the ABI takes no row stride for it)."""
    if t.dtype != torch.uint8:
        raise TypeError(f"{what} must be uint8, got {t.dtype}")
    _shape(t, shape, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _f32_vec(t: torch.Tensor, n: int, what: str):
    if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor of {n} element(s), got {t.dtype} "
                         f"{tuple(t.shape)}")


def _matrix(t: torch.Tensor, shape, dtypes, what: str):
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    _shape(t, shape, what)
    _ld(t)


def _out(out, M: int, N: int, dtype, like: torch.Tensor) -> torch.Tensor:
    """The GEMM / dequantize output: allocated when None, else checked (shape (M, N),
    float32 or bfloat16, unit stride along rows)."""
    if out is None:
        _out_dt(dtype)
        return torch.empty(M, N, dtype=dtype, device=like.device)
    _out_dt(out.dtype)
    _matrix(out, (M, N), (torch.float32, torch.bfloat16), "out")
    return out


def _workspace(ws, need: int, like: torch.Tensor) -> torch.Tensor:
    if ws is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=like.device)
    if ws.dtype != torch.uint8 or ws.dim() != 1 or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous 1-D uint8 tensor")
    if ws.numel() < need:
        raise ValueError(f"workspace holds {ws.numel()} bytes, {need} needed")
    return ws


def _k_match(K: int, cols: int):
    if K != cols:
        raise ValueError(f"A has K = {K} columns but the weight has {cols}")


def _mode(m) -> int:
    if m in ("tensor", PER_TENSOR):
        return PER_TENSOR
    if m in ("row", PER_ROW):
        return PER_ROW
    raise ValueError(f"scale mode must be 'tensor' or 'row', got {m!r}")


def _rule(r) -> int:
    if r in ("ocp", MX_OCP_FLOOR):
        return MX_OCP_FLOOR
    if r in ("ceil", MX_CEIL):
        return MX_CEIL
    raise ValueError(f"MX rule must be 'ocp' or 'ceil', got {r!r}")


def _ld(t: torch.Tensor) -> int:
    """The row stride (leading dimension) of a 2-D tensor with unit stride along its rows.
    A single row's stride is never followed, and torch may report any value for it
    (0 after unsqueeze or expand): it is given as the row length then."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError("expected a 2-D tensor with unit stride along its rows")
    if t.shape[0] <= 1:
        return max(t.stride(0), t.shape[1])
    return t.stride(0)


@dataclasses.dataclass
class PackedNVFP4:
    """NVFP4 tensor [rows, cols]: codes uint8 [rows, cols/2], scales uint8
    [rows, cols/16] (E4M3FN), tscale float32 [1] or [rows]."""
    codes: torch.Tensor
    scales: torch.Tensor
    tscale: torch.Tensor
    rows: int
    cols: int
    per_row: bool = False

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel() + 4 * self.tscale.numel()

    def check(self, what="NVFP4 tensor"):
        _u8(self.codes, (self.rows, self.cols // 2), f"{what} codes")
        _u8(self.scales, (self.rows, self.cols // 16), f"{what} scales")
        _f32_vec(self.tscale, self.rows if self.per_row else 1, f"{what} tensor scale")
        return self


@dataclasses.dataclass
class PackedMXFP4:
    """MXFP4 tensor [rows, cols]: codes uint8 [rows, cols/2], scales uint8 [rows, cols/32] (E8M0)."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def check(self, what="MXFP4 tensor"):
        _u8(self.codes, (self.rows, self.cols // 2), f"{what} codes")
        _u8(self.scales, (self.rows, self.cols // 32), f"{what} scales")
        return self


# --------------------------------------------------------------- NVFP4 -----

def nvfp4_quantize(x: torch.Tensor, mode="tensor", nonfinite: torch.Tensor | None = None,
                   out: PackedNVFP4 | None = None, workspace: torch.Tensor | None = None) -> PackedNVFP4:
    """Quantize a 2-D fp32/bf16 device tensor to NVFP4 (blocks along its rows)."""
    L = lib()
    _dt(x)
    rows, cols = x.shape
    m = _mode(mode)
    if out is None:
        out = PackedNVFP4(torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device),
                          torch.empty(rows, cols // 16, dtype=torch.uint8, device=x.device),
                          torch.empty(rows if m == PER_ROW else 1, dtype=torch.float32, device=x.device),
                          rows, cols, m == PER_ROW)
    if (out.rows, out.cols, out.per_row) != (rows, cols, m == PER_ROW):
        raise ValueError("out does not describe this tensor and scale mode")
    out.check("out")
    if nonfinite is not None and (nonfinite.dtype != torch.int32 or nonfinite.numel() < 1):
        raise ValueError("nonfinite must be an int32 tensor of at least one element")
    wsb = L.nvfp4_quantize_workspace(rows, cols, m)
    workspace = _workspace(workspace, wsb, x) if wsb else workspace
    _need_cuda(x, nonfinite, out.codes, out.scales, out.tscale, workspace)
    _run(L.nvfp4_quantize, _ptr(x), _dt(x), rows, cols, _ld(x), _ptr(out.codes), _ptr(out.scales),
                            _ptr(out.tscale), m, _ptr(workspace), wsb, _ptr(nonfinite), _stream())
    return out


def nvfp4_dequantize(p: PackedNVFP4, dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    L = lib()
    p.check("p")
    out = _out(out, p.rows, p.cols, dtype, p.codes)
    _need_cuda(p.codes, p.scales, p.tscale, out)
    _run(L.nvfp4_dequantize, _ptr(p.codes), _ptr(p.scales), _ptr(p.tscale),
                              PER_ROW if p.per_row else PER_TENSOR, p.rows, p.cols, _ptr(out),
                              _out_dt(out.dtype), _ld(out), _stream())
    return out


def _bf16_a(a: torch.Tensor, fn: str):
    if a.dtype != torch.bfloat16:
        raise TypeError(f"{fn} takes bfloat16 activations")
    if a.dim() != 2:
        raise ValueError(f"{fn} takes a 2-D activation tensor [M, K]")
    _ld(a)
    return a.shape


def _weight_nv(w: PackedNVFP4, K: int):
    if w.per_row:
        raise ValueError("NVFP4 weights carry one tensor scale (quantize them with mode='tensor')")
    w.check("w")
    _k_match(K, w.cols)


def gemm_w4a16(a: torch.Tensor, w: PackedNVFP4, dtype=torch.bfloat16,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """C = A . W^T with bf16 A [M, K] and NVFP4 W [N, K] (per-tensor scale)."""
    L = lib()
    M, K = _bf16_a(a, "gemm_w4a16")
    _weight_nv(w, K)
    out = _out(out, M, w.rows, dtype, a)
    _need_cuda(a, w.codes, w.scales, w.tscale, out)
    _run(L.gemm_w4a16, _ptr(a), M, K, _ld(a), _ptr(w.codes), _ptr(w.scales), _ptr(w.tscale), w.rows,
                        _ptr(out), _out_dt(out.dtype), _ld(out), _stream())
    return out


@dataclasses.dataclass
class DecodeNVFP4:
    """An NVFP4 weight [rows, cols] in the decode layout (see nvfp4_pack_decode):
    codes [cols/128, rows, 64], scales [cols/128, rows, 8], tscale [1]."""
    codes: torch.Tensor
    scales: torch.Tensor
    tscale: torch.Tensor
    rows: int
    cols: int

    def check(self, what="w"):
        _u8(self.codes, (self.cols // 128, self.rows, 64), f"{what} codes")
        _u8(self.scales, (self.cols // 128, self.rows, 8), f"{what} scales")
        _f32_vec(self.tscale, 1, f"{what} tensor scale")
        return self


def nvfp4_pack_decode(w: PackedNVFP4, out: DecodeNVFP4 | None = None) -> DecodeNVFP4:
    """Rewrite a per-tensor NVFP4 weight into the decode layout (segment-major)."""
    L = lib()
    if w.per_row:
        raise ValueError("the decode layout holds weights with a per-tensor scale")
    w.check("w")
    N, K = w.rows, w.cols
    if out is None:
        dev = w.codes.device
        out = DecodeNVFP4(torch.empty(K // 128, N, 64, dtype=torch.uint8, device=dev),
                          torch.empty(K // 128, N, 8, dtype=torch.uint8, device=dev),
                          w.tscale, N, K)
    if (out.rows, out.cols) != (N, K):
        raise ValueError("out does not describe this weight")
    out.check("out")
    _need_cuda(w.codes, w.scales, out.codes, out.scales)
    _run(L.nvfp4_pack_decode, _ptr(w.codes), _ptr(w.scales), N, K, _ptr(out.codes), _ptr(out.scales),
                               _stream())
    return out


def read_ceiling(buf: torch.Tensor, grid: int, sink: torch.Tensor) -> None:
    """Measurement aid: read every byte of `buf` (a contiguous device tensor whose
    size is a multiple of 16 bytes) once, on `grid` workgroups, computing nothing
    from it.  `sink` is a device int32/uint32 tensor of at least one element."""
    L = lib()
    if not buf.is_contiguous() or buf.numel() * buf.element_size() % 16:
        raise ValueError("buf must be contiguous, a multiple of 16 bytes")
    if sink.dtype not in (torch.int32, torch.uint32) or sink.numel() < 1:
        raise ValueError("sink must hold one 32-bit integer")
    _need_cuda(buf, sink)
    _run(L.fp4blk_read_ceiling, _ptr(buf), buf.numel() * buf.element_size(), int(grid), _ptr(sink), _stream())


def gemm_w4a16_decode(a: torch.Tensor, w: DecodeNVFP4, dtype=torch.bfloat16,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """C = A . W^T for bf16 A [M, K] and W in the decode layout: the decode GEMV for M <= 16,
    the prefill GEMM on the same layout for larger M."""
    L = lib()
    M, K = _bf16_a(a, "gemm_w4a16_decode")
    w.check("w")
    _k_match(K, w.cols)
    out = _out(out, M, w.rows, dtype, a)
    _need_cuda(a, w.codes, w.scales, w.tscale, out)
    _run(L.gemm_w4a16_decode, _ptr(a), M, K, _ld(a), _ptr(w.codes), _ptr(w.scales), _ptr(w.tscale), w.rows,
                               _ptr(out), _out_dt(out.dtype), _ld(out), _stream())
    return out


def gemm_w4a4_workspace(M: int, K: int, a_mode="row", device="cuda") -> torch.Tensor:
    n = lib().gemm_w4a4_workspace(M, K, _mode(a_mode))
    return torch.empty(n, dtype=torch.uint8, device=device)


def w4a4_packed_a(ws: torch.Tensor, M: int, K: int, a_mode="row") -> PackedNVFP4:
    """Views of A's NVFP4 form inside a gemm_w4a4 workspace."""
    co, so, to = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    lib().gemm_w4a4_workspace_offsets(M, K, ctypes.byref(co), ctypes.byref(so), ctypes.byref(to))
    per_row = _mode(a_mode) == PER_ROW
    codes = ws[co.value:co.value + M * K // 2].view(M, K // 2)
    scales = ws[so.value:so.value + M * K // 16].view(M, K // 16)
    nt = M if per_row else 1
    tscale = ws[to.value:to.value + 4 * nt].view(torch.float32)
    return PackedNVFP4(codes, scales, tscale, M, K, per_row)


def _w4a4(fn_name: str, a, w, a_mode, dtype, out, workspace, w_check):
    L = lib()
    M, K = _bf16_a(a, fn_name)
    w_check(w, K)
    m = _mode(a_mode)
    out = _out(out, M, w.rows, dtype, a)
    workspace = _workspace(workspace, L.gemm_w4a4_workspace(M, K, m), a)
    _need_cuda(a, w.codes, w.scales, w.tscale, out, workspace)
    _run(getattr(L, fn_name), _ptr(a), M, K, _ld(a), m, _ptr(w.codes), _ptr(w.scales), _ptr(w.tscale), w.rows,
                               _ptr(out), _out_dt(out.dtype), _ld(out), _ptr(workspace), workspace.numel(),
                               _stream())
    return out


def gemm_w4a4(a: torch.Tensor, w: PackedNVFP4, a_mode="row", dtype=torch.bfloat16,
              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """NVFP4 W4A4: quantize bf16 A on the device (per row by default), then C = A_q . W^T."""
    return _w4a4("gemm_w4a4", a, w, a_mode, dtype, out, workspace, _weight_nv)


def gemm_w4a4_noalloc(a: torch.Tensor, w: PackedNVFP4, a_mode="row", dtype=torch.bfloat16,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """gemm_w4a4 with A's packed form in the library's own device scratch (32 MiB per
    device): the library allocates nothing.  Pass `out` to allocate nothing here either.
    Calls that overlap on one device race for the scratch."""
    L = lib()
    M, K = _bf16_a(a, "gemm_w4a4_noalloc")
    _weight_nv(w, K)
    m = _mode(a_mode)
    out = _out(out, M, w.rows, dtype, a)
    _need_cuda(a, w.codes, w.scales, w.tscale, out)
    _run(L.gemm_w4a4_noalloc, _ptr(a), M, K, _ld(a), m, _ptr(w.codes), _ptr(w.scales), _ptr(w.tscale), w.rows,
         _ptr(out), _out_dt(out.dtype), _ld(out), _stream())
    return out


def _prequant_nv(fn_name: str, a: PackedNVFP4, w, dtype, out):
    L = lib()
    a.check("a")
    _k_match(a.cols, w.cols)
    out = _out(out, a.rows, w.rows, dtype, a.codes)
    _need_cuda(a.codes, a.scales, a.tscale, w.codes, w.scales, w.tscale, out)
    _run(getattr(L, fn_name), _ptr(a.codes), _ptr(a.scales), _ptr(a.tscale),
                               PER_ROW if a.per_row else PER_TENSOR, a.rows, a.cols,
                               _ptr(w.codes), _ptr(w.scales), _ptr(w.tscale), w.rows, _ptr(out),
                               _out_dt(out.dtype), _ld(out), _stream())
    return out


def gemm_nvfp4_prequant(a: PackedNVFP4, w: PackedNVFP4, dtype=torch.bfloat16,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    _weight_nv(w, a.cols)
    return _prequant_nv("gemm_nvfp4_w4a4_prequant", a, w, dtype, out)


def _weight_nv_dec(w: DecodeNVFP4, K: int):
    w.check("w")
    _k_match(K, w.cols)


def gemm_w4a4_seg(a: torch.Tensor, w: DecodeNVFP4, a_mode="row", dtype=torch.bfloat16,
                  out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """gemm_w4a4 with W in the decode layout: the same result."""
    return _w4a4("gemm_w4a4_seg", a, w, a_mode, dtype, out, workspace, _weight_nv_dec)


def gemm_nvfp4_prequant_seg(a: PackedNVFP4, w: DecodeNVFP4, dtype=torch.bfloat16,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """gemm_nvfp4_prequant with W in the decode layout."""
    _weight_nv_dec(w, a.cols)
    return _prequant_nv("gemm_nvfp4_w4a4_prequant_seg", a, w, dtype, out)


# --------------------------------------------------------------- MXFP4 -----

def mxfp4_quantize(x: torch.Tensor, rule="ocp", nonfinite: torch.Tensor | None = None,
                   out: PackedMXFP4 | None = None) -> PackedMXFP4:
    L = lib()
    _dt(x)
    rows, cols = x.shape
    if out is None:
        out = PackedMXFP4(torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device),
                          torch.empty(rows, cols // 32, dtype=torch.uint8, device=x.device), rows, cols)
    if (out.rows, out.cols) != (rows, cols):
        raise ValueError("out does not describe this tensor")
    out.check("out")
    if nonfinite is not None and (nonfinite.dtype != torch.int32 or nonfinite.numel() < 1):
        raise ValueError("nonfinite must be an int32 tensor of at least one element")
    _need_cuda(x, nonfinite, out.codes, out.scales)
    _run(L.mxfp4_quantize, _ptr(x), _dt(x), rows, cols, _ld(x), _ptr(out.codes), _ptr(out.scales),
                            _rule(rule), _ptr(nonfinite), _stream())
    return out


def mxfp4_dequantize(p: PackedMXFP4, dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    L = lib()
    p.check("p")
    out = _out(out, p.rows, p.cols, dtype, p.codes)
    _need_cuda(p.codes, p.scales, out)
    _run(L.mxfp4_dequantize, _ptr(p.codes), _ptr(p.scales), p.rows, p.cols, _ptr(out),
                              _out_dt(out.dtype), _ld(out), _stream())
    return out


def _weight_mx(w: PackedMXFP4, K: int):
    w.check("w")
    _k_match(K, w.cols)


def _mx_full(fn_name: str, ws_name: str, a, w, rule, dtype, out, workspace, w_check):
    """The MXFP4 / W4A8 entry points that quantize bf16 A into a workspace first."""
    L = lib()
    M, K = _bf16_a(a, fn_name)
    w_check(w, K)
    r = _rule(rule)
    out = _out(out, M, w.rows, dtype, a)
    workspace = _workspace(workspace, getattr(L, ws_name)(M, K), a)
    _need_cuda(a, w.codes, w.scales, out, workspace)
    _run(getattr(L, fn_name), _ptr(a), M, K, _ld(a), r, _ptr(w.codes), _ptr(w.scales), w.rows,
                               _ptr(out), _out_dt(out.dtype), _ld(out), _ptr(workspace), workspace.numel(),
                               _stream())
    return out


def _mx_prequant(fn_name: str, a, w, dtype, out):
    L = lib()
    a.check("a")
    _k_match(a.cols, w.cols)
    out = _out(out, a.rows, w.rows, dtype, a.codes)
    _need_cuda(a.codes, a.scales, w.codes, w.scales, out)
    _run(getattr(L, fn_name), _ptr(a.codes), _ptr(a.scales), a.rows, a.cols, _ptr(w.codes), _ptr(w.scales),
                               w.rows, _ptr(out), _out_dt(out.dtype), _ld(out), _stream())
    return out


def mxfp4_gemm_w4a4(a: torch.Tensor, w: PackedMXFP4, rule="ocp", dtype=torch.bfloat16,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    return _mx_full("mxfp4_gemm_w4a4", "mxfp4_gemm_w4a4_workspace", a, w, rule, dtype, out, workspace, _weight_mx)


def mxfp4_packed_a(ws: torch.Tensor, M: int, K: int, N: int):
    """Views of A's MXFP4 form inside the workspace of an mxfp4_gemm_w4a4 call
    with W of N rows: segment-major (DecodeMXFP4) or row-major (PackedMXFP4), as
    the library reports for those sizes."""
    if lib().mxfp4_gemm_w4a4_a_segment_major(M, N, K):
        return mxfp4_seg_packed_a(ws, M, K)
    cb = (M * (K // 2) + 255) // 256 * 256
    return PackedMXFP4(ws[:M * K // 2].view(M, K // 2), ws[cb:cb + M * K // 32].view(M, K // 32), M, K)


def mxfp4_gemm_prequant(a: PackedMXFP4, w: PackedMXFP4, dtype=torch.bfloat16,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    w.check("w")
    return _mx_prequant("mxfp4_gemm_prequant", a, w, dtype, out)


def mxfp4_gemm_w4a16(a: torch.Tensor, w: PackedMXFP4, dtype=torch.bfloat16,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """C = A . W^T with bf16 A [M, K] and MXFP4 W [N, K] (K % 128 == 0)."""
    L = lib()
    M, K = _bf16_a(a, "mxfp4_gemm_w4a16")
    _weight_mx(w, K)
    out = _out(out, M, w.rows, dtype, a)
    _need_cuda(a, w.codes, w.scales, out)
    _run(L.mxfp4_gemm_w4a16, _ptr(a), M, K, _ld(a), _ptr(w.codes), _ptr(w.scales), w.rows,
                              _ptr(out), _out_dt(out.dtype), _ld(out), _stream())
    return out


@dataclasses.dataclass
class DecodeMXFP4:
    """An MXFP4 weight [rows, cols] in the decode layout (see mxfp4_pack_decode):
    codes [cols/128, rows, 64], scales [cols/128, rows, 4]."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    def check(self, what="w"):
        _u8(self.codes, (self.cols // 128, self.rows, 64), f"{what} codes")
        _u8(self.scales, (self.cols // 128, self.rows, 4), f"{what} scales")
        return self


def _weight_mx_dec(w: DecodeMXFP4, K: int):
    w.check("w")
    _k_match(K, w.cols)


def mxfp4_pack_decode(w: PackedMXFP4, out: DecodeMXFP4 | None = None) -> DecodeMXFP4:
    """Rewrite an MXFP4 weight into the decode layout (segment-major)."""
    L = lib()
    w.check("w")
    N, K = w.rows, w.cols
    if out is None:
        dev = w.codes.device
        out = DecodeMXFP4(torch.empty(K // 128, N, 64, dtype=torch.uint8, device=dev),
                          torch.empty(K // 128, N, 4, dtype=torch.uint8, device=dev), N, K)
    if (out.rows, out.cols) != (N, K):
        raise ValueError("out does not describe this weight")
    out.check("out")
    _need_cuda(w.codes, w.scales, out.codes, out.scales)
    _run(L.mxfp4_pack_decode, _ptr(w.codes), _ptr(w.scales), N, K, _ptr(out.codes), _ptr(out.scales),
                               _stream())
    return out


def mxfp4_gemm_w4a4_seg_workspace(M: int, K: int, device="cuda") -> torch.Tensor:
    return torch.empty(lib().mxfp4_gemm_w4a4_seg_workspace(M, K), dtype=torch.uint8, device=device)


def mxfp4_seg_packed_a(ws: torch.Tensor, M: int, K: int) -> DecodeMXFP4:
    """Views of A's segment-major MXFP4 form inside an mxfp4_gemm_w4a4_seg workspace."""
    cb = (M * (K // 2) + 255) // 256 * 256
    return DecodeMXFP4(ws[:M * K // 2].view(K // 128, M, 64), ws[cb:cb + M * K // 32].view(K // 128, M, 4), M, K)


def mxfp4_gemm_w4a4_seg(a: torch.Tensor, w: DecodeMXFP4, rule="ocp", dtype=torch.bfloat16,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """MXFP4 W4A4 GEMM with W in the decode (segment-major) layout; A is quantized
    into the workspace in that layout.  The same result as mxfp4_gemm_w4a4."""
    return _mx_full("mxfp4_gemm_w4a4_seg", "mxfp4_gemm_w4a4_seg_workspace", a, w, rule, dtype, out, workspace,
                    _weight_mx_dec)


def mxfp4_gemm_prequant_seg(a: DecodeMXFP4, w: DecodeMXFP4, dtype=torch.bfloat16,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """The GEMM half of mxfp4_gemm_w4a4_seg: A and W both in the segment-major layout."""
    w.check("w")
    return _mx_prequant("mxfp4_gemm_prequant_seg", a, w, dtype, out)


def mxfp4_gemm_w4a16_decode(a: torch.Tensor, w: DecodeMXFP4, dtype=torch.bfloat16,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """C = A . W^T for bf16 A [M, K] and an MXFP4 W in the decode layout (GEMV for M <= 16,
    the prefill GEMM on the same layout for larger M)."""
    L = lib()
    M, K = _bf16_a(a, "mxfp4_gemm_w4a16_decode")
    _weight_mx_dec(w, K)
    out = _out(out, M, w.rows, dtype, a)
    _need_cuda(a, w.codes, w.scales, out)
    _run(L.mxfp4_gemm_w4a16_decode, _ptr(a), M, K, _ld(a), _ptr(w.codes), _ptr(w.scales), w.rows,
                                     _ptr(out), _out_dt(out.dtype), _ld(out), _stream())
    return out


@dataclasses.dataclass
class PackedMXFP8:
    """An MXFP8 tensor [rows, cols]: E4M3FN codes [rows, cols], E8M0 scales [rows, cols/32]."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    def check(self, what="MXFP8 tensor"):
        _u8(self.codes, (self.rows, self.cols), f"{what} codes")
        _u8(self.scales, (self.rows, self.cols // 32), f"{what} scales")
        return self


def mxfp8_quantize(x: torch.Tensor, rule="ocp", nonfinite: torch.Tensor | None = None,
                   out: PackedMXFP8 | None = None) -> PackedMXFP8:
    """MXFP8 (E4M3FN elements, E8M0 per 32) of an fp32 or bf16 [rows, cols] tensor."""
    L = lib()
    _dt(x)
    rows, cols = x.shape
    if out is None:
        out = PackedMXFP8(torch.empty(rows, cols, dtype=torch.uint8, device=x.device),
                          torch.empty(rows, cols // 32, dtype=torch.uint8, device=x.device), rows, cols)
    if (out.rows, out.cols) != (rows, cols):
        raise ValueError("out does not describe this tensor")
    out.check("out")
    if nonfinite is not None and (nonfinite.dtype != torch.int32 or nonfinite.numel() < 1):
        raise ValueError("nonfinite must be an int32 tensor of at least one element")
    _need_cuda(x, nonfinite, out.codes, out.scales)
    _run(L.mxfp8_quantize, _ptr(x), _dt(x), rows, cols, _ld(x), _ptr(out.codes), _ptr(out.scales),
                            _rule(rule), _ptr(nonfinite), _stream())
    return out


def mxfp4_gemm_w4a8_workspace(M: int, K: int, device="cuda") -> torch.Tensor:
    return torch.empty(lib().mxfp4_gemm_w4a8_workspace(M, K), dtype=torch.uint8, device=device)


def mxfp8_packed_a(ws: torch.Tensor, M: int, K: int) -> PackedMXFP8:
    """A's MXFP8 form inside a mxfp4_gemm_w4a8 workspace."""
    cb = (M * K + 255) // 256 * 256
    return PackedMXFP8(ws[:M * K].view(M, K), ws[cb:cb + M * K // 32].view(M, K // 32), M, K)


def mxfp4_gemm_w4a8(a: torch.Tensor, w: PackedMXFP4, rule="ocp", dtype=torch.bfloat16,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """W4A8: bf16 A [M, K] quantized to MXFP8 on the device, MXFP4 W [N, K]."""
    return _mx_full("mxfp4_gemm_w4a8", "mxfp4_gemm_w4a8_workspace", a, w, rule, dtype, out, workspace, _weight_mx)


def mxfp4_gemm_w4a8_prequant(a: PackedMXFP8, w: PackedMXFP4, dtype=torch.bfloat16,
                             out: torch.Tensor | None = None) -> torch.Tensor:
    """The GEMM half of mxfp4_gemm_w4a8 on an MXFP8 A."""
    w.check("w")
    return _mx_prequant("mxfp4_gemm_w4a8_prequant", a, w, dtype, out)


def mxfp4_gemm_w4a8_seg(a: torch.Tensor, w: DecodeMXFP4, rule="ocp", dtype=torch.bfloat16,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """W4A8 with the MXFP4 W in the decode (segment-major) layout; the same result as mxfp4_gemm_w4a8."""
    return _mx_full("mxfp4_gemm_w4a8_seg", "mxfp4_gemm_w4a8_workspace", a, w, rule, dtype, out, workspace,
                    _weight_mx_dec)


def mxfp4_gemm_w4a8_prequant_seg(a: PackedMXFP8, w: DecodeMXFP4, dtype=torch.bfloat16,
                                 out: torch.Tensor | None = None) -> torch.Tensor:
    """The GEMM half of mxfp4_gemm_w4a8_seg on an MXFP8 A."""
    w.check("w")
    return _mx_prequant("mxfp4_gemm_w4a8_prequant_seg", a, w, dtype, out)


# ------------------------------------------------------- grouped (MoE) -----

@dataclasses.dataclass
class ExpertsNVFP4:
    """E NVFP4 expert weights [E, N, K]: codes uint8 [E, N, K/2], scales uint8
    [E, N, K/16], one float32 tensor scale per expert [E]."""
    codes: torch.Tensor
    scales: torch.Tensor
    tscale: torch.Tensor
    experts: int
    rows: int
    cols: int

    def check(self, what="w"):
        _u8(self.codes, (self.experts, self.rows, self.cols // 2), f"{what} codes")
        _u8(self.scales, (self.experts, self.rows, self.cols // 16), f"{what} scales")
        _f32_vec(self.tscale, self.experts, f"{what} tensor scales")
        return self


@dataclasses.dataclass
class ExpertsMXFP4:
    """E MXFP4 expert weights [E, N, K]: codes uint8 [E, N, K/2], scales uint8 [E, N, K/32]."""
    codes: torch.Tensor
    scales: torch.Tensor
    experts: int
    rows: int
    cols: int

    def check(self, what="w"):
        _u8(self.codes, (self.experts, self.rows, self.cols // 2), f"{what} codes")
        _u8(self.scales, (self.experts, self.rows, self.cols // 32), f"{what} scales")
        return self


def nvfp4_quantize_experts(w: torch.Tensor) -> ExpertsNVFP4:
    """Each expert of w [E, N, K] quantized as its own NVFP4 tensor (its own tensor scale)."""
    E, N, K = w.shape
    dev = w.device
    out = ExpertsNVFP4(torch.empty(E, N, K // 2, dtype=torch.uint8, device=dev),
                       torch.empty(E, N, K // 16, dtype=torch.uint8, device=dev),
                       torch.empty(E, dtype=torch.float32, device=dev), E, N, K)
    ws = torch.empty(max(1, lib().nvfp4_quantize_workspace(N, K, PER_TENSOR)), dtype=torch.uint8, device=dev)
    for e in range(E):
        nvfp4_quantize(w[e], out=PackedNVFP4(out.codes[e], out.scales[e], out.tscale[e:e + 1], N, K),
                       workspace=ws)
    return out


def mxfp4_quantize_experts(w: torch.Tensor, rule="ocp") -> ExpertsMXFP4:
    """MXFP4 of expert weights w [E, N, K] (blocks along K; no tensor scale)."""
    E, N, K = w.shape
    p = mxfp4_quantize(w.reshape(E * N, K), rule=rule)
    return ExpertsMXFP4(p.codes.view(E, N, K // 2), p.scales.view(E, N, K // 32), E, N, K)


def _grouped_common(a_rows, K, w, group_offs, row_index):
    """Checks the grouping and the experts; returns (grouped rows, groups)."""
    if group_offs.dtype != torch.int32 or group_offs.dim() != 1 or not group_offs.is_contiguous():
        raise TypeError("group_offs must be a contiguous 1-D int32 device tensor [groups + 1]")
    if row_index is not None and (row_index.dtype != torch.int32 or row_index.dim() != 1
                                  or not row_index.is_contiguous()):
        raise TypeError("row_index must be a contiguous 1-D int32 device tensor [rows]")
    groups = group_offs.numel() - 1
    if groups != w.experts:
        raise ValueError(f"group_offs describes {groups} groups but the weight holds {w.experts} experts")
    w.check("w")
    _k_match(K, w.cols)
    rows = row_index.numel() if row_index is not None else a_rows
    return rows, groups


def nvfp4_grouped_gemm_w4a16(a: torch.Tensor, w: ExpertsNVFP4, group_offs: torch.Tensor,
                             row_index: torch.Tensor | None = None, dtype=torch.bfloat16,
                             out: torch.Tensor | None = None) -> torch.Tensor:
    """C[t] = A[row_index[t]] . W_e^T for the grouped rows t of group e (bf16 A, NVFP4 experts)."""
    L = lib()
    a_rows, K = _bf16_a(a, "nvfp4_grouped_gemm_w4a16")
    rows, groups = _grouped_common(a_rows, K, w, group_offs, row_index)
    out = _out(out, rows, w.rows, dtype, a)
    _need_cuda(a, w.codes, w.scales, w.tscale, group_offs, row_index, out)
    _run(L.nvfp4_grouped_gemm_w4a16, _ptr(a), a_rows, K, _ld(a), _ptr(row_index), _ptr(group_offs),
                                      groups, rows, _ptr(w.codes), _ptr(w.scales), _ptr(w.tscale), w.rows,
                                      _ptr(out), _out_dt(out.dtype), _ld(out), _stream())
    return out


def mxfp4_grouped_gemm_w4a16(a: torch.Tensor, w: ExpertsMXFP4, group_offs: torch.Tensor,
                             row_index: torch.Tensor | None = None, dtype=torch.bfloat16,
                             out: torch.Tensor | None = None) -> torch.Tensor:
    """As nvfp4_grouped_gemm_w4a16 with MXFP4 experts."""
    L = lib()
    a_rows, K = _bf16_a(a, "mxfp4_grouped_gemm_w4a16")
    rows, groups = _grouped_common(a_rows, K, w, group_offs, row_index)
    out = _out(out, rows, w.rows, dtype, a)
    _need_cuda(a, w.codes, w.scales, group_offs, row_index, out)
    _run(L.mxfp4_grouped_gemm_w4a16, _ptr(a), a_rows, K, _ld(a), _ptr(row_index), _ptr(group_offs),
                                      groups, rows, _ptr(w.codes), _ptr(w.scales), w.rows, _ptr(out),
                                      _out_dt(out.dtype), _ld(out), _stream())
    return out


def nvfp4_grouped_gemm_w4a4_workspace(a_rows: int, K: int, device="cuda") -> torch.Tensor:
    return torch.empty(lib().nvfp4_grouped_gemm_w4a4_workspace(a_rows, K), dtype=torch.uint8, device=device)


def nvfp4_grouped_gemm_w4a4(a: torch.Tensor, w: ExpertsNVFP4, group_offs: torch.Tensor,
                            row_index: torch.Tensor | None = None, dtype=torch.bfloat16,
                            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """NVFP4 W4A4 grouped GEMM: every A row quantized once per row, then gathered per group."""
    L = lib()
    a_rows, K = _bf16_a(a, "nvfp4_grouped_gemm_w4a4")
    rows, groups = _grouped_common(a_rows, K, w, group_offs, row_index)
    out = _out(out, rows, w.rows, dtype, a)
    workspace = _workspace(workspace, L.nvfp4_grouped_gemm_w4a4_workspace(a_rows, K), a)
    _need_cuda(a, w.codes, w.scales, w.tscale, group_offs, row_index, out, workspace)
    _run(L.nvfp4_grouped_gemm_w4a4, _ptr(a), a_rows, K, _ld(a), _ptr(row_index), _ptr(group_offs),
                                     groups, rows, _ptr(w.codes), _ptr(w.scales), _ptr(w.tscale), w.rows,
                                     _ptr(out), _out_dt(out.dtype), _ld(out), _ptr(workspace), workspace.numel(),
                                     _stream())
    return out


def nvfp4_grouped_gemm_w4a4_prequant(a: PackedNVFP4, w: ExpertsNVFP4, group_offs: torch.Tensor,
                                     row_index: torch.Tensor | None = None, dtype=torch.bfloat16,
                                     out: torch.Tensor | None = None) -> torch.Tensor:
    """The GEMM half of nvfp4_grouped_gemm_w4a4 on a per-row NVFP4 A."""
    L = lib()
    if not a.per_row:
        raise ValueError("the grouped W4A4 GEMM takes a per-row NVFP4 A")
    a.check("a")
    rows, groups = _grouped_common(a.rows, a.cols, w, group_offs, row_index)
    out = _out(out, rows, w.rows, dtype, a.codes)
    _need_cuda(a.codes, a.scales, a.tscale, w.codes, w.scales, w.tscale, group_offs, row_index, out)
    _run(L.nvfp4_grouped_gemm_w4a4_prequant, _ptr(a.codes), _ptr(a.scales), _ptr(a.tscale), a.rows, a.cols,
                                              _ptr(row_index), _ptr(group_offs), groups, rows, _ptr(w.codes),
                                              _ptr(w.scales), _ptr(w.tscale), w.rows, _ptr(out),
                                              _out_dt(out.dtype), _ld(out), _stream())
    return out


# -------------------------------------------- key-value cache, attention ---

KV_BF16, KV_MXFP8, KV_NVFP4, KV_MXFP4 = 0, 1, 2, 3
_KV_FORMATS = {"bf16": KV_BF16, "mxfp8": KV_MXFP8, "nvfp4": KV_NVFP4, "mxfp4": KV_MXFP4}


class _KvCacheArg(ctypes.Structure):
    """fp4_kv_cache"""
    _fields_ = [("format", ctypes.c_int)] + [(n, ctypes.c_int64) for n in ("pages", "kv_heads", "page_size", "head_dim")] + [
        (n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales", "k_tscale", "v_tscale")]


class KVCache:
    """A paged cache of keys and values in format "bf16", "mxfp8", "nvfp4" or "mxfp4".

    k_codes, v_codes  [pages, kv_heads, page_size, head_dim] bfloat16 ("bf16") or uint8
                      rows of head_dim ("mxfp8") or head_dim / 2 bytes (the 4-bit formats)
    k_scales, v_scales uint8 [pages, kv_heads, head_dim / block, page_size], block 16
                      ("nvfp4", E4M3) or 32 (E8M0); None for "bf16"
    k_tscale, v_tscale float32 [kv_heads], "nvfp4" only: the second-level scales

    A token's slot is page * page_size + offset.  The tensors are checked once, here; the
    cache holds them, and they must not be resized.  `alloc` makes the tensors."""

    def __init__(self, fmt: str, k_codes, v_codes, k_scales=None, v_scales=None, k_tscale=None, v_tscale=None):
        if fmt not in _KV_FORMATS:
            raise ValueError(f"cache format must be one of {sorted(_KV_FORMATS)}, got {fmt!r}")
        self.fmt = fmt
        code = _KV_FORMATS[fmt]
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, kv_heads, page_size, row]")
        pages, heads, page, row = k_codes.shape
        dim = row if code in (KV_BF16, KV_MXFP8) else 2 * row
        if dim not in (64, 128, 256):
            raise ValueError(f"head_dim must be 64, 128 or 256, got {dim}")
        if page < 16 or page > 256 or page & (page - 1):
            raise ValueError(f"page_size must be a power of two in [16, 256], got {page}")
        block = 16 if code == KV_NVFP4 else 32
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            if code != KV_BF16:
                _u8(t, (pages, heads, page, row), name)
            elif t.dtype != torch.bfloat16 or not t.is_contiguous():
                raise TypeError(f"{name} must be contiguous bfloat16")
            else:
                _shape(t, (pages, heads, page, row), name)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if code == KV_BF16:
                if t is not None:
                    raise ValueError(f"a bf16 cache has no {name}")
                continue
            if t is None:
                raise ValueError(f"a {fmt} cache needs {name}")
            _u8(t, (pages, heads, dim // block, page), name)
        for name, t in (("k_tscale", k_tscale), ("v_tscale", v_tscale)):
            if code != KV_NVFP4:
                if t is not None:
                    raise ValueError(f"a {fmt} cache has no {name}")
                continue
            if t is None:
                raise ValueError(f"an nvfp4 cache needs {name}")
            _f32_vec(t, heads, name)
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.k_tscale, self.v_tscale = k_tscale, v_tscale
        _need_cuda(k_codes, v_codes, k_scales, v_scales, k_tscale, v_tscale)
        self.device = k_codes.device
        self._arg = _KvCacheArg(code, pages, heads, page, dim, *(
            None if t is None else t.data_ptr() for t in (k_codes, v_codes, k_scales, v_scales, k_tscale, v_tscale)))
        self._ref = ctypes.byref(self._arg)

    @classmethod
    def alloc(cls, fmt: str, pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda",
              k_tscale=None, v_tscale=None) -> "KVCache":
        """A new cache, its contents unspecified ("nvfp4": with the given second-level scales)."""
        if fmt not in _KV_FORMATS:
            raise ValueError(f"cache format must be one of {sorted(_KV_FORMATS)}, got {fmt!r}")
        row = head_dim if fmt in ("bf16", "mxfp8") else head_dim // 2
        dtype = torch.bfloat16 if fmt == "bf16" else torch.uint8
        codes = [torch.empty(pages, kv_heads, page_size, row, dtype=dtype, device=device) for _ in range(2)]
        scales = [None, None]
        if fmt != "bf16":
            block = 16 if fmt == "nvfp4" else 32
            scales = [torch.empty(pages, kv_heads, head_dim // block, page_size, dtype=torch.uint8, device=device)
                      for _ in range(2)]
        return cls(fmt, *codes, *scales, k_tscale, v_tscale)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k_codes, self.v_codes, self.k_scales, self.v_scales,
                                                          self.k_tscale, self.v_tscale) if t is not None)


def _kv(cache: KVCache):
    """The fp4_kv_cache argument of a cache (kept with recorded calls)."""
    if _recording is not None:
        _recording_keep.append(cache)
    return cache._ref


def _heads(t: torch.Tensor, dtypes, what: str):
    """(tokens, heads, dim, token stride, head stride) of [tokens, heads, dim] with unit stride along dim.
    The stride of a dimension of size 1 is never followed, and torch may report any value for it: it
    is given as `dim` then, which passes every check of strides."""
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{what} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    n, h, d = t.shape
    sn, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{what} needs unit stride along head_dim")
    if h <= 1:
        sh = d
    if n <= 1:
        sn = d
    return n, h, d, sn, sh


_F32_BF16 = (torch.float32, torch.bfloat16)
_BF16 = (torch.bfloat16,)


def _i32_vec(t: torch.Tensor, n: int, what: str):
    if t.dtype != torch.int32:
        raise TypeError(f"{what} must be int32, got {t.dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n} element(s), got {tuple(t.shape)}")


def _out_heads(out, n: int, h: int, d: int, dtype, like, what="out"):
    """(output, token stride, head stride): allocated when None, else checked."""
    if out is None:
        _out_dt(dtype)
        return torch.empty(n, h, d, dtype=dtype, device=like.device), h * d, d
    on, oh, od, st, sh = _heads(out, _F32_BF16, what)
    if (on, oh, od) != (n, h, d):
        raise ValueError(f"{what} has shape {tuple(out.shape)}, expected {(n, h, d)}")
    return out, st, sh


def _lse(lse, n: int, h: int):
    if lse.dtype != torch.float32 or not lse.is_contiguous():
        raise TypeError("lse must be contiguous float32")
    _shape(lse, (n, h), "lse")


def _block_table(block_table, what="block_table"):
    """(sequences, pages of a row, row stride)"""
    if block_table.dtype != torch.int32:
        raise TypeError(f"{what} must be int32, got {block_table.dtype}")
    if block_table.dim() != 2:
        raise ValueError(f"{what} must be [sequences, pages], got {tuple(block_table.shape)}")
    seqs, width = block_table.shape
    stride, unit = block_table.stride()
    if width > 1 and unit != 1:
        raise ValueError(f"{what} needs unit stride along its last dimension")
    return seqs, width, stride if seqs > 1 else width


def kv_cache_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, rule="ocp",
                    nonfinite: torch.Tensor | None = None) -> KVCache:
    """Quantize new tokens' k and v [tokens, kv_heads, head_dim] (fp32 or bf16, any token and
    head strides) into the cache at `slots` (int64 [tokens]; page * page_size + offset,
    negative: the token is skipped).  Slots of one call must differ."""
    n, h, d, kt, kh = _heads(k, _F32_BF16, "k")
    nv, hv, dv, vt, vh = _heads(v, _F32_BF16, "v")
    if n != nv or h != hv or d != dv or k.dtype != v.dtype:
        raise ValueError("k and v must have the same shape and dtype")
    if h != cache.kv_heads or d != cache.head_dim:
        raise ValueError(f"k has {h} heads of {d}, the cache {cache.kv_heads} of {cache.head_dim}")
    if slots.dtype != torch.int64 or slots.dim() != 1 or slots.shape[0] != n or not slots.is_contiguous():
        raise ValueError(f"slots must be a contiguous int64 tensor of {n} element(s)")
    if nonfinite is not None and (nonfinite.dtype != torch.int32 or nonfinite.numel() < 1):
        raise ValueError("nonfinite must be an int32 tensor of at least one element")
    _need_cuda(cache.k_codes, k, v, slots, nonfinite)
    _run(lib().kv_cache_append, _kv(cache), _ptr(k), _ptr(v), _dt(k), n, kt, kh, vt, vh, _ptr(slots), _rule(rule),
         _ptr(nonfinite), _stream())
    return cache


def kv_cache_read(cache: KVCache, block_table: torch.Tensor, cu_seqlens: torch.Tensor, tokens: int,
                  dtype=torch.bfloat16, k_out: torch.Tensor | None = None,
                  v_out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Read cached sequences back as packed rows: k and v [tokens, kv_heads, head_dim], row t
    being position t - cu_seqlens[b] of the sequence b that holds it.  block_table int32
    [sequences, pages], cu_seqlens int32 [sequences + 1], tokens = cu_seqlens[-1] (known to the
    caller, so that nothing waits for the device)."""
    seqs, width, stride = _block_table(block_table)
    _i32_vec(cu_seqlens, seqs + 1, "cu_seqlens")
    tokens, h, d = int(tokens), cache.kv_heads, cache.head_dim
    k_out, kt, kh = _out_heads(k_out, tokens, h, d, dtype, cache.k_codes, "k_out")
    v_out, vt, vh = _out_heads(v_out, tokens, h, d, k_out.dtype, cache.k_codes, "v_out")
    if v_out.dtype != k_out.dtype:
        raise TypeError("k_out and v_out must have the same dtype")
    _need_cuda(cache.k_codes, block_table, cu_seqlens, k_out, v_out)
    _run(lib().kv_cache_read, _kv(cache), _ptr(block_table), seqs, width, stride, _ptr(cu_seqlens), tokens,
         _ptr(k_out), _ptr(v_out), _dt(k_out), kt, kh, vt, vh, _stream())
    return k_out, v_out


def _device() -> int:
    """The current device, which the workspace sizes depend on (-1 where no device is in use)."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -1


@functools.lru_cache(maxsize=4096)
def _decode_need(device, seqs, heads, kv_heads, page_size, head_dim, table_width) -> int:
    """Workspace bytes, by the current device and the sizes."""
    sizes = _KvCacheArg(KV_BF16, 1, kv_heads, page_size, head_dim)
    return lib().attn_decode_paged_workspace(seqs, heads, ctypes.byref(sizes), table_width)


@functools.lru_cache(maxsize=4096)
def _prefill_need(device, q_tokens, heads, k_tokens, kv_heads, head_dim, seqs) -> int:
    return lib().attn_prefill_workspace(q_tokens, heads, k_tokens, kv_heads, head_dim, seqs)


def attn_decode_paged_workspace(cache: KVCache, seqs: int, heads: int, table_width: int) -> torch.Tensor:
    """A workspace for attn_decode_paged calls of these sizes."""
    need = _decode_need(_device(), seqs, heads, cache.kv_heads, cache.page_size, cache.head_dim, table_width)
    return torch.empty(need, dtype=torch.uint8, device=cache.device)


def attn_prefill_workspace(q_tokens: int, heads: int, k_tokens: int, kv_heads: int, head_dim: int, seqs: int,
                           device="cuda") -> torch.Tensor:
    """A workspace for attn_prefill calls of these sizes."""
    need = _prefill_need(_device(), q_tokens, heads, k_tokens, kv_heads, head_dim, seqs)
    return torch.empty(need, dtype=torch.uint8, device=device)


def attn_decode_paged(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                      scale: float | None = None, window: int = 0, dtype=torch.bfloat16,
                      out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of one new token per sequence over the cache: q [sequences, heads, head_dim]
    bf16 (heads a multiple of the cache's), block_table int32 [sequences, pages], seq_lens int32
    [sequences] (the new token included; 0 gives zeros).  scale defaults to head_dim ** -0.5;
    window > 0 attends to the last `window` keys only.  lse: optional float32 [sequences, heads]
    that receives the logarithm of the softmax sum."""
    n, h, d, qt, qh = _heads(q, _BF16, "q")
    seqs, width, stride = _block_table(block_table)
    if seqs != n:
        raise ValueError(f"q has {n} sequences, block_table {seqs}")
    if d != cache.head_dim or h == 0 or h % cache.kv_heads:
        raise ValueError(f"q has {h} heads of {d}, the cache {cache.kv_heads} of {cache.head_dim}")
    _i32_vec(seq_lens, n, "seq_lens")
    out, ot, oh = _out_heads(out, n, h, d, dtype, q)
    if lse is not None:
        _lse(lse, n, h)
    need = _decode_need(_device(), n, h, cache.kv_heads, cache.page_size, d, width)
    if need or workspace is not None:
        workspace = _workspace(workspace, need, q)
    _need_cuda(cache.k_codes, q, block_table, seq_lens, out, lse, workspace)
    _run(lib().attn_decode_paged, _ptr(q), n, h, qt, qh, _kv(cache), _ptr(block_table), width, stride, _ptr(seq_lens),
         d ** -0.5 if scale is None else scale, window, _ptr(out), _dt(out), ot, oh, _ptr(lse), _ptr(workspace),
         need, _stream())
    return out


def attn_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                 cu_seqlens_k: torch.Tensor, causal: bool = True, window: int = 0, scale: float | None = None,
                 dtype=torch.bfloat16, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of packed prompts: q [q_tokens, heads, head_dim], k and v [k_tokens, kv_heads,
    head_dim] bf16, any token and head strides; cu_seqlens_q and cu_seqlens_k int32
    [sequences + 1].  A sequence's last query stands at its last key.  window > 0: a query sees
    the last `window` keys up to its position.  lse: optional float32 [q_tokens, heads]."""
    n, h, d, qt, qh = _heads(q, _BF16, "q")
    nk, hk, dk, kt, kh = _heads(k, _BF16, "k")
    nv, hv, dv, vt, vh = _heads(v, _BF16, "v")
    if nk != nv or hk != hv or dk != dv:
        raise ValueError("k and v must have the same shape")
    if dk != d or hk == 0 or h == 0 or h % hk:
        raise ValueError(f"q has {h} heads of {d}, k {hk} of {dk}")
    if cu_seqlens_q.dim() != 1 or cu_seqlens_q.shape[0] < 2:
        raise ValueError("cu_seqlens_q must hold sequences + 1 offsets")
    seqs = cu_seqlens_q.shape[0] - 1
    _i32_vec(cu_seqlens_q, seqs + 1, "cu_seqlens_q")
    _i32_vec(cu_seqlens_k, seqs + 1, "cu_seqlens_k")
    out, ot, oh = _out_heads(out, n, h, d, dtype, q)
    if lse is not None:
        _lse(lse, n, h)
    need = _prefill_need(_device(), n, h, nk, hk, d, seqs)
    if need or workspace is not None:
        workspace = _workspace(workspace, need, q)
    _need_cuda(q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse, workspace)
    _run(lib().attn_prefill, _ptr(q), n, h, qt, qh, _ptr(k), _ptr(v), nk, hk, d, kt, kh, vt, vh, _ptr(cu_seqlens_q),
         _ptr(cu_seqlens_k), seqs, d ** -0.5 if scale is None else scale, int(bool(causal)), window, _ptr(out),
         _dt(out), ot, oh, _ptr(lse), _ptr(workspace), need, _stream())
    return out


# ------------------------------------------------- around the attention ---

def _run_on(device: int, fn, *args):
    """_run on `device`, the tensors' own, where it is not the current one too (the library launches on the current
    device).  The stream, the device's current one, is the last argument."""
    if device == torch._C._cuda_getDevice():
        _run(fn, *args, torch._C._cuda_getCurrentRawStream(device))
        return
    if _recording is not None:
        raise ValueError("prepare() records calls on the current device only")
    with torch.cuda.device(device):
        _run(fn, *args, torch._C._cuda_getCurrentRawStream(device))


def rope_frequencies(rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The usual angles per position, base ** (-2 i / rot): float64 [rot / 2], made once."""
    return float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / max(rot, 1))


def _head_weight(w, heads: int, dim: int, what: str) -> int:
    """The head stride of a norm's weight: float32 [dim] (0) or [heads, dim]."""
    if w.dtype != torch.float32:
        raise TypeError(f"{what} must be float32, got {w.dtype}")
    if w.is_contiguous():
        if w.shape == (dim,):
            return 0
        if w.shape == (heads, dim):
            return dim
    raise ValueError(f"{what} must be a contiguous [{dim}] or [{heads}, {dim}], got {tuple(w.shape)}")


def _norm_args(n, q_heads, k_heads, d, positions, freqs, q_weight, k_weight, eps):
    """(q weight's and k weight's head strides, eps, rot): the checks that both forms of the norm share."""
    qs = ks = 0
    if eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("weights belong to a norm: give eps")
    else:
        if not 1e-30 <= eps <= 1e30:  # (a smaller one is 0 in fp32: no norm)
            raise ValueError(f"eps must be in [1e-30, 1e30] (None: no norm), got {eps}")
        if q_weight is None or (k_weight is None and k_heads > 0):
            raise ValueError("a norm needs its weights (ones for none)")
        qs = _head_weight(q_weight, q_heads, d, "q_weight")
        if k_heads > 0:
            ks = _head_weight(k_weight, k_heads, d, "k_weight")
    rot = 0
    if freqs is not None:
        if freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
            raise TypeError("freqs must be a contiguous float64 vector [rot / 2]")
        rot = 2 * freqs.shape[0]
        if rot % 16 or rot > d:
            raise ValueError(f"freqs turn {rot} values: a multiple of 16 up to head_dim {d} is needed")
    if rot:
        if positions is None:
            raise ValueError("a rotation needs positions")
        _i32_vec(positions, n, "positions")
    return qs, ks, 0.0 if eps is None else eps, rot


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor | None, freqs: torch.Tensor | None,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float | None = None,
                 interleaved: bool = False, dtype=torch.bfloat16, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None):
    """Every head's row of q [tokens, heads, head_dim] and k [tokens, kv_heads, head_dim] (fp32 or
    bf16, any token and head strides; k may be None) normed by its root mean square (eps None: not)
    with weights float32 [head_dim] or [heads, head_dim], and its first 2 * len(freqs) values
    rotated by positions (int32 [tokens]) times freqs (float64, `rope_frequencies`; None: not):
    value i with i + rot / 2, or neighbours when `interleaved`.  q_out and k_out may be q and k.
    Returns (q_out, k_out)."""
    n, h, d, qt, qh = _heads(q, _F32_BF16, "q")
    hk = kt = kh = kot = koh = 0
    if k is not None:
        nk, hk, dk, kt, kh = _heads(k, _F32_BF16, "k")
        if nk != n or dk != d or k.dtype != q.dtype:
            raise ValueError(f"q is {tuple(q.shape)} {q.dtype}, k {tuple(k.shape)} {k.dtype}")
        if hk == 0:
            raise ValueError("k has no heads (None for no k)")
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out belong to a k")
    qs, ks, eps, rot = _norm_args(n, h, hk, d, positions, freqs, q_weight, k_weight, eps)
    q_out, qot, qoh = _out_heads(q_out, n, h, d, dtype, q, "q_out")
    if k is not None:
        k_out, kot, koh = _out_heads(k_out, n, hk, d, q_out.dtype, k, "k_out")
        if k_out.dtype != q_out.dtype:
            raise TypeError("q_out and k_out must have the same dtype")
    device = _need_cuda(q, k, positions if rot else None, freqs, q_weight, k_weight, q_out, k_out)
    _run_on(device, lib().qk_norm_rope, _ptr(q), _ptr(k), _dt(q), n, h, hk, d, qt, qh, kt, kh, _ptr(q_weight),
            _ptr(k_weight), qs, ks, eps, _ptr(positions) if rot else None, _ptr(freqs), rot, int(bool(interleaved)),
            _ptr(q_out), _ptr(k_out), _dt(q_out), qot, qoh, kot, koh)
    return q_out, k_out


def qk_norm_rope_append(cache: KVCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        positions: torch.Tensor | None, slots: torch.Tensor, freqs: torch.Tensor | None,
                        q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                        eps: float | None = None, interleaved: bool = False, rule="ocp",
                        nonfinite: torch.Tensor | None = None, dtype=torch.bfloat16,
                        q_out: torch.Tensor | None = None) -> torch.Tensor:
    """qk_norm_rope with the keys, and v as it is, quantized into the cache at `slots` as
    kv_cache_append does (the keys from fp32, not from rows rounded before).  q_out may be q.  Returns q_out."""
    n, h, d, qt, qh = _heads(q, _F32_BF16, "q")
    nk, hk, dk, kt, kh = _heads(k, _F32_BF16, "k")
    nv, hv, dv, vt, vh = _heads(v, _F32_BF16, "v")
    if nk != n or nv != n or dk != d or dv != d or hv != hk or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must agree in tokens, head_dim and dtype, k and v in heads")
    if hk != cache.kv_heads or d != cache.head_dim:
        raise ValueError(f"k has {hk} heads of {d}, the cache {cache.kv_heads} of {cache.head_dim}")
    qs, ks, eps, rot = _norm_args(n, h, hk, d, positions, freqs, q_weight, k_weight, eps)
    if slots.dtype != torch.int64 or slots.dim() != 1 or slots.shape[0] != n or not slots.is_contiguous():
        raise ValueError(f"slots must be a contiguous int64 tensor of {n} element(s)")
    if nonfinite is not None and (nonfinite.dtype != torch.int32 or nonfinite.numel() < 1):
        raise ValueError("nonfinite must be an int32 tensor of at least one element")
    q_out, qot, qoh = _out_heads(q_out, n, h, d, dtype, q, "q_out")
    device = _need_cuda(cache.k_codes, q, k, v, positions if rot else None, freqs, slots, q_weight, k_weight, nonfinite,
                        q_out)
    _run_on(device, lib().qk_norm_rope_append, _kv(cache), _ptr(q), _ptr(k), _ptr(v), _dt(q), n, h, qt, qh, kt, kh, vt,
            vh, _ptr(q_weight), _ptr(k_weight), qs, ks, eps, _ptr(positions) if rot else None, _ptr(freqs), rot,
            int(bool(interleaved)), _ptr(slots), _rule(rule), _ptr(nonfinite), _ptr(q_out), _dt(q_out), qot, qoh)
    return q_out


class _KvPagesArg(ctypes.Structure):
    """fp4_kv_pages"""
    _fields_ = [("free_list", ctypes.c_void_p), ("state", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64)]


class KVPages:
    """The free pages of a cache (of all layers' caches, which share block tables).

    free   int32 [pages]: the first state[0] entries are free page ids, dealt from the end
    state  int32 [2]: the number of free pages, and of sequences refused so far

    `alloc` makes a pool in which every page is free."""

    def __init__(self, free: torch.Tensor, state: torch.Tensor, page_size: int):
        if page_size < 16 or page_size > 256 or page_size & (page_size - 1):
            raise ValueError(f"page_size must be a power of two in [16, 256], got {page_size}")
        if free.dim() != 1 or free.shape[0] == 0:
            raise ValueError("free must be [pages]")
        _i32_vec(free, free.shape[0], "free")
        _i32_vec(state, 2, "state")
        _need_cuda(free, state)
        self.free, self.state, self.pages, self.page_size, self.device = free, state, free.shape[0], page_size, free.device
        self._arg = _KvPagesArg(free.data_ptr(), state.data_ptr(), self.pages, page_size)
        self._ref = ctypes.byref(self._arg)

    @classmethod
    def alloc(cls, pages: int, page_size: int, device="cuda") -> "KVPages":
        return cls(torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device),
                   torch.tensor([pages, 0], dtype=torch.int32, device=device), page_size)


def _pool(pages: KVPages):
    if _recording is not None:
        _recording_keep.append(pages)
    return pages._ref


@dataclasses.dataclass
class KVPlan:
    """Where the new tokens of kv_pages_extend go: slots int64 and positions int32 [tokens], the
    offsets cu_q (new tokens) and cu_k (whole contexts) int32 [sequences + 1] (None: not asked
    for), and the lengths and the pool's state after."""
    slots: torch.Tensor
    positions: torch.Tensor
    cu_q: torch.Tensor | None
    cu_k: torch.Tensor | None
    seq_lens: torch.Tensor
    state: torch.Tensor


def kv_pages_extend_workspace(seqs: int, tokens: int, device="cuda") -> torch.Tensor:
    return torch.empty(lib().kv_pages_extend_workspace(seqs, tokens), dtype=torch.uint8, device=device)


def kv_pages_extend(pages: KVPages, block_table: torch.Tensor, seq_lens: torch.Tensor, new_lens: torch.Tensor,
                    tokens: int, in_place: bool = True, offsets: bool = True, out: KVPlan | None = None,
                    workspace: torch.Tensor | None = None) -> KVPlan:
    """Room for new_lens[b] more tokens (int32) behind the seq_lens[b] that sequence b holds: pages are
    dealt from the pool, block_table int32 [sequences, pages] is extended, and the slot and position of every
    new token are listed, packed one sequence behind the other.  tokens = sum(new_lens), or more (known to the
    caller, so that nothing waits for the device).  in_place: seq_lens and the pool's state become
    those after the call; else the plan holds new ones.  A sequence that cannot be served whole is
    left as it is: its slots are -1 and state[1] counts it.  Behind one for which the free pages did not
    suffice, all later ones that need a page are refused too (put decode rows before long prompts).  `out`: a plan
    of the same sizes to write into; lengths, state and offsets then go where its members say, whatever
    in_place and offsets are."""
    seqs, width, stride = _block_table(block_table)
    _i32_vec(seq_lens, seqs, "seq_lens")
    _i32_vec(new_lens, seqs, "new_lens")
    tokens = int(tokens)
    if tokens < 0:
        raise ValueError(f"tokens must not be negative, got {tokens}")
    need = lib().kv_pages_extend_workspace(seqs, tokens)
    if out is None:
        # one allocation: workspace, slots, positions, offsets, lengths, state
        room = need // 4 if workspace is None else 0
        parts = torch.empty(room + 3 * tokens + 3 * seqs + 4, dtype=torch.int32, device=block_table.device).split_with_sizes(
            (room, 2 * tokens, tokens, seqs + 1, seqs + 1, seqs, 2))
        out = KVPlan(parts[1].view(torch.int64), parts[2], *(parts[3:5] if offsets else (None, None)),
                     *((seq_lens, pages.state) if in_place else parts[5:]))
        space = parts[0]
    else:
        if out.slots.dtype != torch.int64 or out.slots.shape != (tokens,) or not out.slots.is_contiguous():
            raise ValueError(f"out.slots must be a contiguous int64 tensor of {tokens} element(s)")
        _i32_vec(out.positions, tokens, "out.positions")
        for x, name in ((out.cu_q, "out.cu_q"), (out.cu_k, "out.cu_k")):
            if x is not None:
                _i32_vec(x, seqs + 1, name)
        _i32_vec(out.seq_lens, seqs, "out.seq_lens")
        _i32_vec(out.state, 2, "out.state")
        space = workspace
    if workspace is not None or (need and space is None):
        space = _workspace(workspace, need, block_table)
    device = _need_cuda(pages.free, block_table, seq_lens, new_lens, out.slots, out.positions, out.cu_q, out.cu_k,
                        out.seq_lens, out.state, space)
    _run_on(device, lib().kv_pages_extend, _pool(pages), _ptr(block_table), seqs, width, stride, _ptr(seq_lens),
            _ptr(new_lens), tokens, _ptr(out.seq_lens), _ptr(out.state), _ptr(out.slots), _ptr(out.positions),
            _ptr(out.cu_q), _ptr(out.cu_k), _ptr(space), need)
    return out


def kv_pages_collect_workspace(pages: KVPages, seqs: int, table_width: int) -> torch.Tensor:
    return torch.empty(lib().kv_pages_collect_workspace(pages.pages, seqs, table_width), dtype=torch.uint8,
                       device=pages.device)


def kv_pages_collect(pages: KVPages, block_table: torch.Tensor, seq_lens: torch.Tensor,
                     workspace: torch.Tensor | None = None) -> KVPages:
    """The pool's free list anew: every page that no row of the block table holds within its
    length, in ascending order.  A sequence that ended gives its pages back by a length of 0.  Whatever holds pages of the
    pool has to stand in this one table (other batches, prompts kept for later use: rows of their own), or its pages
    are dealt a second time."""
    seqs, width, stride = _block_table(block_table)
    _i32_vec(seq_lens, seqs, "seq_lens")
    need = lib().kv_pages_collect_workspace(pages.pages, seqs, width)
    if need or workspace is not None:
        workspace = _workspace(workspace, need, block_table)
    device = _need_cuda(pages.free, block_table, seq_lens, workspace)
    _run_on(device, lib().kv_pages_collect, _pool(pages), _ptr(block_table), seqs, width, stride, _ptr(seq_lens),
            _ptr(workspace), need)
    return pages


def kv_pages_reorder(block_table: torch.Tensor, seq_lens: torch.Tensor, parents: torch.Tensor, page_size: int,
                     out: torch.Tensor | None = None, copies: torch.Tensor | None = None) -> torch.Tensor:
    """Block-table rows of beams after a selection: parents int32 [batch, beams] (beam_select's), row
    j of a group takes the row of beam parents[j], in place or into `out`.  The rows of a group have
    the same length (where the pool ran out under some of them, entries of -1 keep other sequences' pages
    out).  Returns int32 [batch * beams, 3]: what kv_cache_copy has to copy in every layer's cache,
    because a partly filled page belongs to one row only."""
    seqs, width, stride = _block_table(block_table)
    if parents.dtype != torch.int32:
        raise TypeError(f"parents must be int32, got {parents.dtype}")
    if parents.dim() != 2 or not parents.is_contiguous() or parents.numel() != seqs:
        raise ValueError(f"parents must be a contiguous [batch, beams] of {seqs} rows, got {tuple(parents.shape)}")
    batch, beams = parents.shape
    _i32_vec(seq_lens, seqs, "seq_lens")
    ostride = stride
    if out is None:
        out = block_table
    elif out is not block_table:
        oseqs, owidth, ostride = _block_table(out, "out")
        if (oseqs, owidth) != (seqs, width):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(seqs, width)}")
    if copies is None:
        copies = torch.empty(seqs, 3, dtype=torch.int32, device=block_table.device)
    else:
        _copies(copies)
        _shape(copies, (seqs, 3), "copies")
    device = _need_cuda(block_table, seq_lens, parents, out, copies)
    _run_on(device, lib().kv_pages_reorder, _ptr(block_table), batch, beams, width, stride, _ptr(seq_lens),
            _ptr(parents), page_size, _ptr(out), ostride, _ptr(copies))
    return copies


def _copies(t: torch.Tensor):
    if t.dtype != torch.int32:
        raise TypeError(f"copies must be int32, got {t.dtype}")
    if t.dim() != 2 or t.shape[1] != 3 or not t.is_contiguous():
        raise ValueError(f"copies must be a contiguous [n, 3], got {tuple(t.shape)}")


def kv_cache_copy(cache: KVCache, copies: torch.Tensor) -> KVCache:
    """For each row (source page, destination page, tokens) of copies int32 [n, 3] the first `tokens`
    tokens of the source page are copied into the destination page (all heads, keys and values); rows
    with a negative page are skipped."""
    _copies(copies)
    device = _need_cuda(cache.k_codes, copies)
    _run_on(device, lib().kv_cache_copy, _kv(cache), _ptr(copies), copies.shape[0])
    return cache


def beam_select_workspace(batch: int, beams: int, vocab: int, k: int, dtype=torch.bfloat16, device="cuda") -> torch.Tensor:
    return torch.empty(lib().beam_select_workspace(batch, beams, vocab, k, _out_dt(dtype)), dtype=torch.uint8, device=device)


def beam_select(logits: torch.Tensor, scores: torch.Tensor, k: int | None = None, done: torch.Tensor | None = None,
                end_token: int = 0, out=None, workspace: torch.Tensor | None = None):
    """The k (default: beams) best continuations of every group of beams: logits [batch * beams, vocab] fp32 or
    bf16, scores float32 [batch, beams] (the beams' log probabilities so far; -inf: the beam offers
    nothing), done bool or uint8 [batch, beams] (the beam has ended and offers end_token at its own
    score).  Returns (scores float32, parents int32, tokens int32), each [batch, k], best first, ties to the lowest
    beam, then (of one beam) the larger logit, then token; what nothing speaks for (-inf) comes last in the order of beam
    and token.  `out`: those three, to write
    into; its scores may be `scores`."""
    dt = _dt(logits)
    if logits.dim() != 2:
        raise ValueError(f"logits must be [batch * beams, vocab], got {tuple(logits.shape)}")
    if scores.dtype != torch.float32:
        raise TypeError(f"scores must be float32, got {scores.dtype}")
    if scores.dim() != 2 or not scores.is_contiguous():
        raise ValueError(f"scores must be a contiguous [batch, beams], got {tuple(scores.shape)}")
    batch, beams = scores.shape
    rows, vocab = logits.shape
    if rows != batch * beams:
        raise ValueError(f"logits have {rows} rows, scores {batch} x {beams}")
    ld = _ld(logits)
    if done is not None:
        if done.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"done must be bool or uint8, got {done.dtype}")
        _shape(done, (batch, beams), "done")
        if not done.is_contiguous():
            raise ValueError("done must be contiguous")
    k = beams if k is None else k
    need = lib().beam_select_workspace(batch, beams, vocab, k, dt)
    workspace = _workspace(workspace, need, logits)
    if out is None:
        if not 1 <= k <= 64:
            raise ValueError(f"k must be in [1, 64], got {k}")
        parts = torch.empty(3, batch, k, dtype=torch.int32, device=logits.device).unbind(0)
        out = (parts[0].view(torch.float32), parts[1], parts[2])
    else:
        for t, d, name in zip(out, (torch.float32, torch.int32, torch.int32), ("scores", "parents", "tokens"), strict=True):
            if t.dtype != d or not t.is_contiguous():
                raise TypeError(f"out's {name} must be contiguous {d}")
            _shape(t, (batch, k), f"out's {name}")
    device = _need_cuda(logits, scores, done, workspace, *out)
    _run_on(device, lib().beam_select, _ptr(logits), dt, batch, beams, vocab, ld, _ptr(scores), _ptr(done), end_token,
            k, _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), _ptr(workspace), need)
    return out
