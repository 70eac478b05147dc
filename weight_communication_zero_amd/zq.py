"""ctypes binding of libzq (include/zq.h, zq_train.h, zq_layers.h): argument marshalling only.

Every function takes torch tensors (device memory) or, where it reads no size
or element type off the argument, raw integer device pointers, converts them to
the C ABI's plain pointers and sizes, passes the current torch HIP stream unless
one is given, and raises ``ZQError`` on a non-OK status.  All arithmetic happens
in libzq's HIP kernels; there is no fallback path: if ``libzq.so`` is missing or
cannot be loaded, importing this module fails.
"""
from __future__ import annotations

import ctypes as C
import os
import re

import torch  # loaded first: libzq then binds to the HIP runtime torch uses

_HERE = os.path.dirname(os.path.abspath(__file__))
# ZQ_LIB selects another build of the same library (e.g. a tuning variant).
LIB_PATH = os.environ.get("ZQ_LIB") or os.path.join(_HERE, "libzq.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "zq.h")

ZQ_FP32, ZQ_BF16, ZQ_FP16 = 0, 1, 2
ZQ_I32, ZQ_I64 = 0, 1
ZQ_GRAD_WRITE, ZQ_GRAD_ADD, ZQ_GRAD_ADD_SR = 0, 1, 2

STATUS = {
    0: "ZQ_OK", 1: "ZQ_ERR_NULL", 2: "ZQ_ERR_SIZE", 3: "ZQ_ERR_BLOCK", 4: "ZQ_ERR_ALIGN",
    5: "ZQ_ERR_ALIAS", 6: "ZQ_ERR_PEERS", 7: "ZQ_ERR_DTYPE", 8: "ZQ_ERR_LAUNCH",
}
ZQ_OK, ZQ_ERR_NULL, ZQ_ERR_SIZE, ZQ_ERR_BLOCK, ZQ_ERR_ALIGN = 0, 1, 2, 3, 4
ZQ_ERR_ALIAS, ZQ_ERR_PEERS, ZQ_ERR_DTYPE, ZQ_ERR_LAUNCH = 5, 6, 7, 8


class SrSegment(C.Structure):
    """zq_sr_segment of include/zq.h."""
    _fields_ = [("dst", C.c_void_p), ("src", C.c_void_p), ("n", C.c_uint64),
                ("src_offset", C.c_uint64), ("src_len", C.c_uint64), ("seed", C.c_uint64),
                ("counter_base", C.c_uint64)]


class EfqSegment(C.Structure):
    """zq_efq_segment of include/zq.h."""
    _fields_ = [("g", C.c_void_p), ("ef", C.c_void_p), ("codes", C.c_void_p),
                ("scales", C.c_void_p), ("n", C.c_uint64)]


class DrSegment(C.Structure):
    """zq_dr_segment of include/zq.h."""
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("codes_stride", C.c_uint64),
                ("scales_stride", C.c_uint64), ("n", C.c_uint64), ("out", C.c_void_p),
                ("rq_codes", C.c_void_p), ("rq_scales", C.c_void_p), ("rq_ef", C.c_void_p)]


class GradSegment(C.Structure):
    """zq_grad_segment of include/zq_train.h."""
    _fields_ = [("g", C.c_void_p), ("out", C.c_void_p), ("n", C.c_uint64)]


class ZQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {lib.zq_status_str(status).decode()}")
        self.status = status


def _load() -> C.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; build it with `python -c 'import __graft_entry__ as g; g.build()'`"
            " (hipcc, gfx950)")
    L = C.CDLL(LIB_PATH)
    vp, sz, u32, u64, f32, i32 = C.c_void_p, C.c_size_t, C.c_uint32, C.c_uint64, C.c_float, C.c_int
    L.zq_quantize_ef_int4.argtypes = [vp, i32, vp, sz, u32, f32, f32, vp, vp, vp]
    L.zq_dequant_reduce.argtypes = [u32, vp, vp, sz, u32, f32, vp, vp, vp, vp, f32, f32, vp]
    L.zq_quant_int8.argtypes = [vp, i32, sz, u32, vp, vp, vp]
    L.zq_dequant_int8.argtypes = [vp, vp, sz, u32, vp, i32, vp]
    L.zq_sr_accumulate.argtypes = [vp, vp, sz, u64, u64, i32, vp]
    for f in ("zq_quantize_ef_int4", "zq_dequant_reduce", "zq_quant_int8", "zq_dequant_int8",
              "zq_sr_accumulate"):
        getattr(L, f).restype = i32
    L.zq_quantize_ef_int4_permuted.argtypes = [vp, i32, vp, sz, u32, f32, f32, vp, vp, u32, vp,
                                               vp]
    L.zq_quantize_ef_int4_permuted.restype = i32
    L.zq_quantize_ef_int4_batched.argtypes = [vp, u32, i32, u32, f32, f32, vp]
    L.zq_quantize_ef_int4_batched.restype = i32
    L.zq_dequant_reduce_batched.argtypes = [vp, u32, u32, u32, f32, f32, f32, vp]
    L.zq_dequant_reduce_batched.restype = i32
    L.zq_sr_accumulate_batched.argtypes = [vp, u32, i32, vp]
    L.zq_sr_accumulate_batched.restype = i32
    L.zq_zeropp_slots.argtypes = [u32, u32, vp]
    L.zq_zeropp_slots.restype = u32
    L.zq_int4_code_bytes.argtypes = [sz]
    L.zq_int4_code_bytes.restype = sz
    L.zq_num_blocks.argtypes = [sz, u32]
    L.zq_num_blocks.restype = sz
    L.zq_status_str.argtypes = [i32]
    L.zq_status_str.restype = C.c_char_p
    L.zq_embed_lookup.argtypes = [vp, i32, u64, u64, vp, i32, sz, f32, vp, i32, vp]
    L.zq_embed_lookup_int8.argtypes = [vp, vp, u32, u64, u64, vp, i32, sz, f32, vp, i32, vp]
    L.zq_embed_grad.argtypes = [vp, i32, vp, i32, sz, u64, u64, f32, vp, i32, i32, u64, u64, vp, sz,
                                vp]
    L.zq_grad_sumsq_batched.argtypes = [vp, u32, i32, i32, vp, vp, sz, vp]
    L.zq_grad_clip_batched.argtypes = [vp, u32, i32, vp, f32, f32, vp, vp]
    for f in ("zq_embed_lookup", "zq_embed_lookup_int8", "zq_embed_grad", "zq_grad_sumsq_batched",
              "zq_grad_clip_batched"):
        getattr(L, f).restype = i32
    L.zq_embed_grad_workspace.argtypes = [sz, u64, u64]
    L.zq_embed_grad_workspace.restype = sz
    L.zq_grad_sumsq_workspace.argtypes = [u32]
    L.zq_grad_sumsq_workspace.restype = sz
    L.zq_swiglu_int8.argtypes = [vp, vp, i32, sz, u32, vp, vp, vp, vp, vp, vp]
    L.zq_swiglu_grad_int8.argtypes = [vp, vp, vp, vp, u32, vp, i32, sz, vp, vp, vp, vp]
    L.zq_linear_grad_int8.argtypes = [vp, i32, vp, vp, u32, sz, u64, u64, vp, i32, i32, vp, sz, vp]
    L.zq_ce_loss.argtypes = [vp, i32, sz, u64, vp, u64, vp, i32, f32, vp, vp, u64, vp, sz, vp]
    L.zq_ce_loss_int8.argtypes = [vp, i32, sz, u64, vp, vp, u32, u64, vp, i32, f32, vp, vp, u64, vp,
                                  sz, vp]
    L.zq_ce_grad.argtypes = [vp, i32, sz, u64, vp, u64, vp, i32, f32, vp, vp, vp, vp, i32, i32, u64,
                             vp, sz, vp]
    L.zq_ce_grad_int8.argtypes = [vp, i32, sz, u64, vp, vp, u32, u64, vp, i32, f32, vp, vp, vp, vp,
                                  i32, i32, u64, vp, sz, vp]
    for f in ("zq_swiglu_int8", "zq_swiglu_grad_int8", "zq_linear_grad_int8", "zq_ce_loss",
              "zq_ce_loss_int8", "zq_ce_grad", "zq_ce_grad_int8"):
        getattr(L, f).restype = i32
    L.zq_linear_grad_workspace.argtypes = [sz, u64, u64]
    L.zq_ce_loss_workspace.argtypes = [sz, u64, u64, u64]
    L.zq_ce_grad_workspace.argtypes = [sz, u64, u64, u64]
    for f in ("zq_linear_grad_workspace", "zq_ce_loss_workspace", "zq_ce_grad_workspace"):
        getattr(L, f).restype = sz
    L.zq_abi_version.argtypes = []
    L.zq_abi_version.restype = u32
    return L


lib = _load()


def declared_symbols() -> list[str]:
    """Function names declared in include/zq.h."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:zq_status|size_t|const char \*|uint32_t)\s*\*?\s*(zq_\w+)\s*\(",
                                 text, re.M)))


def _p(x) -> int | None:
    """Device pointer of a tensor (or an int already a pointer; None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError("libzq needs contiguous tensors")
    return x.data_ptr()


# torch's own calls for the current stream's handle and the current device;
# the public ones build a Stream object (2.7 us a call) and check for
# initialisation first (0.1 us), which every call here would pay.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_DTYPES = {torch.float32: ZQ_FP32, torch.bfloat16: ZQ_BF16, torch.float16: ZQ_FP16}


def _dtype(t) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return d


def _need(name: str, t, numel: int, dtypes) -> None:
    """Host-side guard before any launch: a tensor argument must be a
    contiguous GPU tensor of an accepted dtype holding at least `numel`
    elements, so no kernel can index past a caller's buffer."""
    if t is None or isinstance(t, int):
        return
    if (t.is_cuda and t.dtype in dtypes and t.is_contiguous() and t.numel() >= numel
            and t.get_device() == _device()):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")


_F32 = (torch.float32,)
_BF16 = (torch.bfloat16,)
_FLOAT = (torch.float32, torch.bfloat16, torch.float16)
_U8 = (torch.uint8,)
_I8 = (torch.int8,)
_F64 = (torch.float64,)
_INDEX = (torch.int32, torch.int64)
_HALF = (torch.bfloat16, torch.float16)


def _check(fn: str, st: int) -> None:
    if st != ZQ_OK:
        raise ZQError(fn, st)


def int4_code_bytes(n: int) -> int:
    return lib.zq_int4_code_bytes(n)


def num_blocks(n: int, block: int) -> int:
    return lib.zq_num_blocks(n, block)


def zq_quantize_ef_int4(g, ef, block: int, beta_e: float, beta_r: float, codes, scales,
                        stream=None, n: int | None = None) -> None:
    """EF int4 quantize: g (fp32/bf16/fp16), ef (fp32 or None, updated in place)
    -> codes (uint8, ceil(n/2)), scales (fp32, ceil(n/block))."""
    n = g.numel() if n is None else n
    nb = (n + block - 1) // block if block > 0 else 0
    _need("g", g, n, _FLOAT)
    _need("ef", ef, n, _F32)
    _need("codes", codes, (n + 1) // 2, _U8)
    _need("scales", scales, nb, _F32)
    _check("zq_quantize_ef_int4",
           lib.zq_quantize_ef_int4(_p(g), _dtype(g), _p(ef), n, block, beta_e, beta_r, _p(codes),
                                   _p(scales), _stream(stream)))


def zeropp_slots(intra: int, inter: int) -> list[int]:
    """ZeRO++'s partition order for `inter` nodes of `intra` GPUs, from
    libzq's zq_zeropp_slots (slot_of_part[r] for rank r)."""
    m = intra * inter
    out = (C.c_uint32 * max(m, 1))()
    got = lib.zq_zeropp_slots(intra, inter, out)
    if got != m or m == 0:
        raise ValueError(f"zq_zeropp_slots rejected intra={intra}, inter={inter}")
    return list(out[:m])


def zq_quantize_ef_int4_permuted(g, ef, block: int, beta_e: float, beta_r: float, codes, scales,
                                 slot_of_part, stream=None, n: int | None = None) -> None:
    """EF int4 quantize whose codes / scales of partition p land in slot
    slot_of_part[p] (g and ef stay in natural order)."""
    n = g.numel() if n is None else n
    nb = (n + block - 1) // block if block > 0 else 0
    _need("g", g, n, _FLOAT)
    _need("ef", ef, n, _F32)
    _need("codes", codes, (n + 1) // 2, _U8)
    _need("scales", scales, nb, _F32)
    slots = (C.c_uint32 * max(len(slot_of_part), 1))(*slot_of_part)
    _check("zq_quantize_ef_int4_permuted",
           lib.zq_quantize_ef_int4_permuted(_p(g), _dtype(g), _p(ef), n, block, beta_e, beta_r,
                                            _p(codes), _p(scales), len(slot_of_part),
                                            C.cast(slots, C.c_void_p), _stream(stream)))


def zq_dequant_reduce(codes_list, scales_list, n_chunk: int, block: int, alpha: float, out=None,
                      rq_codes=None, rq_scales=None, rq_ef=None, rq_beta_e: float = 0.0,
                      rq_beta_r: float = 1.0, stream=None) -> None:
    """Dequantize P int4 chunks, reduce in fp32 (times alpha) into out, and /
    or requantize into rq_codes / rq_scales (with optional rq_ef)."""
    P = len(codes_list)
    if P != len(scales_list):
        raise ValueError("codes_list and scales_list differ in length")
    nb = (n_chunk + block - 1) // block if block > 0 else 0
    for c, sc in zip(codes_list, scales_list):
        _need("codes[p]", c, (n_chunk + 1) // 2, _U8)
        _need("scales[p]", sc, nb, _F32)
    _need("out", out, n_chunk, _F32)
    _need("rq_codes", rq_codes, (n_chunk + 1) // 2, _U8)
    _need("rq_scales", rq_scales, nb, _F32)
    _need("rq_ef", rq_ef, n_chunk, _F32)
    cp = (C.c_void_p * max(P, 1))(*[_p(c) for c in codes_list])
    sp = (C.c_void_p * max(P, 1))(*[_p(s) for s in scales_list])
    _check("zq_dequant_reduce",
           lib.zq_dequant_reduce(P, cp, sp, n_chunk, block, alpha, _p(out), _p(rq_codes),
                                 _p(rq_scales), _p(rq_ef), rq_beta_e, rq_beta_r, _stream(stream)))


def zq_quant_int8(w, block: int, codes, scales, stream=None, n: int | None = None) -> None:
    n = w.numel() if n is None else n
    _need("w", w, n, _FLOAT)
    _need("codes", codes, n, _I8)
    _need("scales", scales, (n + block - 1) // block if block > 0 else 0, _F32)
    _check("zq_quant_int8",
           lib.zq_quant_int8(_p(w), _dtype(w), n, block, _p(codes), _p(scales), _stream(stream)))


def zq_dequant_int8(codes, scales, block: int, out, stream=None, n: int | None = None) -> None:
    n = codes.numel() if n is None else n
    _need("codes", codes, n, _I8)
    _need("scales", scales, (n + block - 1) // block if block > 0 else 0, _F32)
    _need("out", out, n, _FLOAT)
    _check("zq_dequant_int8",
           lib.zq_dequant_int8(_p(codes), _p(scales), n, block, _p(out), _dtype(out),
                               _stream(stream)))


def zq_sr_accumulate(dst, src, seed: int, counter_base: int = 0, zero_src: bool = False,
                     stream=None, n: int | None = None) -> None:
    """bf16 dst += src with stochastic rounding (dst, src: torch.bfloat16)."""
    n = dst.numel() if n is None else n
    _need("dst", dst, n, _BF16)
    _need("src", src, n, _BF16)
    _check("zq_sr_accumulate",
           lib.zq_sr_accumulate(_p(dst), _p(src), n, seed, counter_base, 1 if zero_src else 0,
                                _stream(stream)))


class _SegmentTable:
    """What the marshalled tables share: the device of their tensors, which
    _need has found to be the current one (None: raw pointers only)."""
    device = None

    def note_device(self) -> None:
        self.device = next((t.get_device() for seg in self.segments for t in seg
                            if hasattr(t, "get_device")), None)

    def check_device(self) -> None:
        if self.device is not None and self.device != _device():
            raise ValueError(f"the segment table's tensors are on cuda:{self.device}, the current "
                             f"device is cuda:{_device()}")


class SrSegmentTable(_SegmentTable):
    """A marshalled segment table for zq_sr_accumulate_batched: build it once
    for a fixed set of buffers and pass it to every call (the tensors are
    kept alive by the table)."""

    def __init__(self, segments):
        self.segments = list(segments)
        self.arr = (SrSegment * max(len(self.segments), 1))()
        for i, (dst, src, n, off, seed, cb) in enumerate(self.segments):
            _need("dst", dst, n, _BF16)
            _need("src", src, off + n, _BF16)
            src_len = src.numel() if not isinstance(src, int) else off + n
            self.arr[i] = SrSegment(_p(dst), _p(src), n, off, src_len, seed, cb)
        self.ptr = C.cast(self.arr, C.c_void_p)
        self.note_device()


def zq_sr_accumulate_batched(segments, zero_src: bool = False, stream=None) -> None:
    """Batched SR accumulation.  `segments`: an SrSegmentTable, or an iterable
    of (dst, src, n, src_offset, seed, counter_base) with dst / src bf16
    tensors; src is the whole per-tensor buffer (src_len = src.numel()), of
    which elements [src_offset, src_offset + n) are added into dst[0:n]; with
    zero_src every element of every src buffer is cleared in the same pass."""
    table = segments if isinstance(segments, SrSegmentTable) else SrSegmentTable(segments)
    table.check_device()
    _check("zq_sr_accumulate_batched",
           lib.zq_sr_accumulate_batched(table.ptr, len(table.segments), 1 if zero_src else 0,
                                        _stream(stream)))


class EfqSegmentTable(_SegmentTable):
    """A marshalled segment table for zq_quantize_ef_int4_batched: tuples
    (g, ef or None, codes, scales) of per-tensor buffers (n = g.numel())."""

    def __init__(self, segments, block: int):
        self.segments = list(segments)
        self.arr = (EfqSegment * max(len(self.segments), 1))()
        self.dtype = None
        for i, (g, ef, codes, scales) in enumerate(self.segments):
            n = g.numel()
            _need("g", g, n, _FLOAT)
            _need("ef", ef, n, _F32)
            _need("codes", codes, (n + 1) // 2, _U8)
            _need("scales", scales, (n + block - 1) // block, _F32)
            dt = _dtype(g)
            if self.dtype is not None and dt != self.dtype:
                raise TypeError("all segments of a batch share one gradient dtype")
            self.dtype = dt
            self.arr[i] = EfqSegment(_p(g), _p(ef), _p(codes), _p(scales), n)
        self.block = block
        self.ptr = C.cast(self.arr, C.c_void_p)
        self.note_device()


def zq_quantize_ef_int4_batched(segments, block: int, beta_e: float, beta_r: float,
                                stream=None) -> None:
    """Per-tensor EF int4 quantize of many tensors in one call: `segments` is
    an EfqSegmentTable or an iterable of (g, ef or None, codes, scales)."""
    table = segments if isinstance(segments, EfqSegmentTable) else EfqSegmentTable(segments, block)
    table.check_device()
    if table.block != block:
        raise ValueError(f"the segment table was checked for block {table.block}, not {block}")
    _check("zq_quantize_ef_int4_batched",
           lib.zq_quantize_ef_int4_batched(table.ptr, len(table.segments),
                                           ZQ_FP32 if table.dtype is None else table.dtype, block,
                                           beta_e, beta_r, _stream(stream)))


class DrSegmentTable(_SegmentTable):
    """A marshalled segment table for zq_dequant_reduce_batched.  Each
    segment is (codes, scales, n, codes_stride, scales_stride, out, rq_codes,
    rq_scales, rq_ef): codes a uint8 tensor holding the P peer chunks (peer q
    at byte q * codes_stride), scales a float32 tensor (peer q at element
    q * scales_stride); outputs as in zq_dequant_reduce (None for absent)."""

    def __init__(self, segments, P: int, block: int):
        self.segments = list(segments)
        self.arr = (DrSegment * max(len(self.segments), 1))()
        nbk = lambda n: (n + block - 1) // block
        for i, (codes, scales, n, cst, sst, out, rqc, rqs, rqe) in enumerate(self.segments):
            _need("codes", codes, (P - 1) * cst + (n + 1) // 2 if n else 0, _U8)
            _need("scales", scales, (P - 1) * sst + nbk(n) if n else 0, _F32)
            _need("out", out, n, _F32)
            _need("rq_codes", rqc, (n + 1) // 2, _U8)
            _need("rq_scales", rqs, nbk(n), _F32)
            _need("rq_ef", rqe, n, _F32)
            self.arr[i] = DrSegment(_p(codes), _p(scales), cst, sst, n, _p(out), _p(rqc), _p(rqs),
                                    _p(rqe))
        self.P, self.block = P, block
        self.ptr = C.cast(self.arr, C.c_void_p)
        self.note_device()


def zq_dequant_reduce_batched(segments, P: int, block: int, alpha: float, rq_beta_e: float = 0.0,
                              rq_beta_r: float = 1.0, stream=None) -> None:
    """Per-tensor dequantize-reduce(-requant) of many tensors in one call:
    `segments` is a DrSegmentTable or an iterable of its tuples."""
    table = segments if isinstance(segments, DrSegmentTable) else DrSegmentTable(segments, P, block)
    table.check_device()
    if (table.P, table.block) != (P, block):
        raise ValueError(f"the segment table was checked for P={table.P}, block={table.block}, "
                         f"not P={P}, block={block}")
    _check("zq_dequant_reduce_batched",
           lib.zq_dequant_reduce_batched(table.ptr, len(table.segments), P, block, alpha, rq_beta_e,
                                         rq_beta_r, _stream(stream)))


def _index(t) -> int:
    return ZQ_I64 if t.dtype == torch.int64 else ZQ_I32


def _rows_dim(name: str, t) -> tuple[int, int]:
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions [rows, dim], not {tuple(shape)}")
    return shape


def zq_embed_lookup(table, ids, scale: float, out, stream=None) -> None:
    """out[t] = scale * table[ids[t]] (+0 where ids[t] is outside the table):
    table [rows, dim] fp32/bf16/fp16, ids int32/int64 of any shape, out
    fp32/bf16/fp16 with ids.numel() * dim elements."""
    rows, dim = _rows_dim("table", table)
    n = ids.numel()
    _need("table", table, rows * dim, _FLOAT)
    _need("ids", ids, n, _INDEX)
    _need("out", out, n * dim, _FLOAT)
    _check("zq_embed_lookup",
           lib.zq_embed_lookup(table.data_ptr(), _dtype(table), rows, dim, ids.data_ptr(),
                               _index(ids), n, scale, out.data_ptr(), _dtype(out),
                               _stream(stream)))


def zq_embed_lookup_int8(codes, scales, block: int, ids, scale: float, out, stream=None) -> None:
    """zq_embed_lookup from a table in qwZ's form: codes [rows, dim] int8 and
    scales fp32, as zq_quant_int8 writes them for the flat table."""
    rows, dim = _rows_dim("codes", codes)
    n = ids.numel()
    _need("codes", codes, rows * dim, _I8)
    _need("scales", scales, (rows * dim + block - 1) // block if block > 0 else 0, _F32)
    _need("ids", ids, n, _INDEX)
    _need("out", out, n * dim, _FLOAT)
    _check("zq_embed_lookup_int8",
           lib.zq_embed_lookup_int8(codes.data_ptr(), scales.data_ptr(), block, rows, dim,
                                    ids.data_ptr(), _index(ids), n, scale, out.data_ptr(),
                                    _dtype(out), _stream(stream)))


def embed_grad_workspace(n_tok: int, rows: int, dim: int) -> int:
    """Bytes of workspace zq_embed_grad needs."""
    return lib.zq_embed_grad_workspace(n_tok, rows, dim)


def zq_embed_grad(dout, ids, scale: float, grad, mode: int, workspace, seed: int = 0,
                  counter_base: int = 0, stream=None) -> None:
    """The lookup's gradient by sorted tokens: grad [rows, dim] (fp32/bf16/fp16)
    is written (ZQ_GRAD_WRITE), or added to with rounding to nearest
    (ZQ_GRAD_ADD) or stochastic rounding (ZQ_GRAD_ADD_SR, bf16).  dout has
    ids.numel() * dim elements; workspace is a uint8 tensor of at least
    embed_grad_workspace(ids.numel(), rows, dim) bytes, one for each call that
    may run at the same time."""
    rows, dim = _rows_dim("grad", grad)
    n = ids.numel()
    _need("dout", dout, n * dim, _FLOAT)
    _need("ids", ids, n, _INDEX)
    _need("grad", grad, rows * dim, _FLOAT)
    _need("workspace", workspace, embed_grad_workspace(n, rows, dim), _U8)
    _check("zq_embed_grad",
           lib.zq_embed_grad(_p(dout), _dtype(dout), _p(ids), _index(ids), n, rows, dim, scale,
                             _p(grad), _dtype(grad), mode, seed, counter_base, _p(workspace),
                             workspace.numel() if workspace is not None else 0, _stream(stream)))


class GradSegmentTable(_SegmentTable):
    """A marshalled segment table for zq_grad_sumsq_batched and
    zq_grad_clip_batched: pairs (g, out) of gradient tensors of one dtype,
    where out is g itself, another buffer of g's size, or None (only the sum of
    squares is wanted).  Build it once for a fixed set of buffers."""

    def __init__(self, segments):
        self.segments = list(segments)
        self.arr = (GradSegment * max(len(self.segments), 1))()
        self.dtype = None
        for i, (g, out) in enumerate(self.segments):
            n = g.numel()
            _need("g", g, n, _FLOAT)
            if self.dtype is not None and _dtype(g) != self.dtype:
                raise TypeError("all segments of a batch share one gradient dtype")
            self.dtype = _dtype(g)
            _need("out", out, n, (g.dtype,))
            self.arr[i] = GradSegment(_p(g), _p(out), n)
        self.workspace = grad_sumsq_workspace(len(self.segments))
        self.ptr = C.cast(self.arr, C.c_void_p)
        self.note_device()


def grad_sumsq_workspace(n_seg: int) -> int:
    """Bytes of workspace zq_grad_sumsq_batched needs."""
    return lib.zq_grad_sumsq_workspace(n_seg)


def zq_grad_sumsq_batched(segments, sumsq, workspace, accumulate: bool = False,
                          stream=None) -> None:
    """sumsq (one float64) = [sumsq +] the sum of squares of every segment's g.
    `segments`: a GradSegmentTable or an iterable of (g, out or None);
    workspace: a uint8 tensor of grad_sumsq_workspace(n_seg) bytes."""
    table = segments if isinstance(segments, GradSegmentTable) else GradSegmentTable(segments)
    table.check_device()
    _need("sumsq", sumsq, 1, _F64)
    _need("workspace", workspace, table.workspace, _U8)
    _check("zq_grad_sumsq_batched",
           lib.zq_grad_sumsq_batched(table.ptr, len(table.segments),
                                     ZQ_FP32 if table.dtype is None else table.dtype,
                                     1 if accumulate else 0, _p(sumsq), _p(workspace),
                                     workspace.numel() if workspace is not None else 0,
                                     _stream(stream)))


def zq_grad_clip_batched(segments, sumsq, max_norm: float, eps: float = 1e-6, norm=None,
                         stream=None) -> None:
    """out = g * min(1, max_norm / (sqrt(sumsq) + eps)) for every segment;
    norm (one float32, optional) gets sqrt(sumsq)."""
    table = segments if isinstance(segments, GradSegmentTable) else GradSegmentTable(segments)
    table.check_device()
    _need("sumsq", sumsq, 1, _F64)
    _need("norm", norm, 1, _F32)
    _check("zq_grad_clip_batched",
           lib.zq_grad_clip_batched(table.ptr, len(table.segments),
                                    ZQ_FP32 if table.dtype is None else table.dtype, _p(sumsq),
                                    max_norm, eps, _p(norm), _stream(stream)))


def _blocks(n: int, block: int) -> int:
    return (n + block - 1) // block if block > 0 else 0


def _fits(t, dtype, n: int, device: int) -> bool:
    """_need's checks of one dtype in four attribute reads."""
    return (t.__class__ is not int and t.get_device() == device and t.dtype is dtype
            and t.numel() >= n and t.is_contiguous())


def _current(t) -> int:
    """The device of t where that is the current one, else a number of no device."""
    dev = t.get_device()
    return dev if dev >= 0 and dev == _device() else -2


def _stream_on(stream, device: int) -> int | None:
    """_stream, where a tensor on the current device says that there is one."""
    return _stream(stream) if stream is not None or _raw_stream is None else _raw_stream(device)


_swiglu, _swiglu_grad = lib.zq_swiglu_int8, lib.zq_swiglu_grad_int8


def zq_swiglu_int8(gate, up, block: int, h, gate_codes, gate_scales, up_codes, up_scales,
                   stream=None) -> None:
    """h = gate * sigmoid(gate) * up (fp32/bf16/fp16, all of one dtype), and gate
    and up as zq_quant_int8 blocks for zq_swiglu_grad_int8."""
    n, dt, dev = gate.numel(), gate.dtype, _current(gate)
    nb = _blocks(n, block)
    ptr = torch.Tensor.data_ptr
    if not (_fits(gate, dt, n, dev) and _fits(up, dt, n, dev) and _fits(h, dt, n, dev)
            and _fits(gate_codes, torch.int8, n, dev) and _fits(up_codes, torch.int8, n, dev)
            and _fits(gate_scales, torch.float32, nb, dev)
            and _fits(up_scales, torch.float32, nb, dev)):
        for name, t, m, dtypes in (("gate", gate, n, _FLOAT), ("up", up, n, (dt,)),
                                   ("h", h, n, (dt,)), ("gate_codes", gate_codes, n, _I8),
                                   ("gate_scales", gate_scales, nb, _F32),
                                   ("up_codes", up_codes, n, _I8),
                                   ("up_scales", up_scales, nb, _F32)):
            _need(name, t, m, dtypes)
        ptr, dev = _p, _device()
    st = _swiglu(ptr(gate), ptr(up), _dtype(gate), n, block, ptr(h), ptr(gate_codes),
                 ptr(gate_scales), ptr(up_codes), ptr(up_scales), _stream_on(stream, dev))
    if st:
        _check("zq_swiglu_int8", st)


def zq_swiglu_grad_int8(gate_codes, gate_scales, up_codes, up_scales, block: int, dh, dgate, dup,
                        h=None, stream=None) -> None:
    """dgate and dup of zq_swiglu_int8 at its kept values, for h's gradient dh
    (fp32/bf16/fp16, all of one dtype); h, where given, gets the product of the
    kept values."""
    n, dt, dev = dh.numel(), dh.dtype, _current(dh)
    nb = _blocks(n, block)
    ptr = torch.Tensor.data_ptr
    if not (_fits(dh, dt, n, dev) and _fits(dgate, dt, n, dev) and _fits(dup, dt, n, dev)
            and (h is None or _fits(h, dt, n, dev)) and _fits(gate_codes, torch.int8, n, dev)
            and _fits(up_codes, torch.int8, n, dev) and _fits(gate_scales, torch.float32, nb, dev)
            and _fits(up_scales, torch.float32, nb, dev)):
        for name, t, m, dtypes in (("gate_codes", gate_codes, n, _I8),
                                   ("gate_scales", gate_scales, nb, _F32),
                                   ("up_codes", up_codes, n, _I8),
                                   ("up_scales", up_scales, nb, _F32), ("dh", dh, n, _FLOAT),
                                   ("dgate", dgate, n, (dt,)), ("dup", dup, n, (dt,)),
                                   ("h", h, n, (dt,))):
            _need(name, t, m, dtypes)
        ptr, dev = _p, _device()
    st = _swiglu_grad(ptr(gate_codes), ptr(gate_scales), ptr(up_codes), ptr(up_scales), block,
                      ptr(dh), _dtype(dh), n, ptr(dgate), ptr(dup), None if h is None else ptr(h),
                      _stream_on(stream, dev))
    if st:
        _check("zq_swiglu_grad_int8", st)


def linear_grad_workspace(n_tok: int, out_dim: int, in_dim: int) -> int:
    """Bytes of workspace zq_linear_grad_int8 needs."""
    return lib.zq_linear_grad_workspace(n_tok, out_dim, in_dim)


def _bytes(workspace) -> int:
    return workspace.numel() if workspace is not None else 0


def zq_linear_grad_int8(dy, codes, scales, block: int, grad, mode: int, workspace,
                        stream=None) -> None:
    """grad [out, in] (=, with ZQ_GRAD_ADD +=) dy^T x for dy [tokens, out] (bf16/fp16)
    and the layer's input x [tokens, in] kept as zq_quant_int8 blocks; grad
    fp32/bf16/fp16.  workspace: a uint8 tensor of linear_grad_workspace(tokens, out,
    in) bytes, one for each call that may run at the same time."""
    out_dim, in_dim = _rows_dim("grad", grad)
    n_tok, dy_dim = _rows_dim("dy", dy)
    if dy_dim != out_dim:
        raise ValueError(f"dy has {dy_dim} columns, grad {out_dim} rows")
    _width("codes", codes, in_dim, "grad")
    _need("dy", dy, n_tok * out_dim, _HALF)
    _need("codes", codes, n_tok * in_dim, _I8)
    _need("scales", scales, _blocks(n_tok * in_dim, block), _F32)
    _need("grad", grad, out_dim * in_dim, _FLOAT)
    _need("workspace", workspace, linear_grad_workspace(n_tok, out_dim, in_dim), _U8)
    _check("zq_linear_grad_int8",
           lib.zq_linear_grad_int8(_p(dy), _dtype(dy), _p(codes), _p(scales), block, n_tok, out_dim,
                                   in_dim, _p(grad), _dtype(grad), mode, _p(workspace),
                                   _bytes(workspace), _stream(stream)))


def ce_loss_workspace(n_tok: int, rows: int, dim: int, piece: int = 0) -> int:
    """Bytes of workspace zq_ce_loss and zq_ce_loss_int8 need."""
    return lib.zq_ce_loss_workspace(n_tok, rows, dim, piece)


def ce_grad_workspace(n_tok: int, rows: int, dim: int, piece: int = 0) -> int:
    """Bytes of workspace zq_ce_grad and zq_ce_grad_int8 need."""
    return lib.zq_ce_grad_workspace(n_tok, rows, dim, piece)


def _width(name: str, t, dim: int, of: str) -> None:
    """Refuses a tensor of two or more dimensions whose rows are not `dim` wide (its last
    dimension, or the last few together): there may be enough elements all the same, and
    they would be read at the wrong stride."""
    if t is None or isinstance(t, int):
        return
    shape = t.shape
    if len(shape) < 2 or shape[-1] == dim:
        return
    width = 1
    for m in reversed(shape):
        width *= m
        if width >= dim or m == 0:
            break
    if width != dim and t.numel():
        raise ValueError(f"{name} has {shape[-1]} columns, {of} {dim}")


def _ce_loss(fn, x, w, w_args, rows: int, dim: int, ids, scale, loss, lse, workspace, piece,
             stream) -> None:
    n = ids.numel()
    _width("x", x, dim, "the projection")
    _need("x", x, n * dim, _HALF)
    _need("ids", ids, n, _INDEX)
    _need("loss", loss, n, _F32)
    _need("lse", lse, n, _F32)
    _need("workspace", workspace, ce_loss_workspace(n, rows, dim, piece), _U8)
    _check(fn, getattr(lib, fn)(_p(x), _dtype(x), n, dim, _p(w), *w_args, rows, _p(ids),
                                _index(ids), scale, _p(loss), _p(lse), piece, _p(workspace),
                                _bytes(workspace), _stream(stream)))


def zq_ce_loss(x, w, ids, scale: float, loss, lse, workspace, piece: int = 0, stream=None) -> None:
    """Per-token softmax cross entropy of the logits scale * x w^T, which are never
    kept: x [..., dim] or flat (ids.numel() * dim) and w [rows, dim] bf16 or fp16, ids
    int32/int64 (one outside the vocabulary leaves its token out: loss and lse 0), loss
    and lse fp32.
    workspace: a uint8 tensor of ce_loss_workspace(tokens, rows, dim, piece) bytes;
    piece: vocabulary rows worked on at a time (0: the library's choice)."""
    rows, dim = _rows_dim("w", w)
    _need("w", w, rows * dim, (x.dtype,))
    _ce_loss("zq_ce_loss", x, w, (), rows, dim, ids, scale, loss, lse, workspace, piece, stream)


def zq_ce_loss_int8(x, codes, scales, block: int, ids, scale: float, loss, lse, workspace,
                    piece: int = 0, stream=None) -> None:
    """zq_ce_loss with the projection in qwZ's form: codes [rows, dim] int8 and
    scales fp32, as zq_quant_int8 writes them for the flat matrix."""
    rows, dim = _rows_dim("codes", codes)
    _need("codes", codes, rows * dim, _I8)
    _need("scales", scales, _blocks(rows * dim, block), _F32)
    _ce_loss("zq_ce_loss_int8", x, codes, (_p(scales), block), rows, dim, ids, scale, loss, lse,
             workspace, piece, stream)


def _ce_grad(fn, x, w, w_args, rows: int, dim: int, ids, scale, lse, dloss, dx, dw, mode, workspace,
             piece, stream) -> None:
    n = ids.numel()
    for name, t in (("x", x), ("dx", dx), ("dw", dw)):
        _width(name, t, dim, "the projection")
    _need("x", x, n * dim, _HALF)
    _need("ids", ids, n, _INDEX)
    _need("lse", lse, n, _F32)
    _need("dloss", dloss, n, _F32)
    _need("dx", dx, n * dim, (x.dtype,))
    _need("dw", dw, rows * dim, _FLOAT)
    _need("workspace", workspace, ce_grad_workspace(n, rows, dim, piece), _U8)
    _check(fn, getattr(lib, fn)(_p(x), _dtype(x), n, dim, _p(w), *w_args, rows, _p(ids),
                                _index(ids), scale, _p(lse), _p(dloss), _p(dx), _p(dw),
                                ZQ_FP32 if dw is None else _dtype(dw), mode, piece, _p(workspace),
                                _bytes(workspace), _stream(stream)))


def zq_ce_grad(x, w, ids, scale: float, lse, dloss, dx, dw, mode: int, workspace, piece: int = 0,
               stream=None) -> None:
    """The gradient of zq_ce_loss for the losses' gradients dloss (fp32, a token
    each): dx like x, dw [rows, dim] fp32/bf16/fp16 written (ZQ_GRAD_WRITE) or added
    to (ZQ_GRAD_ADD); dx or dw may be None.  lse is what zq_ce_loss wrote.  workspace:
    a uint8 tensor of ce_grad_workspace(tokens, rows, dim, piece) bytes."""
    rows, dim = _rows_dim("w", w)
    _need("w", w, rows * dim, (x.dtype,))
    _ce_grad("zq_ce_grad", x, w, (), rows, dim, ids, scale, lse, dloss, dx, dw, mode, workspace,
             piece, stream)


def zq_ce_grad_int8(x, codes, scales, block: int, ids, scale: float, lse, dloss, dx, dw, mode: int,
                    workspace, piece: int = 0, stream=None) -> None:
    """zq_ce_grad with the projection in qwZ's form (see zq_ce_loss_int8)."""
    rows, dim = _rows_dim("codes", codes)
    _need("codes", codes, rows * dim, _I8)
    _need("scales", scales, _blocks(rows * dim, block), _F32)
    _ce_grad("zq_ce_grad_int8", x, codes, (_p(scales), block), rows, dim, ids, scale, lse, dloss,
             dx, dw, mode, workspace, piece, stream)
