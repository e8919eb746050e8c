"""Python binding of the mlora C ABI (include/mlora.h) -- argument marshalling only.

Every step of the LoRA branch runs in the CUDA kernels of ``libmlora.so``; this
module only turns PyTorch tensors and numpy arrays into pointers, sizes and
streams.  The library is loaded on first use; if it is missing, that first call
raises ImportError: there is no fallback path.

    import segmented_rank_gemm_02_b200 as mlora
    pool = mlora.Pool(d_in, d_out, n_slots, r_max)
    pool.load_slot(slot, rank, alpha, A, B)              # PEFT layout, bf16
    meta = mlora.build_segments(row_slots, pool)          # host grouping helper
    segs = mlora.DeviceSegments(meta, n_rows, device)     # device metadata
    mlora.apply(pool, segs, X, Y)                         # Y (= X W^T) += LoRA delta
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmlora.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_OUT_OF_MEMORY, ERR_BAD_METADATA, ERR_CUDA, ERR_NO_SLOT = range(7)
(FLAG_BAD_OFFSETS, FLAG_BAD_SLOT, FLAG_BAD_RANK, FLAG_BAD_ROW, FLAG_SLOT_EMPTY, FLAG_TIMEOUT,
 FLAG_STALE_SLOT) = (1, 2, 4, 8, 16, 32, 64)

# Every function the header declares (checked by the CPU test suite).
EXPORTS = ("mlora_pool_create", "mlora_pool_destroy", "mlora_pool_load_slot",
           "mlora_pool_clear_slot", "mlora_pool_slot_info", "mlora_pool_shape",
           "mlora_pool_check", "mlora_shrink", "mlora_expand", "mlora_apply",
           "mlora_apply_noalloc", "mlora_apply_multi", "mlora_apply_ex", "mlora_base_gemm_apply",
           "mlora_build_segments", "mlora_status_string",
           "mlora_version", "mlora_pool_slot_generation", "mlora_slot_cache_create",
           "mlora_slot_cache_destroy", "mlora_slot_cache_acquire", "mlora_slot_cache_release",
           "mlora_mx_scale_bytes", "mlora_mx_quantize", "mlora_mx_dequantize", "mlora_mx_gemm_apply",
           "mlora_group_rows", "mlora_gather_rows", "mlora_combine_rows", "mlora_combine_rows_backward",
           "mlora_slot_cache_invalidate", "mlora_slot_cache_lookup", "mlora_slot_cache_stats")


class MloraError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class SegmentsStruct(ctypes.Structure):
    _fields_ = [("n_segments", ctypes.c_int32), ("n_rows", ctypes.c_int32),
                ("n_tokens", ctypes.c_int32), ("max_segment_rows", ctypes.c_int32),
                ("segment_offsets", ctypes.c_void_p), ("adapter_slots", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("token_indices", ctypes.c_void_p), ("generations", ctypes.c_void_p)]


class MxStruct(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int32), ("n_cols", ctypes.c_int32), ("ld", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class RowGroupsStruct(ctypes.Structure):
    _fields_ = [("offsets", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("ranks", ctypes.c_void_p),
                ("order", ctypes.c_void_p), ("positions", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m segmented_rank_gemm_02_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    i32p = ctypes.POINTER(ctypes.c_int32)
    seg_p = ctypes.POINTER(SegmentsStruct)
    mx_p = ctypes.POINTER(MxStruct)
    sig = {
        "mlora_pool_create": [i32, i32, i32, i32, ctypes.POINTER(vp)],
        "mlora_pool_destroy": [vp],
        "mlora_pool_load_slot": [vp, i32, i32, f32, vp, vp, i32, vp],
        "mlora_pool_clear_slot": [vp, i32, vp],
        "mlora_pool_slot_info": [vp, i32, i32p, ctypes.POINTER(f32), ctypes.POINTER(i64)],
        "mlora_pool_shape": [vp, i32p, i32p, i32p, i32p],
        "mlora_pool_check": [vp, vp, ctypes.POINTER(ctypes.c_uint32)],
        "mlora_shrink": [vp, seg_p, vp, i64, vp, i64, vp],
        "mlora_expand": [vp, seg_p, vp, i64, vp, i64, vp],
        "mlora_apply": [vp, seg_p, vp, i64, vp, i64, vp],
        "mlora_apply_noalloc": [vp, seg_p, vp, i64, vp, i64, vp],
        "mlora_apply_ex": [vp, seg_p, vp, i32, f32, i64, vp, i32, i64, vp],
        "mlora_base_gemm_apply": [vp, seg_p, vp, i64, vp, i64, vp, i64, vp],
        "mlora_apply_multi": [ctypes.POINTER(vp), i32, seg_p, vp, i64, ctypes.POINTER(vp),
                              ctypes.POINTER(i64), vp],
        "mlora_mx_quantize": [vp, i32, i64, mx_p, vp],
        "mlora_mx_dequantize": [mx_p, vp, i32, i64, vp],
        "mlora_mx_gemm_apply": [vp, seg_p, vp, i64, mx_p, mx_p, vp, i32, i64, vp],
        "mlora_group_rows": [vp, vp, i32, i32, ctypes.POINTER(RowGroupsStruct), vp],
        "mlora_gather_rows": [vp, vp, i32, i32, vp, i64, i32, i32, i32, vp, i64, vp],
        "mlora_combine_rows": [vp, vp, vp, i32, i32, vp, i64, i32, i32, i32, vp, i64, vp],
        "mlora_combine_rows_backward": [vp, vp, vp, i32, i32, vp, i64, vp, i64, i32, i32, i32, vp, i64, vp, vp],
        "mlora_build_segments": [vp, i32, vp, vp, vp, i32p, i32p, vp, vp],
        "mlora_pool_slot_generation": [vp, i32, ctypes.POINTER(ctypes.c_uint32)],
        "mlora_slot_cache_create": [i32, ctypes.POINTER(vp)],
        "mlora_slot_cache_destroy": [vp],
        "mlora_slot_cache_acquire": [vp, ctypes.c_uint64, i32p, i32p, ctypes.POINTER(ctypes.c_uint64)],
        "mlora_slot_cache_release": [vp, i32],
        "mlora_slot_cache_invalidate": [vp, i32],
        "mlora_slot_cache_lookup": [vp, ctypes.c_uint64, i32p],
        "mlora_slot_cache_stats": [vp, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i64)],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.mlora_status_string.argtypes = [ctypes.c_int]
    lib.mlora_status_string.restype = ctypes.c_char_p
    lib.mlora_mx_scale_bytes.argtypes = [i32, i32]
    lib.mlora_mx_scale_bytes.restype = i64
    lib.mlora_version.argtypes = []
    lib.mlora_version.restype = ctypes.c_int32
    return lib


_lib_handle = None


def lib():
    """The loaded libmlora.so (loads it on first use; raises if it is not built)."""
    global _lib_handle
    if _lib_handle is None:
        _lib_handle = _load()
    return _lib_handle


def status_string(status: int) -> str:
    return lib().mlora_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != OK:
        raise MloraError(status, what)


_current_device = _raw_stream = None   # torch's, looked up once: a small call is mostly such look-ups


def _look_up() -> None:
    global _current_device, _raw_stream
    if _current_device is None:
        import torch
        _current_device, _raw_stream = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        _look_up()
        return _raw_stream(_current_device())
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    if isinstance(x, np.ndarray):
        return int(x.ctypes.data)
    return int(x)


def _ld(t, what: str, rows: int = 0) -> int:
    """Row stride of a row-major operand that must have `rows` rows or more."""
    st = t.stride()
    if len(st) != 2 or st[1] != 1:
        raise ValueError(f"{what} must be a 2-D row-major tensor")
    if t.shape[0] < rows:
        raise ValueError(f"{what} has {t.shape[0]} rows, the segments are of {rows}")
    return int(st[0])


def as_bf16_tensor(bits: np.ndarray, device=None):
    """bf16 bit patterns (numpy uint16) -> torch.bfloat16 tensor (bit-exact)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)
    return t if device is None else t.to(device)


def bf16_bits(t) -> np.ndarray:
    """torch.bfloat16 tensor -> numpy uint16 bit patterns."""
    import torch
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Pool:
    """A fixed-stride adapter pool for one projection (owns device memory)."""

    def __init__(self, d_in: int, d_out: int, n_slots: int, r_max: int):
        h = ctypes.c_void_p()
        _check(lib().mlora_pool_create(d_in, d_out, n_slots, r_max, ctypes.byref(h)),
               "mlora_pool_create")
        self.handle = h.value
        self.d_in, self.d_out, self.n_slots, self.r_max = d_in, d_out, n_slots, r_max
        import torch
        self.device_index = torch.cuda.current_device()   # where the pool's memory is

    def load_slot(self, slot: int, rank: int, alpha: float, A, B, stream=None) -> None:
        """A: bf16 [rank, d_in], B: bf16 [d_out, rank]; numpy uint16 bits or torch tensors."""
        keep = []

        def src(m):
            if isinstance(m, np.ndarray):
                m = np.ascontiguousarray(m, dtype=np.uint16)
                keep.append(m)
                return int(m.ctypes.data), 0
            m = m.contiguous()
            keep.append(m)
            return int(m.data_ptr()), int(m.is_cuda)

        pa, da = src(A)
        pb, db = src(B)
        if da != db:
            raise ValueError("A and B must both be host or both be device memory")
        _check(lib().mlora_pool_load_slot(self.handle, slot, rank, float(alpha), pa, pb, da,
                                         _stream_ptr(stream)), "mlora_pool_load_slot")
        if not da:
            # host sources are staged by the call itself; keep until it returns
            pass
        self._keep = keep

    def clear_slot(self, slot: int, stream=None) -> None:
        _check(lib().mlora_pool_clear_slot(self.handle, slot, _stream_ptr(stream)),
               "mlora_pool_clear_slot")

    def generation(self, slot: int) -> int:
        """Generation of the slot's contents (mlora_pool_slot_generation)."""
        g = ctypes.c_uint32()
        _check(lib().mlora_pool_slot_generation(self.handle, slot, ctypes.byref(g)),
               "mlora_pool_slot_generation")
        return int(g.value)

    def slot_info(self, slot: int):
        r, a, n = ctypes.c_int32(), ctypes.c_float(), ctypes.c_int64()
        _check(lib().mlora_pool_slot_info(self.handle, slot, ctypes.byref(r), ctypes.byref(a),
                                         ctypes.byref(n)), "mlora_pool_slot_info")
        return r.value, a.value, n.value

    def check(self, stream=None) -> int:
        """Synchronise, read and clear the device status word; returns the flag bits."""
        f = ctypes.c_uint32()
        st = lib().mlora_pool_check(self.handle, _stream_ptr(stream), ctypes.byref(f))
        if st not in (OK, ERR_BAD_METADATA):
            _check(st, "mlora_pool_check")
        return int(f.value)

    def close(self) -> None:
        if getattr(self, "handle", None):
            lib().mlora_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def build_segments(row_slots: np.ndarray, pool: Optional[Pool] = None) -> dict:
    """Host grouping helper (mlora_build_segments): numpy int32 arrays."""
    row_slots = np.ascontiguousarray(row_slots, dtype=np.int32)
    n = int(row_slots.shape[0])
    offsets = np.zeros(n + 1, np.int32)
    slots = np.zeros(max(n, 1), np.int32)
    ti = np.zeros(max(n, 1), np.int32)
    ranks = np.zeros(max(n, 1), np.int32)
    S, longest = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().mlora_build_segments(_ptr(row_slots), n, _ptr(offsets), _ptr(slots), _ptr(ti),
                                     ctypes.byref(S), ctypes.byref(longest),
                                     pool.handle if pool is not None else None,
                                     _ptr(ranks) if pool is not None else None),
           "mlora_build_segments")
    S = S.value
    out = {"offsets": offsets[:S + 1].copy(), "slots": slots[:S].copy(),
           "token_indices": ti[:n].copy(), "max_segment_rows": longest.value}
    if pool is not None:
        out["ranks"] = ranks[:S].copy()
    return out


class DeviceSegments:
    """Segment metadata resident on the device, plus the C struct pointing at it."""

    def __init__(self, meta: dict, n_rows: int, device, scales=None, identity_rows=False,
                 generations=None):
        import torch
        dev = torch.device(device)
        self.offsets = torch.as_tensor(np.asarray(meta["offsets"], np.int32)).to(dev)
        self.slots = torch.as_tensor(np.asarray(meta["slots"], np.int32)).to(dev)
        r = meta.get("ranks")
        self.ranks = None if r is None else torch.as_tensor(np.asarray(r, np.int32)).to(dev)
        self.scales = None if scales is None else torch.as_tensor(
            np.asarray(scales, np.float32)).to(dev)
        ti = meta.get("token_indices")
        self.token_indices = (None if (ti is None or identity_rows)
                              else torch.as_tensor(np.asarray(ti, np.int32)).to(dev))
        n_tokens = int(meta.get("n_tokens", self.offsets[-1].item() if ti is None else len(ti)))
        gens = generations if generations is not None else meta.get("generations")
        self.generations = None if gens is None else torch.as_tensor(
            np.asarray(gens, np.uint32).view(np.int32)).to(dev)
        self.struct = SegmentsStruct(
            int(self.slots.numel()), int(n_rows), n_tokens, int(meta.get("max_segment_rows", 0)),
            _ptr(self.offsets), _ptr(self.slots), _ptr(self.ranks), _ptr(self.scales),
            _ptr(self.token_indices), _ptr(self.generations))

        self._index = self.offsets.get_device()

    @property
    def n_tokens(self) -> int:
        return int(self.struct.n_tokens)


def _seg_ref(pool: Pool, segs):
    """The segments' struct for a call on the pool; their arrays must be where its kernels read them."""
    index = getattr(segs, "_index", None)
    if index is not None and index != pool.device_index and segs.struct.n_segments > 0:
        raise ValueError("the segments must be on the pool's device")
    return ctypes.byref(segs.struct)


def apply(pool: Pool, segs: DeviceSegments, X, Y, stream=None) -> None:
    """Y[t] = bf16(Y[t] + s (X[t] A^T) B^T) in place (mlora_apply)."""
    _check(lib().mlora_apply(pool.handle, _seg_ref(pool, segs), _ptr(X), _ld(X, "X", segs.struct.n_rows),
                            _ptr(Y), _ld(Y, "Y", segs.struct.n_rows), _stream_ptr(stream)), "mlora_apply")


def apply_noalloc(pool: Pool, segs: DeviceSegments, X, Y, stream=None) -> None:
    """mlora_apply with the long-segment scratch in the library's fixed device array
    (mlora_apply_noalloc): allocates nothing; concurrent calls on the GPU race."""
    _check(lib().mlora_apply_noalloc(pool.handle, _seg_ref(pool, segs), _ptr(X), _ld(X, "X", segs.struct.n_rows),
                                     _ptr(Y), _ld(Y, "Y", segs.struct.n_rows), _stream_ptr(stream)),
           "mlora_apply_noalloc")


MAX_FUSED = 4

DTYPE_BF16, DTYPE_FP16, DTYPE_FP32, DTYPE_FP8_E4M3 = 0, 1, 2, 3


def _dtype_code(t) -> int:
    import torch
    codes = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32,
             torch.float8_e4m3fn: DTYPE_FP8_E4M3}
    if t.dtype not in codes:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return codes[t.dtype]


def apply_ex(pool: Pool, segs: DeviceSegments, X, Y, x_scale: float = 1.0, stream=None) -> None:
    """mlora_apply at a quantized base model's dtype boundary (mlora_apply_ex): X bf16 or
    FP8 e4m3 codes (value = code * x_scale), Y bf16, fp16 or fp32, updated in place."""
    _check(lib().mlora_apply_ex(pool.handle, _seg_ref(pool, segs), _ptr(X), _dtype_code(X), float(x_scale),
                                _ld(X, "X", segs.struct.n_rows), _ptr(Y), _dtype_code(Y),
                                _ld(Y, "Y", segs.struct.n_rows), _stream_ptr(stream)),
           "mlora_apply_ex")


def base_gemm_apply(pool: Pool, segs: DeviceSegments, X, W, Y, stream=None) -> None:
    """Y = bf16(X W^T + s (X A^T) B^T) for adapter rows, bf16(X W^T) for the others, in
    one pass (mlora_base_gemm_apply).  X [n_rows, d_in], W [d_out, d_in] (nn.Linear
    layout) and Y [n_rows, d_out], all bf16 on the pool's device; Y is written, not read."""
    _check(lib().mlora_base_gemm_apply(pool.handle, _seg_ref(pool, segs), _ptr(X),
                                       _ld(X, "X", segs.struct.n_rows), _ptr(W), _ld(W, "W"), _ptr(Y),
                                       _ld(Y, "Y", segs.struct.n_rows), _stream_ptr(stream)),
           "mlora_base_gemm_apply")


def apply_multi(pools, segs: DeviceSegments, X, Ys, stream=None) -> None:
    """mlora_apply over several projections sharing X and the segments (q/k/v,
    gate/up): Ys[k] += delta of pools[k], in one pass over X (mlora_apply_multi)."""
    pools, Ys = list(pools), list(Ys)
    if len(pools) != len(Ys):
        raise ValueError("one output per pool")
    n = len(pools)
    for p in pools:
        _seg_ref(p, segs)
    handles = (ctypes.c_void_p * max(n, 1))(*[p.handle for p in pools])
    outs = (ctypes.c_void_p * max(n, 1))(*[_ptr(Y) for Y in Ys])
    lds = (ctypes.c_int64 * max(n, 1))(*[_ld(Y, "Y", segs.struct.n_rows) for Y in Ys])
    _check(lib().mlora_apply_multi(handles, n, ctypes.byref(segs.struct), _ptr(X), _ld(X, "X", segs.struct.n_rows),
                                   outs, lds, _stream_ptr(stream)), "mlora_apply_multi")


def shrink(pool: Pool, segs: DeviceSegments, X, H, stream=None) -> None:
    """H[p, :r] = X[t_p] A^T, fp32, grouped order (mlora_shrink)."""
    _check(lib().mlora_shrink(pool.handle, _seg_ref(pool, segs), _ptr(X), _ld(X, "X", segs.struct.n_rows),
                             _ptr(H), _ld(H, "H", segs.struct.n_tokens), _stream_ptr(stream)), "mlora_shrink")


def expand(pool: Pool, segs: DeviceSegments, H, Y, stream=None) -> None:
    """Y[t_p] = bf16(Y[t_p] + s H[p, :r] B^T) in place (mlora_expand)."""
    _check(lib().mlora_expand(pool.handle, _seg_ref(pool, segs), _ptr(H), _ld(H, "H", segs.struct.n_tokens),
                             _ptr(Y), _ld(Y, "Y", segs.struct.n_rows), _stream_ptr(stream)), "mlora_expand")


_float_codes = {}   # torch dtype -> MLORA_DTYPE_* of the types rows and outputs may have


def _float_code(t, what: str) -> int:
    if not _float_codes:
        import torch
        _float_codes.update({torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32})
    code = _float_codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bf16, fp16 or fp32")
    return code


def _call(fn, what: str, device: int, stream, *args) -> None:
    """fn(*args, stream) with `device` current, on its current stream unless one is given."""
    _look_up()
    if device < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if device != _current_device():
        import torch
        with torch.cuda.device(device):
            return _call(fn, what, device, stream, *args)
    st = fn(*args, _raw_stream(device) if stream is None else _stream_ptr(stream))
    if st != OK:
        raise MloraError(st, what)


def _empty(like, shape, dtype, stream):
    """An output on like's device for a call on `stream`: allocated there, so that its memory is not
    still in use elsewhere."""
    if stream is None:
        return like.new_empty(shape) if dtype is None else like.new_empty(shape, dtype=dtype)
    import torch
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype or like.dtype)


class MxMatrix:
    """A 4-bit microscaled matrix (mlora_mx_matrix): packed codes [n_rows, 16 per block of 32
    columns] and scale tiles [ceil(n_rows / 128), 2 ceil(n_cols / 256), 32, 4, 4], uint8, allocated
    on `device` or given (a checkpoint's own, already in this layout)."""

    def __init__(self, n_rows: int, n_cols: int, device=None, codes=None, scales=None, stream=None, like=None):
        import torch
        n_rows, n_cols = int(n_rows), int(n_cols)
        if not 0 <= n_rows < 1 << 31 or not 0 < n_cols < 1 << 31 or n_cols % 8 != 0:
            raise ValueError("a 4-bit matrix has 0 <= n_rows < 2^31 and n_cols a positive multiple of 8 below 2^31")
        row_bytes = (n_cols + 31) // 32 * 16
        self.n_rows, self.n_cols = n_rows, n_cols
        self._codes, self._scales = codes, scales
        if codes is None and scales is None:
            # one allocation: the scale tiles (whole 1 KB), then the codes; the tensors are made when asked for
            at = (n_rows + 127) // 128 * ((n_cols + 255) // 256) * 1024
            if like is None:
                like = torch.empty(0, dtype=torch.uint8, device=device)
            self._buf = _empty(like, at + n_rows * row_bytes, torch.uint8, stream)
            ptr = self._buf.data_ptr()
            self._index = self._buf.get_device()
            self.struct = MxStruct(n_rows, n_cols, row_bytes, ptr + at, ptr)
            return
        shape = self._scale_shape()
        if codes is None:
            codes = _empty(scales, (n_rows, row_bytes), torch.uint8, stream)
        if scales is None:
            scales = _empty(codes, shape, torch.uint8, stream)
        if codes.dtype != torch.uint8 or tuple(codes.shape) != (n_rows, row_bytes):
            raise ValueError(f"codes must be uint8 [{n_rows}, {row_bytes}]")
        if scales.dtype != torch.uint8 or tuple(scales.shape) != shape or not scales.is_contiguous():
            raise ValueError(f"scales must be contiguous uint8 {list(shape)}")
        if scales.device != codes.device:
            raise ValueError("codes and scales must be on one device")
        self._codes, self._scales = codes, scales
        self._index = codes.get_device()
        ld = _ld(codes, "codes")
        self.struct = MxStruct(n_rows, n_cols, ld if n_rows > 1 else row_bytes, _ptr(codes), _ptr(scales))

    def _scale_shape(self):
        return ((self.n_rows + 127) // 128, 2 * ((self.n_cols + 255) // 256), 32, 4, 4)

    @property
    def codes(self):
        if self._codes is None:
            rows = self.n_rows * ((self.n_cols + 31) // 32 * 16)
            self._codes = self._buf[self._buf.numel() - rows:].view(self.n_rows, (self.n_cols + 31) // 32 * 16)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            shape = self._scale_shape()
            self._scales = self._buf[:shape[0] * shape[1] * 512].view(shape)
        return self._scales

    @property
    def device(self):
        return (self._buf if self._codes is None else self._codes).device


def mx_quantize(X, out: Optional[MxMatrix] = None, stream=None) -> MxMatrix:
    """X [n, d] (bf16, fp16 or fp32, on the GPU) as a 4-bit microscaled matrix (mlora_mx_quantize)."""
    code, (n, d), ld, index = _float_code(X, "X"), X.shape, _ld(X, "X"), X.get_device()
    if index < 0:
        raise ValueError("X must be on a CUDA device")
    if out is None:
        out = MxMatrix(n, d, stream=stream, like=X)
    elif (out.n_rows, out.n_cols, out._index) != (n, d, index):
        raise ValueError("out must have X's shape and device")
    _call(lib().mlora_mx_quantize, "mlora_mx_quantize", index, stream, X.data_ptr(), code,
          ld if n > 1 else max(ld, d), ctypes.byref(out.struct))
    return out


def mx_dequantize(Q: MxMatrix, out=None, dtype=None, stream=None):
    """The values Q stands for, in `dtype` (bf16 unless given) or into `out` (mlora_mx_dequantize)."""
    import torch
    shape = (Q.n_rows, Q.n_cols)
    if out is None:
        out = _empty(Q._buf if Q._codes is None else Q._codes, shape, dtype or torch.bfloat16, stream)
    elif tuple(out.shape) != shape or out.get_device() != Q._index or dtype not in (None, out.dtype):
        raise ValueError("out must have Q's shape and device, and dtype if both are given")
    ld = _ld(out, "out")
    _call(lib().mlora_mx_dequantize, "mlora_mx_dequantize", Q._index, stream, ctypes.byref(Q.struct), out.data_ptr(),
          _float_code(out, "out"), ld if Q.n_rows > 1 else max(ld, Q.n_cols))
    return out


def mx_gemm_apply(pool: Pool, segs: Optional["DeviceSegments"], X, Xq: MxMatrix, W: MxMatrix, Y, stream=None) -> None:
    """Y = round(Xq W^T + s (X A^T) B^T) for adapter rows, round(Xq W^T) for the others, in one pass
    (mlora_mx_gemm_apply).  Xq [n_rows, d_in] and W [d_out, d_in] 4-bit, X the bf16 activations that
    Xq was quantised from (not read, and may be None, if segs is None), Y bf16, fp16 or fp32.
    Nothing is recorded for autograd, and the product has no gradient here."""
    n, index = Xq.n_rows, Y.get_device()
    if tuple(Y.shape) != (n, pool.d_out):
        raise ValueError("Y must be [rows of Xq, d_out]")
    xp, ldx = None, 0
    if segs is not None:
        if X is None or tuple(X.shape) != (n, pool.d_in) or _float_code(X, "X") != DTYPE_BF16:
            raise ValueError("X must be bf16 [rows of Xq, d_in]")
        if X.get_device() != index:
            raise ValueError("X and Y must be on one device")
        xp, ldx = X.data_ptr(), _ld(X, "X")
        ldx = ldx if n > 1 else max(ldx, pool.d_in)
    if Xq._index != index or W._index != index or pool.device_index != index:
        raise ValueError("Xq, W and Y must be on the pool's device")
    ldy = _ld(Y, "Y")
    _call(lib().mlora_mx_gemm_apply, "mlora_mx_gemm_apply", index, stream, pool.handle,
          _seg_ref(pool, segs) if segs is not None else None, xp, ldx, ctypes.byref(Xq.struct),
          ctypes.byref(W.struct), Y.data_ptr(), _float_code(Y, "Y"), ldy if n > 1 else max(ldy, pool.d_out))


class RowGroups:
    """Rows grouped by slot on the device (mlora_group_rows), usable as DeviceSegments: of the
    batch's own rows if they were grouped by row_slots [n_rows], of the rows in grouped order
    (gather_rows) if by [n_rows, top_k], [n_rows, 1] among them.  grouped() gives the latter in
    either case.

    offsets, slots, ranks, order, positions: int32 device tensors (see mlora.h).  ranks are this pool's;
    with_ranks=False leaves them out of the segments, for use with pools whose ranks differ."""

    def __init__(self, pool: Pool, n_rows: int, top_k: int, device=None, max_segment_rows: int = 0, stream=None,
                 with_ranks: bool = True, like=None):
        import torch
        n = n_rows * top_k
        if n > 1 << 30:
            raise ValueError("at most 2^30 entries are grouped")
        S = min(pool.n_slots + 1, n)
        self.pool, self.n_rows, self.top_k, self.n_tokens, self._S = pool, n_rows, top_k, n, S
        # one allocation; the tensors are made when asked for
        if like is None:
            like = torch.empty(0, dtype=torch.int32, device=device)
        self._buf = _empty(like, 3 * S + 1 + 2 * n, torch.int32, stream)
        self._index = self._buf.get_device()
        at = self._buf.data_ptr()
        self._positions = at + 4 * (3 * S + 1 + n)
        self._out = RowGroupsStruct(at, at + 4 * (S + 1), at + 4 * (2 * S + 1), at + 4 * (3 * S + 1), self._positions)
        self._hint, self._with_ranks, self._struct, self._parts = int(max_segment_rows), with_ranks, None, None
        self._own_rows = top_k == 1   # until group_rows sees the shape of its row_slots

    def _segments(self, own_rows: bool) -> SegmentsStruct:
        o, n = self._out, self.n_tokens
        return SegmentsStruct(self._S, n, n, self._hint, o.offsets, o.slots, o.ranks if self._with_ranks else None, None,
                              o.order if own_rows else None, None)

    @property
    def struct(self) -> SegmentsStruct:
        if self._struct is None:
            self._struct = self._segments(self._own_rows)
        return self._struct

    def grouped(self) -> "_GroupedSegments":
        """The segments of the rows in grouped order (those of gather_rows), whatever was grouped."""
        return _GroupedSegments(self)

    def _part(self, i: int):
        if self._parts is None:
            import torch
            self._parts = torch.split(self._buf, (self._S + 1, self._S, self._S, self.n_tokens, self.n_tokens))
        return self._parts[i]

    @property
    def offsets(self):
        return self._part(0)

    @property
    def slots(self):
        return self._part(1)

    @property
    def ranks(self):
        return self._part(2)

    @property
    def order(self):
        return self._part(3)

    @property
    def positions(self):
        return self._part(4)


class _GroupedSegments:
    def __init__(self, groups: RowGroups):
        self.groups, self.n_tokens, self._index = groups, groups.n_tokens, groups._index   # (keeps the arrays)
        self.struct = groups._segments(False)


def group_rows(pool: Pool, row_slots, out: Optional[RowGroups] = None, max_segment_rows: int = 0,
               stream=None, with_ranks: bool = True) -> RowGroups:
    """Sort rows by adapter slot on the device (mlora_group_rows).  row_slots: int32 [n_rows] or
    [n_rows, top_k], contiguous, -1 = base model; which of the two decides what the result is as
    segments (see RowGroups).  `out` reuses a RowGroups of the same sizes (a
    captured graph's).  max_segment_rows: the hint of mlora_segments, if the caller knows one (1 for
    a decode batch used with its own rows, which spares it the launches for long segments);
    with_ranks: see RowGroups (both only without `out`)."""
    import torch
    shape = row_slots.shape
    if row_slots.dtype != torch.int32 or len(shape) not in (1, 2) or not row_slots.is_contiguous():
        raise ValueError("row_slots must be contiguous int32 [n_rows] or [n_rows, top_k]")
    n_rows, top_k, index = shape[0], 1 if len(shape) == 1 else shape[1], row_slots.get_device()
    if top_k < 1 or index < 0 or index != pool.device_index:
        raise ValueError("row_slots needs at least one slot per row, on the pool's device")
    if out is None:
        out = RowGroups(pool, n_rows, top_k, None, max_segment_rows, stream, with_ranks, row_slots)
    elif out.pool is not pool or (out.n_rows, out.top_k, out._index) != (n_rows, top_k, index):
        raise ValueError("out must be of this pool, the same sizes and device")
    _call(lib().mlora_group_rows, "mlora_group_rows", index, stream, pool.handle, row_slots.data_ptr(), n_rows, top_k,
          ctypes.byref(out._out))
    if out._own_rows != (len(shape) == 1):
        out._own_rows, out._struct = len(shape) == 1, None
    return out


def _rows_of(t, n: int, d, dtype, index: int, what: str):
    """Row stride of a [n, d] operand; its dtype and device must be these."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != n or shape[1] != d or t.dtype != dtype or t.get_device() != index:
        raise ValueError(f"{what} has the wrong shape, dtype or device")
    ld = _ld(t, what)
    return ld if n > 1 else max(ld, d)


def _weights_ptr(groups: RowGroups, w, index: int, what: str):
    import torch
    if w is None:
        return None
    shape = tuple(w.shape)
    if (w.dtype != torch.float32 or not w.is_contiguous() or w.get_device() != index
            or shape not in ((groups.n_rows, groups.top_k), (groups.n_tokens,))):
        raise ValueError(f"{what} must be contiguous fp32 [n_rows, top_k] (or flat) on the rows' device")
    return w.data_ptr()


def gather_rows(groups: RowGroups, X, Xs=None, stream=None):
    """Xs[positions[t, j]] = X[t]: the rows in grouped order (mlora_gather_rows).  The gradient of X
    is combine_rows(groups, dXs); nothing is recorded for autograd.  Entries whose slot is not the
    pool's have no row: as many at the end of Xs, from offsets[-1] on, are left as they were, that
    is uninitialised in a new Xs."""
    code, d, n, index = _float_code(X, "X"), X.shape[-1], groups.n_tokens, groups._index
    ldx = _rows_of(X, groups.n_rows, d, X.dtype, index, "X")
    if Xs is None:
        Xs, ldxs = _empty(X, (n, d), None, stream), d
    else:
        ldxs = _rows_of(Xs, n, d, X.dtype, index, "Xs")
    _call(lib().mlora_gather_rows, "mlora_gather_rows", index, stream, groups.pool.handle, groups._positions,
          groups.n_rows, groups.top_k, X.data_ptr(), ldx, code, d, n, Xs.data_ptr(), ldxs)
    return Xs


def combine_rows(groups: RowGroups, Ys, weights=None, Y=None, stream=None):
    """Y[t] = sum_j weights[t, j] Ys[positions[t, j]] (mlora_combine_rows); weights fp32 or None (ones).
    Nothing is recorded for autograd: the gradients are combine_rows_backward."""
    code, d, n, index = _float_code(Ys, "Ys"), Ys.shape[-1], groups.n_tokens, groups._index
    ldys = _rows_of(Ys, n, d, Ys.dtype, index, "Ys")
    w = _weights_ptr(groups, weights, index, "weights")
    if Y is None:
        Y, ldy = _empty(Ys, (groups.n_rows, d), None, stream), d
    else:
        ldy = _rows_of(Y, groups.n_rows, d, Ys.dtype, index, "Y")
    _call(lib().mlora_combine_rows, "mlora_combine_rows", index, stream, groups.pool.handle, groups._positions, w,
          groups.n_rows, groups.top_k, Ys.data_ptr(), ldys, code, d, n, Y.data_ptr(), ldy)
    return Y


def combine_rows_backward(groups: RowGroups, dY, Ys, weights=None, dYs=None, dweights=None, stream=None):
    """(dYs, dweights) of combine_rows from dY (mlora_combine_rows_backward).  Without weights only dYs
    is computed (dweights is None, Ys may be None) unless a dweights tensor is given.  Rows of dYs from
    groups.offsets[-1] on (there are some only where a slot was not the pool's) are left as they were,
    that is uninitialised in a new dYs: leave them out of sums over rows, or give a dYs of zeros."""
    import torch
    code, d, n, index = _float_code(dY, "dY"), dY.shape[-1], groups.n_tokens, groups._index
    lddy = _rows_of(dY, groups.n_rows, d, dY.dtype, index, "dY")
    w = _weights_ptr(groups, weights, index, "weights")
    if dYs is None:
        dYs, lddys = _empty(dY, (n, d), None, stream), d
    else:
        lddys = _rows_of(dYs, n, d, dY.dtype, index, "dYs")
    if dweights is None and weights is not None:
        dweights = _empty(dY, (groups.n_rows, groups.top_k), torch.float32, stream)
    dw = _weights_ptr(groups, dweights, index, "dweights")
    if dw is not None and Ys is None:
        raise ValueError("the gradient of the weights needs Ys")
    ysp, ldys = (None, 0) if Ys is None else (Ys.data_ptr(), _rows_of(Ys, n, d, dY.dtype, index, "Ys"))
    _call(lib().mlora_combine_rows_backward, "mlora_combine_rows_backward", index, stream, groups.pool.handle,
          groups._positions, w, groups.n_rows, groups.top_k, dY.data_ptr(), lddy, ysp, ldys, code, d, n, dYs.data_ptr(),
          lddys, dw)
    return dYs, dweights


class SlotCache:
    """Host-side adapter cache over a pool's slots (mlora_slot_cache): LRU order among
    unpinned slots, pin counts for in-flight batches.  Needs no GPU."""

    NONE = 2 ** 64 - 1

    def __init__(self, n_slots: int):
        h = ctypes.c_void_p()
        _check(lib().mlora_slot_cache_create(int(n_slots), ctypes.byref(h)), "mlora_slot_cache_create")
        self.handle = h.value

    def acquire(self, adapter_id: int):
        """(slot, needs_load, evicted_id or None); pins the slot."""
        s, nl, ev = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_uint64()
        _check(lib().mlora_slot_cache_acquire(self.handle, ctypes.c_uint64(adapter_id), ctypes.byref(s),
                                             ctypes.byref(nl), ctypes.byref(ev)),
               "mlora_slot_cache_acquire")
        return s.value, bool(nl.value), (None if ev.value == self.NONE else int(ev.value))

    def release(self, slot: int) -> None:
        _check(lib().mlora_slot_cache_release(self.handle, int(slot)), "mlora_slot_cache_release")

    def invalidate(self, slot: int) -> None:
        _check(lib().mlora_slot_cache_invalidate(self.handle, int(slot)), "mlora_slot_cache_invalidate")

    def lookup(self, adapter_id: int) -> int:
        s = ctypes.c_int32()
        _check(lib().mlora_slot_cache_lookup(self.handle, ctypes.c_uint64(adapter_id), ctypes.byref(s)),
               "mlora_slot_cache_lookup")
        return s.value

    def stats(self):
        h, m, e = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib().mlora_slot_cache_stats(self.handle, ctypes.byref(h), ctypes.byref(m), ctypes.byref(e)),
               "mlora_slot_cache_stats")
        return h.value, m.value, e.value

    def close(self) -> None:
        if getattr(self, "handle", None):
            lib().mlora_slot_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def version() -> int:
    return int(lib().mlora_version())
