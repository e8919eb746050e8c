"""The form that the library chooses for a 4-bit product, asked of the library itself."""
import ctypes

import segmented_rank_gemm_02_b200 as mlora


class _Plan(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("ksplit", ctypes.c_int32)]


def planned(n_rows, d_in, d_out, n_tokens=0):
    """(rows of a tile, its columns, CTAs a tile): 128 rows are the few-rows form, 256 the pair tiles.
    n_tokens: the grouped positions of the segments, 0 without adapters."""
    fn = mlora.lib()._ZN5mlora12plan_mx_gemmEiiii
    fn.argtypes, fn.restype = [ctypes.c_int32] * 4, _Plan
    p = fn(n_rows, d_in, d_out, n_tokens)
    return p.rows, p.cols, p.ksplit
