"""Host-side refusals of the 4-bit and grouped-row entry points (nothing is launched, no GPU is
needed), the scale layout, and the references that the GPU tests use."""
import ctypes

import numpy as np
import pytest

import mx_ref


@pytest.fixture(scope="module")
def mlora():
    from segmented_rank_gemm_02_b200 import build
    build.build()
    import segmented_rank_gemm_02_b200 as m
    m.lib()
    return m


def test_reference_known_values():
    x = np.zeros((1, 40))
    x[0, :8] = [7.9, 6.0, 5.0, 3.5, 2.5, 0.25, -0.75, -7.0]
    x[0, 32:] = 2.0 ** -10 * np.arange(8)
    codes, scale, values = mx_ref.quantize(x)
    assert scale.tolist() == [[127, 127 - 10]]                  # 2^(floor(log2 7.9) - 2), 2^(-8 - 2)
    assert values[0, :8].tolist() == [6.0, 6.0, 4.0, 4.0, 2.0, 0.0, -1.0, -6.0]
    assert codes[0, :8].tolist() == [7, 7, 6, 6, 4, 0, 10, 15]
    assert (values[0, 32:] * 2.0 ** 10).tolist() == [0, 1, 2, 3, 4, 4, 6, 6]


def test_scale_bytes_and_layout(mlora):
    L = mlora.lib()
    for n, d in [(1, 8), (128, 256), (129, 264), (300, 4096), (0, 32)]:
        want = -(-n // 128) * 2 * -(-d // 256) * 512
        assert L.mlora_mx_scale_bytes(n, d) == want
        Q = mlora.MxMatrix(n, d, "cpu")
        assert Q.scales.numel() == want and Q.codes.shape == (n, -(-d // 32) * 16)
    assert L.mlora_mx_scale_bytes(-1, 8) == -1
    # the byte offset that the header gives, against the reference's tiles
    scale = np.arange(200 * 10, dtype=np.uint32).reshape(200, 10)
    scale = (scale % 251 + 1).astype(np.uint8)
    flat = mx_ref.tile_scales(scale).reshape(-1)
    for r, b in [(0, 0), (31, 3), (32, 4), (127, 9), (128, 0), (199, 7)]:
        at = ((r // 128) * 2 * -(-320 // 256) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
        assert flat[at] == scale[r, b]


def _mx(mlora, rows=4, cols=64, ld=None, codes=256, scales=512):
    return mlora.MxStruct(rows, cols, (cols + 31) // 32 * 16 if ld is None else ld, codes, scales)


def test_quantize_refusals(mlora):
    L, bad, unsupported = mlora.lib(), mlora.ERR_INVALID_ARG, mlora.ERR_UNSUPPORTED

    def both(x, dtype, ldx, q):
        p = ctypes.byref(q) if q is not None else None
        got = L.mlora_mx_quantize(x, dtype, ldx, p, None), L.mlora_mx_dequantize(p, x, dtype, ldx, None)
        assert got[0] == got[1]
        return got[0]

    assert both(256, 0, 64, None) == bad
    assert both(None, 0, 64, _mx(mlora)) == bad
    assert both(256, mlora.DTYPE_FP8_E4M3, 64, _mx(mlora)) == bad
    assert both(256, 7, 64, _mx(mlora)) == bad
    assert both(256, 0, 56, _mx(mlora)) == bad                 # rows overlap
    assert both(256, 0, 68, _mx(mlora)) == bad                 # rows not of whole vectors
    assert both(256, mlora.DTYPE_FP32, 66, _mx(mlora)) == bad
    assert both(264, 0, 64, _mx(mlora)) == bad                 # misaligned
    assert both(256, 0, 64, _mx(mlora, rows=-1)) == bad
    assert both(256, 0, 64, _mx(mlora, cols=0)) == bad
    assert both(256, 0, 64, _mx(mlora, cols=60)) == unsupported
    assert both(256, 0, 64, _mx(mlora, ld=16)) == bad
    assert both(256, 0, 64, _mx(mlora, ld=40)) == bad
    assert both(256, 0, 64, _mx(mlora, codes=None)) == bad
    assert both(256, 0, 64, _mx(mlora, scales=None)) == bad
    assert both(256, 0, 64, _mx(mlora, codes=264)) == bad
    assert both(None, 0, 64, _mx(mlora, rows=0, codes=None, scales=None)) == mlora.OK


def test_null_pool_refusals(mlora):
    L, bad = mlora.lib(), mlora.ERR_INVALID_ARG
    q = ctypes.byref(_mx(mlora))
    seg = mlora.SegmentsStruct(0, 0, 0, 0, None, None, None, None, None)
    assert L.mlora_mx_gemm_apply(None, ctypes.byref(seg), None, 0, q, q, 256, 0, 64, None) == bad
    out = mlora.RowGroupsStruct(256, 256, None, 256, 256)
    assert L.mlora_group_rows(None, 256, 1, 1, ctypes.byref(out), None) == bad
    assert L.mlora_gather_rows(None, 256, 1, 1, 256, 8, 0, 8, 1, 256, 8, None) == bad
    assert L.mlora_combine_rows(None, 256, None, 1, 1, 256, 8, 0, 8, 1, 256, 8, None) == bad
    assert L.mlora_combine_rows_backward(None, 256, None, 1, 1, 256, 8, 256, 8, 0, 8, 1, 256, 8, 256, None) == bad


def test_binding_refusals(mlora):
    import torch
    with pytest.raises(ValueError):
        mlora.MxMatrix(4, 60, "cpu")
    with pytest.raises(ValueError):
        mlora.MxMatrix(4, 64, codes=torch.zeros(4, 16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mlora.MxMatrix(4, 64, codes=torch.zeros(4, 32, dtype=torch.uint8), scales=torch.zeros(3, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mlora.mx_quantize(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        mlora.mx_quantize(torch.zeros(4, 64))                  # not on a GPU
    with pytest.raises(ValueError):
        mlora.mx_quantize(torch.zeros(4, 64).to(torch.float8_e4m3fn))
    for slots in (torch.zeros(4, dtype=torch.int64), torch.zeros(4, 2, 2, dtype=torch.int32),
                  torch.zeros(4, 4, dtype=torch.int32)[:, :2], torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError):
            mlora.group_rows(None, slots)


def test_reference_grouping():
    offsets, slots, order, positions = mx_ref.group(np.array([[2, -1], [0, 2], [9, 2]]), 3)
    assert slots.tolist() == [-1, 0, 2, -1] and offsets.tolist() == [0, 1, 2, 5, 5]
    assert order.tolist() == [1, 2, 0, 3, 5, 4] and positions.tolist() == [2, 0, 1, 3, -1, 4]
