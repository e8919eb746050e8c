"""Operands that the binding of the 4-bit and grouped-row calls refuses (no GPU is needed)."""
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def mlora():
    from segmented_rank_gemm_02_b200 import build
    build.build()
    import segmented_rank_gemm_02_b200 as m
    m.lib()
    return m


def _groups(mlora, n, k):
    return mlora.RowGroups(SimpleNamespace(handle=None, n_slots=3, device_index=-1), n, k, "cpu")


def test_weights_of_another_shape_are_refused(mlora):
    """As many weights in another arrangement would be read as other choices' weights."""
    gr, Ys, dY = _groups(mlora, 6, 2), torch.zeros(12, 8), torch.zeros(6, 8)
    for shape in ((2, 6), (12, 1), (1, 12), (3, 4), (6, 2, 1)):
        w = torch.ones(shape)
        with pytest.raises(ValueError, match="weights must be"):
            mlora.combine_rows(gr, Ys, w)
        with pytest.raises(ValueError, match="weights must be"):
            mlora.combine_rows_backward(gr, dY, Ys, w)
        with pytest.raises(ValueError, match="dweights must be"):
            mlora.combine_rows_backward(gr, dY, Ys, None, dweights=w)
    for shape in ((6, 2), (12,)):   # get as far as the device
        with pytest.raises(ValueError, match="CUDA device"):
            mlora.combine_rows(gr, Ys, torch.ones(shape))


@pytest.mark.parametrize("n", [1, 3])
def test_codes_whose_bytes_are_apart_are_refused(mlora, n):
    """A row's codes have to be consecutive, of a matrix of one row too."""
    scales = torch.zeros(1, 2, 32, 4, 4, dtype=torch.uint8)
    apart = torch.zeros(n, 64, dtype=torch.uint8)[:, ::2]
    with pytest.raises(ValueError, match="codes must be"):
        mlora.MxMatrix(n, 64, codes=apart, scales=scales)
    with pytest.raises(ValueError, match="codes must be"):
        mlora.MxMatrix(n, 64, codes=apart)
    assert mlora.MxMatrix(n, 64, codes=apart.contiguous(), scales=scales).struct.ld == 32


def test_a_matrix_allocates_on_its_stream(mlora, monkeypatch):
    """Whatever part of a matrix is allocated belongs to the stream that the matrix is for."""
    seen = []

    def empty(like, shape, dtype, stream):
        seen.append(stream)
        return torch.zeros(shape, dtype=dtype)

    monkeypatch.setattr(mlora, "_empty", empty)
    mlora.MxMatrix(3, 64, "cpu", stream=7)
    mlora.MxMatrix(3, 64, codes=torch.zeros(3, 32, dtype=torch.uint8), stream=8)
    mlora.MxMatrix(3, 64, scales=torch.zeros(1, 2, 32, 4, 4, dtype=torch.uint8), stream=9)
    assert seen == [7, 8, 9]


def test_sizes_past_32_bits_are_refused(mlora):
    """Sizes reach the library as 32-bit numbers: larger ones would arrive as others."""
    codes, scales = torch.empty(0, dtype=torch.uint8), torch.empty(0, dtype=torch.uint8)
    for n, d in ((1 << 31, 8), ((1 << 32) + 5, 8), (1, 1 << 31), (1, (1 << 32) + 8)):
        with pytest.raises(ValueError, match="4-bit matrix has"):
            mlora.MxMatrix(n, d, codes=codes, scales=scales)
    for n, k in (((1 << 30) + 1, 1), ((1 << 32) + 5, 1), (1 << 16, (1 << 14) + 1)):
        with pytest.raises(ValueError, match="entries"):
            mlora.RowGroups(SimpleNamespace(n_slots=3), n, k, "meta")


def test_plan_of_the_longest_matrices(mlora):
    from mx_plan import planned
    for n in ((1 << 31) - 1, (1 << 31) - 100, (1 << 31) - 257):
        assert planned(n, 64, 64) == (256, 256, 1)


def test_plan_of_a_long_list_of_rows(mlora):
    """With adapters the few-rows form's time grows with the square of the list: it is left to short ones,
    few rows named by a long list included."""
    from mx_plan import planned
    for n, d_in, d_out in ((60000, 512, 128), (1 << 24, 8, 8), (16384, 64, 64), (8, 4096, 128)):
        if n < 1 << 24:
            assert planned(n, d_in, d_out)[0] == 128
        assert planned(n, d_in, d_out, max(n, 60000))[0] == 256
    assert planned(256, 4096, 4096, 256) == planned(256, 4096, 4096)
