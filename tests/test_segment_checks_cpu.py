"""The binding's checks of operands against the segments they are used with (nothing is launched,
no GPU is needed: every call here is refused before the library sees it)."""
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


def _calls(m, pool, segs, X, Y, H):
    W = torch.zeros(16, 8, dtype=torch.bfloat16)
    return {
        "apply": lambda: m.apply(pool, segs, X, Y),
        "apply_noalloc": lambda: m.apply_noalloc(pool, segs, X, Y),
        "apply_ex": lambda: m.apply_ex(pool, segs, X, Y),
        "base_gemm_apply": lambda: m.base_gemm_apply(pool, segs, X, W, Y),
        "apply_multi": lambda: m.apply_multi([pool], segs, X, [Y]),
        "shrink": lambda: m.shrink(pool, segs, X, H),
        "expand": lambda: m.expand(pool, segs, H, Y),
    }


OPERANDS = [("apply", "X"), ("apply", "Y"), ("apply_noalloc", "X"), ("apply_noalloc", "Y"), ("apply_ex", "X"),
            ("apply_ex", "Y"), ("base_gemm_apply", "X"), ("base_gemm_apply", "Y"), ("apply_multi", "X"),
            ("apply_multi", "Y"), ("shrink", "X"), ("shrink", "H"), ("expand", "H"), ("expand", "Y")]


@pytest.mark.parametrize("call,short", OPERANDS)
def test_operands_shorter_than_the_segments_are_refused(mlora, call, short):
    """A router's groups (N = n_rows * top_k grouped rows) with the batch's own n_rows instead of the
    gathered ones would be read and written past their ends."""
    n, k = 6, 2
    struct = mlora.SegmentsStruct(2, n * k, n * k, 0, None, None, None, None, None)
    segs, pool = SimpleNamespace(struct=struct), SimpleNamespace(handle=None, d_in=8, d_out=16)
    rows = {name: n if name == short else n * k for name in "XYH"}
    X = torch.zeros(rows["X"], 8, dtype=torch.bfloat16)
    Y = torch.zeros(rows["Y"], 16, dtype=torch.bfloat16)
    H = torch.zeros(rows["H"], 16)
    with pytest.raises(ValueError, match=f"{short} has 6 rows"):
        _calls(mlora, pool, segs, X, Y, H)[call]()


@pytest.mark.parametrize("call", ["apply", "apply_noalloc", "apply_ex", "base_gemm_apply", "apply_multi", "shrink",
                                  "expand", "mx_gemm_apply"])
def test_segments_elsewhere_are_refused(mlora, call):
    """Segments whose arrays are not on the pool's device (here: in host memory) would be read by its kernels
    all the same."""
    meta = {"offsets": [0, 2, 4], "slots": [0, 1], "token_indices": [3, 1, 0, 2]}
    pool = SimpleNamespace(handle=None, d_in=8, d_out=16, n_slots=2, device_index=-2)   # no tensor is there
    groups = mlora.RowGroups(pool, 4, 1, "cpu")
    X, Y, H = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(4, 16)
    for segs in (mlora.DeviceSegments(meta, 4, "cpu"), groups, groups.grouped()):
        calls = _calls(mlora, pool, segs, X, Y, H)
        calls["mx_gemm_apply"] = lambda segs=segs: mlora.mx_gemm_apply(
            SimpleNamespace(handle=None, d_in=8, d_out=16, device_index=-1), segs, X, mlora.MxMatrix(4, 8, "cpu"),
            mlora.MxMatrix(16, 8, "cpu"), Y)
        if call == "mx_gemm_apply":
            segs._index = 0   # the matrices' device is looked at first
        with pytest.raises(ValueError, match="segments must be on the pool's device"):
            calls[call]()
