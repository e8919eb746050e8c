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
