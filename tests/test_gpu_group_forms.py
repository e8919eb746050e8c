"""What a batch grouped on the device is as segments: of its own rows for row_slots [n_rows], of the
gathered rows for [n_rows, top_k], a router's single choice [n_rows, 1] among them.

Operands are small integers: sums are exact in fp32, results are compared bit for bit."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_02_b200 as mlora
from gpu_harness import DEVICE

pytestmark = pytest.mark.gpu

N, D_IN, D_OUT, SLOTS, RANK = 150, 256, 136, 6, 8


def _case(k, seed):
    rng = np.random.default_rng(seed)
    ints = lambda *s: rng.integers(-2, 3, s).astype(np.float64)   # noqa: E731
    X, W = ints(N, D_IN), ints(D_OUT, D_IN)
    X[:, ::32] = W[:, ::32] = 4.0    # the block's largest: a scale of 1
    A, B = ints(SLOTS, RANK, D_IN), ints(SLOTS, D_OUT, RANK)
    A[rng.random(A.shape) < 0.9] = 0
    pool = mlora.Pool(D_IN, D_OUT, SLOTS, RANK)
    bf = lambda a: torch.from_numpy(a).to(DEVICE, torch.bfloat16)   # noqa: E731
    for a in range(SLOTS):
        pool.load_slot(a, RANK, float(RANK), bf(A[a]), bf(B[a]))   # scale 1
    slots = np.stack([rng.permutation(SLOTS + 1)[:k] - 1 for _ in range(N)]).astype(np.int32)
    each = np.empty((N, k, D_OUT))
    for t in range(N):
        for j in range(k):
            a = slots[t, j]
            each[t, j] = W @ X[t] + (B[a] @ (A[a] @ X[t]) if a >= 0 else 0)
    assert np.abs(each).max() < 2 ** 20
    return pool, bf(X), mlora.mx_quantize(bf(W)), slots, each


@pytest.mark.parametrize("explicit", [False, True])
@pytest.mark.parametrize("k", [1, 2, 3])
def test_a_routers_choices(k, explicit):
    """group -> gather -> quantise -> product -> combine, the groups passed themselves or grouped()."""
    pool, X, Wq, slots, each = _case(k, k)
    gr = mlora.group_rows(pool, torch.from_numpy(slots).to(DEVICE))
    for _ in range(2):   # the second time into the same arrays
        Xs = mlora.gather_rows(gr, X)
        Ys = torch.full((N * k, D_OUT), float("nan"), device=DEVICE)
        mlora.mx_gemm_apply(pool, gr.grouped() if explicit else gr, Xs, mlora.mx_quantize(Xs), Wq, Ys)
        assert torch.equal(mlora.combine_rows(gr, Ys).cpu().double(), torch.from_numpy(each.sum(1)))
        mlora.group_rows(pool, torch.from_numpy(slots).to(DEVICE), out=gr)
    assert pool.check() == 0


def test_one_slot_a_row_and_a_reused_result():
    pool, X, Wq, slots, each = _case(1, 9)
    flat = torch.from_numpy(slots[:, 0].copy()).to(DEVICE)
    Xq = mlora.mx_quantize(X)
    for gr in (mlora.group_rows(pool, flat), mlora.RowGroups(pool, N, 1, torch.device(DEVICE))):
        for form in (flat, flat.view(N, 1), flat):   # the form follows the row_slots of the last call
            mlora.group_rows(pool, form, out=gr)
            Y = torch.full((N, D_OUT), float("nan"), device=DEVICE)
            if form.dim() == 1:
                mlora.mx_gemm_apply(pool, gr, X, Xq, Wq, Y)
            else:
                Xs, Ys = mlora.gather_rows(gr, X), torch.full_like(Y, float("nan"))
                mlora.mx_gemm_apply(pool, gr, Xs, mlora.mx_quantize(Xs), Wq, Ys)
                mlora.combine_rows(gr, Ys, Y=Y)
            assert torch.equal(Y.cpu().double(), torch.from_numpy(each[:, 0]))
    assert pool.check() == 0
