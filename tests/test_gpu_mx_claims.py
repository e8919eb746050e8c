"""Rows named by several grouped positions (an error of the caller, flagged): the lowest position in a
valid adapter segment has the row, in every tile, every CTA of a cluster and every run, and the rows
named once get their own adapter as ever.

The sums are of small integers, exact in fp32: results are compared bit for bit."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_02_b200 as mlora
from gpu_harness import DEVICE, free
from mx_plan import planned

pytestmark = pytest.mark.gpu

SLOTS, RANK = 5, 8


def _case(n, n_tokens, d_in, d_out, run, seed):
    """Integer operands, and segments of `run` positions whose rows are drawn with repetition; one
    segment in five is of the base model, one row in nine is named once."""
    rng = np.random.default_rng(seed)
    ints = lambda *s: rng.integers(-2, 3, s).astype(np.float32)   # noqa: E731
    X, W = ints(n, d_in), ints(d_out, d_in)
    X[:, ::32] = W[:, ::32] = 4.0    # the block's largest: a scale of 1
    A = [np.where(rng.random((RANK, d_in)) < 16 / d_in, ints(RANK, d_in), 0) for _ in range(SLOTS)]
    B = [ints(d_out, RANK) for _ in range(SLOTS)]
    pool = mlora.Pool(d_in, d_out, SLOTS, RANK)
    bf = lambda a: torch.from_numpy(a).to(DEVICE, torch.bfloat16)   # noqa: E731
    for a in range(SLOTS):
        pool.load_slot(a, RANK, float(RANK), bf(A[a].astype(np.float32)), bf(B[a]))   # scale 1
    once = np.arange(0, n, 9)
    many = np.setdiff1d(np.arange(n), once)
    rows = np.concatenate([once, rng.choice(many, n_tokens - once.size)])
    rows = rows[rng.permutation(n_tokens)].astype(np.int32)
    offsets = np.append(np.arange(0, n_tokens, run), n_tokens).astype(np.int32)
    slots = rng.integers(-1, SLOTS, offsets.size - 1).astype(np.int32)
    seg = np.repeat(np.arange(slots.size), np.diff(offsets))
    slot = np.full(n, -1)
    for q in np.flatnonzero(slots[seg] >= 0)[::-1]:
        slot[rows[q]] = slots[seg[q]]
    meta = {"offsets": offsets, "slots": slots, "token_indices": rows, "max_segment_rows": 1}
    segs = mlora.DeviceSegments(meta, n, DEVICE)
    want = X.astype(np.float64) @ W.T.astype(np.float64)
    for a in range(SLOTS):
        at = slot == a
        want[at] += (X[at].astype(np.float64) @ A[a].T) @ B[a].T.astype(np.float64)
    assert np.abs(want).max() < 2 ** 20
    return pool, segs, bf(X), bf(W), want


CASES = [
    # few rows, d_in split over a cluster; with more adapters than CTAs, and with one tile or several
    (4, 700, 3584, 136, 7, (128, 128, 2)), (8, 700, 4096, 128, 7, (128, 128, 4)),
    (100, 1000, 8192, 264, 16, (128, 128, 4)), (9, 300, 14336, 64, 16, (128, 128, 8)),
    # few rows, whole tiles: the column tiles of one row block look their rows up separately
    (300, 2000, 256, 520, 16, (128, 128, 1)),
    # many rows: lookup in one launch, and in two
    (2600, 9000, 256, 4104, 16, (256, 384, 1)), (2600, 40000, 256, 4104, 64, (256, 384, 1)),
]


@pytest.mark.parametrize("n,n_tokens,d_in,d_out,run,form", CASES)
def test_lowest_position_has_the_row(n, n_tokens, d_in, d_out, run, form):
    assert planned(n, d_in, d_out, n_tokens) == form
    pool, segs, X, W, want = _case(n, n_tokens, d_in, d_out, run, n + n_tokens)
    Xq, Wq = mlora.mx_quantize(X), mlora.mx_quantize(W)
    for _ in range(4):
        Y = torch.full((n, d_out), float("nan"), dtype=torch.float32, device=DEVICE)
        mlora.mx_gemm_apply(pool, segs, X, Xq, Wq, Y)
        assert pool.check() == mlora.FLAG_BAD_ROW
        assert torch.equal(Y.cpu().double(), torch.from_numpy(want))
    free()


@pytest.mark.parametrize("n,n_tokens,run", [(300, 3000, 16), (1000, 40000, 64)])   # one launch, two
def test_lowest_position_in_the_bf16_product(n, n_tokens, run):
    pool, segs, X, W, want = _case(n, n_tokens, 256, 512, run, n)
    for _ in range(4):
        Y = torch.full((n, 512), float("nan"), dtype=torch.bfloat16, device=DEVICE)
        mlora.base_gemm_apply(pool, segs, X, W, Y)
        assert pool.check() == mlora.FLAG_BAD_ROW
        assert torch.equal(Y.cpu(), torch.from_numpy(want).to(torch.bfloat16))
    free()
