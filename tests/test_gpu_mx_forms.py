"""The 4-bit product in each of its forms, with adapters: the cases are chosen by the form that the
library plans for them, which is checked.

The operands are small integers whose sums stay below 2^24, exact in fp32, so an output is the
64-bit result rounded once to its type: compared bit for bit."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_02_b200 as mlora
from gpu_harness import DEVICE, free
from mx_plan import planned

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def _ints(gen, *shape):
    return torch.randint(-2, 3, shape, generator=gen, device=DEVICE).double()


class _Case:
    """A pool of `ranks` (slot a has rank ranks[a % len]), its adapters, and integer rows and weights."""

    def __init__(self, n, d_in, d_out, n_slots, ranks, seed, r_max=None):
        g = torch.Generator(device=DEVICE)
        g.manual_seed(seed)
        self.n, self.d_out, self.n_slots = n, d_out, n_slots
        self.X, self.W = _ints(g, n, d_in), _ints(g, d_out, d_in)
        self.X[:, ::32] = self.W[:, ::32] = 4.0    # the block's largest: a scale of 1
        self.pool = mlora.Pool(d_in, d_out, n_slots, r_max or max(ranks))
        self.A, self.B = [], []
        for a in range(n_slots):
            r = ranks[a % len(ranks)]
            A, B = _ints(g, r, d_in), _ints(g, d_out, r)
            A[torch.rand(A.shape, generator=g, device=DEVICE) > 8 / d_in] = 0
            self.A.append(A), self.B.append(B)
            self.pool.load_slot(a, r, float(r), A.bfloat16(), B.bfloat16())   # scale 1
        self.Xb = self.X.bfloat16()
        self.Xq, self.Wq = mlora.mx_quantize(self.Xb), mlora.mx_quantize(self.W.float())

    def want(self, slot):
        Y = self.X @ self.W.T
        for a in range(self.n_slots):
            at = torch.from_numpy(np.flatnonzero(slot == a)).to(DEVICE)
            Y[at] += (self.X[at] @ self.A[a].T) @ self.B[a].T
        assert Y.abs().max() < 60000    # fp16's range too
        return Y

    def check(self, segs, slot, dtypes=DTYPES):
        want = self.want(slot)
        for dtype in dtypes:
            Y = torch.full((self.n, self.d_out), float("nan"), dtype=dtype, device=DEVICE)
            mlora.mx_gemm_apply(self.pool, segs, self.Xb, self.Xq, self.Wq, Y)
            assert torch.equal(Y, want.to(dtype))
        assert self.pool.check() == 0


def _slots(n, n_slots, runs, seed, base=0.15):
    rng = np.random.default_rng(seed)
    slot = rng.integers(0, n_slots, n).astype(np.int32)
    slot[rng.random(n) < base] = -1
    return np.sort(slot) if runs else slot


def _segments(c, slot):
    return mlora.DeviceSegments(mlora.build_segments(slot, c.pool), c.n, DEVICE)


@pytest.mark.parametrize("n,d_in,d_out,n_slots,ranks,runs", [
    (4608, 4096, 2048, 8, (64,), True),
    (2560, 512, 1032, 12, (16,), False),
    (1300, 1024, 2056, 70, (1, 8), False),       # more slots a row block than one ring stage holds
    (2048, 256, 2048, 9, (5, 16, 24, 40, 64), False),
    (2600, 264, 1032, 5, (32,), True),
])
def test_256_column_pair_tiles(n, d_in, d_out, n_slots, ranks, runs):
    assert planned(n, d_in, d_out, n) == (256, 256, 1)
    c = _Case(n, d_in, d_out, n_slots, ranks, n)
    slot = _slots(n, n_slots, runs, n)
    c.check(_segments(c, slot), slot)
    free()


@pytest.mark.parametrize("n,d_in,d_out,form", [(100, 264, 136, (128, 128, 1)), (40, 8192, 136, (128, 128, 4)),
                                               (1300, 520, 2056, (256, 256, 1)), (2600, 256, 4104, (256, 384, 1))])
@pytest.mark.parametrize("r_max,ranks", [(8, (1, 3, 8)), (16, (16, 9)), (32, (32, 17, 8)), (64, (64, 33, 2))])
def test_each_rank_bucket_in_each_form(n, d_in, d_out, form, r_max, ranks):
    """Pools whose largest bucket is 8, 16, 32 and 64; rows standing together and scattered."""
    assert planned(n, d_in, d_out, n) == form
    c = _Case(n, d_in, d_out, 6, ranks, n + r_max, r_max)
    for runs in (True, False):
        slot = _slots(n, 6, runs, r_max)
        c.check(_segments(c, slot), slot, [torch.float32, torch.bfloat16])
    free()


@pytest.mark.parametrize("n,d_in,d_out,ksplit", [(4, 3584, 136, 2), (2, 3584, 64, 2), (60, 8192, 256, 4),
                                                 (5, 8192, 128, 4), (128, 8192, 200, 4), (9, 14336, 64, 8)])
@pytest.mark.parametrize("n_slots", [1, 3, 40])
def test_adapters_divided_over_a_cluster(n, d_in, d_out, ksplit, n_slots):
    """d_in split over 2, 4 and 8 CTAs, whose slots are every ksplit-th: fewer of them than CTAs, and more."""
    assert planned(n, d_in, d_out, n) == (128, 128, ksplit)
    c = _Case(n, d_in, d_out, n_slots, (8, 64, 16, 20), n + n_slots)
    for base in (0.0, 0.5):
        slot = _slots(n, n_slots, False, n_slots, base)
        c.check(_segments(c, slot), slot)
    free()


def test_pair_tiles_with_a_list_of_rows_past_one_lookup():
    """More grouped positions than the one-launch lookup of the pair form takes."""
    n, d_in, d_out = 34000, 64, 1032
    assert planned(n, d_in, d_out, n)[0] == 256
    c = _Case(n, d_in, d_out, 9, (8, 16), 3)
    for runs in (True, False):
        slot = _slots(n, 9, runs, 5)
        c.check(_segments(c, slot), slot, [torch.float32])
    free()


@pytest.mark.parametrize("n,d_in,d_out", [(8192, 64, 64), (8193, 64, 64), (16400, 512, 128), (40000, 256, 64)])
def test_a_long_list_of_rows_leaves_the_few_rows_form(n, d_in, d_out):
    assert planned(n, d_in, d_out)[0] == 128 and planned(n, d_in, d_out, n)[0] == (128 if n <= 8192 else 256)
    c = _Case(n, d_in, d_out, 7, (8, 16), n)
    slot = _slots(n, 7, False, 2)
    c.check(_segments(c, slot), slot, [torch.float32, torch.bfloat16])
    free()


def _many_segments(n, run, n_slots, seed):
    """Segments of `run` positions of shuffled rows, neighbours with equal slots among them."""
    rng = np.random.default_rng(seed)
    offsets = np.append(np.arange(0, n, run), n).astype(np.int32)
    slots = rng.integers(-1, n_slots, offsets.size - 1).astype(np.int32)
    rows = rng.permutation(n).astype(np.int32)
    slot = np.empty(n, np.int32)
    slot[rows] = np.repeat(slots, np.diff(offsets))
    return {"offsets": offsets, "slots": slots, "token_indices": rows, "max_segment_rows": 1}, slot


@pytest.mark.parametrize("n,run", [(4000, 2), (2048, 2), (36000, 5)])   # 2000, 1024, 7200 segments
def test_more_segments_than_the_lookups_keep(n, run):
    """Segment lists longer than the pair form's and the bf16 product's shared-memory tables."""
    meta, slot = _many_segments(n, run, 7, n)
    assert planned(n, 256, 1544, n)[0] == 256 and len(meta["slots"]) > 1023
    c = _Case(n, 256, 1544, 7, (8, 12), n)
    segs = mlora.DeviceSegments(meta, n, DEVICE)
    c.check(segs, slot, [torch.float32])
    Y = torch.full((n, 1544), float("nan"), dtype=torch.bfloat16, device=DEVICE)
    mlora.base_gemm_apply(c.pool, segs, c.Xb, c.W.bfloat16(), Y)
    assert c.pool.check() == 0 and torch.equal(Y, c.want(slot).bfloat16())
    free()


def test_quantize_the_longest_row():
    """A row of 2^31 - 8 columns: padding and chunk counts that 32-bit sums would not hold."""
    d = (1 << 31) - 8
    g = torch.Generator(device=DEVICE)
    g.manual_seed(1)
    X = torch.zeros(1, d, dtype=torch.bfloat16, device=DEVICE)
    spots = torch.tensor([0, 255, 256, 1 << 30, d - 257, d - 32, d - 25, d - 24, d - 9, d - 1], device=DEVICE)
    X[0, spots] = torch.randn(spots.numel(), generator=g, device=DEVICE).bfloat16()
    Q = mlora.mx_quantize(X)
    for lo in (0, d - 24 - 256):     # the last block has 24 columns; a piece of whole blocks before it
        piece = X[:, lo: lo + 280].contiguous()
        part = mlora.mx_quantize(piece)
        assert torch.equal(Q.codes[:, lo // 2: lo // 2 + 144], part.codes)
        out = torch.empty(1, 280, dtype=torch.bfloat16, device=DEVICE)
        mlora.mx_dequantize(part, out=out)
        X[:, lo: lo + 280] = out
    back = torch.zeros_like(X)
    mlora.mx_dequantize(Q, out=back)
    for lo in (0, d - 24 - 256):
        assert torch.equal(back[:, lo: lo + 280], X[:, lo: lo + 280])
    for at in ((1 << 30), d - 300):  # between them: what stands alone in its block, and zeros
        block = back[0, at: at + 20].float()
        assert torch.equal(block != 0, X[0, at: at + 20] != 0)
    del X, Q, back
    free()
