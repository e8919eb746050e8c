"""4-bit microscaled matrices and their product with the LoRA delta, against 64-bit references.

Tolerances.  Quantisation and its inverse are exact functions of their inputs: bit equality.
The product of integers whose sums stay below 2^24 is exact in fp32: equality.  Otherwise an
element may be off by its one rounding (half a step of the output's type, relative), by the
fp32 sums (at most one step of 2^-23 of the sum of magnitudes for each of the d_in products),
and by the low-rank product's operand split (bf16 hi + lo keep s H to 2^-17) plus its sums.
"""
import numpy as np
import pytest
import torch

import mx_ref
import oracle
import segmented_rank_gemm_02_b200 as mlora
from gpu_harness import DEVICE, free

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# below the smallest normal number steps are absolute: half of the smallest subnormal (fp16 counts)
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def _rows(n, d, dtype, seed=0, spread=6.0):
    """Normal rows whose blocks differ in scale by up to 2^spread either way."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, d)) * np.exp2(rng.uniform(-spread, spread, (n, -(-d // 8))).repeat(8, 1)[:, :d])
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 8), (1, 32), (3, 40), (33, 256), (127, 264), (128, 288), (129, 1032), (300, 4096)])
def test_quantize_bits_and_back(n, d, dtype):
    X = _rows(n, d, dtype, seed=n + d)
    X[0, 0] = 0.0
    if n > 2:
        X[1] = 0                    # blocks of zeros
        X[2, : d // 2] = 2.0 ** -24  # a tiny block (fp16's smallest)
    codes, scale, values = mx_ref.quantize(X.double().numpy())
    Q = mlora.mx_quantize(X.to(DEVICE))
    assert np.array_equal(Q.codes.cpu().numpy(), mx_ref.pack(codes))
    tiles, want = Q.scales.cpu().numpy(), mx_ref.tile_scales(scale)
    assert np.array_equal(tiles, want)
    back = mlora.mx_dequantize(Q, dtype=torch.float32)
    assert np.array_equal(back.cpu().double().numpy(), values)
    assert torch.equal(mlora.mx_dequantize(Q).double().cpu(), torch.from_numpy(values).to(torch.bfloat16).double())


def test_quantize_ties_and_saturation():
    # every midpoint between neighbouring levels, the values beside it, and what saturates
    a = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.96875])
    x = np.zeros((4, 32), np.float32)
    x[0, :9], x[0, 9:18] = a, -a
    x[1, :9] = np.nextafter(a.astype(np.float32), np.float32(0))
    x[2, :9] = np.nextafter(a.astype(np.float32), np.float32(8))
    x[:3, 31] = 4.0                 # scale 1 in every block
    x[3, :3] = [1.0, -0.2, 0.25]
    codes, scale, values = mx_ref.quantize(x)
    assert scale[0, 0] == 127 and values[0, 7] == 6.0 and values[0, 0] == 0.0 and values[0, 1] == 1.0
    Q = mlora.mx_quantize(torch.from_numpy(x).to(DEVICE))
    assert np.array_equal(Q.codes.cpu().numpy(), mx_ref.pack(codes))
    assert np.array_equal(mlora.mx_dequantize(Q, dtype=torch.float32).cpu().double().numpy(), values)


def test_quantize_extremes():
    # the largest and smallest fp32 magnitudes, subnormal blocks, infinities and NaN
    x = np.zeros((6, 64), np.float32)
    x[0, :4] = [3.4028235e38, -1e38, 1e30, 1.0]
    x[1, :3] = [1e-45, 1.1754944e-38, -5.9e-39]
    x[2, 5], x[2, 40] = np.inf, 1.0
    x[3, 5], x[3, 40] = np.nan, -2.0
    x[4, :2] = [2.0 ** -125, 2.0 ** -126]
    x[5, 33] = -np.inf
    codes, scale, values = mx_ref.quantize(x)
    Q = mlora.mx_quantize(torch.from_numpy(x).to(DEVICE))
    assert np.array_equal(Q.codes.cpu().numpy(), mx_ref.pack(codes))
    assert np.array_equal(Q.scales.cpu().numpy(), mx_ref.tile_scales(scale))
    back = mlora.mx_dequantize(Q, dtype=torch.float32).cpu().double().numpy()
    assert np.array_equal(back, values, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantize_special_rows_beside_others(dtype):
    # rows 32 apart are quantised together: infinities, NaN of either sign, zeros, subnormals and the
    # largest numbers of one row leave the rows beside it alone
    X = _rows(160, 328, dtype, seed=9, spread=3.0)
    info = torch.finfo(dtype)
    special = [float("inf"), float("-inf"), float("nan"), info.max, -info.max, info.smallest_normal, 2.0 ** -24, 0.0]
    for i, v in enumerate(special):
        X[i + 32 * (i % 4), 32 * (i % 8): 32 * (i % 8) + 32] = 0
        X[i + 32 * (i % 4), 32 * (i % 8) + 5 * (i % 6)] = v
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    negative_nan = X[40:41, 7:8].view(bits)
    negative_nan.fill_(-1)               # every bit set: a NaN with its sign
    codes, scale, values = mx_ref.quantize(X.double().numpy())
    assert np.isnan(values).any() and (scale == 255).sum() == 4
    Q = mlora.mx_quantize(X.to(DEVICE))
    assert np.array_equal(Q.codes.cpu().numpy(), mx_ref.pack(codes))
    assert np.array_equal(Q.scales.cpu().numpy(), mx_ref.tile_scales(scale))
    back = mlora.mx_dequantize(Q, dtype=torch.float32).cpu().double().numpy()
    assert np.array_equal(back, values, equal_nan=True)


def test_quantize_strided_rows_and_reused_output():
    wide = _rows(70, 320, torch.bfloat16, seed=4).to(DEVICE)
    X = wide[:, 32:32 + 200]        # a slice of wider rows (32 columns in: 64 bytes)
    out = mlora.MxMatrix(70, 200, DEVICE)
    out.codes.fill_(0xff)
    out.scales.fill_(0xff)
    assert mlora.mx_quantize(X, out=out) is out
    codes, scale, values = mx_ref.quantize(X.double().cpu().numpy())
    assert np.array_equal(out.codes.cpu().numpy(), mx_ref.pack(codes))
    assert np.array_equal(out.scales.cpu().numpy(), mx_ref.tile_scales(scale))
    back = torch.full((70, 264), 7.0, dtype=torch.float16, device=DEVICE)
    mlora.mx_dequantize(out, out=back[:, 8:208])
    assert torch.equal(back[:, 8:208].double().cpu(), torch.from_numpy(values).to(torch.float16).double())
    assert (back[:, :8] == 7).all() and (back[:, 208:] == 7).all()


def _integers(n, d, seed):
    """Small integers times block scales 1 or 2: every code exact, sums far below 2^24."""
    rng = np.random.default_rng(seed)
    x = rng.choice([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], (n, d)).astype(np.float64)
    x[:, ::32] = 4.0                # block maximum 4 or 6: scale 1 before the factor
    return x * np.exp2(rng.integers(0, 2, (n, -(-d // 32))).repeat(32, 1)[:, :d])


SHAPES = [(1, 8, 8), (1, 32, 128), (1, 4096, 4096), (5, 72, 40), (17, 256, 136), (128, 512, 128), (129, 320, 264),
          (256, 4096, 512), (300, 1000, 200), (64, 8192, 1024), (513, 2048, 2056), (257, 14336, 384),
          # many rows: pair tiles, with rows, columns and K blocks off the tile sizes (4481 rows: the last
          # pair's second half is empty)
          (4000, 520, 3000), (4481, 1032, 2056), (9000, 64, 1032), (4608, 4096, 2048)]


@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_base_product_exact_integers(n, d_in, d_out):
    X, W = _integers(n, d_in, 1), _integers(d_out, d_in, 2)
    want = X @ W.T
    assert np.abs(X) .max() * np.abs(W).max() * d_in < 2 ** 24
    pool = mlora.Pool(d_in, d_out, 1, 8)
    Xq = mlora.mx_quantize(torch.from_numpy(X).to(DEVICE, torch.bfloat16))
    Wq = mlora.mx_quantize(torch.from_numpy(W).to(DEVICE, torch.bfloat16))
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        Y = torch.full((n, d_out), float("nan"), dtype=dtype, device=DEVICE)
        mlora.mx_gemm_apply(pool, None, None, Xq, Wq, Y)
        assert torch.equal(Y.cpu().double(), torch.from_numpy(want).to(dtype).double())
    assert pool.check() == 0
    free()


def _case(n, d_in, d_out, n_slots, ranks, base, runs, seed):
    rng = np.random.default_rng(seed)
    slot_rank = np.array([ranks[i % len(ranks)] for i in range(n_slots)], np.int32)
    slot = rng.integers(0, n_slots, n).astype(np.int32)
    if runs:
        slot = np.sort(slot)
    slot[rng.random(n) < base] = -1
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s) * 0.1).to(torch.bfloat16)   # noqa: E731
    A = {a: bf(int(slot_rank[a]), d_in) for a in range(n_slots)}
    B = {a: bf(d_out, int(slot_rank[a])) for a in range(n_slots)}
    pool = mlora.Pool(d_in, d_out, n_slots, max(ranks))
    for a in range(n_slots):
        pool.load_slot(a, int(slot_rank[a]), 2.0 * a + 1.0, A[a].to(DEVICE), B[a].to(DEVICE))
    X = _rows(n, d_in, torch.bfloat16, seed + 1, spread=1.0)
    W = _rows(d_out, d_in, torch.float32, seed + 2, spread=1.0) * 0.05
    return pool, slot, slot_rank, A, B, X, W


def _reference(slot, slot_rank, A, B, X, W, rows=None):
    """Y and the bound's magnitudes, in 64 bits: the base products' and the low-rank products'."""
    rows = np.arange(len(slot)) if rows is None else rows
    x = mx_ref.quantize(X.double().numpy()[rows])[2]
    w = mx_ref.quantize(W.double().numpy())[2]
    Y, mag, lora = x @ w.T, np.abs(x) @ np.abs(w).T, np.zeros((len(rows), w.shape[0]))
    for i, t in enumerate(rows):
        a = int(slot[t])
        if a < 0:
            continue
        s = (2.0 * a + 1.0) / float(slot_rank[a])
        xt, Aa, Ba = X[t].double().numpy(), A[a].double().numpy(), B[a].double().numpy()
        Y[i] += s * (Ba @ (Aa @ xt))
        lora[i] = s * (np.abs(Ba) @ (np.abs(Aa) @ np.abs(xt)))
    return Y, mag, lora


def _assert_product(Y, ref, mag, lora, d_in, rank=64):
    got = Y.cpu().double().numpy()
    assert not np.isnan(got).any(), "rows left unwritten"
    # lora: H sums d_in products in fp32, the operand split 2^-17, rank products, the scale's rounding
    sums = d_in * 2.0 ** -23 * mag + (d_in * 2.0 ** -23 + 2.0 ** -17 + (rank + 4) * 2.0 ** -23) * lora
    bound = HALF_STEP[Y.dtype] * (np.abs(ref) + sums) + sums + TINY[Y.dtype]
    worst = (np.abs(got - ref) / bound).max()
    assert worst <= 1.0, worst
    # and far closer than that bound in the mean: sums of d_in terms do not all err one way
    rms = np.sqrt(np.mean((got - ref) ** 2)) / np.sqrt(np.mean(ref ** 2))
    assert rms <= HALF_STEP[Y.dtype] + 2.0 ** -16, rms


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,d_in,d_out,slots,ranks,base,runs", [
    (1, 256, 136, 1, (8,), 0.0, False),
    (1, 4096, 1024, 3, (1,), 0.0, False),
    (2, 64, 8, 2, (16,), 0.0, False),
    (40, 1024, 264, 7, (1, 7, 12, 16), 0.2, False),
    (130, 520, 200, 5, (8, 24, 64), 0.3, False),
    (256, 2048, 512, 64, (16,), 0.1, False),
    (300, 200, 200, 7, (1, 7, 12, 24, 40, 64), 0.1, True),
    (700, 768, 640, 3, (64,), 0.0, True),
    (140, 512, 128, 140, (4,), 0.0, False),      # every row its own adapter
    (64, 512, 128, 2, (32,), 1.0, False),        # base rows only
    (4481, 200, 3080, 9, (8, 24, 64), 0.2, True),      # pair tiles: requests standing together
    (4000, 776, 2568, 40, (1, 8, 16), 0.2, False),     # and scattered rows of many slots
])
def test_product_with_adapters(n, d_in, d_out, slots, ranks, base, runs, dtype):
    pool, slot, slot_rank, A, B, X, W = _case(n, d_in, d_out, slots, ranks, base, runs, 11)
    segs = mlora.DeviceSegments(mlora.build_segments(slot, pool), n, DEVICE)
    Xd = X.to(DEVICE)
    Xq, Wq = mlora.mx_quantize(Xd), mlora.mx_quantize(W.to(DEVICE))
    Y = torch.full((n, d_out), float("nan"), dtype=dtype, device=DEVICE)
    mlora.mx_gemm_apply(pool, segs, Xd, Xq, Wq, Y)
    assert pool.check() == 0
    rows = None
    if n > 1000:   # the reference of some rows: each tile's first and last, and every 37th
        rows = np.unique(np.concatenate([np.arange(0, n, 128), np.arange(127, n, 128), np.arange(0, n, 37), [n - 1]]))
        assert not torch.isnan(Y).any()
        Y = Y[torch.from_numpy(rows).to(DEVICE)]
    _assert_product(Y, *_reference(slot, slot_rank, A, B, X, W, rows), d_in)
    free()


def test_product_strided_operands():
    n, d_in, d_out = 77, 264, 144
    pool, slot, slot_rank, A, B, X, W = _case(n, d_in, d_out, 4, (16,), 0.2, False, 31)
    segs = mlora.DeviceSegments(mlora.build_segments(slot, pool), n, DEVICE)
    Xw = torch.zeros(n, 400, dtype=torch.bfloat16, device=DEVICE)
    Xd = Xw[:, 64:64 + d_in]
    Xd.copy_(X)
    codes = torch.full((n, 192), 0xff, dtype=torch.uint8, device=DEVICE)[:, 16:160]   # rows 192 bytes apart
    Xq = mlora.mx_quantize(Xd, out=mlora.MxMatrix(n, d_in, codes=codes))
    Wq = mlora.mx_quantize(W.to(DEVICE))
    Yw = torch.full((n, 200), 7.0, dtype=torch.bfloat16, device=DEVICE)
    Y = Yw[:, 8:8 + d_out]
    mlora.mx_gemm_apply(pool, segs, Xd, Xq, Wq, Y)
    _assert_product(Y, *_reference(slot, slot_rank, A, B, X, W), d_in)
    assert (Yw[:, :8] == 7).all() and (Yw[:, 8 + d_out:] == 7).all()


def test_product_rejected_segments_get_the_base_product():
    n, d_in, d_out = 200, 256, 256
    pool, slot, slot_rank, A, B, X, W = _case(n, d_in, d_out, 4, (16,), 0.0, False, 41)
    meta = mlora.build_segments(slot, pool)
    pool.clear_slot(2)
    segs = mlora.DeviceSegments(meta, n, DEVICE)
    Xd = X.to(DEVICE)
    Y = torch.full((n, d_out), float("nan"), dtype=torch.float32, device=DEVICE)
    mlora.mx_gemm_apply(pool, segs, Xd, mlora.mx_quantize(Xd), mlora.mx_quantize(W.to(DEVICE)), Y)
    assert pool.check() & mlora.FLAG_SLOT_EMPTY
    slot2 = np.where(slot == 2, -1, slot)
    _assert_product(Y, *_reference(slot2, slot_rank, A, B, X, W), d_in)


def test_nan_scale_and_nan_rows_stay_in_their_row():
    n, d_in, d_out = 130, 512, 128
    X, W = _integers(n, d_in, 5), _integers(d_out, d_in, 6)
    Xt = torch.from_numpy(X).to(DEVICE, torch.bfloat16)
    Xt[129, 3] = float("nan")
    Xt[7, 500] = float("inf")
    pool = mlora.Pool(d_in, d_out, 1, 8)
    Y = torch.zeros(n, d_out, dtype=torch.float32, device=DEVICE)
    mlora.mx_gemm_apply(pool, None, None, mlora.mx_quantize(Xt), mlora.mx_quantize(torch.from_numpy(W).float().to(DEVICE)), Y)
    want = torch.from_numpy(X @ W.T)
    good = torch.ones(n, dtype=torch.bool)
    good[[7, 129]] = False
    assert torch.equal(Y.cpu().double()[good], want[good])
    assert torch.isnan(Y[[7, 129]]).all()


def test_capture_replay_and_other_stream():
    n, d_in, d_out = 96, 512, 384
    pool, slot, slot_rank, A, B, X, W = _case(n, d_in, d_out, 6, (16,), 0.1, False, 51)
    segs = mlora.DeviceSegments(mlora.build_segments(slot, pool), n, DEVICE)
    Wq = mlora.mx_quantize(W.to(DEVICE))
    Xd = X.to(DEVICE)
    Xq = mlora.MxMatrix(n, d_in, DEVICE)
    Y = torch.zeros(n, d_out, dtype=torch.float32, device=DEVICE)

    def step():
        mlora.mx_quantize(Xd, out=Xq)
        mlora.mx_gemm_apply(pool, segs, Xd, Xq, Wq, Y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                       # the workspace grows outside the capture
    torch.cuda.current_stream().wait_stream(side)
    _assert_product(Y, *_reference(slot, slot_rank, A, B, X, W), d_in)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    X2 = _rows(n, d_in, torch.bfloat16, 99, spread=1.0)
    Xd.copy_(X2)
    Y.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    _assert_product(Y, *_reference(slot, slot_rank, A, B, X2, W), d_in)
    assert pool.check() == 0


def test_results_do_not_vary():
    n, d_in, d_out = 256, 4096, 512
    pool, slot, slot_rank, A, B, X, W = _case(n, d_in, d_out, 9, (16,), 0.1, False, 61)
    segs = mlora.DeviceSegments(mlora.build_segments(slot, pool), n, DEVICE)
    Xd = X.to(DEVICE)
    Xq, Wq = mlora.mx_quantize(Xd), mlora.mx_quantize(W.to(DEVICE))
    Ys = []
    for _ in range(3):
        Y = torch.zeros(n, d_out, dtype=torch.float32, device=DEVICE)
        mlora.mx_gemm_apply(pool, segs, Xd, Xq, Wq, Y)
        Ys.append(Y)
    assert torch.equal(Ys[0], Ys[1]) and torch.equal(Ys[0], Ys[2])


def test_matches_the_oracle_entry():
    # the base term as the oracle's, on the quantised values: the library's own reference of W
    n, d_in, d_out = 64, 256, 128
    pool, slot, slot_rank, A, B, X, W = _case(n, d_in, d_out, 3, (16,), 0.2, False, 71)
    segs = mlora.DeviceSegments(mlora.build_segments(slot, pool), n, DEVICE)
    Xd = X.to(DEVICE)
    Xq, Wq = mlora.mx_quantize(Xd), mlora.mx_quantize(W.to(DEVICE))
    Y = torch.zeros(n, d_out, dtype=torch.bfloat16, device=DEVICE)
    mlora.mx_gemm_apply(pool, segs, Xd, Xq, Wq, Y)
    y0 = (mlora.mx_dequantize(Xq, dtype=torch.float32).double() @ mlora.mx_dequantize(Wq, dtype=torch.float32).double().T)
    bits = {a: mlora.bf16_bits(A[a]) for a in A}, {a: mlora.bf16_bits(B[a]) for a in B}
    alpha = np.array([2.0 * a + 1.0 for a in range(3)], np.float32)
    ref, flags = oracle.apply_rows_xf64(X.double().numpy(), y0.cpu().numpy(), slot, None, slot_rank, alpha, *bits)
    assert flags == 0
    err = np.abs(Y.cpu().double().numpy() - ref)
    assert (err <= 1e-2 * (1 + np.abs(ref))).all()


def test_graph_outlives_a_grown_workspace():
    # a graph captured while the pool's workspace was small still runs after a larger batch grew it
    n, d_in, d_out = 40, 64, 64
    pool, slot, slot_rank, A, B, X, W = _case(n, d_in, d_out, 3, (64,), 0.0, False, 81)
    segs = mlora.DeviceSegments(mlora.build_segments(slot, pool), n, DEVICE)
    Xd = X.to(DEVICE)
    Xq, Wq = mlora.mx_quantize(Xd), mlora.mx_quantize(W.to(DEVICE))
    Y = torch.zeros(n, d_out, dtype=torch.float32, device=DEVICE)
    mlora.mx_gemm_apply(pool, segs, Xd, Xq, Wq, Y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mlora.mx_gemm_apply(pool, segs, Xd, Xq, Wq, Y)
    big = 9000                      # 9000 x 64 fp32 of H: more than the first MiB
    slot2 = np.resize(slot, big).astype(np.int32)
    X2 = _rows(big, d_in, torch.bfloat16, 5, spread=1.0)
    segs2 = mlora.DeviceSegments(mlora.build_segments(slot2, pool), big, DEVICE)
    X2d = X2.to(DEVICE)
    Y2 = torch.full((big, d_out), float("nan"), dtype=torch.float32, device=DEVICE)
    mlora.mx_gemm_apply(pool, segs2, X2d, mlora.mx_quantize(X2d), Wq, Y2)
    filler = [torch.full((1 << 18,), float("nan"), device=DEVICE) for _ in range(8)]
    Y.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    _assert_product(Y, *_reference(slot, slot_rank, A, B, X, W), d_in)
    rows = np.arange(0, big, 111)
    _assert_product(Y2[torch.from_numpy(rows).to(DEVICE)], *_reference(slot2, slot_rank, A, B, X2, W, rows), d_in)
    assert pool.check() == 0
    del filler


@pytest.mark.parametrize("n_rows", [200, 34000])
def test_row_lookup_of_many_segments_and_rows(n_rows):
    """More segments than a block keeps in shared memory, and more rows than the one-launch lookup
    takes: every row its own segment (200 rows; the adapters' slots repeat), or runs of 16."""
    d, n_slots = 64, 7
    run = 1 if n_rows <= 1024 else 16
    pool, _, slot_rank, A, B, X, W = _case(n_rows, d, d, n_slots, (8, 16), 0.0, False, 91)
    seg_slot = np.random.default_rng(5).integers(-1, n_slots, n_rows // run).astype(np.int32)
    # 200 rows: pad with empty segments, so that the list is longer than any table in shared memory
    pad = 3000 if n_rows <= 1024 else 0
    offsets = np.concatenate([np.arange(0, n_rows + 1, run), np.full(pad, n_rows)]).astype(np.int32)
    perm = np.random.default_rng(6).permutation(n_rows).astype(np.int32)
    meta = {"offsets": offsets, "slots": np.concatenate([seg_slot, np.full(pad, -1)]).astype(np.int32),
            "token_indices": perm, "max_segment_rows": run}
    slot = np.empty(n_rows, np.int32)
    slot[perm] = seg_slot.repeat(run)
    segs = mlora.DeviceSegments(meta, n_rows, DEVICE)
    Xd = X.to(DEVICE)
    Y = torch.full((n_rows, d), float("nan"), dtype=torch.float32, device=DEVICE)
    mlora.mx_gemm_apply(pool, segs, Xd, mlora.mx_quantize(Xd), mlora.mx_quantize(W.to(DEVICE)), Y)
    assert pool.check() == 0 and not torch.isnan(Y).any()
    rows = np.arange(0, n_rows, max(1, n_rows // 300))
    _assert_product(Y[torch.from_numpy(rows).to(DEVICE)], *_reference(slot, slot_rank, A, B, X, W, rows), d)
    free()


def test_rows_claimed_twice_or_missing_are_flagged():
    n, d = 96, 64
    pool, _, slot_rank, A, B, X, W = _case(n, d, d, 2, (16,), 0.0, False, 95)
    ti = np.arange(n, dtype=np.int32)
    ti[50] = 3                       # row 3 named twice, row 50 not at all
    ti[60] = n + 5                   # no such row
    meta = {"offsets": np.array([0, 40, n], np.int32), "slots": np.array([0, 1], np.int32), "token_indices": ti,
            "max_segment_rows": 1}
    segs = mlora.DeviceSegments(meta, n, DEVICE)
    Xd = X.to(DEVICE)
    Y = torch.full((n, d), float("nan"), dtype=torch.float32, device=DEVICE)
    mlora.mx_gemm_apply(pool, segs, Xd, mlora.mx_quantize(Xd), mlora.mx_quantize(W.to(DEVICE)), Y)
    assert pool.check() & mlora.FLAG_BAD_ROW
    slot = np.where(np.arange(n) < 40, 0, 1)
    slot[[50, 60]] = -1
    rows = np.array([t for t in range(n) if t != 3])
    _assert_product(Y[torch.from_numpy(rows).to(DEVICE)], *_reference(slot, slot_rank, A, B, X, W, rows), d)


@pytest.mark.parametrize("n,d_out", [(70, 136), (2600, 4104)])   # few rows, and pair tiles
def test_infinities_stay_with_their_rows(n, d_out):
    """An adapter with an infinity in B and an activation row with a NaN reach the rows of that
    adapter and that row alone, although tiles mix rows of many adapters."""
    d_in = 256
    rng = np.random.default_rng(2)
    slot = rng.integers(-1, 5, n).astype(np.int32)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s) * 0.1).to(torch.bfloat16)   # noqa: E731
    A, B = {a: bf(16, d_in) for a in range(5)}, {a: bf(d_out, 16) for a in range(5)}
    B[3][7, 2] = float("inf")
    pool = mlora.Pool(d_in, d_out, 5, 16)
    for a in range(5):
        pool.load_slot(a, 16, 2.0 * a + 1.0, A[a].to(DEVICE), B[a].to(DEVICE))
    X, W = _rows(n, d_in, torch.bfloat16, 7, spread=1.0), _rows(d_out, d_in, torch.float32, 8, spread=1.0) * 0.05
    nan_row = int(np.nonzero(slot == 1)[0][0])
    clean = X.clone()
    X[nan_row, 9] = float("nan")
    segs = mlora.DeviceSegments(mlora.build_segments(slot, pool), n, DEVICE)
    Xd = X.to(DEVICE)
    Y = torch.zeros(n, d_out, dtype=torch.float32, device=DEVICE)
    mlora.mx_gemm_apply(pool, segs, Xd, mlora.mx_quantize(Xd), mlora.mx_quantize(W.to(DEVICE)), Y)
    assert pool.check() == 0
    bad = ~torch.isfinite(Y).cpu().numpy()
    want = np.zeros((n, d_out), bool)
    want[slot == 3, 7] = True
    want[nan_row] = True
    assert np.array_equal(bad, want)
    rows = np.array([t for t in range(0, n, max(1, n // 200)) if slot[t] != 3 and t != nan_row])
    _assert_product(Y[torch.from_numpy(rows).to(DEVICE)], *_reference(slot, slot_rank_of(16, 5), A, B, clean, W, rows), d_in)


def slot_rank_of(rank, n):
    return np.full(n, rank, np.int32)


def test_other_stream_and_two_pools_at_once():
    """Two pools' products on two streams at once, each with its own workspace."""
    cases = []
    for seed, n in ((3, 150), (4, 300)):
        pool, slot, slot_rank, A, B, X, W = _case(n, 512, 256, 5, (16,), 0.1, False, 100 + seed)
        segs = mlora.DeviceSegments(mlora.build_segments(slot, pool), n, DEVICE)
        cases.append((pool, slot, slot_rank, A, B, X, W, segs, X.to(DEVICE), mlora.mx_quantize(W.to(DEVICE)),
                      torch.full((n, 256), float("nan"), device=DEVICE)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for st, (pool, _, _, _, _, _, _, segs, Xd, Wq, Y) in zip(streams, cases):
            Xq = mlora.mx_quantize(Xd, stream=st)
            mlora.mx_gemm_apply(pool, segs, Xd, Xq, Wq, Y, stream=st)
    torch.cuda.synchronize()
    for pool, slot, slot_rank, A, B, X, W, _, _, _, Y in cases:
        assert pool.check() == 0
        _assert_product(Y, *_reference(slot, slot_rank, A, B, X, W), 512)


def test_a_long_matrix_passes_32_bits():
    """Offsets past 2^32 bytes: rows near the end of a matrix of 4.3 G elements."""
    n, d = 524300, 8192                # 8.6 GB of bf16, 2.1 GB of codes
    X = torch.zeros(n, d, dtype=torch.bfloat16, device=DEVICE)
    tail = _rows(40, d, torch.bfloat16, 3).to(DEVICE)
    X[-40:] = tail
    Q = mlora.mx_quantize(X)
    values = mx_ref.quantize(tail.double().cpu().numpy())[2]
    back = mlora.mx_dequantize(Q, out=X)
    assert torch.equal(back[-40:].double().cpu(), torch.from_numpy(values)) and not back[:1000].any()
    pool = mlora.Pool(d, 64, 1, 8)
    W = _rows(64, d, torch.float32, 4, spread=1.0)
    Wq = mlora.mx_quantize(W.to(DEVICE))
    Y = torch.full((n, 64), float("nan"), dtype=torch.float32, device=DEVICE)
    mlora.mx_gemm_apply(pool, None, None, Q, Wq, Y)
    assert pool.check() == 0 and not Y[:-40].any()
    w = mx_ref.quantize(W.double().numpy())[2]
    _assert_product(Y[-40:], values @ w.T, np.abs(values) @ np.abs(w).T, np.zeros((40, 64)), d)
    del X, Q, back, Y
    free()
