"""Rows grouped by slot on the device, gathered and combined, against plain references.

Grouping and gathering are exact.  combine sums top_k products in fp32: at most top_k + 1
roundings of 2^-24 of the sum of magnitudes, and one to the output's type; a weight's gradient
sums d products in fp32, at most d roundings of 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import mx_ref
import segmented_rank_gemm_02_b200 as mlora
from gpu_harness import DEVICE, free

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def _slots(n, k, n_slots, seed, base=0.1):
    rng = np.random.default_rng(seed)
    s = np.minimum(rng.zipf(1.3, (n, k)) - 1, n_slots - 1).astype(np.int32)
    s[rng.random((n, k)) < base] = -1
    return s


def _check_groups(gr, slots, n_slots):
    offsets, ids, order, positions = mx_ref.group(slots, n_slots)
    assert np.array_equal(gr.offsets.cpu().numpy(), offsets)
    assert np.array_equal(gr.slots.cpu().numpy(), ids)
    assert np.array_equal(gr.order.cpu().numpy(), order)
    assert np.array_equal(gr.positions.cpu().numpy(), positions)


@pytest.mark.parametrize("n,k,n_slots", [(1, 1, 1), (1, 1, 64), (1, 8, 3), (31, 1, 5), (32, 1, 1), (33, 2, 40), (256, 1, 64),
                                         (1000, 3, 7), (1024, 1, 1024), (1025, 1, 4), (4099, 2, 128), (8192, 4, 1000),
                                         (20000, 1, 12000), (70001, 8, 33)])
def test_group_rows(n, k, n_slots):
    pool = mlora.Pool(8, 8, n_slots, 8)
    slots = _slots(n, k, n_slots, n + k)
    gr = mlora.group_rows(pool, torch.from_numpy(slots).to(DEVICE))
    _check_groups(gr, slots, n_slots)
    assert pool.check() == 0
    # one slot for everything, and every slot in turn
    for s in (np.full((n, k), n_slots - 1, np.int32), np.full((n, k), -1, np.int32),
              (np.arange(n * k, dtype=np.int32)[::-1] % n_slots).reshape(n, k).copy()):
        mlora.group_rows(pool, torch.from_numpy(s).to(DEVICE), out=gr)
        _check_groups(gr, s, n_slots)
    free()


def test_group_rows_no_rows_and_bad_slots():
    pool = mlora.Pool(8, 8, 5, 8)
    gr = mlora.group_rows(pool, torch.empty(0, dtype=torch.int32, device=DEVICE))
    assert gr.offsets.tolist() == [0] and gr.n_tokens == 0
    s = np.array([3, 7, -1, 5, -2, 0, 2 ** 31 - 1, -2 ** 31, 3], np.int32)
    gr = mlora.group_rows(pool, torch.from_numpy(s).to(DEVICE))
    assert pool.check() == mlora.FLAG_BAD_SLOT
    _check_groups(gr, s, 5)
    assert gr.positions.tolist() == [2, -1, 0, -1, -1, 1, -1, -1, 3] and gr.order.tolist()[4:] == [1, 3, 4, 6, 7]
    X = torch.arange(9 * 8, dtype=torch.float32, device=DEVICE).view(9, 8)
    Xs = torch.full((9, 8), -1.0, device=DEVICE)
    mlora.gather_rows(gr, X, Xs)
    assert torch.equal(Xs[:4], X[gr.order[:4].long()]) and (Xs[4:] == -1).all()   # rows behind the last: as they were
    Y = mlora.combine_rows(gr, Xs, torch.full((9, 1), 2.0, device=DEVICE))
    want = 2 * X
    want[gr.positions < 0] = 0
    assert torch.equal(Y, want)
    dYs, dw = mlora.combine_rows_backward(gr, X, Xs, torch.ones(9, 1, device=DEVICE), dYs=torch.full_like(Xs, 5.0))
    assert (dYs[4:] == 5).all() and (dw.view(-1)[gr.positions < 0] == 0).all()
    assert pool.check() == 0


def test_group_ranks_and_apply():
    """The groups of one slot per row are a batch's segments: same results as the host helper's."""
    rng = np.random.default_rng(3)
    n, d = 300, 256
    pool = mlora.Pool(d, d, 9, 16)
    for a in range(9):
        if a != 4:
            bf = lambda *s: torch.from_numpy(rng.standard_normal(s) * 0.1).to(DEVICE, torch.bfloat16)   # noqa: E731
            pool.load_slot(a, 8 + (a % 2) * 8, 16.0, bf(8 + (a % 2) * 8, d), bf(d, 8 + (a % 2) * 8))
    slots = _slots(n, 1, 9, 5)
    slots[slots == 4] = 2
    X = torch.from_numpy(rng.standard_normal((n, d))).to(DEVICE, torch.bfloat16)
    Y0 = torch.from_numpy(rng.standard_normal((n, d))).to(DEVICE, torch.bfloat16)
    gr = mlora.group_rows(pool, torch.from_numpy(slots[:, 0].copy()).to(DEVICE))
    used = [a for a in gr.slots.tolist()]
    assert gr.ranks.tolist() == [0 if a < 0 else pool.slot_info(a)[0] for a in used]
    Y1, Y2 = Y0.clone(), Y0.clone()
    mlora.apply(pool, gr, X, Y1)
    mlora.apply(pool, mlora.DeviceSegments(mlora.build_segments(slots[:, 0], pool), n, DEVICE), X, Y2)
    assert pool.check() == 0
    # each row's result depends on its adapter alone, and both paths sum in fp32 before one rounding
    assert ((Y1.double() - Y2.double()).abs() <= 2.0 ** -7 * (Y2.double().abs() + 2.0 ** -6)).all()
    base = torch.from_numpy(slots[:, 0] < 0).to(DEVICE)
    assert torch.equal(Y1[base], Y0[base])
    # the rows in grouped order, where a slot's rows stand together, and back
    Ys = mlora.gather_rows(gr, Y0)
    mlora.apply(pool, gr.grouped(), mlora.gather_rows(gr, X), Ys)
    Y3 = mlora.combine_rows(gr, Ys)
    assert pool.check() == 0
    assert ((Y3.double() - Y2.double()).abs() <= 2.0 ** -7 * (Y2.double().abs() + 2.0 ** -6)).all()
    # ranks of another pool may differ: its segments go without them
    other = mlora.Pool(d, 64, 9, 8)
    for a in range(9):
        other.load_slot(a, 4, 4.0, torch.zeros(4, d, dtype=torch.bfloat16, device=DEVICE),
                        torch.zeros(64, 4, dtype=torch.bfloat16, device=DEVICE))
    Z = torch.ones(n, 64, dtype=torch.bfloat16, device=DEVICE)
    mlora.apply(other, mlora.group_rows(pool, torch.from_numpy(slots[:, 0].copy()).to(DEVICE), with_ranks=False), X, Z)
    assert other.check() == 0 and (Z == 1).all()


ROWS = [(1, 1, 8), (1, 2, 4096), (5, 3, 40), (64, 1, 512), (33, 2, 1032), (257, 4, 2048), (100, 8, 256), (40, 5, 8192),
        (9, 2, 16384), (2000, 2, 128)]


def _operands(n, k, d, dtype, seed):
    rng = np.random.default_rng(seed)
    slots = _slots(n, k, 6, seed)
    Ys = torch.from_numpy(rng.standard_normal((n * k, d))).to(dtype)
    w = torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32))
    dY = torch.from_numpy(rng.standard_normal((n, d))).to(dtype)
    return slots, Ys, w, dY


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,k,d", ROWS)
def test_gather_combine_and_gradients(n, k, d, dtype):
    pool = mlora.Pool(8, 8, 6, 8)
    slots, Ys, w, dY = _operands(n, k, d, dtype, n * k + d)
    gr = mlora.group_rows(pool, torch.from_numpy(slots).to(DEVICE))
    pos = torch.from_numpy(mx_ref.group(slots, 6)[3]).view(n, k)
    Xs = mlora.gather_rows(gr, dY.to(DEVICE))
    want = torch.empty(n * k, d, dtype=dtype)
    want[pos.view(-1)] = dY.repeat_interleave(k, 0)
    assert torch.equal(Xs.cpu(), want)
    for weights in (w, None):
        wv = (w if weights is not None else torch.ones(n, k)).double()
        parts = wv.unsqueeze(2) * Ys.double()[pos]
        ref, mag = parts.sum(1), parts.abs().sum(1)
        got = mlora.combine_rows(gr, Ys.to(DEVICE), None if weights is None else w.to(DEVICE)).cpu()
        sums = (k + 1) * 2.0 ** -24 * mag
        assert got.dtype == dtype
        assert ((got.double() - ref).abs() <= HALF_STEP[dtype] * (ref.abs() + sums) + sums + TINY[dtype]).all()
        dYs, dw = mlora.combine_rows_backward(gr, dY.to(DEVICE), Ys.to(DEVICE), None if weights is None else w.to(DEVICE))
        want = torch.empty(n * k, d, dtype=dtype)
        # one product in fp32, one rounding
        want[pos.view(-1)] = (wv.float().unsqueeze(2) * dY.float().unsqueeze(1)).to(dtype).view(n * k, d)
        assert torch.equal(dYs.cpu(), want)
        if weights is None:
            assert dw is None
            continue
        prod = Ys.double()[pos] * dY.double().unsqueeze(1)
        assert ((dw.cpu().double() - prod.sum(2)).abs() <= (d + 1) * 2.0 ** -24 * prod.abs().sum(2)).all()
    assert pool.check() == 0
    free()


def test_gradients_against_differences():
    """Along a random direction the loss <G, combine> changes by <gradient, direction>: it is
    linear in Ys and in the weights, so a difference quotient is exact but for rounding."""
    n, k, d = 50, 3, 64
    pool = mlora.Pool(8, 8, 6, 8)
    slots, Ys, w, G = _operands(n, k, d, torch.float32, 77)
    gr = mlora.group_rows(pool, torch.from_numpy(slots).to(DEVICE))
    Ys, w, G = Ys.to(DEVICE), w.to(DEVICE), G.to(DEVICE)
    dYs, dw = mlora.combine_rows_backward(gr, G, Ys, w)
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(1)
    V, v = torch.randn(Ys.shape, generator=gen, device=DEVICE), torch.randn(w.shape, generator=gen, device=DEVICE)
    loss = lambda a, b: (G.double() * mlora.combine_rows(gr, a, b).double()).sum()   # noqa: E731
    # fp32 roundings: 2 (k + 2) 2^-24 of the magnitudes' sum per loss, over a step of 1
    slack = 4 * (k + 2) * 2.0 ** -24 * float((G.abs().double() * mlora.combine_rows(
        gr, Ys.abs() + V.abs(), w.abs() + v.abs()).double()).sum())
    assert abs(float(loss(Ys + V, w) - loss(Ys, w) - (dYs.double() * V.double()).sum())) <= slack
    assert abs(float(loss(Ys, w + v) - loss(Ys, w) - (dw.double() * v.double()).sum())) <= slack
    # gather's gradient: <gather(X), H> = <X, combine(H)>
    X, H = torch.randn(n, d, generator=gen, device=DEVICE), torch.randn(n * k, d, generator=gen, device=DEVICE)
    a = (mlora.gather_rows(gr, X).double() * H.double()).sum()
    b = (X.double() * mlora.combine_rows(gr, H).double()).sum()
    assert abs(float(a - b)) <= (k + 2) * 2.0 ** -24 * float((X.abs().double() * mlora.combine_rows(gr, H.abs()).double()).sum())


def test_strided_rows_and_special_values():
    n, k, d = 21, 2, 72
    pool = mlora.Pool(8, 8, 6, 8)
    slots, Ys, w, dY = _operands(n, k, d, torch.bfloat16, 5)
    gr = mlora.group_rows(pool, torch.from_numpy(slots).to(DEVICE))
    pos = torch.from_numpy(mx_ref.group(slots, 6)[3]).view(n, k)
    wide = torch.full((n * k, 104), 9.0, dtype=torch.bfloat16, device=DEVICE)
    view = wide[:, 16:16 + d]
    view.copy_(Ys)
    Yw = torch.full((n, 88), 9.0, dtype=torch.bfloat16, device=DEVICE)
    mlora.combine_rows(gr, view, w.to(DEVICE), Y=Yw[:, 8:8 + d])
    want = mlora.combine_rows(gr, Ys.to(DEVICE), w.to(DEVICE))
    assert torch.equal(Yw[:, 8:8 + d], want) and (Yw[:, :8] == 9).all() and (Yw[:, 80:] == 9).all()
    # an infinity reaches its own row only, and a weight of zero makes it NaN, as the formula says
    Ys2, w2 = Ys.clone(), w.clone()
    Ys2[pos[3, 1], 7] = float("inf")
    w2[3, 1] = 0.0
    got = mlora.combine_rows(gr, Ys2.to(DEVICE), w2.to(DEVICE)).cpu()
    assert torch.isnan(got[3, 7]) and torch.isfinite(got).sum() == got.numel() - 1


def test_bad_positions_are_skipped_and_flagged():
    pool = mlora.Pool(8, 8, 6, 8)
    gr = mlora.group_rows(pool, torch.zeros(4, 2, dtype=torch.int32, device=DEVICE))
    gr.positions[3] = 8          # outside [0, 8)
    gr.positions[5] = -7
    X = torch.ones(4, 16, device=DEVICE)
    Xs = torch.zeros(8, 16, device=DEVICE)
    mlora.gather_rows(gr, X, Xs)
    assert pool.check() == mlora.FLAG_BAD_ROW
    assert Xs.sum(1).cpu().tolist() == [16, 16, 16, 0, 16, 0, 16, 16]
    assert torch.equal(mlora.combine_rows(gr, Xs)[:, 0].cpu(), torch.tensor([2.0, 1.0, 1.0, 2.0]))
    assert pool.check() == mlora.FLAG_BAD_ROW


def test_mixture_of_adapters_over_a_4bit_layer():
    """The operators together, as a routed layer runs them, captured once and replayed for
    another batch: group -> gather -> quantise -> 4-bit product with each segment's adapter ->
    combine, against 64 bits."""
    n, k, d_in, d_out, n_slots, r = 90, 2, 512, 384, 5, 8
    rng = np.random.default_rng(8)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s) * 0.1).to(torch.bfloat16)   # noqa: E731
    A, B = [bf(r, d_in) for _ in range(n_slots)], [bf(d_out, r) for _ in range(n_slots)]
    pool = mlora.Pool(d_in, d_out, n_slots, r)
    for a in range(n_slots):
        pool.load_slot(a, r, 16.0, A[a].to(DEVICE), B[a].to(DEVICE))
    W = bf(d_out, d_in)
    Wq = mlora.mx_quantize(W.to(DEVICE))
    w64 = mx_ref.quantize(W.double().numpy())[2]
    X = torch.empty(n, d_in, dtype=torch.bfloat16, device=DEVICE)
    slots = torch.empty(n, k, dtype=torch.int32, device=DEVICE)
    weights = torch.empty(n, k, device=DEVICE)
    gr = mlora.RowGroups(pool, n, k, torch.device(DEVICE))
    Xs = torch.empty(n * k, d_in, dtype=torch.bfloat16, device=DEVICE)
    Xq = mlora.MxMatrix(n * k, d_in, DEVICE)
    Ys = torch.empty(n * k, d_out, device=DEVICE)
    Y = torch.empty(n, d_out, device=DEVICE)

    def layer():
        mlora.group_rows(pool, slots, out=gr)
        mlora.gather_rows(gr, X, Xs)
        mlora.mx_quantize(Xs, out=Xq)
        mlora.mx_gemm_apply(pool, gr, Xs, Xq, Wq, Ys)
        mlora.combine_rows(gr, Ys, weights, Y)

    def fill(seed):
        g = np.random.default_rng(seed)
        s = g.permuted(np.tile(np.arange(n_slots), (n, 1)), axis=1)[:, :k].astype(np.int32)
        s[g.random((n, k)) < 0.1] = -1
        x = torch.from_numpy(g.standard_normal((n, d_in))).to(torch.bfloat16)
        w = torch.softmax(torch.from_numpy(g.standard_normal((n, k)).astype(np.float32)), 1)
        X.copy_(x), slots.copy_(torch.from_numpy(s)), weights.copy_(w)
        ref = np.zeros((n, d_out))
        xq = mx_ref.quantize(x.double().numpy())[2]
        for t in range(n):
            for j in range(k):
                y = w64 @ xq[t]
                if s[t, j] >= 0:
                    y = y + 16.0 / r * (B[s[t, j]].double().numpy() @ (A[s[t, j]].double().numpy() @ x[t].double().numpy()))
                ref[t] += float(w[t, j]) * y
        return ref

    def check(ref):
        err = np.abs(Y.cpu().double().numpy() - ref)
        # fp32 sums of d_in products and the low-rank operand's 2^-17, of sums of magnitudes that
        # are at most 2^6 times the largest result here (sqrt(d_in) below 2^5)
        assert (err <= (d_in * 2.0 ** -23 + 2.0 ** -17) * 2.0 ** 6 * np.abs(ref).max()).all()

    ref = fill(1)
    layer()
    check(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for seed in (2, 3):
        ref = fill(seed)
        Y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check(ref)
    assert pool.check() == 0


def test_refusals_with_a_pool():
    """Argument errors that need a pool: returned by the host, nothing launched."""
    import ctypes
    L, bad, unsupported = mlora.lib(), mlora.ERR_INVALID_ARG, mlora.ERR_UNSUPPORTED
    pool = mlora.Pool(64, 128, 3, 8)
    h = pool.handle
    out = ctypes.byref(mlora.RowGroupsStruct(256, 256, None, 256, 256))
    assert L.mlora_group_rows(h, None, 4, 1, out, None) == bad
    assert L.mlora_group_rows(h, 256, -1, 1, out, None) == bad
    assert L.mlora_group_rows(h, 256, 4, 0, out, None) == bad
    assert L.mlora_group_rows(h, 256, 2 ** 30, 4, out, None) == bad
    assert L.mlora_group_rows(h, 256, 4, 1, None, None) == bad
    assert L.mlora_group_rows(h, 256, 4, 1, ctypes.byref(mlora.RowGroupsStruct(256, 256, None, None, 256)), None) == bad
    big = mlora.Pool(8, 8, 12799, 8)
    assert L.mlora_group_rows(big.handle, 256, 4, 1, out, None) == unsupported

    def rows(x=256, ldx=16, dtype=0, d=16, n=4, k=1, xs=512, ldxs=16, pos=256):
        got = (L.mlora_gather_rows(h, pos, n, k, x, ldx, dtype, d, 4, xs, ldxs, None),
               L.mlora_combine_rows(h, pos, None, n, k, xs, ldxs, dtype, d, 4, x, ldx, None),
               L.mlora_combine_rows_backward(h, pos, None, n, k, x, ldx, 1024, 16, dtype, d, 4, xs, ldxs, 2048, None)
               if xs is not None else bad)
        assert got[0] == got[1] == got[2]
        return got[0]

    assert rows(x=None) == bad and rows(xs=None) == bad and rows(pos=None) == bad
    assert rows(ldx=8) == bad and rows(ldxs=8) == bad and rows(ldx=20) == bad and rows(x=264) == bad
    assert rows(dtype=3) == bad and rows(d=0) == bad and rows(k=0) == bad and rows(n=-1) == bad
    assert rows(d=12, ldx=16) == unsupported
    assert rows(n=0) == mlora.OK
    assert L.mlora_combine_rows_backward(h, 256, None, 4, 1, 256, 16, None, 0, 0, 16, 4, None, 0, None, None) == bad
    assert L.mlora_combine_rows_backward(h, 256, None, 4, 1, 256, 16, None, 0, 0, 16, 4, 512, 16, 1024, None) == bad

    q = lambda n, d: mlora.MxStruct(n, d, (d + 31) // 32 * 16, 256, 512)   # noqa: E731
    ref = ctypes.byref

    def gemm(xq=q(4, 64), w=q(128, 64), segs=None, x=None, ldx=64, y=1024, dtype=0, ldy=128):
        return L.mlora_mx_gemm_apply(h, ref(segs) if segs else None, x, ldx, ref(xq), ref(w), y, dtype, ldy, None)

    assert gemm(xq=q(4, 72)) == bad and gemm(w=q(128, 72)) == bad and gemm(w=q(120, 64)) == bad
    assert gemm(y=None) == bad and gemm(y=1032) == bad and gemm(ldy=120) == bad and gemm(ldy=132) == bad
    assert gemm(dtype=mlora.DTYPE_FP8_E4M3) == bad
    seg = mlora.SegmentsStruct(1, 4, 4, 0, 256, 256, None, None, None)
    assert gemm(segs=seg) == bad                              # LoRA without X
    assert gemm(segs=seg, x=256, ldx=60) == bad
    assert gemm(segs=mlora.SegmentsStruct(1, 5, 5, 0, 256, 256, None, None, None), x=256) == bad
    assert gemm(xq=mlora.MxStruct(0, 64, 32, None, None)) == mlora.OK
    assert pool.check() == 0


def test_rows_past_32_bits():
    """Grouped rows whose byte offsets pass 2^32."""
    n, k, d = 140000, 2, 8192            # 280000 grouped rows of 16 KB
    pool = mlora.Pool(8, 8, 3, 8)
    slots = _slots(n, k, 3, 1)
    gr = mlora.group_rows(pool, torch.from_numpy(slots).to(DEVICE))
    pos = gr.positions.view(n, k).long()
    X = torch.zeros(n, d, dtype=torch.bfloat16, device=DEVICE)
    X[:, 5] = (torch.arange(n, device=DEVICE) % 251).to(torch.bfloat16)
    Xs = mlora.gather_rows(gr, X)
    assert torch.equal(Xs[pos.view(-1), 5].view(n, k), X[:, 5:6].expand(n, k))
    Y = mlora.combine_rows(gr, Xs)
    assert torch.equal(Y[:, 5], (2 * X[:, 5].float()).to(torch.bfloat16)) and not Y[:, 6:].any()
    dYs, dw = mlora.combine_rows_backward(gr, X, Xs, torch.ones(n, k, device=DEVICE), dYs=Xs.clone().fill_(7.0))
    assert torch.equal(dYs[pos.view(-1), 5], Xs[pos.view(-1), 5])
    assert torch.equal(dw, (X[:, 5:6].float() ** 2).expand(n, k))
    assert pool.check() == 0
    del X, Xs, Y, dYs
    free()


def test_streams_of_their_own():
    """Outputs allocated for a call on another stream belong to that stream."""
    pool = mlora.Pool(8, 8, 6, 8)
    st = torch.cuda.Stream()
    slots, Ys, w, dY = _operands(500, 2, 256, torch.bfloat16, 9)
    sd, Yd, wd, dYd = (t.to(DEVICE) for t in (torch.from_numpy(slots), Ys, w, dY))
    torch.cuda.synchronize()
    gr = mlora.group_rows(pool, sd, stream=st)
    Xs = mlora.gather_rows(gr, dYd, stream=st)
    Y = mlora.combine_rows(gr, Yd, wd, stream=st)
    dYs, dw = mlora.combine_rows_backward(gr, dYd, Yd, wd, stream=st.cuda_stream)
    torch.cuda.synchronize()
    _check_groups(gr, slots, 6)
    assert torch.equal(Xs, mlora.gather_rows(gr, dYd)) and torch.equal(Y, mlora.combine_rows(gr, Yd, wd))
    a, b = mlora.combine_rows_backward(gr, dYd, Yd, wd)
    assert torch.equal(dYs, a) and torch.equal(dw, b)
