"""Timed cases of the 4-bit microscaled base layer and of the device-side row grouping.

Each case names one operator and its sizes; `run` computes it either in plain torch
(`own` false) or through this library's entry points (`own` true):

  round_trip   mx_quantize, then mx_dequantize: rows to 4-bit e2m1 codes with one
               power-of-two scale per 32 elements, and back to the values they stand for
  product      mx_quantize of the activations, then mx_gemm_apply: the base projection of
               4-bit activations and 4-bit weights plus each row's LoRA delta
  group        group_rows, then gather_rows: rows (or a router's top-k choices) sorted by
               adapter slot on the device, and the rows brought into that order
  combine      combine_rows: every row's weighted sum over its choices, back in row order
  combine_grad combine_rows_backward: its gradients, to the grouped rows and the weights

The 4-bit format (OCP microscaling, MXFP4): a block of 32 consecutive elements of a row
has the scale 2^e, e = floor(log2(max|x|)) - 2 clamped to [-127, 127], stored as e + 127;
each element is x / 2^e rounded to the nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6} (ties to the
even code, larger values to 6), two codes to a byte, the first in the low half.  The scales
are kept in tiles of 128 rows x 4 blocks: [ceil(n/128)][2 ceil(d/256)][32][4][4], where
row r of a tile and block b are at [r % 32][r // 32][b].
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's activations on their way into a 4096-wide 4-bit layer
        {"name": "round_trip_decode", "op": "round_trip", "n": 256, "d": 4096, "dtype": "bf16"},
        # an up projection's weights being quantised when a model is loaded
        {"name": "round_trip_weight", "op": "round_trip", "n": 14336, "d": 4096, "dtype": "bf16"},
        # one new token of one request through a 4096 x 4096 projection
        {"name": "product_one_row", "op": "product", "n": 1, "d_in": 4096, "d_out": 4096, "slots": 64, "rank": 16,
         "base": 0.0, "runs": False, "dtype": "bf16"},
        # the decode batch of the q projection: 256 rows in arrival order over 64 adapters
        {"name": "product_decode", "op": "product", "n": 256, "d_in": 4096, "d_out": 4096, "slots": 64, "rank": 16,
         "base": 0.1, "runs": False, "dtype": "bf16"},
        # prefill of a few requests, a total that fits no tile, into an fp16 model's up projection
        {"name": "product_prefill_odd", "op": "product", "n": 1999, "d_in": 4096, "d_out": 14336, "slots": 8,
         "rank": 64, "base": 0.0, "runs": True, "dtype": "fp16"},
        # a full prefill batch of the 8192-wide model's up projection
        {"name": "product_prefill", "op": "product", "n": 4096, "d_in": 8192, "d_out": 28672, "slots": 8, "rank": 64,
         "base": 0.0, "runs": True, "dtype": "bf16"},
        # a decode batch whose adapters are known on the device only
        {"name": "group_decode", "op": "group", "n": 256, "k": 1, "d": 4096, "slots": 64, "dtype": "bf16"},
        # a prefill batch routed to two of 128 adapters a token
        {"name": "group_prefill", "op": "group", "n": 8192, "k": 2, "d": 8192, "slots": 128, "dtype": "bf16"},
        # the way back, for a decode batch and for a prefill batch with four choices a token
        {"name": "combine_decode", "op": "combine", "n": 256, "k": 2, "d": 4096, "slots": 64, "dtype": "bf16"},
        {"name": "combine_prefill", "op": "combine", "n": 8192, "k": 4, "d": 8192, "slots": 128, "dtype": "bf16"},
        # a training step of the router: a small ragged batch in 32 bits, a large one in bf16
        {"name": "combine_grad_small", "op": "combine_grad", "n": 509, "k": 2, "d": 4096, "slots": 16, "dtype": "fp32"},
        {"name": "combine_grad_large", "op": "combine_grad", "n": 8192, "k": 4, "d": 8192, "slots": 128,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["round_trip", "product", "product", "product", "group", "combine", "combine_grad"])
    if op == "round_trip":
        while True:
            n, d = _log(rng, 1, 14336), 8 * _log(rng, 1, 1024)
            if 8 <= n * d <= 14336 * 4096:
                return {"op": op, "n": n, "d": d, "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "product":
        while True:
            n, d_in, d_out = _log(rng, 1, 4096), 8 * _log(rng, 32, 1024), 8 * _log(rng, 32, 3584)
            if n * d_in * d_out <= 4096 * 8192 * 28672 // 2:
                return {"op": op, "n": n, "d_in": d_in, "d_out": d_out, "slots": _log(rng, 1, 64),
                        "rank": rng.choice([1, 8, 12, 16, 32, 64]), "base": rng.choice([0.0, 0.1, 0.5]),
                        "runs": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    while True:
        n, k, d = _log(rng, 1, 32768), rng.choice([1, 2, 3, 4, 8]), 8 * _log(rng, 16, 1024)
        slots = _log(rng, max(2, k), 1024)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if n * k * d * SIZES[dtype] <= 8192 * 4 * 8192 * 2 and n * slots <= 1 << 24:
            return {"op": op, "n": n, "k": k, "d": d, "slots": slots, "dtype": dtype}


# ------------------------------------------------------------------ inputs
def _zipf(n, device):
    return torch.arange(1, n + 1, dtype=torch.float32, device=device) ** -1.1


def _activations(n, d, dtype, g):
    """Rows as a transformer layer's input has them: normal, with a few large channels."""
    x = torch.randn(n, d, generator=g, device=DEVICE)
    gain = torch.ones(d, device=DEVICE)
    gain[torch.randint(0, d, (max(1, d // 256),), generator=g, device=DEVICE)] = 12.0
    return (x * gain).to(DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    s = {"case": dict(case)}
    op = case["op"]
    if op == "round_trip":
        s["X"] = _activations(case["n"], case["d"], case["dtype"], g)
        return s
    if op == "product":
        n, d_in, d_out, slots, rank = case["n"], case["d_in"], case["d_out"], case["slots"], case["rank"]
        s["X"] = _activations(n, d_in, "bf16", g)
        # the weights as a checkpoint in this format keeps them
        W = torch.randn(d_out, d_in, generator=g, device=DEVICE).mul_(0.02)
        s["codes"], s["scales"] = _pack(*_quantize(W))
        del W
        s["A"] = (0.02 * torch.randn(slots, rank, d_in, generator=g, device=DEVICE)).to(torch.bfloat16)
        s["B"] = (0.02 * torch.randn(slots, d_out, rank, generator=g, device=DEVICE)).to(torch.bfloat16)
        s["alpha"] = 2.0 * rank
        slot = torch.multinomial(_zipf(slots, DEVICE), n, replacement=True, generator=g).to(torch.int32)
        if case["runs"]:
            slot = torch.sort(slot).values   # each request's rows stand together
        base = torch.rand(n, generator=g, device=DEVICE) < case["base"]
        s["slot"] = torch.where(base, torch.full_like(slot, -1), slot)
        s["Y"] = torch.empty(n, d_out, dtype=DTYPES[case["dtype"]], device=DEVICE)
        if own:   # what a serving program keeps: the adapter pool, the batch's segments, the weights' handle
            import segmented_rank_gemm_02_b200 as mlora
            s["pool"] = mlora.Pool(d_in, d_out, slots, rank)
            for a in range(slots):
                s["pool"].load_slot(a, rank, s["alpha"], s["A"][a], s["B"][a])
            meta = mlora.build_segments(s["slot"].cpu().numpy(), s["pool"])
            s["segs"] = mlora.DeviceSegments(meta, n, DEVICE)
            s["W"] = mlora.MxMatrix(d_out, d_in, codes=s["codes"], scales=s["scales"])
        return s
    n, k, d, slots = case["n"], case["k"], case["d"], case["slots"]
    p = _zipf(slots, DEVICE).expand(n, slots)
    slot = torch.multinomial(p, k, replacement=False, generator=g).to(torch.int32)
    base = torch.rand(n, k, generator=g, device=DEVICE) < 0.05
    s["slot"] = torch.where(base, torch.full_like(slot, -1), slot).contiguous()
    if op == "group":
        s["X"] = _activations(n, d, case["dtype"], g)
    else:
        s["Ys"] = torch.randn(n * k, d, generator=g, device=DEVICE).to(DTYPES[case["dtype"]])
        s["weights"] = torch.softmax(torch.randn(n, k, generator=g, device=DEVICE), 1)
        order = torch.sort(s["slot"].reshape(-1), stable=True).indices
        s["positions"] = torch.empty(n * k, dtype=torch.int64, device=DEVICE)
        s["positions"][order] = torch.arange(n * k, device=DEVICE)
        if op == "combine_grad":
            s["dY"] = torch.randn(n, d, generator=g, device=DEVICE).to(DTYPES[case["dtype"]])
    if own:   # the pool whose slots the rows are grouped by; the forward pass's groups
        import segmented_rank_gemm_02_b200 as mlora
        s["pool"] = mlora.Pool(8, 8, slots, 8)
        if op != "group":
            s["groups"] = mlora.group_rows(s["pool"], s["slot"])
    return s


# ------------------------------------------------------------------ plain forms
def _blocks(X):
    n, d = X.shape
    return torch.nn.functional.pad(X.float(), (0, -d % 32)).view(n, -1, 32)


def _times_pow2(x, e):
    """x 2^e for whole e, without rounding: two factors, each a normal fp32 power of two."""
    half = torch.div(e, 2, rounding_mode="floor")
    return x * ((half + 127) << 23).view(torch.float32) * ((e - half + 127) << 23).view(torch.float32)


def _quantize(X):
    """Codes 0..15 (uint8) [n, d rounded up to 32] and scale exponents (int32) [n, blocks]."""
    x = _blocks(X)
    amax = x.abs().amax(2)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32))
    e = e.clamp(-127, 127)
    a = _times_pow2(x, -e.unsqueeze(2))
    neg = torch.signbit(a)
    a = a.abs_()
    code = (a > 0.25).to(torch.uint8)
    for t, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= t) if even else (a > t)
    return (code + 8 * neg.to(torch.uint8)).view(x.shape[0], -1), e


def _pack(code, e):
    """Two codes to a byte; the scale bytes in tiles."""
    n, blocks = e.shape
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    tiles = 2 * -(-blocks // 8)
    b = torch.zeros(-(-n // 128) * 128, tiles * 4, dtype=torch.uint8, device=e.device)
    b[:n, :blocks] = (e + 127).to(torch.uint8)
    return packed.contiguous(), b.view(-1, 4, 32, tiles, 4).permute(0, 3, 2, 1, 4).contiguous()


def _values(code, e, d):
    """The fp32 values that codes and exponents stand for."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=code.device)
    v = table[code.to(torch.int32)].view(code.shape[0], -1, 32)
    return _times_pow2(v, e.unsqueeze(2)).view(code.shape[0], -1)[:, :d]


def _unpack(codes, scales, n, d):
    code = torch.stack((codes & 15, codes >> 4), 2).view(n, -1)
    e = scales.permute(0, 3, 2, 1, 4).reshape(scales.shape[0] * 128, -1)[:n, :code.shape[1] // 32].to(torch.int32) - 127
    return _values(code, e, d)


def _delta(X, slot, A, B, alpha):
    """s (X A^T) B^T of each row's own adapter: all adapters' products, the others' masked out."""
    S, r, d_in = A.shape
    h = (X.float() @ A.float().view(S * r, d_in).T).view(-1, S, r)
    mine = slot.unsqueeze(1) == torch.arange(S, device=slot.device)
    h = (h * mine.unsqueeze(2) * (alpha / r)).view(-1, S * r)
    return h @ B.float().transpose(0, 1).reshape(-1, S * r).T


def _group(slot, n_slots):
    flat = slot.reshape(-1)
    N = flat.numel()
    order = torch.sort(flat, stable=True).indices
    positions = torch.empty_like(order)
    positions[order] = torch.arange(N, device=order.device)
    counts = torch.zeros(n_slots + 1, dtype=torch.int64, device=flat.device)
    counts.scatter_add_(0, (flat + 1).long(), torch.ones_like(flat, dtype=torch.int64))
    first = torch.sort((counts == 0).to(torch.int32), stable=True).indices[:min(n_slots + 1, N)]
    slots = torch.where(counts[first] > 0, first - 1, torch.full_like(first, -1))
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device=flat.device), torch.cumsum(counts[first], 0)))
    return tuple(t.to(torch.int32) for t in (offsets, slots, order, positions))


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import segmented_rank_gemm_02_b200 as mlora
        if op == "round_trip":
            return mlora.mx_dequantize(mlora.mx_quantize(state["X"]), dtype=state["X"].dtype)
        if op == "product":
            Xq = mlora.mx_quantize(state["X"])
            mlora.mx_gemm_apply(state["pool"], state["segs"], state["X"], Xq, state["W"], state["Y"])
            return state["Y"]
        if op == "group":
            gr = mlora.group_rows(state["pool"], state["slot"])
            rows = mlora.gather_rows(gr, state["X"])
            return {"offsets": gr.offsets, "slots": gr.slots, "order": gr.order, "positions": gr.positions, "rows": rows}
        if op == "combine":
            return mlora.combine_rows(state["groups"], state["Ys"], state["weights"])
        dYs, dw = mlora.combine_rows_backward(state["groups"], state["dY"], state["Ys"], state["weights"])
        return {"dYs": dYs, "dweights": dw}
    if op == "round_trip":
        code, e = _quantize(state["X"])
        return _values(code, e, c["d"]).to(state["X"].dtype)
    if op == "product":
        code, e = _quantize(state["X"])
        W = _unpack(state["codes"], state["scales"], c["d_out"], c["d_in"])
        Y = _values(code, e, c["d_in"]) @ W.T
        Y += _delta(state["X"], state["slot"], state["A"], state["B"], state["alpha"])
        state["Y"].copy_(Y)
        return state["Y"]
    if op == "group":
        offsets, slots, order, positions = _group(state["slot"], c["slots"])
        rows = state["X"][torch.div(order, c["k"], rounding_mode="floor").long()]
        return {"offsets": offsets, "slots": slots, "order": order, "positions": positions, "rows": rows}
    mine = state["Ys"][state["positions"]].float().view(c["n"], c["k"], c["d"])
    if op == "combine":
        return (mine * state["weights"].unsqueeze(2)).sum(1).to(state["Ys"].dtype)
    dY = state["dY"].float()
    dYs = torch.empty_like(state["Ys"])
    dYs[state["positions"]] = (state["weights"].unsqueeze(2) * dY.unsqueeze(1)).to(dYs.dtype).view(-1, c["d"])
    return {"dYs": dYs, "dweights": (mine * dY.unsqueeze(1)).sum(2)}


# ------------------------------------------------------------------ work
def _mx_bytes(n, d):
    return n * (-(-d // 32)) * 17


def work(case):
    op = case["op"]
    size = SIZES[case["dtype"]]
    n = case["n"]
    if op == "round_trip":
        d = case["d"]
        return {"bytes": 2 * n * d * size + _mx_bytes(n, d), "flops": 4 * n * d}
    if op == "product":
        d_in, d_out, r = case["d_in"], case["d_out"], case["rank"]
        rows = n * (1 - case["base"])
        used = min(case["slots"], max(1, rows))
        return {"bytes": 2 * n * d_in + _mx_bytes(n, d_in) + _mx_bytes(d_out, d_in) + used * r * (d_in + d_out) * 2
                + n * d_out * size, "flops": 2 * n * d_in * d_out + 2 * rows * r * (d_in + d_out)}
    k, d = case["k"], case["d"]
    if op == "group":
        return {"bytes": 4 * n * k * 3 + n * d * size + n * k * d * size, "flops": n * k}
    if op == "combine":
        return {"bytes": n * k * d * size + n * d * size + 8 * n * k, "flops": 2 * n * k * d}
    return {"bytes": 2 * n * k * d * size + n * d * size + 12 * n * k, "flops": 3 * n * k * d}


# ------------------------------------------------------------------ in 64 bits
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _power(e):
    """2^e in fp64 for whole e: the number whose bits have that exponent."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(X):
    """The definition, element by element: the power of two below the block's largest
    magnitude, and the nearer of the two neighbouring levels."""
    n, d = X.shape
    x = torch.zeros(n, -(-d // 32) * 32, dtype=torch.float64, device=X.device)
    x[:, :d] = X.double()
    x = x.view(n, -1, 32)
    big = x.abs().max(2).values
    e = (big.view(torch.int64) >> 52) - 1023.0 - 2   # the exponent in a positive fp64's bits
    e = torch.where(big > 0, e, torch.full_like(e, -127.0)).clamp(-127, 127)
    step = _power(e).unsqueeze(2)
    a = (x / step).abs()
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=X.device)
    lo = torch.searchsorted(levels, a, right=True) - 1
    hi = (lo + 1).clamp(max=7)
    down, up = a - levels[lo], levels[hi] - a
    take_up = (up < down) | ((up == down) & (lo % 2 == 1))
    v = torch.where(take_up, levels[hi], levels[lo])
    return (torch.sign(x) * v * step).view(n, -1)[:, :d]


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], case["op"]
    if op == "round_trip":
        return _exact_values(s["X"])
    if op == "product":
        t = s["scales"]
        rows, blocks = c["d_out"], -(-c["d_in"] // 32)
        r = torch.arange(rows, device=t.device).unsqueeze(1)
        b = torch.arange(blocks, device=t.device).unsqueeze(0)
        e = t[r // 128, b // 4, r % 32, (r % 128) // 32, b % 4].double() - 127
        levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64, device=t.device)
        W = torch.empty(rows, blocks * 32, dtype=torch.float64, device=t.device)
        W[:, 0::2] = levels[(s["codes"] % 16).int()]
        W[:, 1::2] = levels[torch.div(s["codes"], 16, rounding_mode="floor").int()]
        W = (W.view(rows, blocks, 32) * _power(e).unsqueeze(2)).view(rows, -1)[:, :c["d_in"]]
        Y = torch.matmul(_exact_values(s["X"]), W.t())
        slot = s["slot"].cpu()
        for a in range(c["slots"]):
            at = torch.nonzero(slot == a).view(-1).to(t.device)
            if at.numel():
                h = s["X"][at].double() @ s["A"][a].double().t()
                Y[at] += (s["alpha"] / c["rank"]) * (h @ s["B"][a].double().t())
        return Y
    if op == "group":
        rows = s["X"].double().repeat_interleave(c["k"], 0)
        order = torch.argsort(s["slot"].view(-1).long() * (c["n"] * c["k"])
                              + torch.arange(c["n"] * c["k"], device=rows.device))
        return {"offsets": None, "slots": None, "order": None, "positions": None, "rows": rows[order]}
    pos = s["positions"].view(c["n"], c["k"])
    if op == "combine":
        Y = torch.zeros(c["n"], c["d"], dtype=torch.float64, device=pos.device)
        for j in range(c["k"]):
            Y.addcmul_(s["weights"][:, j:j + 1].double(), s["Ys"][pos[:, j]].double())
        return Y
    dY = s["dY"].double()
    dYs = torch.zeros(c["n"] * c["k"], c["d"], dtype=torch.float64, device=pos.device)
    dw = torch.zeros(c["n"], c["k"], dtype=torch.float64, device=pos.device)
    for j in range(c["k"]):
        dYs[pos[:, j]] = s["weights"][:, j:j + 1].double() * dY
        dw[:, j] = torch.linalg.vecdot(s["Ys"][pos[:, j]].double(), dY)
    return {"dYs": dYs, "dweights": dw}
