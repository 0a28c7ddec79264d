"""Cases for measuring the 8-bit floating-point products on packed weights and the mixture-of-experts layer for a few
tokens.

Four operators, each in a plain form (elementary torch operations in 32 bits) and as calls of this package:

    moe       router logits and activations of a few tokens -> the whole gated layer's output
    product8  one packed weight with 8-bit values times activations rounded to 8 bits token by token
    experts8  the same, one product per expert over its own ragged range of columns
    quantize8 packed values -> 8-bit values, a scale for each block of 128 (returned as the values they stand for)

Activations are [channels, tokens]; weights are hierarchical N:M (dense, 2:4 and pruned column vectors in
tiles of 64 rows) with a random channel permutation per tile, and importance |W|.  Weight shapes are the
4096 / 11008 linear layers this repository is benchmarked on, and small experts; the sparsities are those of its
workloads.  8-bit values are E4M3 codes times a power of two: the smallest one, within 2^-124 .. 2^119, at which no
value of the block exceeds 448.
"""
import math

import torch

own = False

TILE_ROWS = 64
ALIGN = 8                       # an expert's columns start at a multiple of this
SPARSITIES = ((0.5, 0.25), (0.75, 0.55), (0.75, 0.5), (0.7, 0.51))


def listed():
    return [
        # one sequence's next token through a layer of 8 experts, two of them chosen
        {"name": "moe-token", "op": "moe", "values": "bf16", "hidden": 4096, "inter": 11008, "t_s": 0.75, "v_s": 0.55,
         "experts": 8, "tokens": 1, "top_k": 2, "dtype": "bf16", "renormalize": True, "idle": 0.0},
        # the same through a layer of many small experts: latency
        {"name": "moe-token-small", "op": "moe", "values": "bf16", "hidden": 2048, "inter": 1024, "t_s": 0.5,
         "v_s": 0.25, "experts": 64, "tokens": 1, "top_k": 8, "dtype": "fp32", "renormalize": True, "idle": 0.0},
        # a decode step of 7 slots, some of them without a sequence, 4-bit weights of odd sizes
        {"name": "moe-odd-mx4", "op": "moe", "values": "mx4", "hidden": 1088, "inter": 1472, "t_s": 0.7, "v_s": 0.51,
         "experts": 10, "tokens": 7, "top_k": 3, "dtype": "fp32", "renormalize": False, "idle": 0.3},
        # a decode step of 16 sequences with 8-bit weights: every expert is met
        {"name": "moe-batch-fp8", "op": "moe", "values": "fp8", "hidden": 4096, "inter": 11008, "t_s": 0.75,
         "v_s": 0.55, "experts": 8, "tokens": 16, "top_k": 2, "dtype": "bf16", "renormalize": True, "idle": 0.0},
        # a decode step of 32 sequences
        {"name": "moe-batch", "op": "moe", "values": "bf16", "hidden": 4096, "inter": 11008, "t_s": 0.75, "v_s": 0.55,
         "experts": 8, "tokens": 32, "top_k": 2, "dtype": "bf16", "renormalize": True, "idle": 0.0},
        # one sequence's next token through a down projection
        {"name": "product8-token", "op": "product8", "cout": 4096, "cin": 11008, "t_s": 0.75, "v_s": 0.55, "batch": 1},
        # a decode step of 16 sequences through an up projection
        {"name": "product8-batch", "op": "product8", "cout": 11008, "cin": 4096, "t_s": 0.75, "v_s": 0.55, "batch": 16},
        # a prompt through a down projection, odd length
        {"name": "product8-prompt", "op": "product8", "cout": 4096, "cin": 11008, "t_s": 0.75, "v_s": 0.55,
         "batch": 2047},
        # up projections of 8 experts for a decode step of 33 sequences
        {"name": "experts8-decode", "op": "experts8", "cout": 11008, "cin": 4096, "t_s": 0.75, "v_s": 0.55,
         "experts": 8, "tokens": 33, "top_k": 2},
        # down projections for a prompt: uneven, odd counts
        {"name": "experts8-prompt", "op": "experts8", "cout": 4096, "cin": 11008, "t_s": 0.75, "v_s": 0.55,
         "experts": 8, "tokens": 2047, "top_k": 2},
        # quantising one square projection
        {"name": "quantize8-one", "op": "quantize8", "cout": 4096, "cin": 4096, "t_s": 0.5, "v_s": 0.25, "weights": 1},
        # quantising a layer's 8 experts
        {"name": "quantize8-experts", "op": "quantize8", "cout": 11008, "cin": 4096, "t_s": 0.75, "v_s": 0.55,
         "weights": 8},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _weight(rng):
    while True:
        cout, cin = 64 * _log(rng, 2, 172), 4 * _log(rng, 64, 2752)
        if cout * cin <= 11008 * 4096:
            t_s, v_s = rng.choice(SPARSITIES)
            return {"cout": cout, "cin": cin, "t_s": t_s, "v_s": v_s}


def draw(rng):
    op = rng.choice(["moe", "moe", "moe", "product8", "product8", "experts8", "quantize8"])
    if op == "moe":
        while True:
            hidden, inter, experts = 64 * _log(rng, 2, 64), 64 * _log(rng, 2, 172), _log(rng, 2, 64)
            if hidden * inter * experts <= 4096 * 11008 * 8:
                break
        t_s, v_s = rng.choice(SPARSITIES)
        return {"op": op, "values": rng.choice(["bf16", "mx4", "fp8"]), "hidden": hidden, "inter": inter, "t_s": t_s,
                "v_s": v_s, "experts": experts, "tokens": _log(rng, 1, 32), "top_k": rng.randint(1, min(8, experts)),
                "dtype": rng.choice(["bf16", "fp32"]), "renormalize": rng.random() < 0.5,
                "idle": rng.choice([0.0, 0.0, 0.3])}
    if op == "product8":
        return {"op": op, **_weight(rng), "batch": _log(rng, 1, 2047)}
    if op == "experts8":
        return {"op": op, **_weight(rng), "experts": rng.randint(2, 8), "tokens": _log(rng, 1, 2047),
                "top_k": rng.randint(1, 2)}
    return {"op": op, **_weight(rng), "weights": rng.randint(1, 8)}


# --------------------------------------------------------------------------- inputs

def _counts(cin, t, v):
    """Region counts of a row: dense and 2:4 channels by the closed form."""
    z = math.floor(t * cin + 0.5)
    g = max(0, min(math.floor((t - v) * cin / 2 + 0.5), min(z, cin - z) // 2))
    return cin - z - 2 * g, 4 * g


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _draw_weight(cout, cin, gen):
    """bf16 weight with log-normal channel scales, importance |W|, one channel order per tile."""
    scale = torch.randn(cin, generator=gen, device="cuda").exp()
    w = (torch.randn(cout, cin, generator=gen, device="cuda") * (0.02 * scale)).bfloat16()
    perm = torch.rand(cout // TILE_ROWS, cin, generator=gen, device="cuda").argsort(dim=1)
    return w, w.float().abs(), perm


def _draw_x(channels, columns, gen):
    """Activations: some channels are louder than others."""
    loud = (torch.randn(channels, 1, generator=gen, device="cuda") * 0.5).exp()
    return (torch.randn(channels, columns, generator=gen, device="cuda") * loud).bfloat16()


def _draw_logits(case, gen):
    e, n = case["experts"], case["tokens"]
    logits = torch.randn(e, n, generator=gen, device="cuda") * 2 + torch.randn(e, 1, generator=gen, device="cuda")
    idle = torch.rand(n, generator=gen, device="cuda") < case["idle"]
    logits[:, idle] = float("-inf")                       # slots without a sequence
    return logits.bfloat16() if case["dtype"] == "bf16" else logits


def _draw_ids(case, gen):
    """Experts of every token, [tokens, top_k]: some experts are liked better than others."""
    e, n, k = case["experts"], case["tokens"], case["top_k"]
    like = torch.randn(e, generator=gen, device="cuda") * 0.7
    score = torch.randn(n, e, generator=gen, device="cuda") + like
    return score.topk(k, 1).indices


def _capacity(tokens, top_k, experts):
    """Columns that any routing of these sizes fits into."""
    used = tokens * top_k
    return -(-(used + min(experts, used) * (ALIGN - 1)) // ALIGN) * ALIGN


def _arrange(ids, experts, tokens, top_k):
    """Columns in the order (expert, token), each expert's first column a multiple of ALIGN."""
    hot = torch.zeros(tokens, experts, dtype=torch.int64, device=ids.device).scatter_(1, ids, 1)
    counts = hot.sum(0)
    padded = (counts + ALIGN - 1) // ALIGN * ALIGN
    starts = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    slots = starts[ids] + (hot.cumsum(0) - hot).gather(1, ids)
    src = torch.full((_capacity(tokens, top_k, experts),), -1, dtype=torch.int64, device=ids.device)
    src[slots] = torch.arange(tokens, device=ids.device)[:, None].expand_as(slots)
    return [t.int() for t in (slots, starts, counts, src)]


def _regions(imp, perm, nd, n24):
    """Dense and 2:4 channels of every tile, in the tile's channel order."""
    tiles, cin = perm.shape
    score = imp.view(tiles, TILE_ROWS, cin).double().sum(1)
    order = score.argsort(dim=1, descending=True, stable=True)
    region = torch.full_like(order, 2)
    region.scatter_(1, order[:, :nd], 0)
    region.scatter_(1, order[:, nd:nd + n24], 1)
    cols = perm.gather(1, region.gather(1, perm).argsort(dim=1, stable=True))
    return cols[:, :nd], cols[:, nd:nd + n24]


def _kept(w, imp, perm, nd, n24):
    """Kept values in packed order [tiles, rows, n] with their channels, dense and 2:4."""
    tiles, cin = perm.shape
    idx_d, idx_s = _regions(imp, perm, nd, n24)
    wt, it = w.view(tiles, TILE_ROWS, cin), imp.view(tiles, TILE_ROWS, cin)
    at_d = idx_d[:, None, :].expand(tiles, TILE_ROWS, nd)
    at_s = idx_s[:, None, :].expand(tiles, TILE_ROWS, n24)
    four = it.gather(2, at_s).view(tiles, TILE_ROWS, n24 // 4, 4)
    two = four.argsort(dim=3, descending=True, stable=True)[..., :2].sort(dim=3).values
    val_s = wt.gather(2, at_s).view_as(four).gather(3, two).flatten(2)
    col_s = at_s.reshape(four.shape).gather(3, two).flatten(2)
    return wt.gather(2, at_d), at_d, val_s, col_s


def _pad(v, block):
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % block))


def _power(n):
    """2.0**n in float64 for whole numbers n of the normal range, from its bits."""
    return (n.long() + 1023 << 52).view(torch.float64)


def _fp8(v, top):
    """bf16 values rounded to E4M3 times a power of two; top is the largest magnitude of each one's block."""
    part, power = torch.frexp(top.double())                # top = part * 2**power, part in [0.5, 1)
    scale = torch.where(top > 0, power - 9 + (part > 0.875).int(), -124).clamp(-124, 119)
    a = v.double().abs() * _power(-scale)
    step = _power(torch.frexp(a).exponent.clamp(min=-5) - 4)
    q = ((a / step).round() * step).clamp(max=448.0)
    return (q * v.sign() * _power(scale)).bfloat16()       # exact


def _fp8_rows(v):
    """Values [..., n] in blocks of 128 along n."""
    b = _pad(v, 128)
    b = b.unflatten(-1, (b.shape[-1] // 128, 128))
    return _fp8(b, b.abs().amax(-1, keepdim=True)).flatten(-2)[..., :v.shape[-1]]


def _fp8_columns(x):
    """Activations [channels, tokens] with one scale a token."""
    return _fp8(x, x.abs().amax(0, keepdim=True))


def _mx4_rows(v):
    """Values [..., n] rounded to 4-bit microscaled values in blocks of 32 along n."""
    b = _pad(v, 32).double()
    b = b.unflatten(-1, (b.shape[-1] // 32, 32))
    top = b.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(min=-127)
    a = b.abs() * _power(-scale)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = ((a / step).round() * step).clamp(max=6.0)
    return (q * b.sign() * _power(scale)).bfloat16().flatten(-2)[..., :v.shape[-1]]


_ROUND = {"bf16": lambda v: v, "mx4": _mx4_rows, "fp8": _fp8_rows}


def _dense(w, imp, perm, t_s, v_s, values):
    """The masked weight as a dense bf16 matrix, its kept values rounded to the type of `values`."""
    nd, n24 = _counts(w.shape[1], t_s, v_s)
    val_d, col_d, val_s, col_s = _kept(w, imp, perm, nd, n24)
    out = torch.zeros_like(w).view(perm.shape[0], TILE_ROWS, perm.shape[1])
    out.scatter_(2, col_d, _ROUND[values](val_d))
    out.scatter_(2, col_s, _ROUND[values](val_s))
    return out.view_as(w)


def _blocks(v):
    """[tiles, rows, n] -> the packed layout [tiles, n/32, rows, 32]."""
    v = _pad(v, 32)
    return v.unflatten(2, (v.shape[2] // 32, 32)).transpose(1, 2).contiguous()


def _pack(w, imp, perm, t_s, v_s):
    import structured_sparse_gemm_amd as hinm
    return hinm.pack(w, imp, TILE_ROWS, t_s, v_s, perm.int())


def _stack(packed, values):
    import structured_sparse_gemm_amd as hinm
    stack = hinm.Experts.stack(packed)
    return {"bf16": lambda s: s, "mx4": hinm.quantize_mx4, "fp8": hinm.quantize_fp8}[values](stack)


def _moe_shapes(case):
    """(cout, cin) of the gate, up and down projections."""
    return (case["inter"], case["hidden"]), (case["inter"], case["hidden"]), (case["hidden"], case["inter"])


def prepare(case, seed):
    gen, op = _gen(seed), case["op"]
    state = {"case": case}
    sparse = case["t_s"], case["v_s"]
    if op == "moe":
        state["logits"] = _draw_logits(case, gen)
        state["x"] = _draw_x(case["hidden"], case["tokens"], gen)
        state["w"] = []
        for cout, cin in _moe_shapes(case):
            drawn = (_draw_weight(cout, cin, gen) for _ in range(case["experts"]))
            if own:
                state["w"].append(_stack([_pack(*d, *sparse) for d in drawn], case["values"]))
            else:
                state["w"].append([_dense(*d, *sparse, case["values"]) for d in drawn])
    elif op == "experts8":
        n, k, e = case["tokens"], case["top_k"], case["experts"]
        ids = _draw_ids(case, gen)
        slots, starts, counts, src = _arrange(ids, e, n, k)
        cap = src.numel()
        state["x"] = _draw_x(case["cin"], cap, gen)
        state["y"] = torch.zeros(case["cout"], cap, dtype=torch.bfloat16, device="cuda")
        drawn = (_draw_weight(case["cout"], case["cin"], gen) for _ in range(e))
        if own:
            import structured_sparse_gemm_amd as hinm
            state["routing"] = hinm.Routing(ids=ids.int(), weights=torch.ones(n, k, device="cuda") / k, slots=slots,
                                            starts=starts, counts=counts, src=src)
            state["w"] = _stack([_pack(*d, *sparse) for d in drawn], "fp8")
        else:
            state["ranges"] = list(zip(starts.tolist(), counts.tolist()))
            state["w"] = [_dense(*d, *sparse, "fp8") for d in drawn]
    elif op == "quantize8":
        drawn = (_draw_weight(case["cout"], case["cin"], gen) for _ in range(case["weights"]))
        if own:
            import structured_sparse_gemm_amd as hinm
            state["w"] = hinm.Experts.stack([_pack(*d, *sparse) for d in drawn])
        else:
            kept = [_kept(*d, *_counts(case["cin"], *sparse)) for d in drawn]
            state["w"] = [torch.stack([_blocks(k[i]) for k in kept]) for i in (0, 2)]
    else:
        drawn = _draw_weight(case["cout"], case["cin"], gen)
        state["x"] = _draw_x(case["cin"], case["batch"], gen)
        if own:
            import structured_sparse_gemm_amd as hinm
            state["w"] = hinm.quantize_fp8(_pack(*drawn, *sparse))
        else:
            state["w"] = _dense(*drawn, *sparse, "fp8")
    return state


# --------------------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import structured_sparse_gemm_amd as hinm
    case, op = state["case"], state["case"]["op"]
    if op == "moe":
        return hinm.moe_layer(state["x"], state["logits"], *state["w"], top_k=case["top_k"],
                              renormalize=case["renormalize"])
    if op == "experts8":
        return hinm.spmm_experts(state["w"], state["x"], state["routing"], out=state["y"])
    if op == "quantize8":
        back = hinm.quantize_fp8(state["w"]).dequantize()
        return [back.val_dense.view(torch.bfloat16), back.val_24.view(torch.bfloat16)]
    return hinm.spmm(state["w"], state["x"])


def _router_weights(logits, top_k, renormalize):
    """[experts, tokens]: the chosen experts' weights, 0 elsewhere."""
    key = torch.where(logits.isnan(), float("-inf"), logits)
    top, ids = key.sort(dim=0, descending=True, stable=True)
    top, ids = top[:top_k], ids[:top_k]
    ok = top > float("-inf")
    best = torch.where(ok[:1], top[:1], 0.0)
    part = torch.exp(top - best)
    whole = part if renormalize else torch.exp(key - best)
    weights = torch.where(ok, part / whole.sum(0), 0.0)
    return torch.zeros_like(logits).scatter(0, ids, weights)


def _run_plain(state):
    case, op = state["case"], state["case"]["op"]
    if op == "moe":
        weights = _router_weights(state["logits"].float(), case["top_k"], case["renormalize"])
        x = state["x"].float()
        y = torch.zeros_like(x)
        for gate, up, down, weight in zip(*state["w"], weights):
            g, u = gate.float() @ x, up.float() @ x
            y += torch.where(weight > 0, (down.float() @ (g / (1 + torch.exp(-g)) * u)) * weight, 0.0)
        return y.bfloat16()
    if op == "experts8":
        x = _fp8_columns(state["x"]).float()
        for w, (start, count) in zip(state["w"], state["ranges"]):
            if count:
                state["y"][:, start:start + count] = w.float() @ x[:, start:start + count]
        return state["y"]
    if op == "quantize8":
        out = []
        for v in state["w"]:                               # [weights, tiles, blocks of 32, rows, 32]
            rows = v.transpose(2, 3).flatten(3)
            out.append(_fp8_rows(rows).unflatten(3, (-1, 32)).transpose(2, 3).contiguous() if v.numel() else v)
        return out
    return (state["w"].float() @ _fp8_columns(state["x"]).float()).bfloat16()


# --------------------------------------------------------------------------- the definition in 64 bits

def _e4m3_grid():
    """The 127 magnitudes of E4M3, ascending: 8 below the normal ones, then 8 to a power of two, without 480."""
    grid = [i / 512 for i in range(8)]
    grid += [(8 + m) / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return torch.tensor(grid[:127], dtype=torch.float64, device="cuda")


def _nearest(a, grid):
    """The nearest of an ascending grid's values, half-way cases to the even place in it."""
    half = (grid[1:] + grid[:-1]) / 2
    a = a.contiguous()
    low, high = torch.searchsorted(half, a), torch.searchsorted(half, a, right=True)
    return grid[torch.where(low % 2 == 0, low, high)]


def _exact_fp8(v, dim):
    """float64 values whose blocks lie along `dim`: the scale found by doubling up to the first that fits."""
    top = v.abs().amax(dim, keepdim=True)
    at = torch.full_like(top, 2.0 ** -124)
    for jump in (128, 64, 32, 16, 8, 4, 2, 1):             # the largest scale that is too small, times 2
        at = torch.where(top > 448.0 * at * 2.0 ** (jump - 1), at * 2.0 ** jump, at)
    at = at.clamp(max=2.0 ** 119)
    return _nearest(v.abs() / at, _e4m3_grid()) * at * v.sign()


def _exact_mx4(v):
    top = v.abs().amax(-1, keepdim=True)
    field = top.view(torch.int64) >> 52                    # 1023 + floor(log2(top)) in float64
    unit = (torch.clamp(field - 2, 1023 - 127, 1023 + 127) << 52).view(torch.float64)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    return _nearest(v.abs() / unit, grid) * unit * v.sign()


def _exact_rows(v, values):
    """Kept values [rows, n] of one region in the type of `values`."""
    if values == "bf16":
        return v
    size, n = (128 if values == "fp8" else 32), v.shape[1]
    b = _pad(v, size)
    b = b.view(v.shape[0], b.shape[1] // size, size)
    return (_exact_fp8(b, 2) if values == "fp8" else _exact_mx4(b)).flatten(1)[:, :n]


def _exact_weight(drawn, t_s, v_s, values):
    """Per tile: rank every channel by counting those that beat it; in each 2:4 group keep an entry that fewer
    than two others beat.  Returns the masked weight in float64, and the packed-order values."""
    w, imp, perm = drawn
    cout, cin = w.shape
    nd, n24 = _counts(cin, t_s, v_s)
    out = torch.zeros(cout, cin, dtype=torch.float64, device="cuda")
    dense, pairs = [], []
    low = torch.arange(cin, device="cuda")
    for t in range(perm.shape[0]):
        rows = slice(t * TILE_ROWS, (t + 1) * TILE_ROWS)
        wt, it = w[rows].double(), imp[rows].double()
        score = it.sum(0)
        by = score.sort().values
        ahead = cin - torch.searchsorted(by, score, right=True)
        if bool((by[1:] == by[:-1]).any()):                # equal scores: the lower channel first
            same = (score[:, None] == score[None, :]) & (low[None, :] < low[:, None])
            ahead = ahead + same.sum(1)
        rank = ahead[perm[t]]
        cols_d = perm[t][rank < nd]
        cols_s = perm[t][(rank >= nd) & (rank < nd + n24)]
        fours = it[:, cols_s].view(TILE_ROWS, -1, 4)
        beats = torch.zeros_like(fours)
        for i in range(4):
            for j in range(4):
                if i != j:
                    a, b = fours[..., j], fours[..., i]
                    beats[..., i] += ((a > b) | ((a == b) & (j < i))).double()
        keep = (beats < 2).view(TILE_ROWS, -1)
        vs = wt[:, cols_s]
        vd, packed = _exact_rows(wt[:, cols_d], values), _exact_rows(vs[keep].view(TILE_ROWS, n24 // 2), values)
        out[rows, cols_d] = vd
        full = torch.zeros_like(vs)
        full[keep] = packed.reshape(-1)
        out[rows, cols_s] = full
        dense.append(vd)
        pairs.append(packed)
    return out, torch.stack(dense), torch.stack(pairs)


def _exact_router(logits, top_k, renormalize):
    l = torch.where(logits.isnan(), float("-inf"), logits)
    left, weights = l.clone(), torch.zeros_like(l)
    for _ in range(top_k):
        top = left.max(0).values
        hit = (left == top) & (top > float("-inf"))
        first = hit & (hit.long().cumsum(0) == 1)
        weights += torch.where(first, torch.exp(top - l.max(0).values), 0.0)
        left = torch.where(first, float("-inf"), left)
    live = torch.where(l > float("-inf"), torch.exp(l - l.max(0).values), 0.0)
    total = (weights if renormalize else live).sum(0)
    return weights / torch.where(total > 0, total, 1.0)


def exact(case, seed):
    gen, op = _gen(seed), case["op"]
    sparse = case["t_s"], case["v_s"]
    if op == "moe":
        n, e = case["tokens"], case["experts"]
        weights = _exact_router(_draw_logits(case, gen).double(), case["top_k"], case["renormalize"])
        x = _draw_x(case["hidden"], n, gen).double()
        met = [weights[i].nonzero().flatten() for i in range(e)]
        inner = {}
        out = torch.zeros(case["hidden"], n, dtype=torch.float64, device="cuda")
        for part, (cout, cin) in enumerate(_moe_shapes(case)):
            for i in range(e):
                drawn = _draw_weight(cout, cin, gen)
                if not met[i].numel():
                    continue
                w = _exact_weight(drawn, *sparse, case["values"])[0]
                if part == 0:
                    g = w @ x[:, met[i]]
                    inner[i] = g * torch.sigmoid(g)
                elif part == 1:
                    inner[i] = inner[i] * (w @ x[:, met[i]])
                else:
                    out[:, met[i]] += (w @ inner[i]) * weights[i, met[i]]
        return out
    if op == "experts8":
        n, k, e = case["tokens"], case["top_k"], case["experts"]
        count = torch.bincount(_draw_ids(case, gen).flatten(), minlength=e).tolist()
        cap = _capacity(n, k, e)
        x = _exact_fp8(_draw_x(case["cin"], cap, gen).double(), 0)
        out = torch.zeros(case["cout"], cap, dtype=torch.float64, device="cuda")
        at = 0
        for c in count:
            w = _exact_weight(_draw_weight(case["cout"], case["cin"], gen), *sparse, "fp8")[0]
            out[:, at:at + c] = w @ x[:, at:at + c]
            at += -(-c // ALIGN) * ALIGN
        return out
    if op == "quantize8":
        dense, pairs = [], []
        for _ in range(case["weights"]):
            _, d, s = _exact_weight(_draw_weight(case["cout"], case["cin"], gen), *sparse, "fp8")
            for out, v in ((dense, d), (pairs, s)):
                v = _pad(v, 32)
                out.append(v.view(v.shape[0], TILE_ROWS, v.shape[2] // 32, 32).permute(0, 2, 1, 3))
        return [torch.stack(dense), torch.stack(pairs)]
    drawn = _draw_weight(case["cout"], case["cin"], gen)
    x = _exact_fp8(_draw_x(case["cin"], case["batch"], gen).double(), 0)
    return _exact_weight(drawn, *sparse, "fp8")[0] @ x


# --------------------------------------------------------------------------- what a pass cannot do without

def _kept_count(cout, cin, case):
    nd, n24 = _counts(cin, case["t_s"], case["v_s"])
    return cout * (nd + n24 // 2)


def _packed_bytes(cout, cin, case, values):
    """Bytes of one packed weight: values (with scales), 2-bit positions, channel lists."""
    nd, n24 = _counts(cin, case["t_s"], case["v_s"])
    each = {"bf16": 2, "fp8": 1 + 1 / 128, "mx4": 1 / 2 + 1 / 32}[values]
    return (_kept_count(cout, cin, case) * each + cout * n24 / 8 + cout // TILE_ROWS * (nd + n24) * 4)


def work(case):
    op = case["op"]
    if op == "moe":
        n, k, e = case["tokens"], case["top_k"], case["experts"]
        met = min(e, n * k)
        packed = sum(_packed_bytes(*s, case, case["values"]) for s in _moe_shapes(case))
        kept = sum(_kept_count(*s, case) for s in _moe_shapes(case))
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": met * packed + n * case["hidden"] * 4 + n * e * size, "flops": 2 * kept * n * k}
    kept = _kept_count(case["cout"], case["cin"], case)
    if op == "quantize8":
        return {"bytes": case["weights"] * kept * 4, "flops": case["weights"] * kept * 2}
    if op == "experts8":
        n = case["tokens"] * case["top_k"]
        packed = min(case["experts"], n) * _packed_bytes(case["cout"], case["cin"], case, "fp8")
    else:
        n = case["batch"]
        packed = _packed_bytes(case["cout"], case["cin"], case, "fp8")
    return {"bytes": packed + n * 2 * (case["cin"] + case["cout"]), "flops": 2 * kept * n}
