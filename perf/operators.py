"""Cases for measuring the mixture-of-experts operators on packed weights and the 4-bit microscaled values.

Five operators, each in a plain form (elementary torch operations in 32 bits) and as calls of this package:

    route     logits -> top-k experts, softmax weights, column order by expert
    dispatch  token columns -> columns in the order of their experts
    combine   weighted sum of each token's expert columns
    experts   one product per expert over its own ragged range of columns
    quantize  packed values -> 4-bit microscaled values (returned as the values they stand for)
    product   one packed weight with 4-bit microscaled values times activations

Activations are [channels, tokens]; weights are hierarchical N:M (dense, 2:4 and pruned column vectors in
tiles of 64 rows) with a random channel permutation per tile, and importance |W|.  Weight shapes are the
4096 / 11008 linear layers this repository is benchmarked on; the sparsities are those of its workloads.
"""
import math

import torch

own = False

TILE_ROWS = 64
ALIGN = 8                       # an expert's columns start at a multiple of this
SPARSITIES = ((0.5, 0.25), (0.75, 0.55), (0.75, 0.5), (0.7, 0.51))


def listed():
    return [
        # a decode step: 16 sequences meet a small router
        {"name": "route-decode", "op": "route", "tokens": 16, "experts": 8, "top_k": 2, "dtype": "bf16",
         "renormalize": True, "idle": 0.0},
        # a long prompt over many small experts; a twentieth of the columns are padding that no expert may take
        {"name": "route-prompt", "op": "route", "tokens": 8192, "experts": 128, "top_k": 8, "dtype": "fp32",
         "renormalize": False, "idle": 0.05},
        # 16 sequences' activations on their way to two experts each
        {"name": "dispatch-decode", "op": "dispatch", "channels": 4096, "tokens": 16, "experts": 8, "top_k": 2},
        # a prompt of 4096 tokens
        {"name": "dispatch-prompt", "op": "dispatch", "channels": 4096, "tokens": 4096, "experts": 8, "top_k": 2},
        # the same prompt coming back, one token short of even
        {"name": "combine-prompt", "op": "combine", "channels": 4096, "tokens": 4095, "experts": 8, "top_k": 2},
        # up projections of 8 experts for a decode step of 16 sequences: every expert's weight is read
        {"name": "experts-decode", "op": "experts", "values": "bf16", "cout": 11008, "cin": 4096, "t_s": 0.75,
         "v_s": 0.55, "experts": 8, "tokens": 16, "top_k": 2},
        # down projections for a prompt: uneven, odd counts
        {"name": "experts-prompt", "op": "experts", "values": "bf16", "cout": 4096, "cin": 11008, "t_s": 0.75,
         "v_s": 0.55, "experts": 8, "tokens": 2047, "top_k": 2},
        # the decode step with 4-bit weights
        {"name": "experts-mx4-decode", "op": "experts", "values": "mx4", "cout": 11008, "cin": 4096, "t_s": 0.75,
         "v_s": 0.55, "experts": 8, "tokens": 32, "top_k": 2},
        # quantising one square projection
        {"name": "quantize-one", "op": "quantize", "cout": 4096, "cin": 4096, "t_s": 0.5, "v_s": 0.25, "weights": 1},
        # quantising a layer's 8 experts
        {"name": "quantize-experts", "op": "quantize", "cout": 11008, "cin": 4096, "t_s": 0.75, "v_s": 0.55,
         "weights": 8},
        # one sequence's next token through a down projection
        {"name": "product-token", "op": "product", "cout": 4096, "cin": 11008, "t_s": 0.75, "v_s": 0.55, "batch": 1},
        # a prompt through an up projection, odd length
        {"name": "product-prompt", "op": "product", "cout": 11008, "cin": 4096, "t_s": 0.75, "v_s": 0.55,
         "batch": 2047},
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
    op = rng.choice(["route", "dispatch", "combine", "experts", "experts", "quantize", "product"])
    if op == "route":
        experts = _log(rng, 2, 256)
        return {"op": op, "tokens": _log(rng, 1, 8192), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
                "dtype": rng.choice(["bf16", "fp32"]), "renormalize": rng.random() < 0.5,
                "idle": rng.choice([0.0, 0.05, 0.3])}
    if op in ("dispatch", "combine"):
        experts = _log(rng, 2, 64)
        return {"op": op, "channels": _log(rng, 64, 4096), "tokens": _log(rng, 1, 4096), "experts": experts,
                "top_k": rng.randint(1, 2)}
    if op == "experts":
        return {"op": op, "values": rng.choice(["bf16", "mx4"]), **_weight(rng), "experts": rng.randint(2, 8),
                "tokens": _log(rng, 1, 2047), "top_k": rng.randint(1, 2)}
    if op == "quantize":
        return {"op": op, **_weight(rng), "weights": rng.randint(1, 8)}
    return {"op": op, **_weight(rng), "batch": _log(rng, 1, 2047)}


# --------------------------------------------------------------------------- inputs

def _counts(case):
    """Region counts of a row: dense, 2:4 and pruned channels by the closed form."""
    cin, t, v = case["cin"], case["t_s"], case["v_s"]
    z = math.floor(t * cin + 0.5)
    g = max(0, min(math.floor((t - v) * cin / 2 + 0.5), min(z, cin - z) // 2))
    return cin - z - 2 * g, 4 * g, z


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _draw_weight(case, gen):
    """bf16 weight with log-normal channel scales, importance |W|, one channel order per tile."""
    cout, cin = case["cout"], case["cin"]
    scale = torch.randn(cin, generator=gen, device="cuda").exp()
    w = (torch.randn(cout, cin, generator=gen, device="cuda") * (0.02 * scale)).bfloat16()
    perm = torch.rand(cout // TILE_ROWS, cin, generator=gen, device="cuda").argsort(dim=1)
    return w, w.float().abs(), perm


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
    n = ids.shape[0]
    hot = torch.zeros(n, experts, dtype=torch.int64, device=ids.device)
    ok = ids >= 0
    hot.scatter_add_(1, ids.clamp(min=0).long(), ok.long())
    counts = hot.sum(0)
    padded = (counts + ALIGN - 1) // ALIGN * ALIGN
    starts = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    before = hot.cumsum(0) - hot
    slots = torch.where(ok, starts[ids.clamp(min=0).long()] + before.gather(1, ids.clamp(min=0).long()), -1)
    src = torch.full((_capacity(tokens, top_k, experts),), -1, dtype=torch.int64, device=ids.device)
    token = torch.arange(n, device=ids.device)[:, None].expand_as(slots)
    src[slots[ok]] = token[ok]
    return [t.int() for t in (slots, starts, counts, src)]


def _routing(ids, weights, experts, tokens, top_k):
    slots, starts, counts, src = _arrange(ids, experts, tokens, top_k)
    return {"ids": ids.int(), "weights": weights, "slots": slots, "starts": starts, "counts": counts, "src": src}


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


def _pad32(v):
    return torch.nn.functional.pad(v, (0, -v.shape[2] % 32))


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


def _mx4(v):
    """Values [tiles, rows, n] rounded to 4-bit microscaled values in blocks of 32 along n."""
    n = v.shape[2]
    b = _pad32(v).float().unflatten(2, (-1, 32))
    top = b.abs().amax(3, keepdim=True).bfloat16()                   # exact: the values are bf16
    exp = ((top.view(torch.int16).long() >> 7) - 2).clamp(min=0)     # its exponent field, less 2: 2**(exp - 127)
    scale = ((exp - 127 + 1023) << 52).view(torch.float64)
    a = (b.double() / scale).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = ((a / step).round() * step).clamp(max=6.0)
    return (q * scale * b.sign()).bfloat16().flatten(2)[..., :n]


def _dense(w, imp, perm, case, four_bit):
    """The masked weight as a dense bf16 matrix, with 4-bit values on request."""
    nd, n24, _ = _counts(case)
    val_d, col_d, val_s, col_s = _kept(w, imp, perm, nd, n24)
    if four_bit:
        val_d, val_s = _mx4(val_d), _mx4(val_s)
    out = torch.zeros_like(w).view(perm.shape[0], TILE_ROWS, perm.shape[1])
    out.scatter_(2, col_d, val_d)
    out.scatter_(2, col_s, val_s)
    return out.view_as(w)


def _blocks(v):
    """[tiles, rows, n] -> the packed layout [tiles, n/32, rows, 32]."""
    return _pad32(v).unflatten(2, (-1, 32)).transpose(1, 2).contiguous()


def _pack(w, imp, perm, case):
    import structured_sparse_gemm_amd as hinm
    return hinm.pack(w, imp, TILE_ROWS, case["t_s"], case["v_s"], perm.int())


def _as_routing(r, experts, tokens):
    import structured_sparse_gemm_amd as hinm
    return hinm.Routing(ids=r["ids"], weights=r["weights"], slots=r["slots"], starts=r["starts"], counts=r["counts"],
                        src=r["src"])


def prepare(case, seed):
    gen, op = _gen(seed), case["op"]
    state = {"case": case}
    if op == "route":
        e, n = case["experts"], case["tokens"]
        logits = torch.randn(e, n, generator=gen, device="cuda") * 2 + torch.randn(e, 1, generator=gen, device="cuda")
        if case["idle"]:
            idle = torch.rand(n, generator=gen, device="cuda") < case["idle"]
            logits[:, idle] = float("-inf")
        state["logits"] = logits.bfloat16() if case["dtype"] == "bf16" else logits
    elif op in ("dispatch", "combine"):
        n, k, e = case["tokens"], case["top_k"], case["experts"]
        ids = _draw_ids(case, gen)
        weights = torch.rand(n, k, generator=gen, device="cuda") + 0.1
        weights = weights / weights.sum(1, keepdim=True)
        state["routing"] = _routing(ids, weights, e, n, k)
        cols = n if op == "dispatch" else state["routing"]["src"].numel()
        state["x"] = torch.randn(case["channels"], cols, generator=gen, device="cuda").bfloat16()
        if own:
            state["routing"] = _as_routing(state["routing"], e, n)
    elif op == "experts":
        n, k, e = case["tokens"], case["top_k"], case["experts"]
        ids = _draw_ids(case, gen)
        routing = _routing(ids, torch.ones(n, k, device="cuda") / k, e, n, k)
        cap = routing["src"].numel()
        state["x"] = torch.randn(case["cin"], cap, generator=gen, device="cuda").bfloat16()
        state["y"] = torch.zeros(case["cout"], cap, dtype=torch.bfloat16, device="cuda")
        weights = []
        for _ in range(e):
            w, imp, perm = _draw_weight(case, gen)
            weights.append(_pack(w, imp, perm, case) if own else _dense(w, imp, perm, case, case["values"] == "mx4"))
        if own:
            import structured_sparse_gemm_amd as hinm
            state["routing"] = _as_routing(routing, e, n)
            state["w"] = hinm.Experts.stack(weights)
            if case["values"] == "mx4":
                state["w"] = hinm.quantize_mx4(state["w"])
        else:
            state["ranges"] = list(zip(routing["starts"].tolist(), routing["counts"].tolist()))
            state["w"] = weights
    elif op == "quantize":
        nd, n24, _ = _counts(case)
        weights = []
        for _ in range(case["weights"]):
            w, imp, perm = _draw_weight(case, gen)
            if own:
                weights.append(_pack(w, imp, perm, case))
            else:
                val_d, _, val_s, _ = _kept(w, imp, perm, nd, n24)
                weights.append((_blocks(val_d), _blocks(val_s)))
        if own:
            import structured_sparse_gemm_amd as hinm
            state["w"] = hinm.Experts.stack(weights)
        else:
            state["w"] = [torch.stack(v) for v in zip(*weights)]
    else:
        w, imp, perm = _draw_weight(case, gen)
        state["x"] = torch.randn(case["cin"], case["batch"], generator=gen, device="cuda").bfloat16()
        if own:
            import structured_sparse_gemm_amd as hinm
            state["w"] = hinm.quantize_mx4(_pack(w, imp, perm, case))
        else:
            state["w"] = _dense(w, imp, perm, case, True)
    return state


# --------------------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import structured_sparse_gemm_amd as hinm
    case, op = state["case"], state["case"]["op"]
    if op == "route":
        r = hinm.route(state["logits"], case["top_k"], renormalize=case["renormalize"], align=ALIGN)
        return {"ids": r.ids, "weights": r.weights, "slots": r.slots, "starts": r.starts, "counts": r.counts,
                "src": r.src}
    if op == "dispatch":
        return hinm.dispatch(state["x"], state["routing"])
    if op == "combine":
        return hinm.combine(state["x"], state["routing"])
    if op == "experts":
        return hinm.spmm_experts(state["w"], state["x"], state["routing"], out=state["y"])
    if op == "quantize":
        back = hinm.quantize_mx4(state["w"]).dequantize()
        return [back.val_dense.view(torch.bfloat16), back.val_24.view(torch.bfloat16)]
    return hinm.spmm(state["w"], state["x"])


def _run_plain(state):
    case, op = state["case"], state["case"]["op"]
    if op == "route":
        logits = state["logits"].float()
        key = torch.where(logits.isnan(), float("-inf"), logits)
        top, ids = key.sort(dim=0, descending=True, stable=True)
        top, ids = top[:case["top_k"]].t(), ids[:case["top_k"]].t()
        ok = top > float("-inf")
        best = torch.where(ok[:, :1], top[:, :1], 0.0)
        part = torch.exp(top - best)
        whole = part if case["renormalize"] else torch.exp(key.t() - best)
        weights = torch.where(ok, part / whole.sum(1, keepdim=True), 0.0)
        r = _routing(torch.where(ok, ids, -1), weights, case["experts"], case["tokens"], case["top_k"])
        return {k: r[k].contiguous() for k in ("ids", "weights", "slots", "starts", "counts", "src")}
    if op == "dispatch":
        src = state["routing"]["src"]
        return torch.where(src >= 0, state["x"][:, src.clamp(min=0).long()], 0.0)
    if op == "combine":
        slots, weights = state["routing"]["slots"].long(), state["routing"]["weights"]
        acc = torch.zeros(case["channels"], case["tokens"], device="cuda")
        for j in range(case["top_k"]):
            acc += state["x"][:, slots[:, j].clamp(min=0)].float() * torch.where(slots[:, j] >= 0, weights[:, j], 0.0)
        return acc.bfloat16()
    if op == "experts":
        for w, (start, count) in zip(state["w"], state["ranges"]):
            if count:
                state["y"][:, start:start + count] = w.float() @ state["x"][:, start:start + count].float()
        return state["y"]
    if op == "quantize":
        return [_mx4(v.flatten(0, 2)).view_as(v) for v in state["w"]]
    return (state["w"].float() @ state["x"].float()).bfloat16()


# --------------------------------------------------------------------------- the definition in 64 bits

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_four_bit(v):
    """Nearest representable value, half-way cases to the even code, by the table of all eight magnitudes."""
    v = v.double()
    top = v.abs().amax(-1, keepdim=True)
    field = top.view(torch.int64) >> 52                              # 1023 + floor(log2(top)) in float64
    unit = (torch.clamp(field - 2, 1023 - 127, 1023 + 127) << 52).view(torch.float64)
    a, out = v.abs() / unit, torch.zeros_like(v)
    for code in range(1, 8):
        half = (_GRID[code - 1] + _GRID[code]) / 2
        out = torch.where((a > half) | ((a == half) & (code % 2 == 0)), _GRID[code], out)
    return out * unit * v.sign()


def _exact_weight(case, gen, four_bit):
    """Per tile: rank every channel by counting those that beat it; in each 2:4 group keep an entry that fewer
    than two others beat.  Returns the masked weight in float64, and the packed-order values."""
    w, imp, perm = _draw_weight(case, gen)
    nd, n24, _ = _counts(case)
    tiles, cin = perm.shape
    out = torch.zeros(case["cout"], cin, dtype=torch.float64, device="cuda")
    dense, pairs = [], []
    low = torch.arange(cin, device="cuda")
    for t in range(tiles):
        rows = slice(t * TILE_ROWS, (t + 1) * TILE_ROWS)
        wt, it = w[rows].double(), imp[rows].double()
        score = it.sum(0)
        by = score.sort(stable=True).values
        ahead = cin - torch.searchsorted(by, score, right=True)
        if by.unique().numel() < cin:                      # equal scores: the lower channel first
            same = (score[:, None] == score[None, :]) & (low[None, :] < low[:, None])
            ahead = ahead + same.sum(1)
        rank = ahead[perm[t]]
        cols_d = perm[t][rank < nd]
        cols_s = perm[t][(rank >= nd) & (rank < nd + n24)]
        vd = wt[:, cols_d]
        fours = it[:, cols_s].view(TILE_ROWS, -1, 4)
        beats = torch.zeros_like(fours)
        for i in range(4):
            for j in range(4):
                if i != j:
                    a, b = fours[..., j], fours[..., i]
                    beats[..., i] += ((a > b) | ((a == b) & (j < i))).double()
        keep = (beats < 2).view(TILE_ROWS, -1)
        vs = wt[:, cols_s]
        packed = vs[keep].view(TILE_ROWS, -1)
        if four_bit:
            def blocks(v):
                n = v.shape[1]
                p = torch.nn.functional.pad(v, (0, -n % 32)).view(TILE_ROWS, -1, 32)
                return _exact_four_bit(p).view(TILE_ROWS, -1)[:, :n]
            vd, packed = blocks(vd), blocks(packed)
        out[rows, cols_d] = vd
        full = torch.zeros_like(vs)
        full[keep] = packed.reshape(-1)
        out[rows, cols_s] = full
        dense.append(vd)
        pairs.append(packed)
    return out, torch.stack(dense), torch.stack(pairs)


def exact(case, seed):
    gen, op = _gen(seed), case["op"]
    if op == "route":
        state = prepare(case, seed)
        l = state["logits"].double()
        k, n = case["top_k"], case["tokens"]
        l = torch.where(l.isnan(), float("-inf"), l)
        weights = torch.zeros(n, k, dtype=torch.float64, device="cuda")
        left = l.clone()
        total = torch.zeros(n, dtype=torch.float64, device="cuda")
        for j in range(k):
            top = left.max(0).values
            hit = (left == top[None]) & (top[None] > float("-inf"))
            first = hit & (hit.long().cumsum(0) == 1)
            weights[:, j] = torch.where(top > float("-inf"), torch.exp(top - l.max(0).values), 0.0)
            total += weights[:, j]
            left = torch.where(first, float("-inf"), left)
        if not case["renormalize"]:
            live = l > float("-inf")
            total = torch.where(live, torch.exp(l - l.max(0).values[None]), 0.0).sum(0)
        weights /= torch.where(total > 0, total, 1.0)[:, None]
        return {"ids": None, "weights": weights, "slots": None, "starts": None, "counts": None, "src": None}
    if op in ("dispatch", "combine"):
        n, k, e = case["tokens"], case["top_k"], case["experts"]
        ids = _draw_ids(case, gen)
        weights = torch.rand(n, k, generator=gen, device="cuda") + 0.1
        weights = weights / weights.sum(1, keepdim=True)
        # columns by a stable sort of the (token, choice) pairs by expert
        order = ids.flatten().argsort(stable=True)
        owner = ids.flatten()[order]
        count = torch.bincount(owner, minlength=e)
        start = (torch.ceil(count / ALIGN) * ALIGN).long().cumsum(0)
        start = torch.cat([start.new_zeros(1), start[:-1]])
        place = torch.arange(n * k, device="cuda") - (count.cumsum(0) - count)[owner] + start[owner]
        cap = _capacity(n, k, e)
        cols = n if op == "dispatch" else cap
        x = torch.randn(case["channels"], cols, generator=gen, device="cuda").bfloat16().double()
        if op == "dispatch":
            out = torch.zeros(case["channels"], cap, dtype=torch.float64, device="cuda")
            out[:, place] = x[:, order // k]
            return out
        out = torch.zeros(case["channels"], n, dtype=torch.float64, device="cuda")
        out.index_add_(1, order // k, x[:, place] * weights.flatten()[order].double())
        return out
    if op == "experts":
        n, k, e = case["tokens"], case["top_k"], case["experts"]
        count = torch.bincount(_draw_ids(case, gen).flatten(), minlength=e).tolist()
        cap = _capacity(n, k, e)
        x = torch.randn(case["cin"], cap, generator=gen, device="cuda").bfloat16().double()
        out = torch.zeros(case["cout"], cap, dtype=torch.float64, device="cuda")
        at = 0
        for c in count:
            w, _, _ = _exact_weight(case, gen, case["values"] == "mx4")
            out[:, at:at + c] = w @ x[:, at:at + c]
            at += -(-c // ALIGN) * ALIGN
        return out
    if op == "quantize":
        nd, n24, _ = _counts(case)
        dense, pairs = [], []
        for _ in range(case["weights"]):
            _, d, s = _exact_weight(case, gen, True)
            for out, v in ((dense, d), (pairs, s)):
                v = torch.nn.functional.pad(v, (0, -v.shape[2] % 32))
                out.append(v.view(v.shape[0], TILE_ROWS, -1, 32).permute(0, 2, 1, 3))
        return [torch.stack(dense), torch.stack(pairs)]
    weight, _, _ = _exact_weight(case, gen, True)
    x = torch.randn(case["cin"], case["batch"], generator=gen, device="cuda").bfloat16().double()
    return weight @ x


# --------------------------------------------------------------------------- what a pass cannot do without

def _packed_bytes(case, four_bit):
    """Bytes of one packed weight: values (with scales when 4-bit), 2-bit positions, channel lists."""
    nd, n24, _ = _counts(case)
    kept = case["cout"] * (nd + n24 // 2)
    values = kept / 2 + kept / 32 if four_bit else kept * 2
    return values + case["cout"] * n24 / 8 + case["cout"] // TILE_ROWS * (nd + n24) * 4


def work(case):
    op = case["op"]
    if op == "route":
        n, k, e = case["tokens"], case["top_k"], case["experts"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * e * size + n * k * 12 + _capacity(n, k, e) * 4 + e * 8, "flops": n * e * 4}
    if op in ("dispatch", "combine"):
        n, k, c = case["tokens"], case["top_k"], case["channels"]
        cap = _capacity(n, k, case["experts"])
        if op == "dispatch":
            return {"bytes": c * n * 2 + c * cap * 2 + cap * 4, "flops": 0}
        return {"bytes": c * n * k * 2 + c * n * 2 + n * k * 8, "flops": 2 * c * n * k}
    nd, n24, _ = _counts(case)
    kept = case["cout"] * (nd + n24 // 2)
    if op == "experts":
        n = case["tokens"] * case["top_k"]
        packed = min(case["experts"], n) * _packed_bytes(case, case["values"] == "mx4")
        return {"bytes": packed + n * 2 * (case["cin"] + case["cout"]), "flops": 2 * kept * n}
    if op == "quantize":
        return {"bytes": case["weights"] * kept * 4, "flops": case["weights"] * kept * 2}
    n = case["batch"]
    return {"bytes": _packed_bytes(case, True) + n * 2 * (case["cin"] + case["cout"]), "flops": 2 * kept * n}
