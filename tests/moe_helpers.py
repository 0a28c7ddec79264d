"""Plain 64-bit forms of the mixture-of-experts operators and of the 4-bit microscaled values, for the tests."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_to_f64(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def route(logits: np.ndarray, top_k: int, renormalize: bool, align: int, n_cols: int) -> dict:
    """logits float64 [experts, tokens]; one token at a time."""
    E, N = logits.shape
    ids = np.full((N, top_k), -1, np.int64)
    weights = np.zeros((N, top_k))
    for n in range(N):
        l = logits[:, n]
        ok = [e for e in range(E) if not np.isnan(l[e]) and l[e] > -np.inf]
        best = sorted(ok, key=lambda e: (-l[e], e))[:top_k]
        if not best:
            continue
        m = l[best[0]]
        part = {e: 1.0 if l[e] == m else float(np.exp(l[e] - m)) for e in ok}
        total = sum(part[e] for e in (best if renormalize else ok))
        for j, e in enumerate(best):
            ids[n, j], weights[n, j] = e, part[e] / total
    counts = np.array([(ids == e).sum() for e in range(E)], np.int64)
    starts = np.zeros(E + 1, np.int64)
    for e in range(E):
        starts[e + 1] = starts[e] + -(-counts[e] // align) * align
    slots = np.full((N, top_k), -1, np.int64)
    src = np.full(n_cols, -1, np.int64)
    seen = np.zeros(E, np.int64)
    for n in range(N):
        for j in range(top_k):
            e = ids[n, j]
            if e >= 0:
                slots[n, j] = starts[e] + seen[e]
                src[slots[n, j]] = n
                seen[e] += 1
    return {"ids": ids, "weights": weights, "slots": slots, "starts": starts, "counts": counts, "src": src}


def mx4_block(v: np.ndarray):
    """One block of 32 float64 values -> (scale byte, codes, the values they stand for)."""
    if not np.all(np.isfinite(v)):
        return 255, None, np.full(32, np.nan)
    top = np.abs(v).max()
    if top == 0:
        return 0, np.where(np.signbit(v), 8, 0), v * 0.0
    e = max(int(np.frexp(top)[1]) - 1 - 2, -127)
    a = np.abs(v) / 2.0 ** e
    code = np.zeros(32, np.int64)
    for i, x in enumerate(a):
        d = np.abs(GRID - x)
        near = np.flatnonzero(d == d.min())                # one, or two at a half-way case
        code[i] = next(c for c in near if len(near) == 1 or c % 2 == 0)
    value = GRID[code] * 2.0 ** e * np.where(np.signbit(v), -1.0, 1.0)
    return e + 127, code | np.where(np.signbit(v), 8, 0), value


def mx4_buffers(val_bits: np.ndarray, meta: np.ndarray | None):
    """Packed bf16 values [T, kb, R, 32] (uint16) -> codes uint32 [T,kb,R/64,4,16,4], scales uint8 [T,kb,R/64,16,4],
    metadata uint16 [T,kb,R/64,4,16,4] or None, and the values they stand for [T, kb, R, 32]."""
    T, K, R, _ = val_bits.shape
    G = R // 64
    code = np.zeros((T, K, G, 4, 16, 4), np.uint32)
    scale = np.zeros((T, K, G, 16, 4), np.uint8)
    m16 = np.zeros((T, K, G, 4, 16, 4), np.uint16) if meta is not None else None
    value = np.zeros((T, K, R, 32))
    v = bf16_to_f64(val_bits)
    for t in range(T):
        for k in range(K):
            for r in range(R):
                g, f, i = r // 64, r % 64 // 16, r % 16
                s, c, value[t, k, r] = mx4_block(v[t, k, r])
                scale[t, k, g, i, f] = s
                if c is not None:
                    for q in range(4):
                        code[t, k, g, q, i, f] = sum(int(c[8 * q + u]) << (4 * u) for u in range(8))
                if meta is not None:
                    for q in range(4):
                        m16[t, k, g, q, i, f] = (int(meta[t, k, r]) >> (16 * q)) & 0xffff
    return code, scale, m16, value


def dense_from_packed(p, bufs: dict, val_dense: np.ndarray, val_24: np.ndarray) -> np.ndarray:
    """The weight [cout, cin] in float64 that packed buffers stand for, given their values in float64."""
    T, R = p.n_tiles, p.tile_rows
    w = np.zeros((p.cout, p.cin))
    rows = np.arange(R)
    for t in range(T):
        for j, c in enumerate(bufs["idx_dense"][t]):
            if c >= 0:
                w[t * R:(t + 1) * R, c] = val_dense[t, j // 32, :, j % 32]
        for g in range(p.n_24_pad // 4):
            cols = bufs["idx_24"][t, 4 * g:4 * g + 4]
            if (cols < 0).all():
                continue
            nib = (bufs["meta_24"][t, g // 16] >> np.uint64(4 * (g % 16))) & np.uint64(15)
            for h in range(2):
                at = ((nib >> np.uint64(2 * h)) & np.uint64(3)).astype(np.int64)
                w[t * R + rows, cols[at]] = val_24[t, g // 16, :, 2 * (g % 16) + h]
    return w


# Tolerance of a product with bf16 output: every fp32 addition is off by at most half a step, 2^-24 of the running
# sum, itself at most sum |w||x|; the matrix instructions add in an order and rounding of their own, so a whole step
# (2^-23) is granted to each of the kept terms; then one rounding to bf16, 2^-8 of the value.
def product_bound(w: np.ndarray, x: np.ndarray, kept: int) -> np.ndarray:
    mag = np.abs(w) @ np.abs(x)
    acc = (kept + 64) * 2.0 ** -23 * mag
    return acc + 2.0 ** -8 * (np.abs(w @ x) + acc) + 2.0 ** -133
