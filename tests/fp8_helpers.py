"""Plain 64-bit forms of the 8-bit values and of the mixture-of-experts layer, for the tests."""
from __future__ import annotations

import numpy as np

import moe_helpers as mh


def e4m3_table() -> np.ndarray:
    """Values of the 256 codes by the format's definition: sign, 4 exponent bits (bias 7), 3 mantissa bits; the
    largest code is NaN."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = (np.nan if (c & 127) == 127 else a) * (-1 if c & 128 else 1)
    return v


E4M3 = e4m3_table()
GRID = E4M3[:127]


def scale_byte(top: float, last: int = 246) -> int:
    """The smallest E8M0 byte of 3 .. last at which top does not exceed 448."""
    for e in range(3, last + 1):
        if top <= 448.0 * 2.0 ** (e - 127):
            return e
    return last


def round_codes(v: np.ndarray, e: int):
    """float64 values -> codes and the values they stand for at the scale 2^(e - 127)."""
    a = np.abs(v) / 2.0 ** (e - 127)
    code = np.zeros(v.shape, np.int64)
    bad = ~np.isfinite(v)
    a = np.where(bad, 0.0, np.minimum(a, 448.0))
    hi = np.searchsorted(GRID, a, side="left")             # first grid value >= a
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(bad, 127, code) | np.where(np.signbit(v) & ~bad, 128, 0)
    return code, E4M3[code] * 2.0 ** (e - 127)


def finite_top(v: np.ndarray) -> float:
    f = np.abs(v[np.isfinite(v)])
    return float(f.max()) if f.size else 0.0


def weight_buffers(val_bits: np.ndarray):
    """Packed bf16 values [T, kb, R, 32] (uint16) -> codes uint8 of the same shape, scales uint8 [T, ceil(kb/4), R] and
    the values they stand for."""
    T, K, R, _ = val_bits.shape
    v = mh.bf16_to_f64(val_bits)
    code, value = np.zeros(v.shape, np.uint8), np.zeros(v.shape)
    scale = np.zeros((T, -(-K // 4), R), np.uint8)
    for t in range(T):
        for g in range(scale.shape[1]):
            for r in range(R):
                b = v[t, 4 * g:4 * g + 4, r]
                scale[t, g, r] = e = scale_byte(finite_top(b))
                c, value[t, 4 * g:4 * g + 4, r] = round_codes(b, int(e))
                code[t, 4 * g:4 * g + 4, r] = c
    return code, scale, value


def columns(x: np.ndarray) -> np.ndarray:
    """Activations [channels, tokens] as the values that their codes stand for, one scale a token."""
    out = np.zeros(x.shape)
    for n in range(x.shape[1]):
        out[:, n] = round_codes(x[:, n], scale_byte(finite_top(x[:, n]), 247))[1]
    return out


def values_of(code: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """Codes [..., kb, R, 32] and scales [..., ceil(kb/4), R] as float64."""
    s = np.repeat(scale.astype(np.float64), 4, axis=-2)[..., :code.shape[-3], :]
    return E4M3[code] * 2.0 ** (s[..., None] - 127)


def moe_layer(logits, x, gate, up, down, top_k: int, renormalize: bool, kept):
    """One token at a time in float64: gate, up, down lists of dense weights; kept = kept values of a row of (up,
    down).  Returns the output and a bound of the kernel's error.

    Bound: a sum of k products is off by (k + 64) 2^-23 of the sum of magnitudes (as moe_helpers.product_bound); silu's
    slope is at most 1.1, its exponential, addition and division add less than 2^-20 of the result; h is the
    sum of two bf16 values (2^-16: the second is off by half a step, 2^-8, of at most 2^-8 of h); a router weight is off by (2 |l - m| + 10) 2^-24; one rounding to bf16 of the output."""
    E, N = logits.shape
    r = mh.route(logits, top_k, renormalize, 1, N * top_k)
    out, tol = np.zeros((down[0].shape[0], N)), np.zeros((down[0].shape[0], N))
    for n in range(N):
        l = logits[:, n][np.isfinite(logits[:, n])]
        span = l.max() - l.min() if l.size else 0.0
        for j in range(top_k):
            e = r["ids"][n, j]
            if e < 0:
                continue
            w = r["weights"][n, j]
            g, u = gate[e] @ x[:, n], up[e] @ x[:, n]
            dg, du = [(kept[0] + 64) * 2.0 ** -23 * (np.abs(m[e]) @ np.abs(x[:, n])) for m in (gate, up)]
            with np.errstate(over="ignore"):
                s = g / (1 + np.exp(-g))
            h = s * u
            dh = (1.1 * dg) * (np.abs(u) + du) + (np.abs(s) + 1.1 * dg) * du + (2.0 ** -20 + 2.0 ** -16) * np.abs(h)
            dh += 2.0 ** -16 * dh + 2.0 ** -133
            mag = np.abs(down[e]) @ (np.abs(h) + dh)
            out[:, n] += w * (down[e] @ h)
            tol[:, n] += w * (np.abs(down[e]) @ dh + (kept[1] + 64) * 2.0 ** -23 * mag)
            tol[:, n] += (2 * span + 10) * 2.0 ** -24 * w * mag + (top_k + 4) * 2.0 ** -24 * w * mag
    return out, tol + 2.0 ** -8 * (np.abs(out) + tol) + 2.0 ** -133
