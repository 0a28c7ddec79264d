"""Router, dispatch, combine, expert products and 4-bit microscaled values on the GPU against plain 64-bit forms.

Tolerances count roundings: whole numbers and copied bits are equal; a router weight is a quotient of fp32
exponentials of an exact or once-rounded difference; a combined value is top_k fused multiply-adds and one rounding
to bf16; a product's bound is moe_helpers.product_bound.
"""
import numpy as np
import pytest
import torch

import synth
from helpers import bits_of, device_packed_numpy
import moe_helpers as mh

pytestmark = pytest.mark.gpu
hinm = pytest.importorskip("structured_sparse_gemm_amd")
DEV = torch.device("cuda:0")


def _np(t):
    return t.detach().cpu().numpy()


def _f64(t):
    return t.detach().double().cpu().numpy()


# --------------------------------------------------------------------------- router

def _check_route(logits: torch.Tensor, k: int, renorm: bool, align: int):
    e, n = logits.shape
    r = hinm.route(logits.to(DEV), k, renormalize=renorm, align=align)
    torch.cuda.synchronize()
    want = mh.route(_f64(logits), k, renorm, align, hinm.route_columns(n, e, k, align))
    for f in ("ids", "counts", "starts", "slots", "src"):
        assert np.array_equal(_np(getattr(r, f)), want[f]), f
    # exp(d), d = l - m rounded once: off by |d| 2^-24 from d and 2 steps (2^-23 each) from expf; the sum adds the
    # same for its terms; division and the last rounding half a step each
    l = np.where(np.isfinite(_f64(logits)), _f64(logits), np.nan)
    span = np.nan_to_num(np.nanmax(l, 0) - np.nanmin(l, 0)) if n and np.isfinite(l).any() else np.zeros(n)
    tol = (2 * span[:, None] + 10) * 2.0 ** -24 * want["weights"] + 2.0 ** -140
    assert np.all(np.abs(_f64(r.weights) - want["weights"]) <= tol)
    return r


@pytest.mark.parametrize("n", [0, 1, 5, 63, 64, 65, 200])
@pytest.mark.parametrize("e,k,align", [(8, 2, 8), (1, 1, 1), (3, 3, 4), (7, 4, 1), (130, 8, 16), (33, 16, 8)])
def test_route(n, e, k, align):
    g = torch.Generator().manual_seed(17 * n + e)
    logits = torch.randn(e, n, generator=g) * 3
    print(f"[route] n={n} e={e} k={k} align={align}", flush=True)
    for renorm in (True, False):
        _check_route(logits, k, renorm, align)
        _check_route(logits.bfloat16(), k, renorm, align)      # bf16: equal logits are common


@pytest.mark.parametrize("n,e,k", [(2048, 4, 2), (2049, 5, 1), (4200, 300, 2), (130, 1024, 3)])
def test_route_many_blocks(n, e, k):
    """Past 32 blocks of 64 tokens the counts are summed in groups; 1024 experts are the most."""
    g = torch.Generator().manual_seed(n)
    print(f"[route] n={n} e={e} k={k}", flush=True)
    _check_route(torch.randn(e, n, generator=g).bfloat16(), k, False, 8)


def test_route_special_logits():
    """NaN and -inf are not eligible, +inf shares the weight, tokens without any expert go nowhere, equal logits
    take the lower expert."""
    inf, nan = float("inf"), float("nan")
    rows = torch.tensor([[0.0, 0.0, 0.0, 0.0], [-inf, -inf, -inf, -inf], [nan, 1.0, nan, -inf], [nan, nan, nan, nan],
                         [inf, 3.0, inf, inf], [5.0, inf, 5.0, -inf], [-inf, 2.0, 2.0, 2.0], [1e38, -1e38, 0.0, 3e38],
                         [-3e38, -inf, -3e38, -3e38], [0.0, -0.0, 0.0, -0.0]])
    print("[route] special logits", flush=True)
    for dt in (torch.float32, torch.bfloat16):
        for k in (1, 2, 3, 4):
            for renorm in (True, False):
                r = _check_route(rows.to(dt).t().contiguous(), k, renorm, 8)
                assert torch.isfinite(r.weights).all()
    sums = hinm.route(rows.t().contiguous().to(DEV), 4, renormalize=True).weights.sum(1)
    assert torch.equal((sums > 0.5).cpu(), torch.tensor([1, 0, 1, 0, 1, 1, 1, 1, 1, 1], dtype=torch.bool))


def test_route_strided_logits():
    g = torch.Generator().manual_seed(5)
    big = torch.randn(6, 301, generator=g).bfloat16().to(DEV)
    a, b = hinm.route(big[:, 7:207], 2), hinm.route(big[:, 7:207].contiguous(), 2)
    for f in ("ids", "weights", "slots", "starts", "counts", "src"):
        assert torch.equal(getattr(a, f), getattr(b, f)), f


# --------------------------------------------------------------------------- dispatch and combine

def _routing(n, e, k, seed, align=8, idle=0.1):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(e, n, generator=g)
    if n:
        logits[:, torch.rand(n, generator=g) < idle] = float("-inf")
    return hinm.route(logits.to(DEV), k, align=align)


@pytest.mark.parametrize("c,n,e,k,align", [(1, 1, 1, 1, 1), (5, 17, 3, 2, 8), (64, 300, 8, 2, 8), (130, 1025, 4, 1, 1),
                                           (3, 40, 16, 16, 4), (33, 9000, 6, 3, 8), (3, 15000, 4, 2, 8), (2, 70000, 2, 2, 8)])
@pytest.mark.parametrize("pad", [0, 3])
def test_dispatch_and_combine(c, n, e, k, align, pad):
    """Contiguous matrices and slices of wider ones whose surroundings stay as they were."""
    print(f"[move] c={c} n={n} e={e} k={k} align={align} pad={pad}", flush=True)
    r = _routing(n, e, k, c + n, align)
    g = torch.Generator().manual_seed(n)
    wide = torch.randn(c, n + 2 * pad, generator=g).bfloat16().to(DEV)
    x = wide[:, pad:pad + n]
    src = _np(r.src)
    box = torch.full((c, r.n_cols + 2 * pad), 7.0, dtype=torch.bfloat16, device=DEV)
    xs = hinm.dispatch(x, r, out=box[:, pad:pad + r.n_cols])
    torch.cuda.synchronize()
    want = np.where(src >= 0, bits_of(x)[:, np.maximum(src, 0)], 0)
    assert np.array_equal(bits_of(xs), want)
    assert pad == 0 or (bool((box[:, :pad] == 7).all()) and bool((box[:, -pad:] == 7).all()))

    ys = torch.randn(c, r.n_cols + 2 * pad, generator=g).bfloat16().to(DEV)[:, pad:pad + r.n_cols]
    ys[:, torch.from_numpy(src < 0).to(DEV)] = float("nan")              # columns without a token add nothing
    box = torch.full((c, n + 2 * pad), 7.0, dtype=torch.bfloat16, device=DEV)
    y = hinm.combine(ys, r, out=box[:, pad:pad + n])
    torch.cuda.synchronize()
    slots, w, yf = _np(r.slots), _f64(r.weights), _f64(ys)
    ref, mag = np.zeros((c, n)), np.zeros((c, n))
    for j in range(k):
        v = np.where(slots[:, j] >= 0, yf[:, np.maximum(slots[:, j], 0)], 0.0)
        ref += w[:, j] * v
        mag += np.abs(w[:, j] * v)
    acc = k * 2.0 ** -24 * mag * 1.01                                    # one rounding a fused multiply-add
    assert np.all(np.abs(_f64(y) - ref) <= acc + 2.0 ** -8 * (np.abs(ref) + acc) + 2.0 ** -134)
    assert pad == 0 or (bool((box[:, :pad] == 7).all()) and bool((box[:, -pad:] == 7).all()))


def test_dispatch_copies_bits_and_ignores_wild_sources():
    """NaN payloads are copied; sources and slots outside their range count as none."""
    x = torch.tensor([[0x7fc1, 0x3f80, 0xffff, 0x8000]], dtype=torch.int32).to(torch.int16).view(torch.bfloat16).to(DEV)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    r = hinm.Routing(i32([[0], [0], [0], [0]]), torch.ones(4, 1, device=DEV), i32([[3], [-5], [99], [0]]), i32([0, 8]),
                     i32([4]), i32([2, 0, -7, 4, 3, 1 << 30, 1, -(1 << 31)]))
    xs = hinm.dispatch(x, r)
    assert bits_of(xs).tolist() == [[0xffff, 0x7fc1, 0, 0, 0x8000, 0, 0x3f80, 0]]
    ys = torch.arange(8, device=DEV).float().bfloat16()[None]
    assert hinm.combine(ys, r).tolist() == [[3.0, 0.0, 0.0, 0.0]]


# --------------------------------------------------------------------------- weights

def _pack(cout, cin, rows, t, v, seed, **kw):
    w = synth.small(cout, cin, rows, t, v, 1, seed=seed, **kw)
    return hinm.pack(w.w_bf16.to(DEV), w.importance.to(DEV), rows, t, v, w.perm.to(DEV))


def _dense(pk):
    b = device_packed_numpy(pk)
    return mh.dense_from_packed(pk.plan, b, mh.bf16_to_f64(b["val_dense"]), mh.bf16_to_f64(b["val_24"]))


def _check_mx4(q, pk):
    b = device_packed_numpy(pk)
    out = []
    for val, meta, names in (("val_dense", None, ("val_dense", "scale_dense", None)),
                             ("val_24", "meta_24", ("val_24", "scale_24", "meta_24"))):
        code, scale, m16, value = mh.mx4_buffers(b[val], b[meta] if meta else None)
        live = scale[..., None, :, :] != 255                              # codes of a NaN block say nothing
        assert np.array_equal(_np(getattr(q, names[1])), scale), names[1]
        got = _np(getattr(q, names[0])).view(np.uint32)
        # the sign of a value that rounds to zero is kept; compare all code bits
        assert np.array_equal(np.where(live, got, 0), np.where(live, code, 0)), names[0]
        if m16 is not None:
            assert np.array_equal(_np(q.meta_24).view(np.uint16), m16)
        out.append(value)
    assert np.array_equal(_np(q.idx_dense), b["idx_dense"]) and np.array_equal(_np(q.idx_24), b["idx_24"])
    back = q.dequantize()
    torch.cuda.synchronize()
    got = device_packed_numpy(back)
    for name, value in zip(("val_dense", "val_24"), out):
        g = mh.bf16_to_f64(got[name])
        assert np.array_equal(g, value, equal_nan=True), name
    for name in ("meta_24", "idx_dense", "idx_24"):
        assert np.array_equal(got[name], b[name]), name
    return out


@pytest.mark.parametrize("cout,cin,rows,t,v", [(64, 128, 64, 0.75, 0.55), (128, 300, 64, 0.5, 0.25),
                                               (256, 68, 128, 0.75, 0.5), (192, 260, 192, 0.0, 0.0),
                                               (64, 8, 64, 0.5, 0.0), (128, 132, 64, 0.6, 0.6)])
def test_quantize(cout, cin, rows, t, v):
    print(f"[mx4] {cout}x{cin} R={rows} t={t} v={v}", flush=True)
    pk = _pack(cout, cin, rows, t, v, seed=cin)
    _check_mx4(hinm.quantize_mx4(pk), pk)


def test_quantize_every_scale_and_code():
    """Blocks around every power of two a bf16 can hold, half-way cases, subnormals, zeros, infinities and NaN."""
    pk = _pack(256, 512, 64, 0.0, 0.0, seed=1)                            # all dense: T 4, 16 blocks, 64 rows
    v = np.zeros((4, 16, 64, 32), np.float64)
    rng = np.random.default_rng(0)
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9, 0.24, 0.26, 1.24]
    e = np.arange(4 * 16 * 64).reshape(4, 16, 64) % 255 - 126             # 2^-126 .. 2^128 as the largest
    v[..., 0] = np.where(e > 127, 0.0, 1.0)
    v[..., 1:13] = np.array(mids) / 4
    v[..., 13:] = rng.uniform(-2, 2, (4, 16, 64, 19)) * (rng.uniform(size=(4, 16, 64, 19)) < 0.8)
    with np.errstate(over="ignore"):
        f = np.ldexp(v, e[..., None]).astype(np.float32)
    bits = (f.view(np.uint32) >> 16).astype(np.uint16)                    # cut to bf16
    bits[0, 0, 0] = 0
    bits[0, 0, 1] = 0x8000                                                # -0 everywhere
    bits[0, 0, 2, 5] = 0x7f80                                             # an infinity
    bits[0, 0, 3, 31] = 0xffc0                                            # a NaN
    bits[0, 0, 4] = 1                                                     # the smallest subnormal
    bits[0, 0, 5] = 0x7f7f                                                # the largest
    bits[0, 0, 6, :2] = [0x0080, 0x8001]                                  # the smallest normal and subnormal
    pk.val_dense.copy_(torch.from_numpy(bits.view(np.int16)))
    print("[mx4] every scale", flush=True)
    out = _check_mx4(hinm.quantize_mx4(pk), pk)
    assert np.isnan(out[0][0, 0, 2]).all() and np.isnan(out[0][0, 0, 3]).all()


def test_quantize_a_stack_and_its_own_lists():
    pk = [_pack(128, 132, 64, 0.7, 0.51, seed=s) for s in range(3)]
    q = hinm.quantize_mx4(hinm.Experts.stack(pk))
    for i, p in enumerate(pk):
        one = hinm.quantize_mx4(p)
        for b in hinm._MX4_BUFFERS:
            assert torch.equal(getattr(q, b)[i], getattr(one, b)), b
    # the lists are copies: translating the source's leaves the 4-bit weight alone
    one = hinm.quantize_mx4(pk[0])
    before = one.idx_24.clone()
    hinm.translate_indices(pk[0], torch.randperm(132, generator=torch.Generator().manual_seed(0)).int().to(DEV))
    assert torch.equal(one.idx_24, before) and not torch.equal(pk[0].idx_24, before)
    st = q.dequantize()
    assert isinstance(st, hinm.Experts) and st.n_experts == 3


# --------------------------------------------------------------------------- products

def _check_product(y, w, x, kept, what):
    wf, xf = w, _f64(x)
    err = np.abs(_f64(y) - wf @ xf)
    bound = mh.product_bound(wf, xf, kept)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} outputs off, the first at {np.argwhere(bad)[0].tolist()}"


@pytest.mark.parametrize("batch", [1, 2, 7, 8, 16, 17, 31, 33, 64, 65, 128, 130, 257, 300, 1031, 1040])
@pytest.mark.parametrize("cout,cin,rows,t,v", [(128, 300, 64, 0.75, 0.55), (192, 2052, 64, 0.5, 0.25)])
def test_product_with_four_bit_values(batch, cout, cin, rows, t, v):
    print(f"[mx4 spmm] {cout}x{cin} batch={batch}", flush=True)
    q = hinm.quantize_mx4(_pack(cout, cin, rows, t, v, seed=cin + 1))
    x = torch.randn(cin, batch, generator=torch.Generator().manual_seed(batch)).bfloat16().to(DEV)
    y = hinm.spmm(q, x)
    y2 = hinm.spmm(q, x)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))          # the same bits on every call
    _check_product(y, _dense(q.dequantize()), x, cin - q.plan.z, f"batch {batch}")


@pytest.mark.parametrize("cout,cin,rows,t,v", [(64, 4, 64, 0.0, 0.0), (256, 68, 128, 0.75, 0.5), (64, 64, 64, 0.9, 0.9),
                                               (192, 260, 192, 0.0, 0.0), (64, 8, 64, 0.5, 0.0),
                                               (64, 4100, 64, 0.6, 0.38), (128, 32, 64, 0.99, 0.99)])
@pytest.mark.parametrize("batch", [1, 5, 40, 200])
def test_product_corner_shapes(cout, cin, rows, t, v, batch):
    print(f"[mx4 spmm] {cout}x{cin} R={rows} t={t} v={v} batch={batch}", flush=True)
    q = hinm.quantize_mx4(_pack(cout, cin, rows, t, v, seed=7))
    x = torch.randn(cin, batch, generator=torch.Generator().manual_seed(batch)).bfloat16().to(DEV)
    y = hinm.spmm(q, x)
    torch.cuda.synchronize()
    _check_product(y, _dense(q.dequantize()), x, cin - q.plan.z, f"{cout}x{cin}")


def _ranges(counts, align, gap=0, lead=0):
    starts, at = [], lead
    for c in counts:
        starts.append(at)
        at += -(-c // align) * align + gap
    return starts, at


COUNTS = [([3, 0, 1, 9], 8), ([0, 0, 0, 0], 8), ([16, 17, 0, 15], 1), ([1, 1, 1, 1], 1), ([70, 5, 33, 64], 8),
          ([0, 300, 0, 2], 8), ([129, 128, 127, 130], 1), ([0, 0, 0, 600], 8), ([40, 257, 64, 65], 4), ([700, 3, 1025, 0], 8), ([1023, 65, 1, 300], 1)]


@pytest.mark.parametrize("counts,align", COUNTS)
@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("layout", ["tight", "gaps", "odd"])
def test_expert_products(counts, align, mx4, layout):
    """Ragged ranges, empty experts, columns between ranges left as they were, and unaligned layouts: "odd" has an
    odd row stride, an odd first column and odd starts."""
    cout, cin, t, v = 192, 516, 0.75, 0.55
    print(f"[experts] counts={counts} align={align} mx4={mx4} {layout}", flush=True)
    pk = [_pack(cout, cin, 64, t, v, seed=50 + i) for i in range(4)]
    st = hinm.Experts.stack(pk)
    if mx4:
        st = hinm.quantize_mx4(st)
        pk = [hinm.quantize_mx4(p).dequantize() for p in pk]
    gap, lead = {"tight": (0, 0), "gaps": (8, 16), "odd": (3, 1)}[layout]
    starts, cols = _ranges(counts, align, gap, lead)
    cols = max(cols, 1)
    g = torch.Generator().manual_seed(sum(counts) + align)
    ld = cols + (cols + 1) % 2 if layout == "odd" else -(-cols // 8) * 8
    store = torch.randn(cin * ld + 1, generator=g).bfloat16().to(DEV)
    off = 1 if layout == "odd" else 0
    x = store[off:off + cin * ld].view(cin, ld)[:, :cols]
    mine = torch.zeros(cols, dtype=torch.bool)
    for s, c in zip(starts, counts):
        mine[s:s + c] = True
    x[:, ~mine.to(DEV)] = float("nan")                                     # no other range's business
    i32 = lambda q: torch.tensor(q, dtype=torch.int32, device=DEV)
    r = hinm.Routing(i32([[0]]), torch.ones(1, 1, device=DEV), i32([[0]]), i32(starts + [cols]), i32(counts),
                     i32([0] * cols))
    ystore = torch.full((cout * ld + 1,), 7.0, dtype=torch.bfloat16, device=DEV)
    y = ystore[off:off + cout * ld].view(cout, ld)[:, :cols]
    hinm.spmm_experts(st, x, r, out=y)
    first = ystore.clone()
    hinm.spmm_experts(st, x, r, out=y)
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), ystore.view(torch.int16))  # the same bits on every call
    seen = torch.zeros_like(ystore, dtype=torch.bool)
    seen[off:off + cout * ld].view(cout, ld)[:, :cols][:, mine.to(DEV)] = True
    assert bool((ystore[~seen] == 7).all())                                # everything else as it was
    for e, (s, c) in enumerate(zip(starts, counts)):
        if c:
            _check_product(y[:, s:s + c], _dense(pk[e]), x[:, s:s + c], cin - pk[e].plan.z, f"expert {e}")


@pytest.mark.parametrize("mx4", [False, True])
def test_expert_products_clip_wild_ranges(mx4):
    """Ranges that leave the buffer are clipped to it; negative starts and counts give nothing."""
    pk = [_pack(64, 128, 64, 0.75, 0.55, seed=i) for i in range(5)]
    st = hinm.Experts.stack(pk)
    st = hinm.quantize_mx4(st) if mx4 else st
    x = torch.randn(128, 48, generator=torch.Generator().manual_seed(0)).bfloat16().to(DEV)
    i32 = lambda q: torch.tensor(q, dtype=torch.int32, device=DEV)
    r = hinm.Routing(i32([[0]]), torch.ones(1, 1, device=DEV), i32([[0]]), i32([-8, 8, 40, 16, 1 << 30, 0]),
                     i32([16, -3, 2 ** 31 - 1, 4, 7]), i32([0] * 48))
    y = torch.full((64, 48), 7.0, dtype=torch.bfloat16, device=DEV)
    print("[experts] wild ranges", flush=True)
    hinm.spmm_experts(st, x, r, out=y)
    torch.cuda.synchronize()
    keep = torch.ones(48, dtype=torch.bool, device=DEV)
    keep[40:], keep[16:20] = False, False
    assert bool((y[:, keep] == 7).all())
    d = st.dequantize() if mx4 else st
    one = lambda e: hinm.HinmPacked(d.plan, *[getattr(d, b)[e] for b in hinm._BUFFERS])
    _check_product(y[:, 40:], _dense(one(2)), x[:, 40:], 128, "expert 2")
    _check_product(y[:, 16:20], _dense(one(3)), x[:, 16:20], 128, "expert 3")


def test_pruned_rows_may_hold_nan():
    """A pruned X row that is not finite reaches no output, and neither does the row that a pad index stands for."""
    pk = _pack(64, 128, 64, 0.75, 0.55, seed=3)
    q = hinm.quantize_mx4(pk)
    used = set(_np(pk.idx_dense).ravel().tolist()) | set(_np(pk.idx_24).ravel().tolist())
    for batch in (1, 20, 150):
        x = torch.randn(128, batch, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
        x[[c for c in range(128) if c not in used]] = float("nan")
        y = hinm.spmm(q, x)
        torch.cuda.synchronize()
        assert torch.isfinite(y.float()).all()


# --------------------------------------------------------------------------- a layer

class Layer:
    """8 experts of gate, up and down projections: route, dispatch, two products, a gated activation, a product,
    combine."""

    def __init__(self, mx4, d=256, h=384, e=8, k=2, seed=0):
        mk = lambda a, b, s: hinm.Experts.stack([_pack(a, b, 64, 0.5, 0.25, seed=s + i) for i in range(e)])
        self.gate, self.up, self.down = mk(h, d, seed), mk(h, d, seed + 100), mk(d, h, seed + 200)
        if mx4:
            self.gate, self.up, self.down = map(hinm.quantize_mx4, (self.gate, self.up, self.down))
        self.k, self.e = k, e

    def __call__(self, x, logits):
        r = hinm.route(logits, self.k)
        xs = hinm.dispatch(x, r)
        g, u = hinm.spmm_experts(self.gate, xs, r), hinm.spmm_experts(self.up, xs, r)
        h = torch.nn.functional.silu(g) * u
        y = hinm.combine(hinm.spmm_experts(self.down, h, r), r)
        return r, xs, g, u, h, y


def _one(stack, e):
    d = stack.dequantize() if isinstance(stack, hinm.HinmMx4) else stack
    return _dense(hinm.HinmPacked(d.plan, *[getattr(d, b)[e] for b in hinm._BUFFERS]))


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("tokens", [1, 13, 200])
def test_layer(mx4, tokens):
    layer = Layer(mx4)
    gen = torch.Generator().manual_seed(tokens)
    x = torch.randn(256, tokens, generator=gen).bfloat16().to(DEV)
    logits = torch.randn(8, tokens, generator=gen).bfloat16().to(DEV)
    if tokens > 1:
        logits[:, 0] = float("-inf")                                       # a padded place of the batch
    print(f"[layer] tokens={tokens} mx4={mx4}", flush=True)
    r, xs, g, u, h, y = layer(x, logits)
    torch.cuda.synchronize()
    starts, counts = _np(r.starts), _np(r.counts)
    for stack, src, dst in ((layer.gate, xs, g), (layer.up, xs, u)):
        for e in range(8):
            s, c = int(starts[e]), int(counts[e])
            if c:
                _check_product(dst[:, s:s + c], _one(stack, e), src[:, s:s + c], stack.plan.cin, f"expert {e}")
    down = hinm.spmm_experts(layer.down, h, r)
    ref = np.zeros((256, tokens))
    mag = np.zeros((256, tokens))
    slots, w = _np(r.slots), _f64(r.weights)
    for e in range(8):
        s, c = int(starts[e]), int(counts[e])
        if c:
            _check_product(down[:, s:s + c], _one(layer.down, e), h[:, s:s + c], layer.down.plan.cin, f"down {e}")
    yd = _f64(down)
    for n in range(tokens):
        for j in range(2):
            if slots[n, j] >= 0:
                ref[:, n] += w[n, j] * yd[:, slots[n, j]]
                mag[:, n] += np.abs(w[n, j] * yd[:, slots[n, j]])
    acc = 2 * 2.0 ** -24 * mag * 1.01
    assert np.all(np.abs(_f64(y) - ref) <= acc + 2.0 ** -8 * (np.abs(ref) + acc) + 2.0 ** -134)
    if tokens > 1:
        assert bool((y[:, 0] == 0).all())


@pytest.mark.parametrize("mx4", [False, True])
def test_layer_in_graphs_on_two_streams(mx4):
    """Two captured layers of different sizes, replayed several times at once on two streams with eager calls
    between, against the eager results."""
    layer = Layer(mx4, seed=7)
    gen = torch.Generator().manual_seed(9)
    sizes = (24, 150)
    xs = [torch.randn(256, n, generator=gen).bfloat16().to(DEV) for n in sizes]
    ls = [torch.randn(8, n, generator=gen).bfloat16().to(DEV) for n in sizes]
    fresh = [[(torch.randn(256, n, generator=gen).bfloat16().to(DEV), torch.randn(8, n, generator=gen).bfloat16().to(DEV))
              for n in sizes] for _ in range(4)]
    for x, l in zip(xs, ls):
        layer(x, l)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, l in zip(xs, ls):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = layer(x, l)
        graphs.append(graph)
        outs.append((res[0].counts, res[-1]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        print(f"[layer] graph replay {rep}", flush=True)
        want = []
        for i in range(2):
            xs[i].copy_(fresh[rep][i][0])
            ls[i].copy_(fresh[rep][i][1])
            res = layer(xs[i], ls[i])
            want.append((res[0].counts.clone(), res[-1].clone()))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i][0], want[i][0]), (rep, i)
            assert torch.equal(outs[i][1].view(torch.int16), want[i][1].view(torch.int16)), (rep, i)


def test_layer_on_two_streams():
    layer = Layer(True, seed=3)
    gen = torch.Generator().manual_seed(4)
    args = [(torch.randn(256, n, generator=gen).bfloat16().to(DEV), torch.randn(8, n, generator=gen).to(DEV))
            for n in (16, 40)]
    want = [layer(*a)[-1].clone() for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    print("[layer] two streams", flush=True)
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(layer(*args[i])[-1])
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y.view(torch.int16), want[i].view(torch.int16))


# --------------------------------------------------------------------------- X held in LDS

@pytest.mark.parametrize("batch", [1, 2, 3, 4, 5, 8, 9, 15, 16])
@pytest.mark.parametrize("cout,cin,t,v", [(1024, 4100, 0.6, 0.38), (12800, 260, 0.75, 0.55), (4096, 1028, 0.5, 0.25)])
def test_product_of_few_tokens(cout, cin, t, v, batch):
    """Shapes on which the rows of X are held in LDS: row blocks cut between waves and between workgroups, and many
    row blocks a wave; contiguous X, and a slice whose rows are not aligned and whose buffer ends with an odd
    element."""
    print(f"[mx4 spmm] {cout}x{cin} batch={batch}", flush=True)
    q = hinm.quantize_mx4(_pack(cout, cin, 64, t, v, seed=cin))
    w = _dense(q.dequantize())
    g = torch.Generator().manual_seed(batch)
    for ld, first in ((batch, 0), (batch + 1 + batch % 2, 1)):
        store = torch.randn(cin * ld, generator=g).bfloat16().to(DEV)
        x = store.view(cin, ld)[:, ld - batch:]                 # the last row's last element ends the buffer
        y = hinm.spmm(q, x)
        y2 = hinm.spmm(q, x)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
        _check_product(y, w, x, cin - q.plan.z, f"batch {batch} ld {ld}")


@pytest.mark.parametrize("counts,align", [([2, 0, 16, 1, 5, 9, 0, 3], 8), ([0, 0, 0, 1, 0, 0, 0, 0], 8),
                                          ([7, 7, 7, 7, 7, 7, 7, 7], 1), ([40, 0, 0, 3, 0, 17, 0, 0], 8),
                                          ([0, 3, 0, 0, 0, 0, 0, 0], 1)])
@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("odd", [False, True])
def test_expert_products_of_few_tokens(counts, align, mx4, odd):
    cout, cin, t, v = 6400, 260, 0.75, 0.55
    print(f"[experts] few tokens counts={counts} align={align} mx4={mx4} odd={odd}", flush=True)
    pk = [_pack(cout, cin, 64, t, v, seed=80 + i) for i in range(8)]
    st = hinm.Experts.stack(pk)
    if mx4:
        st = hinm.quantize_mx4(st)
        pk = [hinm.quantize_mx4(p).dequantize() for p in pk]
    starts, cols = _ranges(counts, align, 3 if odd else 0, 1 if odd else 0)
    ld = cols + (cols + 1) % 2 if odd else -(-cols // 8) * 8
    g = torch.Generator().manual_seed(sum(counts))
    x = torch.randn(cin, ld, generator=g).bfloat16().to(DEV)[:, ld - cols:]
    i32 = lambda q: torch.tensor(q, dtype=torch.int32, device=DEV)
    r = hinm.Routing(i32([[0]]), torch.ones(1, 1, device=DEV), i32([[0]]), i32(starts + [cols]), i32(counts),
                     i32([0] * cols))
    mine = torch.zeros(cols, dtype=torch.bool)
    for s, c in zip(starts, counts):
        mine[s:s + c] = True
    x[:, ~mine.to(DEV)] = float("nan")
    y = torch.full((cout, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    hinm.spmm_experts(st, x, r, out=y)
    first = y.clone()
    hinm.spmm_experts(st, x, r, out=y)
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), y.view(torch.int16))
    assert bool((y[:, ~mine.to(DEV)] == 7).all())
    for e, (s, c) in enumerate(zip(starts, counts)):
        if c:
            _check_product(y[:, s:s + c], _dense(pk[e]), x[:, s:s + c], cin - pk[e].plan.z, f"expert {e}")


@pytest.mark.parametrize("mx4", [False, True])
def test_expert_products_past_32_bit_offsets(mx4):
    """Rows 2^24 bytes apart and more, the last of them past 2^32 bytes from the first, and a result as far apart."""
    cout, cin, ld, counts = 64, 264, (1 << 23) + 8, [5, 0, 33]
    pk = [_pack(cout, cin, 64, 0.5, 0.25, seed=90 + i) for i in range(3)]
    st = hinm.Experts.stack(pk)
    if mx4:
        st = hinm.quantize_mx4(st)
        pk = [hinm.quantize_mx4(p).dequantize() for p in pk]
    starts, cols = _ranges(counts, 8)
    x = torch.empty(cin * ld, dtype=torch.bfloat16, device=DEV).view(cin, ld)[:, :cols]
    y = torch.empty(cout * ld, dtype=torch.bfloat16, device=DEV).view(cout, ld)[:, :cols]
    x.copy_(torch.randn(cin, cols, generator=torch.Generator().manual_seed(4)).bfloat16())
    y.fill_(7.0)
    i32 = lambda q: torch.tensor(q, dtype=torch.int32, device=DEV)
    r = hinm.Routing(i32([[0]]), torch.ones(1, 1, device=DEV), i32([[0]]), i32(starts + [cols]), i32(counts),
                     i32([0] * cols))
    hinm.spmm_experts(st, x, r, out=y)
    for e, (s, c) in enumerate(zip(starts, counts)):
        if c:
            _check_product(y[:, s:s + c], _dense(pk[e]), x[:, s:s + c], cin - pk[e].plan.z, f"expert {e}")
        assert bool((y[:, s + c:starts[e + 1] if e < 2 else cols] == 7).all())
    if mx4:
        one = hinm.spmm(hinm.quantize_mx4(_pack(cout, cin, 64, 0.5, 0.25, seed=90)), x[:, :5], out=y[:, 8:13])
        assert torch.equal(one.view(torch.int16), y[:, :5].view(torch.int16))


@pytest.mark.parametrize("given", [False, True])
def test_products_of_one_workspace(given):
    """A product that copies X into the workspace, then one that counts arrivals there, each several times; the
    first is long enough that it does not split."""
    cout, cin, n = 2048, 1028, 3 * 2048 + 1
    q = hinm.quantize_mx4(_pack(cout, cin, 64, 0.5, 0.25, seed=5))
    gen = torch.Generator().manual_seed(6)
    xs = [torch.randn(cin, b, generator=gen).bfloat16().to(DEV) for b in (n, 1, 33, 300)]
    need = max(hinm.spmm_experts_workspace_bytes(q.plan, 1, x.shape[1], x.shape[1] % 8 == 0) for x in xs)
    want = [hinm.spmm(q, x, workspace=torch.zeros(need, dtype=torch.uint8, device=DEV)) for x in xs]
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV) if given else None
    for _ in range(3):
        for x, w in zip(xs, want):
            assert torch.equal(hinm.spmm(q, x, workspace=ws).view(torch.int16), w.view(torch.int16))
    if given:
        assert not bool(ws[:65536].any())


def test_workspaces_are_checked():
    q = hinm.quantize_mx4(_pack(64, 68, 64, 0.5, 0.25, seed=1))
    st = hinm.Experts.stack([_pack(64, 68, 64, 0.5, 0.25, seed=2)])
    x = torch.zeros(68, 8, dtype=torch.bfloat16, device=DEV)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    r = hinm.Routing(i32([[0]]), torch.ones(1, 1, device=DEV), i32([[0]]), i32([0, 8]), i32([8]), i32([0] * 8))
    for bad in (torch.zeros(1 << 24, dtype=torch.uint8), torch.zeros(1 << 24, dtype=torch.float32, device=DEV),
                torch.zeros(1 << 24, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError):
            hinm.spmm(q, x, workspace=bad)
        with pytest.raises(ValueError):
            hinm.spmm_experts(st, x, r, workspace=bad)
    for small in (0, 65536):
        with pytest.raises(hinm.HinmError):
            hinm.spmm_experts(st, x, r, workspace=torch.zeros(small, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("mx4", [False, True])
def test_layer_without_tokens(mx4):
    st = hinm.Experts.stack([_pack(128, 68, 64, 0.5, 0.25, seed=i) for i in range(3)])
    st = hinm.quantize_mx4(st) if mx4 else st
    r = hinm.route(torch.zeros(3, 0, dtype=torch.bfloat16, device=DEV), 2)
    xs = hinm.dispatch(torch.zeros(68, 0, dtype=torch.bfloat16, device=DEV), r)
    ys = hinm.spmm_experts(st, xs, r)
    y = hinm.combine(ys, r)
    torch.cuda.synchronize()
    assert r.counts.tolist() == [0, 0, 0] and y.shape == (128, 0)


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("e,most", [(300, 3), (1024, 1), (65, 90)])
def test_many_experts(e, most, mx4):
    """More experts than a wave has lanes, most of them with few columns or none, in both kernels."""
    pk = [_pack(64, 36, 64, 0.5, 0.25, seed=i) for i in range(5)]
    st = hinm.Experts.stack([pk[i % 5] for i in range(e)])
    if mx4:
        st = hinm.quantize_mx4(st)
        pk = [hinm.quantize_mx4(p).dequantize() for p in pk]
    g = torch.Generator().manual_seed(e)
    counts = torch.randint(0, most + 1, (e,), generator=g).tolist()
    starts, cols = _ranges(counts, 1, lead=2)
    x = torch.randn(36, cols, generator=g).bfloat16().to(DEV)
    i32 = lambda q: torch.tensor(q, dtype=torch.int32, device=DEV)
    r = hinm.Routing(i32([[0]]), torch.ones(1, 1, device=DEV), i32([[0]]), i32(starts + [cols]), i32(counts),
                     i32([0] * cols))
    y = hinm.spmm_experts(st, x, r)
    w = [_dense(p) for p in pk]
    for i, (s, c) in enumerate(zip(starts, counts)):
        if c:
            _check_product(y[:, s:s + c], w[i % 5], x[:, s:s + c], 36 - pk[0].plan.z, f"expert {i}")


def test_products_that_copy_x_in_graphs_on_two_streams():
    """Two graphs of a long product with unaligned rows and a split one, replayed together several times with eager
    work between."""
    q = hinm.quantize_mx4(_pack(2048, 1028, 64, 0.5, 0.25, seed=5))
    gen = torch.Generator().manual_seed(7)
    streams, graphs, outs, want = [torch.cuda.Stream() for _ in range(2)], [], [], []
    for s in streams:
        xs = [torch.randn(1028, b, generator=gen).bfloat16().to(DEV) for b in (6145, 1, 301)]
        want.append([hinm.spmm(q, x) for x in xs])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append([hinm.spmm(q, x) for x in xs])
        graphs.append((g, xs))
    for _ in range(4):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for (g, xs), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = hinm.spmm(q, graphs[0][1][1])
        torch.cuda.synchronize()
        assert torch.equal(eager.view(torch.int16), want[0][1].view(torch.int16))
        for o, w in zip(outs, want):
            for a, b in zip(o, w):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16))
