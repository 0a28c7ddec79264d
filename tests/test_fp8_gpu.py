"""8-bit values and their products on the GPU against plain 64-bit forms (fp8_helpers).

Codes and scales are equal to the definition's; a product's bound is moe_helpers.product_bound with the rounded
operands: products of codes and powers of two are exact, so the sums are those of a bf16 product.
"""
import numpy as np
import pytest
import torch

import fp8_helpers as fh
import moe_helpers as mh
from helpers import device_packed_numpy

pytestmark = pytest.mark.gpu
hinm = pytest.importorskip("structured_sparse_gemm_amd")
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def _np(t):
    return t.detach().cpu().numpy()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _packed(cout, cin, t_s=0.75, v_s=0.55, seed=0, tile_rows=64, scale=0.02):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(cout, cin, generator=g) * torch.exp(torch.randn(cin, generator=g)) * scale).bfloat16().to(DEV)
    perm = torch.stack([torch.randperm(cin, generator=g) for _ in range(cout // tile_rows)]).int().to(DEV)
    return hinm.pack(w, w.float().abs(), tile_rows, t_s, v_s, perm)


def _dense(packed8):
    """The weight an 8-bit packed weight stands for, float64 [cout, cin], from its buffers."""
    full = packed8.dequantize()
    code = {k: _np(getattr(packed8, k).view(torch.uint8)) for k in ("val_dense", "val_24")}
    return mh.dense_from_packed(packed8.plan, device_packed_numpy(full), fh.values_of(code["val_dense"], _np(packed8.scale_dense)),
                                fh.values_of(code["val_24"], _np(packed8.scale_24)))


def _kept_mask(packed8):
    """Where the weight keeps a value, whatever it is."""
    full = device_packed_numpy(packed8.dequantize())
    one = {k: np.ones(full[k].shape) for k in ("val_dense", "val_24")}
    return mh.dense_from_packed(packed8.plan, full, one["val_dense"], one["val_24"]) != 0


def _x(cin, n, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(cin, n, generator=g) * torch.exp(0.5 * torch.randn(cin, 1, generator=g))
    return x.bfloat16()


def _check(y, w, x, kept):
    xq = fh.columns(_f64(x))
    err = np.abs(_f64(y) - w @ xq)
    assert np.all(err <= mh.product_bound(w, xq, kept)), float((err / mh.product_bound(w, xq, kept)).max())


SHAPES = [(64, 64, 0.5, 0.25), (128, 256, 0.75, 0.55), (192, 132, 0.7, 0.51), (64, 1500, 0.75, 0.5),
          (128, 700, 0.5, 0.5), (128, 320, 0.5, 0.0), (64, 48, 0.0, 0.0), (64, 16, 0.99, 0.98)]


@pytest.mark.parametrize("cout,cin,t_s,v_s", SHAPES)
def test_quantize(cout, cin, t_s, v_s):
    """Every code and scale, and the exact way back; the lists are copied."""
    print(f"[fp8] quantize {cout}x{cin} {t_s} {v_s}", flush=True)
    pk = _packed(cout, cin, t_s, v_s, seed=cin)
    q = hinm.quantize_fp8(pk)
    back = q.dequantize()
    torch.cuda.synchronize()
    for k in ("val_dense", "val_24"):
        bits = _np(getattr(pk, k)).view(np.uint16)
        code, scale, value = fh.weight_buffers(bits)
        assert np.array_equal(_np(getattr(q, k).view(torch.uint8)), code), k
        assert np.array_equal(_np(getattr(q, k.replace("val", "scale"))), scale), k
        assert np.array_equal(mh.bf16_to_f64(_np(getattr(back, k)).view(np.uint16)), value), k
    for k in ("idx_dense", "idx_24", "meta_24"):
        assert torch.equal(getattr(q, k), getattr(pk, k)) and torch.equal(getattr(back, k), getattr(pk, k)), k
    assert back.flags == pk.flags


def test_quantize_special_values():
    """Zeros, the smallest and largest magnitudes, half-way cases, values past 448 * 2^119, NaN and infinities."""
    pk = _packed(64, 512, 0.5, 0.25, seed=3)
    g = np.random.default_rng(0)
    for name in ("val_dense", "val_24"):
        bits = g.integers(0, 1 << 16, getattr(pk, name).shape, dtype=np.uint16)
        bits[:, :, 0] = 0
        bits[:, :, 1] = 0x8000
        bits[:, :, 2] = g.integers(0, 128, bits[:, :, 2].shape)                       # subnormal
        bits[:, :, 3] = 0x7f7f
        bits[:, :, 4] = 0x7f80
        bits[:, :, 5] = np.where(g.random(bits[:, :, 5].shape) < 0.1, 0x7fc0, 0x3f80 + g.integers(0, 256, bits[:, :, 5].shape))
        bits[:, :, 6] = 0x3f80 | g.integers(0, 128, bits[:, :, 6].shape)               # [1, 2): every half-way case
        bits[:, :, 7] = (g.integers(100, 140, bits[:, :, 7].shape) << 7) | 0x60        # 1.75 * 2^k
        bits[:, :, 8] = 0xff80
        getattr(pk, name).copy_(torch.from_numpy(bits.view(np.int16)).to(DEV))
    q = hinm.quantize_fp8(pk)
    back = q.dequantize()
    torch.cuda.synchronize()
    for k in ("val_dense", "val_24"):
        code, scale, value = fh.weight_buffers(_np(getattr(pk, k)).view(np.uint16))
        assert np.array_equal(_np(getattr(q, k).view(torch.uint8)), code), k
        assert np.array_equal(_np(getattr(q, k.replace("val", "scale"))), scale), k
        got = mh.bf16_to_f64(_np(getattr(back, k)).view(np.uint16))
        assert np.array_equal(got, value, equal_nan=True), k


def test_quantize_stack():
    packed = [_packed(128, 300, seed=s) for s in range(3)]
    q = hinm.quantize_fp8(hinm.Experts.stack(packed))
    for e, p in enumerate(packed):
        one = hinm.quantize_fp8(p)
        for k in hinm._MX4_BUFFERS:
            a, b = getattr(q, k)[e], getattr(one, k)
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k
    back = q.dequantize()
    assert isinstance(back, hinm.Experts) and back.n_experts == 3


@pytest.mark.parametrize("n", [1, 2, 5, 8, 9, 16, 17, 33, 64, 100, 200, 257])
@pytest.mark.parametrize("cout,cin,t_s,v_s", SHAPES)
def test_product(cout, cin, t_s, v_s, n):
    print(f"[fp8] product {cout}x{cin} {t_s} {v_s} n={n}", flush=True)
    q = hinm.quantize_fp8(_packed(cout, cin, t_s, v_s, seed=cin + 1))
    x = _x(cin, n, n).to(DEV)
    y = hinm.spmm(q, x)
    torch.cuda.synchronize()
    _check(y, _dense(q), x, q.plan.n_dense + q.plan.n_24 // 2)
    assert torch.equal(hinm.spmm(q, x), y)


@pytest.mark.parametrize("n", [1, 7, 16, 31, 130])
@pytest.mark.parametrize("pad", [(1, 0), (3, 5), (8, 8)])
def test_product_strided(n, pad):
    """Slices of wider matrices, their surroundings NaN and left as they were."""
    q = hinm.quantize_fp8(_packed(128, 600, seed=9))
    x = _x(600, n, n).to(DEV)
    box = torch.full((600, n + sum(pad)), float("nan"), dtype=BF16, device=DEV)
    box[:, pad[0]:pad[0] + n] = x
    out = torch.full((128, n + sum(pad)), 7.0, dtype=BF16, device=DEV)
    y = hinm.spmm(q, box[:, pad[0]:pad[0] + n], out=out[:, pad[0]:pad[0] + n])
    torch.cuda.synchronize()
    assert torch.equal(y, hinm.spmm(q, x))
    assert bool((out[:, :pad[0]] == 7).all()) and bool((out[:, pad[0] + n:] == 7).all())


@pytest.mark.parametrize("n", [4, 40, 150])
def test_product_non_finite(n):
    """A NaN or an infinity makes NaN of its token's outputs whose rows keep its channel and leaves all others, and
    the other tokens, as they are; a token of zeros gives zeros."""
    q = hinm.quantize_fp8(_packed(192, 320, seed=4))
    w = _dense(q)
    x = _x(320, n, 5)
    x[17, 1], x[200, 2], x[:, 3] = float("nan"), float("-inf"), 0.0
    y = _f64(hinm.spmm(q, x.to(DEV)))
    kept = q.plan.n_dense + q.plan.n_24 // 2
    clean = x.clone()
    clean[17, 1], clean[200, 2] = 0.0, 0.0
    xq = fh.columns(_f64(clean))
    bad = np.zeros(y.shape, bool)
    bad[:, 1], bad[:, 2] = _kept_mask(q)[:, 17], _kept_mask(q)[:, 200]
    assert bad.any() and np.isnan(y[bad]).all()
    assert np.all(np.abs(y - w @ xq)[~bad] <= mh.product_bound(w, xq, kept)[~bad])
    assert np.all(y[:, 3] == 0)


@pytest.mark.parametrize("power", [-120, -60, 60, 110])
def test_product_far_scales(power):
    """Tokens of very different sizes: the scale is the token's own."""
    q = hinm.quantize_fp8(_packed(64, 256, seed=6))
    x = _x(256, 20, 6).float()
    x[:, ::2] *= 2.0 ** power
    x = x.bfloat16().to(DEV)
    y = hinm.spmm(q, x)
    _check(y, _dense(q), x, q.plan.n_dense + q.plan.n_24 // 2)


def _ranges(counts, starts, n_cols):
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    s = torch.tensor([*starts, n_cols], dtype=torch.int32, device=DEV)
    z = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    return hinm.Routing(z, z.float(), z, s, c, torch.zeros(n_cols, dtype=torch.int32, device=DEV))


CASES = [([3, 0, 17, 1], [0, 8, 8, 32], 40), ([0, 0, 0, 0], [0, 0, 0, 0], 8), ([5, 300, 2, 130], [0, 8, 308, 312], 450),
         ([40, 40, 40, 40], [1, 43, 90, 131], 171), ([600, 1, 0, 0], [0, 600, 608, 608], 608)]


@pytest.mark.parametrize("counts,starts,cols", CASES)
@pytest.mark.parametrize("cout,cin,t_s,v_s", [(128, 256, 0.75, 0.55), (64, 1500, 0.75, 0.5), (192, 132, 0.5, 0.25)])
def test_experts(cout, cin, t_s, v_s, counts, starts, cols):
    """Ragged ranges, aligned and not; columns between them keep what they held."""
    print(f"[fp8] experts {cout}x{cin} counts={counts}", flush=True)
    packed = [_packed(cout, cin, t_s, v_s, seed=s) for s in range(4)]
    q = hinm.quantize_fp8(hinm.Experts.stack(packed))
    x = _x(cin, cols, cols).to(DEV)
    out = torch.full((cout, cols), 7.0, dtype=BF16, device=DEV)
    hinm.spmm_experts(q, x, _ranges(counts, starts, cols), out=out)
    torch.cuda.synchronize()
    rest = np.ones(cols, bool)
    for e in range(4):
        at = slice(starts[e], starts[e] + counts[e])
        rest[at] = False
        _check(out[:, at], _dense(hinm.quantize_fp8(packed[e])), x[:, at], q.plan.n_dense + q.plan.n_24 // 2)
    assert bool((out[:, torch.from_numpy(rest).to(DEV)] == 7).all())


def test_experts_out_of_range():
    """Ranges past the buffer are clipped to it."""
    q = hinm.quantize_fp8(hinm.Experts.stack([_packed(64, 256, seed=s) for s in range(3)]))
    x = _x(256, 30, 1).to(DEV)
    out = torch.full((64, 30), 7.0, dtype=BF16, device=DEV)
    hinm.spmm_experts(q, x, _ranges([9, 5, 9], [-4, 3, 25], 30), out=out)
    one = [hinm.quantize_fp8(_packed(64, 256, seed=s)) for s in range(3)]
    want = torch.full((64, 30), 7.0, dtype=BF16, device=DEV)
    want[:, 3:8], want[:, 25:30] = hinm.spmm(one[1], x[:, 3:8].contiguous()), hinm.spmm(one[2], x[:, 25:30].contiguous())
    kept = q.plan.n_dense + q.plan.n_24 // 2
    _check(out[:, 3:8], _dense(one[1]), x[:, 3:8], kept)
    _check(out[:, 25:30], _dense(one[2]), x[:, 25:30], kept)
    assert bool((out[:, :3] == 7).all()) and bool((out[:, 8:25] == 7).all())


def test_zero_columns():
    q = hinm.quantize_fp8(_packed(64, 256))
    assert hinm.spmm(q, torch.zeros(256, 0, dtype=BF16, device=DEV)).shape == (64, 0)


def test_checkpoint(tmp_path):
    q = hinm.quantize_fp8(_packed(128, 300, seed=2))
    torch.save(q.state_dict(), tmp_path / "w.pt")
    r = hinm.HinmFp8.from_state_dict(torch.load(tmp_path / "w.pt", weights_only=True), DEV)
    x = _x(300, 9, 1).to(DEV)
    assert torch.equal(hinm.spmm(q, x), hinm.spmm(r, x)) and r.flags == q.flags


@pytest.mark.parametrize("n", [1, 16, 300])
def test_graph_and_streams(n):
    """Captured with its own workspace and replayed between eager calls; two streams at once."""
    q = hinm.quantize_fp8(_packed(128, 1500, seed=8))
    x = _x(1500, n, 3).to(DEV)
    want = hinm.spmm(q, x).clone()
    out = torch.empty_like(want)
    other = _x(1500, n, 4).to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        hinm.spmm(q, x, out=out)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hinm.spmm(q, x, out=out)
    for _ in range(4):
        out.zero_()
        g.replay()
        hinm.spmm(q, other)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    ys = []
    for k in range(4):
        with torch.cuda.stream(s if k % 2 else torch.cuda.current_stream()):
            ys.append(hinm.spmm(q, x))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)


@pytest.mark.parametrize("cin", [4096, 4100, 8192, 8196, 9428, 9432, 18860, 18864, 20000])
def test_product_many_channels(cin):
    """Channel counts at which LDS holds 16, 8 or no columns, and one pass of loads or more cover them."""
    q = hinm.quantize_fp8(_packed(64, cin, 0.75, 0.55, seed=cin))
    w = _dense(q)
    for n in (1, 2, 7, 8, 9, 15, 16, 23, 40):
        print(f"[fp8] channels {cin} n={n}", flush=True)
        x = _x(cin, n, n).to(DEV)
        y = hinm.spmm(q, x)
        torch.cuda.synchronize()
        _check(y, w, x, q.plan.n_dense + q.plan.n_24 // 2)


@pytest.mark.parametrize("n", [1, 6, 8, 13, 16])
def test_product_last_channels(n):
    """Kept channels at the very end of X, of whose rows the loads begin early."""
    p = _packed(64, 64, 0.0, 0.0, seed=n)
    q = hinm.quantize_fp8(p)
    x = torch.zeros(64, n, dtype=BF16)
    x[-9:] = _x(9, n, n)
    x = x.to(DEV)
    _check(hinm.spmm(q, x), _dense(q), x, q.plan.n_dense + q.plan.n_24 // 2)


@pytest.mark.parametrize("experts", [1, 2, 31, 33, 64, 300])
@pytest.mark.parametrize("most", [1, 8, 19, 45])
def test_experts_few_tokens(experts, most):
    """Up to 32 segments share the workgroups evenly, more in contiguous ranges; some of none."""
    rng = np.random.default_rng(experts + most)
    counts = rng.integers(0, most + 1, experts)
    starts = np.cumsum(counts + rng.integers(0, 3, experts)) - counts
    cols = int(starts[-1] + counts[-1] + 2)
    print(f"[fp8] few tokens E={experts} counts up to {most} columns {cols}", flush=True)
    made = [_packed(128, 260, seed=s) for s in range(min(experts, 5))]
    q = hinm.quantize_fp8(hinm.Experts.stack([made[e % len(made)] for e in range(experts)]))
    dense = [_dense(hinm.quantize_fp8(m)) for m in made]
    x = _x(260, cols, cols).to(DEV)
    out = torch.full((128, cols), 7.0, dtype=BF16, device=DEV)
    hinm.spmm_experts(q, x, _ranges(counts.tolist(), starts.tolist(), cols), out=out)
    torch.cuda.synchronize()
    rest = np.ones(cols, bool)
    for e in range(experts):
        at = slice(int(starts[e]), int(starts[e] + counts[e]))
        rest[at] = False
        if counts[e]:
            _check(out[:, at], dense[e % len(made)], x[:, at], q.plan.n_dense + q.plan.n_24 // 2)
    assert bool((out[:, torch.from_numpy(rest).to(DEV)] == 7).all())


@pytest.mark.parametrize("cin", [7892, 7896, 8916, 8920, 15788, 15792, 17836, 17840])
def test_experts_many_channels(cin):
    """Items of 64, 32 and 16 rows: the sums of more rows leave LDS less room for channels."""
    one = _packed(256, cin, 0.75, 0.55, seed=cin)
    q = hinm.quantize_fp8(hinm.Experts.stack([one] * 64))
    rng = np.random.default_rng(cin)
    counts = rng.integers(*((9, 17) if cin < 9000 else (0, 9)), 64)
    starts = np.cumsum(counts) - counts
    cols = int(counts.sum())
    print(f"[fp8] experts of {cin} channels, {cols} columns", flush=True)
    x = _x(cin, cols, cin).to(DEV)
    out = hinm.spmm_experts(q, x, _ranges(counts.tolist(), starts.tolist(), cols))
    torch.cuda.synchronize()
    _check(out, _dense(hinm.quantize_fp8(one)), x, q.plan.n_dense + q.plan.n_24 // 2)


@pytest.mark.parametrize("rows", [128, 192])
@pytest.mark.parametrize("n", [1, 20, 200])
def test_product_tile_heights(rows, n):
    q = hinm.quantize_fp8(_packed(384, 700, 0.75, 0.55, seed=rows, tile_rows=rows))
    x = _x(700, n, n).to(DEV)
    _check(hinm.spmm(q, x), _dense(q), x, q.plan.n_dense + q.plan.n_24 // 2)


def test_same_weight_on_two_streams():
    """Workspaces are the stream's: long and short products on two streams at once."""
    q = hinm.quantize_fp8(_packed(256, 1500, seed=3))
    xs = [_x(1500, n, n).to(DEV) for n in (300, 4, 150, 1)]
    want = [hinm.spmm(q, x).clone() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(16):
        with torch.cuda.stream(streams[i % 2]):
            got.append((i % 4, hinm.spmm(q, xs[i % 4])))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for k, y in got)


def _check_some(y, q, x, cols):
    """Of a product with many columns, those."""
    xs = x[:, cols]
    _check(y[:, cols], _dense(q), xs, q.plan.n_dense + q.plan.n_24 // 2)


def test_product_in_windows():
    """So many columns that their rounded values are made and multiplied in two windows of 16384."""
    q = hinm.quantize_fp8(_packed(64, 65536, 0.99, 0.985, seed=1))
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(65536, 16500, device=DEV, generator=g, dtype=BF16)
    print("[fp8] windows, one weight", flush=True)
    y = hinm.spmm(q, x)
    torch.cuda.synchronize()
    _check_some(y, q, x, [0, 1, 8191, 16383, 16384, 16385, 16499])


def test_experts_in_windows():
    """A range that two windows share, one in each, and a gap between the windows' last and first columns."""
    one = _packed(64, 65536, 0.99, 0.985, seed=2)
    q, e = hinm.quantize_fp8(hinm.Experts.stack([one] * 4)), hinm.quantize_fp8(one)
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(65536, 16600, device=DEV, generator=g, dtype=BF16)
    for starts, counts in (([0, 300, 16400, 16500], [290, 16080, 90, 100]), ([5, 8000, 16390, 16390], [7000, 8380, 0, 210])):
        print(f"[fp8] windows, experts {starts} {counts}", flush=True)
        out = torch.full((64, 16600), 7.0, dtype=BF16, device=DEV)
        hinm.spmm_experts(q, x, _ranges(counts, starts, 16600), out=out)
        torch.cuda.synchronize()
        used = np.zeros(16600, bool)
        for s, c in zip(starts, counts):
            used[s:s + c] = True
        _check_some(out, e, x, [c for c in (5, 301, 8100, 16379, 16383, 16384, 16400, 16599) if used[c]])
        assert bool((out[:, torch.from_numpy(~used).to(DEV)] == 7).all())


@pytest.mark.parametrize("n", [65, 95, 96, 97])
def test_product_several_segments(n):
    """One weight's columns in up to six segments of sixteen, and the first count that takes the other kernel."""
    q = hinm.quantize_fp8(_packed(320, 600, 0.75, 0.55, seed=n))
    x = _x(600, n, n).to(DEV)
    y = hinm.spmm(q, x)
    torch.cuda.synchronize()
    _check(y, _dense(q), x, q.plan.n_dense + q.plan.n_24 // 2)
    assert torch.equal(hinm.spmm(q, x), y)
