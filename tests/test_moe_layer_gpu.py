"""The mixture-of-experts layer for a few tokens on the GPU against a plain 64-bit form (fp8_helpers.moe_layer, which
derives the tolerance), and against the same layer made of router, dispatch, expert products and combine."""
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
QUANT = {"bf16": lambda s: s, "mx4": hinm.quantize_mx4, "fp8": hinm.quantize_fp8}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _stack(cout, cin, experts, t_s, v_s, values, seed, tile_rows=64):
    """A stack of random weights and the dense float64 weights it stands for."""
    g = torch.Generator().manual_seed(seed)
    packed = []
    for _ in range(experts):
        w = (torch.randn(cout, cin, generator=g) * torch.exp(0.5 * torch.randn(cin, generator=g)) * cin ** -0.5).bfloat16().to(DEV)
        perm = torch.stack([torch.randperm(cin, generator=g) for _ in range(cout // tile_rows)]).int().to(DEV)
        packed.append(hinm.pack(w, w.float().abs(), tile_rows, t_s, v_s, perm))
    dense = []
    for p in packed:
        full = p if values == "bf16" else QUANT[values](p).dequantize()
        bufs = device_packed_numpy(full)
        dense.append(mh.dense_from_packed(p.plan, bufs, mh.bf16_to_f64(bufs["val_dense"]), mh.bf16_to_f64(bufs["val_24"])))
    return QUANT[values](hinm.Experts.stack(packed)), dense


class Layer:
    def __init__(self, hidden, inter, experts, t_s=0.75, v_s=0.55, values="bf16", seed=0, rows=(64, 64)):
        self.gate, self.dg = _stack(inter, hidden, experts, t_s, v_s, values, seed, rows[0])
        self.up, self.du = _stack(inter, hidden, experts, t_s, v_s, values, seed + 1, rows[0])
        self.down, self.dd = _stack(hidden, inter, experts, t_s, v_s, values, seed + 2, rows[1])
        self.hidden, self.experts = hidden, experts
        self.kept = [p.n_dense + p.n_24 // 2 for p in (self.up.plan, self.down.plan)]

    def __call__(self, x, logits, k, renorm=True, **kw):
        return hinm.moe_layer(x, logits, self.gate, self.up, self.down, k, renormalize=renorm, **kw)

    def want(self, x, logits, k, renorm=True):
        return fh.moe_layer(_f64(logits), _f64(x), self.dg, self.du, self.dd, k, renorm, self.kept)


def _inputs(layer, n, seed, idle=0.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(layer.hidden, n, generator=g) * torch.exp(0.3 * torch.randn(layer.hidden, 1, generator=g))).bfloat16()
    logits = torch.randn(layer.experts, n, generator=g) * 2
    logits[:, torch.rand(n, generator=g) < idle] = float("-inf")
    return x.to(DEV), logits.to(dtype).to(DEV)


def _check(y, want, tol):
    err = np.abs(_f64(y) - want)
    assert np.all(err <= tol), float(np.nanmax(err / tol))


SHAPES = [(64, 64, 1, 1, 0.75, 0.55), (128, 192, 4, 2, 0.75, 0.55), (192, 128, 7, 3, 0.5, 0.25), (64, 320, 70, 8, 0.75, 0.5),
          (320, 64, 3, 3, 0.5, 0.5), (256, 128, 5, 2, 0.0, 0.0)]


@pytest.mark.parametrize("values", ["bf16", "mx4", "fp8"])
@pytest.mark.parametrize("hidden,inter,experts,k,t_s,v_s", SHAPES)
def test_layer(hidden, inter, experts, k, t_s, v_s, values):
    layer = Layer(hidden, inter, experts, t_s, v_s, values)
    for n in (1, 2, 4, 5, 8, 9, 16, 17, 31, 32):
        print(f"[moe] {hidden}x{inter} E={experts} k={k} {values} n={n}", flush=True)
        x, logits = _inputs(layer, n, n, idle=0.2 if n > 4 else 0.0, dtype=BF16 if n % 2 else torch.float32)
        renorm = n % 3 != 0
        y = layer(x, logits, k, renorm)
        torch.cuda.synchronize()
        _check(y, *layer.want(x, logits, k, renorm))
        assert torch.equal(layer(x, logits, k, renorm), y)


@pytest.mark.parametrize("rows", [(128, 64), (64, 128), (192, 128)])
@pytest.mark.parametrize("values", ["bf16", "mx4", "fp8"])
def test_tile_heights(rows, values):
    layer = Layer(384, 384, 3, values=values, rows=rows)
    x, logits = _inputs(layer, 6, 1)
    _check(layer(x, logits, 2), *layer.want(x, logits, 2))


def test_all_tokens_one_expert():
    """More tokens than a segment holds."""
    layer = Layer(128, 192, 4)
    x, logits = _inputs(layer, 32, 2)
    logits[:] = torch.tensor([0.0, 3.0, -float("inf"), 1.0], device=DEV)[:, None]
    for k in (1, 2, 4):
        _check(layer(x, logits, k), *layer.want(x, logits, k))


def test_wide_channels():
    """Channel counts at which a segment holds 16, 8 or 4 tokens."""
    for hidden, inter in ((4096, 128), (4160, 64), (64, 8192), (64, 8256), (64, 11008), (64, 16384), (16384, 64)):
        print(f"[moe] {hidden}x{inter}", flush=True)
        layer = Layer(hidden, inter, 2, seed=hidden + inter)
        for n in (1, 7, 20):
            x, logits = _inputs(layer, n, n)
            _check(layer(x, logits, 1 + n % 2), *layer.want(x, logits, 1 + n % 2))


def test_special_logits():
    """NaN and -inf are not eligible, +inf shares the weight, a token without an expert gives +0, equal logits take the
    lower expert."""
    inf, nan = float("inf"), float("nan")
    rows = torch.tensor([[0.0, 0.0, 0.0, 0.0], [-inf, -inf, -inf, -inf], [nan, 1.0, nan, -inf], [nan, nan, nan, nan],
                         [inf, 3.0, inf, inf], [5.0, inf, 5.0, -inf], [-inf, 2.0, 2.0, 2.0], [1e38, -1e38, 0.0, 3e38],
                         [-3e38, -inf, -3e38, -3e38], [0.0, -0.0, 0.0, -0.0]])
    layer = Layer(128, 64, 4)
    x, _ = _inputs(layer, 10, 3)
    for dt in (torch.float32, BF16):
        logits = rows.to(dt).t().contiguous().to(DEV)
        for k in (1, 2, 4):
            for renorm in (True, False):
                y = layer(x, logits, k, renorm)
                ref = _f64(logits)
                want, tol = fh.moe_layer(ref, _f64(x), layer.dg, layer.du, layer.dd, k, renorm, layer.kept)
                _check(y, want, tol)
                assert bool((y.view(torch.int16)[:, [1, 3]] == 0).all())


def test_non_finite_stays_with_its_token():
    """NaN in one token, and in the weights of an expert that other tokens did not choose."""
    layer = Layer(128, 192, 4)
    x, logits = _inputs(layer, 12, 4)
    logits[:, :6] = torch.tensor([1.0, 0.0, -float("inf"), -float("inf")], device=DEV)[:, None]
    logits[:, 6:] = torch.tensor([1.0, -float("inf"), 0.0, -float("inf")], device=DEV)[:, None]
    clean = layer(x, logits, 2).clone()
    bad = x.clone()
    bad[:, 3] = float("nan")
    y = layer(bad, logits, 2)
    keep = [i for i in range(12) if i != 3]
    assert torch.equal(y[:, keep], clean[:, keep]) and bool(y[:, 3].isnan().all())
    for w in (layer.gate, layer.up, layer.down):
        w.val_24[1:2].fill_(0x7fc0)
        w.val_24[3:4].fill_(0x7fc0)
    y = layer(x, logits, 2)
    assert torch.equal(y[:, 6:], clean[:, 6:]) and bool(y[:, :6].isnan().all())


@pytest.mark.parametrize("pad", [(0, 0), (1, 3), (8, 8)])
def test_strided(pad):
    """Slices of wider matrices, their surroundings NaN and left as they were."""
    layer = Layer(192, 128, 5)
    n = 11
    x, logits = _inputs(layer, n, 5)
    want = layer(x, logits, 2)

    def wide(t):
        box = torch.full((t.shape[0], n + sum(pad)), float("nan"), dtype=t.dtype, device=DEV)
        box[:, pad[0]:pad[0] + n] = t
        return box[:, pad[0]:pad[0] + n]
    out = torch.full((192, n + sum(pad)), 7.0, dtype=BF16, device=DEV)
    y = layer(wide(x), wide(logits), 2, out=out[:, pad[0]:pad[0] + n])
    assert torch.equal(y, want)
    assert bool((out[:, :pad[0]] == 7).all()) and bool((out[:, pad[0] + n:] == 7).all())


@pytest.mark.parametrize("values", ["bf16", "mx4", "fp8"])
def test_against_the_chain(values):
    """route -> dispatch -> three expert products -> combine: more roundings (g, u and each expert's output to bf16;
    with 8-bit values the activations to 8 bits), so close, not equal."""
    layer = Layer(256, 384, 6, values=values)
    x, logits = _inputs(layer, 24, 6)
    y = layer(x, logits, 2).double()
    r = hinm.route(logits, 2)
    xs = hinm.dispatch(x, r)
    g, u = (hinm.spmm_experts(w, xs, r).float() for w in (layer.gate, layer.up))
    h = torch.where(r.src >= 0, torch.nn.functional.silu(g) * u, 0.0).bfloat16()
    z = hinm.combine(hinm.spmm_experts(layer.down, h, r), r).double()
    # 8-bit activations: x and h off by 2^-4 of the value at most, three products deep
    assert (y - z).norm() <= (0.15 if values == "fp8" else 0.02) * y.norm()


def test_zero_tokens():
    layer = Layer(64, 64, 2)
    x, logits = _inputs(layer, 0, 1)
    assert layer(x, logits, 1).shape == (64, 0)


@pytest.mark.parametrize("n,k", [(1, 1), (9, 2), (32, 4)])
def test_graph_and_streams(n, k):
    """Captured with its own workspace and replayed between eager calls on new inputs; two streams at once."""
    layer = Layer(256, 320, 6)
    x, logits = _inputs(layer, n, 7)
    want = layer(x, logits, k).clone()
    x2, logits2 = _inputs(layer, n, 8)
    want2 = layer(x2, logits2, k).clone()
    sx, sl, out = x.clone(), logits.clone(), torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(sx, sl, k, out=out)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(sx, sl, k, out=out)
    for i in range(5):
        sx.copy_(x2 if i % 2 else x)
        sl.copy_(logits2 if i % 2 else logits)
        g.replay()
        layer(x, logits, k)
        torch.cuda.synchronize()
        assert torch.equal(out, want2 if i % 2 else want)
    torch.cuda.synchronize()
    ys = []
    for i in range(6):
        with torch.cuda.stream(s if i % 2 else torch.cuda.current_stream()):
            ys.append(layer(x, logits, k))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)


@pytest.mark.parametrize("experts,k", [(16, 16), (40, 16), (260, 4), (520, 8)])
def test_many_pairs(experts, k):
    """Up to 512 pairs of a token and an expert, and more segments than share the workgroups evenly."""
    layer = Layer(64, 64, experts, seed=experts)
    for n in (1, 3, 32):
        print(f"[moe] E={experts} k={k} n={n}", flush=True)
        x, logits = _inputs(layer, n, n)
        _check(layer(x, logits, k), *layer.want(x, logits, k))


@pytest.mark.parametrize("values", ["bf16", "mx4", "fp8"])
def test_many_blocks(values):
    """Several turns of every wave, in both kernels, and shares that end inside an expert."""
    layer = Layer(1024, 1088, 5, values=values, seed=3)
    for n in (1, 2, 6, 21, 32):
        print(f"[moe] blocks {values} n={n}", flush=True)
        x, logits = _inputs(layer, n, n)
        _check(layer(x, logits, 2), *layer.want(x, logits, 2))


def test_tokens_of_one_column_block():
    """Tokens 8 g .. 8 g + 7 are loaded together: an expert's tokens from one, two and all such groups."""
    layer = Layer(128, 128, 2, seed=5)
    x, logits = _inputs(layer, 30, 5)
    for mine in (range(24, 30), range(6, 10), range(0, 30, 3), range(29, 30), range(7, 8)):
        logits[0], logits[1] = 0.0, 1.0
        logits[0, list(mine)] = 2.0
        _check(layer(x, logits, 1), *layer.want(x, logits, 1))


def test_layers_on_two_streams():
    layer = Layer(128, 192, 4, seed=8)
    ins = [_inputs(layer, n, n) for n in (1, 32, 2, 9)]
    want = [layer(x, l, 2).clone() for x, l in ins]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(16):
        with torch.cuda.stream(streams[i % 2]):
            got.append((i % 4, layer(*ins[i % 4], 2)))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for k, y in got)


@pytest.mark.parametrize("values", ["bf16", "mx4", "fp8"])
def test_infinite_products(values):
    """A token whose inner values pass bf16's range gets infinities of the right signs, or NaN where they meet; the
    other tokens keep their results."""
    layer = Layer(128, 64, 2, t_s=0.0, v_s=0.0, values=values, seed=9)
    x, logits = _inputs(layer, 5, 9)
    want = layer(x, logits, 1)
    x[:, 2] *= 2.0 ** 70
    with np.errstate(over="ignore", invalid="ignore"):
        w = layer.dg, layer.du, layer.dd
        e = int(_f64(logits)[:, 2].argmax())
        g, u = (m[e] @ _f64(x[:, 2]) for m in w[:2])
        h = np.where(g > 0, g, 0.0) * u                        # silu(g) of so large a g
        hot = np.abs(h) > 2.0 ** 129                           # infinite in fp32 and bf16; others finite
        assert hot.any() and np.all(hot | (np.abs(h) < 2.0 ** 127))
    y = layer(x, logits, 1)
    keep = [0, 1, 3, 4]
    assert torch.equal(y[:, keep], want[:, keep])
    part = w[2][e][:, hot] * np.sign(h[hot])
    up, down = (part > 0).any(1), (part < 0).any(1)
    got = _f64(y[:, 2])
    assert np.all(np.isnan(got[up & down])) and np.all(got[up & ~down] == np.inf) and np.all(got[~up & down] == -np.inf)
