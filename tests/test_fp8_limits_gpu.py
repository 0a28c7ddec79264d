"""8-bit products at the upper end of bf16's range: no finite activation becomes infinite.

The activations' scale is at most 2^119, as the weights' is, and larger values saturate at 448 * 2^119 = 1.75 * 2^127,
so that every code times its scale is a bf16 value (256 * 2^120 would be 2^128, which bf16 does not have).  The bound
is moe_helpers.product_bound with the rounded operands: codes times powers of two are exact, and the weights are small
enough for every sum to stay below 2^127.
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
# 448 * 2^119, the next value, the last that rounds to code 240 at 2^120, the first that would round to 256, the largest
TOPS = (0x7f60, 0x7f61, 0x7f77, 0x7f78, 0x7f7f)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _bits(v):
    return torch.tensor([v], dtype=torch.int32).to(torch.int16).view(BF16)[0]


def _weight(cout, cin, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(cout, cin, generator=g) * 2.0 ** -14).bfloat16().to(DEV)
    perm = torch.stack([torch.randperm(cin, generator=g) for _ in range(cout // 64)]).int().to(DEV)
    return hinm.quantize_fp8(hinm.pack(w, w.float().abs(), 64, 0.5, 0.25, perm))


def _dense(q):
    full = q.dequantize()
    code = {k: getattr(q, k).view(torch.uint8).cpu().numpy() for k in ("val_dense", "val_24")}
    return mh.dense_from_packed(q.plan, device_packed_numpy(full), fh.values_of(code["val_dense"], q.scale_dense.cpu().numpy()),
                                fh.values_of(code["val_24"], q.scale_24.cpu().numpy()))


def _columns(x):
    """What the codes stand for, by the definition: scales up to 2^119, saturating there."""
    out = np.zeros(x.shape)
    for n in range(x.shape[1]):
        out[:, n] = fh.round_codes(x[:, n], fh.scale_byte(fh.finite_top(x[:, n])))[1]
    return out


def _x(cin, n, seed):
    """Ordinary tokens; every other one with a far value in some channels, or in all of them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(cin, n, generator=g).bfloat16()
    for i in range(0, n, 2):
        top = TOPS[(i // 2) % len(TOPS)]
        if i % 4:
            x[:, i] = (torch.randn(cin, generator=g) * 2.0 ** 125).clamp(-2.0 ** 127, 2.0 ** 127).bfloat16()
        rows = torch.randperm(cin, generator=g)[:max(1, cin // 16)]
        x[rows, i] = torch.where(torch.rand(rows.numel(), generator=g) < 0.5, _bits(top), -_bits(top))
    return x


def _check(y, w, x, kept):
    xq = _columns(_f64(x))
    assert np.abs(xq).max() <= 448 * 2.0 ** 119 and (np.abs(w) @ np.abs(xq)).max() < 2.0 ** 127
    got = _f64(y)
    assert np.isfinite(got).all()
    err, bound = np.abs(got - w @ xq), mh.product_bound(w, xq, kept)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 40, 130, 300])
@pytest.mark.parametrize("cin", [64, 700, 9000])
def test_product(cin, n):
    """One token, up to eight, sixteen, several segments and the many-token kernel; one pass over the channels and more."""
    print(f"[fp8 limits] {cin} channels, {n} tokens", flush=True)
    q = _weight(128, cin, cin)
    w, kept = _dense(q), q.plan.n_dense + q.plan.n_24 // 2
    for seed in range(5 if n == 1 else 1):
        x = _x(cin, n, seed)
        if n == 1:
            x[cin // 2, 0] = _bits(TOPS[seed])
        y = hinm.spmm(q, x.to(DEV))
        torch.cuda.synchronize()
        _check(y, w, x, kept)


@pytest.mark.parametrize("counts", [[9, 0, 3], [17, 8, 23], [200, 150, 40]])
def test_experts(counts):
    print(f"[fp8 limits] experts {counts}", flush=True)
    one = [_weight(64, 320, s) for s in range(3)]
    q = hinm.HinmFp8(one[0].plan, **{k: torch.stack([getattr(w, k).view(torch.uint8) if "val" in k else getattr(w, k) for w in one])
                                     .view(getattr(one[0], k).dtype) for k in hinm._MX4_BUFFERS}, n_experts=3)
    starts = np.cumsum([0] + counts)
    x = _x(320, int(starts[-1]), 3)
    z = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    r = hinm.Routing(z, z.float(), z, torch.tensor(starts, dtype=torch.int32, device=DEV),
                     torch.tensor(counts, dtype=torch.int32, device=DEV), torch.zeros(int(starts[-1]), dtype=torch.int32, device=DEV))
    y = hinm.spmm_experts(q, x.to(DEV), r)
    torch.cuda.synchronize()
    for e, c in enumerate(counts):
        at = slice(int(starts[e]), int(starts[e]) + c)
        if c:
            _check(y[:, at], _dense(one[e]), x[:, at], q.plan.n_dense + q.plan.n_24 // 2)


@pytest.mark.parametrize("n", [1, 12, 130])
def test_not_finite_beside_far_values(n):
    """A NaN or an infinity of a saturating token stays NaN, and reaches no other token."""
    q = _weight(64, 256, 1)
    w = _dense(q)
    x = torch.zeros(256, n, dtype=BF16)
    x[3], x[5] = _bits(0x7f7f), 1.0
    clean = hinm.spmm(q, x.to(DEV))
    x[200, 0] = float("inf") if n % 2 else float("nan")
    y = hinm.spmm(q, x.to(DEV))
    keeps = torch.from_numpy(w[:, 200] != 0).to(DEV)
    assert bool(keeps.any()) and bool(y[keeps, 0].isnan().all()) and torch.equal(y[:, 1:], clean[:, 1:])
    assert bool(clean.isfinite().all())
