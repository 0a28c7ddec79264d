"""Host-side refusals and plain helpers of the mixture-of-experts operators and the 4-bit values (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as hinm
from moe_helpers import GRID, mx4_block, route

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return hinm.library()


def _packed(p, **kw):
    k = hinm.PackedT(p.raw, FAKE, FAKE, FAKE, FAKE, FAKE)
    for name, v in kw.items():
        setattr(k, name, v)
    return k


def _mx4(p, **kw):
    k = hinm.Mx4T(p.raw, *([FAKE] * 7))
    for name, v in kw.items():
        setattr(k, name, v)
    return k


def _err(lib):
    return lib.hinm_last_error().decode()


@pytest.mark.parametrize("n,e,k,align", [(1, 1, 1, 1), (16, 8, 2, 8), (0, 4, 2, 8), (3, 64, 8, 8), (8192, 128, 8, 16),
                                         (5, 3, 3, 1), (7, 1024, 16, 256)])
def test_route_columns_hold_every_routing(lib, n, e, k, align):
    got = hinm.route_columns(n, e, k, align)
    # the fullest: one token in as many experts as there are pairs, the rest anywhere
    used = n * k
    want = used + min(e, used) * (align - 1)
    assert got == -(-want // align) * align


def test_route_columns_hold_random_routings(lib):
    rng = np.random.default_rng(3)
    for _ in range(200):
        n, e = int(rng.integers(0, 40)), int(rng.integers(1, 12))
        k, align = int(rng.integers(1, e + 1)), int(2 ** rng.integers(0, 5))
        r = route(rng.standard_normal((e, n)), k, True, align, hinm.route_columns(n, e, k, align))
        assert r["starts"][-1] <= hinm.route_columns(n, e, k, align)


@pytest.mark.parametrize("args,status", [((4, 0, 1, 8), 2), ((4, 1025, 1, 8), 2), ((-1, 4, 1, 8), 2), ((4, 4, 0, 8), 2),
                                         ((4, 4, 5, 8), 2), ((4, 64, 17, 8), 2), ((4, 4, 2, 3), 1), ((4, 4, 2, 0), 1),
                                         ((4, 4, 2, 512), 1), ((1 << 27, 4, 2, 8), 2)])
def test_route_columns_refuses(lib, args, status):
    n = ctypes.c_int64()
    assert lib.hinm_route_columns(*args, ctypes.byref(n)) == status
    assert _err(lib)


def test_route_refuses(lib):
    cols = hinm.route_columns(100, 8, 2, 8)
    ws = ctypes.c_size_t()
    assert lib.hinm_route_workspace_bytes(100, 8, ctypes.byref(ws)) == 0 and ws.value == (2 + 1) * 8 * 4

    def call(**kw):
        a = dict(logits=FAKE, type=1, n=100, ldl=100, e=8, k=2, renorm=1, align=8, ids=FAKE, w=FAKE, slots=FAKE,
                 starts=FAKE, counts=FAKE, src=FAKE, cols=cols, ws=FAKE, wsn=ws.value)
        a.update(kw)
        return lib.hinm_route(*a.values(), None)

    assert call(type=2) == 1 and call(logits=None) == 1 and call(ids=None) == 1 and call(starts=None) == 1
    assert call(src=None) == 1 and call(ldl=99) == 2 and call(cols=cols - 1) == 2 and call(k=9) == 2
    assert call(logits=FAKE + 2) == 5 and call(slots=FAKE + 2) == 5 and call(ws=FAKE + 16) == 5
    assert call(ws=None) == 6 and call(wsn=ws.value - 1) == 6
    assert lib.hinm_route_workspace_bytes(64, 8, ctypes.byref(ws)) == 0 and ws.value == 0
    assert lib.hinm_route_workspace_bytes(64, 8, None) == 1


def test_dispatch_and_combine_refuse(lib):
    def dispatch(x=FAKE, c=4, n=8, ldx=8, src=FAKE, cols=16, xs=FAKE, ldxs=16):
        return lib.hinm_dispatch(x, c, n, ldx, src, cols, xs, ldxs, None)

    assert dispatch(ldx=7) == 2 and dispatch(ldxs=15) == 2 and dispatch(c=-1) == 2 and dispatch(c=1 << 31) == 2
    assert dispatch(x=None) == 1 and dispatch(src=None) == 1 and dispatch(xs=None) == 1
    assert dispatch(x=FAKE + 1) == 5 and dispatch(src=FAKE + 2) == 5
    assert dispatch(c=0) == 0 and dispatch(cols=0) == 0
    big = (1 << 30) + 1
    assert dispatch(cols=big, ldxs=big) == 2 and dispatch(n=big, ldx=big) == 2

    def combine(ys=FAKE, c=4, cols=16, ldys=16, slots=FAKE, w=FAKE, n=8, k=2, y=FAKE, ldy=8):
        return lib.hinm_combine(ys, c, cols, ldys, slots, w, n, k, y, ldy, None)

    assert combine(cols=big, ldys=big) == 2 and combine(n=big, ldy=big) == 2
    assert combine(ldys=15) == 2 and combine(ldy=7) == 2 and combine(k=0) == 2 and combine(k=17) == 2
    assert combine(ys=None) == 1 and combine(slots=None) == 1 and combine(w=None) == 1 and combine(y=None) == 1
    assert combine(y=FAKE + 1) == 5 and combine(w=FAKE + 2) == 5
    assert combine(c=0) == 0 and combine(n=0, ldy=0) == 0


@pytest.mark.parametrize("mx4", [False, True])
def test_experts_refuse(lib, mx4):
    p = hinm.plan(128, 256, 64, 0.75, 0.55)
    need = hinm.spmm_experts_workspace_bytes(p, 4, 40)
    make, fn = (_mx4, lib.hinm_spmm_experts_mx4) if mx4 else (_packed, lib.hinm_spmm_experts)

    def call(k=None, e=4, x=FAKE, cols=40, ldx=40, starts=FAKE, counts=FAKE, y=FAKE, ldy=40, ws=FAKE, wsn=need):
        return fn(ctypes.byref(make(p) if k is None else k), e, x, cols, ldx, starts, counts, y, ldy, ws, wsn, None)

    assert fn(None, 4, FAKE, 40, 40, FAKE, FAKE, FAKE, 40, FAKE, need, None) == 1
    assert call(e=0) == 2 and call(e=1025) == 2 and call(cols=-1) == 2 and call(ldx=39) == 2 and call(ldy=39) == 2
    assert call(cols=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25) == 2
    assert call(starts=None) == 1 and call(counts=None) == 1 and call(x=None) == 1 and call(y=None) == 1
    assert call(starts=FAKE + 2) == 5 and call(x=FAKE + 1) == 5
    assert call(k=make(p, val_24=None)) == 1 and call(k=make(p, idx_dense=FAKE + 4)) == 5
    if mx4:
        assert call(k=make(p, scale_24=None)) == 1
    if need:
        assert call(ws=None) == 6 and call(wsn=need - 1) == 6 and call(ws=FAKE + 16) == 5
    # many tokens, unaligned rows: the workspace also holds a copy of X with aligned rows
    many = hinm.spmm_experts_workspace_bytes(p, 1, 30001)
    assert hinm.spmm_experts_workspace_bytes(p, 1, 30001, x_aligned=False) == max(many, 65536) + 256 * 30008 * 2
    # without splits too the counters' 64 KiB are kept free for other calls with the same workspace
    none = 256 * 64 * 2 * 256
    assert hinm.spmm_experts_workspace_bytes(p, 1, none) == 0
    assert hinm.spmm_experts_workspace_bytes(p, 1, none, x_aligned=False) == 65536 + 256 * none * 2
    assert call(e=1, cols=1001, ldx=1001, ldy=1001, wsn=many) == 6
    q = hinm.plan(96, 256, 32, 0.75, 0.55)                       # tile_rows 32
    assert call(k=make(q)) == 2 and "tile_rows" in _err(lib)
    assert call(cols=0, x=None, y=None, ldx=0, ldy=0) == 0       # no columns: nothing to do
    bad = make(p)
    bad.plan.n_dense += 1
    assert call(k=bad) == 1
    n = ctypes.c_size_t()
    assert lib.hinm_spmm_experts_workspace_bytes(ctypes.byref(p.raw), 0, 40, 1, ctypes.byref(n)) == 2
    assert lib.hinm_spmm_experts_workspace_bytes(ctypes.byref(p.raw), 4, -1, 1, ctypes.byref(n)) == 2
    assert lib.hinm_spmm_experts_workspace_bytes(ctypes.byref(p.raw), 4, 40, 1, None) == 1
    assert lib.hinm_spmm_experts_workspace_bytes(ctypes.byref(q.raw), 4, 40, 1, ctypes.byref(n)) == 2


def test_mx4_refuses(lib):
    p = hinm.plan(128, 256, 64, 0.75, 0.55)
    q = hinm.plan(96, 256, 32, 0.75, 0.55)
    ref = ctypes.byref
    assert lib.hinm_mx4_quantize(None, 1, ref(_mx4(p)), None) == 1
    assert lib.hinm_mx4_quantize(ref(_packed(p)), 1, None, None) == 1
    assert lib.hinm_mx4_quantize(ref(_packed(p)), 0, ref(_mx4(p)), None) == 1
    assert lib.hinm_mx4_quantize(ref(_packed(q)), 1, ref(_mx4(q)), None) == 2
    assert lib.hinm_mx4_quantize(ref(_packed(p)), 1, ref(_mx4(p, scale_dense=None)), None) == 1
    assert lib.hinm_mx4_quantize(ref(_packed(p, val_24=FAKE + 8)), 1, ref(_mx4(p)), None) == 5
    assert lib.hinm_mx4_dequantize(ref(_mx4(p, meta_24=None)), 1, ref(_packed(p)), None) == 1
    assert lib.hinm_mx4_dequantize(ref(_mx4(q)), 1, ref(_packed(q)), None) == 2
    n = ctypes.c_size_t()
    assert lib.hinm_spmm_mx4_workspace_bytes(ref(p.raw), 16, 1, ref(n)) == 0
    assert lib.hinm_spmm_mx4(ref(_mx4(p)), FAKE, 16, 15, FAKE, 16, FAKE, n.value, None) == 2
    assert lib.hinm_spmm_mx4(ref(_mx4(p)), None, 16, 16, FAKE, 16, FAKE, n.value, None) == 1
    assert lib.hinm_spmm_mx4(ref(_mx4(q)), FAKE, 16, 16, FAKE, 16, FAKE, n.value, None) == 2
    assert lib.hinm_spmm_mx4(ref(_mx4(p)), None, 0, 0, None, 0, None, 0, None) == 0


def _routing(n=6, k=2, e=4, cols=40):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)
    return hinm.Routing(z(n, k), torch.zeros(n, k), z(n, k), z(e + 1), z(e), z(cols))


def test_binding_refuses_wrong_tensors():
    with pytest.raises(ValueError):
        hinm.route(torch.zeros(4, 8), 2)                                     # not on a GPU
    r = _routing()
    with pytest.raises(ValueError):
        hinm.dispatch(torch.zeros(16, 6), r)                                 # fp32
    with pytest.raises(ValueError):
        hinm.dispatch(torch.zeros(16, 5, dtype=torch.bfloat16), r)           # tokens
    with pytest.raises(ValueError):
        hinm.dispatch(torch.zeros(6, 16, dtype=torch.bfloat16).t(), r)       # column stride
    with pytest.raises(ValueError):
        hinm.dispatch(torch.zeros(1, 6, dtype=torch.bfloat16).expand(16, 6), r)   # rows that overlap
    with pytest.raises(ValueError):
        hinm.combine(torch.zeros(16, 39, dtype=torch.bfloat16), r)
    with pytest.raises(ValueError):
        r2 = _routing()
        r2.weights = r2.weights.double()
        hinm.combine(torch.zeros(16, 40, dtype=torch.bfloat16), r2)
    with pytest.raises(ValueError):
        hinm.Experts.stack([])
    with pytest.raises(ValueError):
        hinm.quantize_mx4(torch.zeros(4))
    with pytest.raises(ValueError):
        hinm.spmm_experts(torch.zeros(4), torch.zeros(4, 4, dtype=torch.bfloat16), r)


def test_stored_stacks_and_four_bit_weights_round_trip():
    p = hinm.plan(128, 256, 64, 0.75, 0.55)
    pk = [hinm.alloc_packed(p, "cpu") for _ in range(3)]
    for i, k in enumerate(pk):
        for b in hinm._BUFFERS:
            getattr(k, b).fill_(i + 1)
    st = hinm.Experts.stack(pk)
    assert st.n_experts == 3 and st.nbytes() == 3 * p.packed_bytes
    back = hinm.Experts.from_state_dict(st.state_dict())
    assert all(torch.equal(getattr(back, b), getattr(st, b)) for b in hinm._BUFFERS)
    bad = st.state_dict()
    bad["n_experts"] = 2
    with pytest.raises(ValueError):
        hinm.Experts.from_state_dict(bad)
    with pytest.raises(ValueError):
        hinm.Experts.stack([pk[0], hinm.alloc_packed(hinm.plan(128, 256, 64, 0.5, 0.25), "cpu")])
    for n in (None, 2):
        lead = () if n is None else (n,)
        q = hinm.HinmMx4(p, **{k: torch.zeros((*lead, *s), dtype=t) for k, (s, t) in hinm._mx4_shapes(p).items()},
                         n_experts=n)
        # 17 of 64 bytes of the bf16 values, and the metadata and lists as they are
        vals = p.bytes_val_dense + p.bytes_val_24
        assert q.nbytes() == (n or 1) * (vals * 17 // 64 + p.packed_bytes - vals)
        b2 = hinm.HinmMx4.from_state_dict(q.state_dict())
        assert b2.n_experts == n
        bad = q.state_dict()
        bad["format_version"] = 99
        with pytest.raises(ValueError):
            hinm.HinmMx4.from_state_dict(bad)
        bad = q.state_dict()
        bad["scale_24"] = bad["scale_24"][..., :2]
        with pytest.raises(ValueError):
            hinm.HinmMx4.from_state_dict(bad)


def test_plain_four_bit_rule():
    """The tests' plain rounding: half-way cases to the even code, saturation, scales of powers of two."""
    v = np.zeros(32)
    v[:9] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.75, 5.0]
    s, c, val = mx4_block(v)
    assert s == 127 and c[:9].tolist() == [6, 0, 2, 2, 4, 4, 6, 10, 6]
    assert val[:9].tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, -1.0, 4.0]
    s, c, val = mx4_block(np.full(32, 7.96875))                    # 7.97 saturates at 6
    assert s == 127 and (c == 7).all() and (val == 6).all()
    s, c, val = mx4_block(np.full(32, 8.0))
    assert s == 128 and (c == 6).all() and (val == 8).all()
    assert mx4_block(np.zeros(32))[0] == 0
    assert mx4_block(np.full(32, 2.0 ** -130))[0] == 0 and mx4_block(np.full(32, np.inf))[0] == 255
    assert set(GRID) == {0, .5, 1, 1.5, 2, 3, 4, 6}


def test_binding_refuses_weights_on_the_host():
    """Everything else about these calls is right: only the place of the tensors is refused."""
    p = hinm.plan(128, 256, 64, 0.75, 0.55)
    st = hinm.Experts.stack([hinm.alloc_packed(p, "cpu") for _ in range(4)])
    q = hinm.HinmMx4(p, **{k: torch.zeros(s, dtype=t) for k, (s, t) in hinm._mx4_shapes(p).items()})
    r, b = _routing(), torch.bfloat16
    for call in (lambda: hinm.dispatch(torch.zeros(16, 6, dtype=b), r),
                 lambda: hinm.combine(torch.zeros(16, 40, dtype=b), r),
                 lambda: hinm.spmm_experts(st, torch.zeros(256, 40, dtype=b), r),
                 lambda: hinm.spmm(q, torch.zeros(256, 3, dtype=b)),
                 lambda: hinm.quantize_mx4(st), lambda: hinm.quantize_mx4(hinm.alloc_packed(p, "cpu")),
                 q.dequantize):
        with pytest.raises(ValueError, match="on a GPU"):
            call()
