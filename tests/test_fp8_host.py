"""8-bit weights and the mixture-of-experts layer: refusals, workspace sizes and stored weights (CPU only: tensors in
host memory, and pointers that nothing reads, are refused last)."""
import ctypes

import pytest
import torch

import structured_sparse_gemm_amd as hinm

BF16 = torch.bfloat16


def _plan(cout=128, cin=256, rows=64, t_s=0.75, v_s=0.55):
    return hinm.plan(cout, cin, rows, t_s, v_s)


def _eight(p=None, n=None):
    p = p or _plan()
    lead = () if n is None else (n,)
    return hinm.HinmFp8(p, **{k: torch.zeros((*lead, *s), dtype=t) for k, (s, t) in hinm._fp8_shapes(p).items()}, n_experts=n)


def _four(p=None, n=None):
    p = p or _plan()
    return hinm.HinmMx4(p, **{k: torch.zeros((n, *s), dtype=t) for k, (s, t) in hinm._mx4_shapes(p).items()}, n_experts=n)


def _sixteen(p=None, n=4):
    return hinm.Experts.stack([hinm.alloc_packed(p or _plan(), "cpu") for _ in range(n)])


def _routing(e=4, cols=40):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)
    return hinm.Routing(z(6, 2), torch.zeros(6, 2), z(6, 2), z(e + 1), z(e), z(cols))


# --- products -------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("x,message", [
    (torch.zeros(255, 3, dtype=BF16), r"x must be bf16 \[256, columns\]"), (torch.zeros(256, 3), r"x must be bf16 \[256, columns\]"),
    (torch.zeros(3, 256, dtype=BF16).t(), "unit column stride"), (torch.zeros(256, 3, dtype=BF16), "on a GPU")])
def test_product(x, message):
    with pytest.raises(ValueError, match=message):
        hinm.spmm(_eight(), x)


def test_product_kinds():
    x = torch.zeros(256, 3, dtype=BF16)
    with pytest.raises(ValueError, match="multiply a stack with spmm_experts"):
        hinm.spmm(_eight(n=4), x)
    with pytest.raises(ValueError, match="out_rows is not supported with 8-bit values"):
        hinm.spmm(_eight(), x, out_rows=torch.arange(128, dtype=torch.int32))
    with pytest.raises(ValueError, match="takes an Experts stack"):
        hinm.spmm_experts(_eight(), torch.zeros(256, 40, dtype=BF16), _routing())
    for call in (lambda w: hinm.Group([w]), lambda w: hinm.spmm_noalloc(w, x, torch.zeros(128, 3, dtype=BF16)),
                 lambda w: hinm.translate_indices(w, torch.arange(256, dtype=torch.int32))):
        with pytest.raises(ValueError, match="8-bit weights are multiplied one at a time by spmm"):
            call(_eight())
        with pytest.raises(ValueError, match="stack of experts"):
            call(_eight(n=2))


@pytest.mark.parametrize("e,cols,message", [(3, 40, "3 experts"), (4, 39, "x has 39 columns, the routing 40"), (4, 40, "on a GPU")])
def test_experts(e, cols, message):
    with pytest.raises(ValueError, match=message):
        hinm.spmm_experts(_eight(n=4), torch.zeros(256, cols, dtype=BF16), _routing(e=e))


@pytest.mark.parametrize("what,message", [
    (torch.zeros(4), "takes a HinmPacked weight or an Experts stack"), (_eight(), "takes a HinmPacked weight or an Experts stack"),
    (hinm.alloc_packed(_plan(), "cpu"), "on a GPU")])
def test_quantize(what, message):
    with pytest.raises(ValueError, match=message):
        hinm.quantize_fp8(what)


def _fake(p, cls=hinm.Fp8T, base=1 << 20, n=7):
    """A struct whose pointers nothing reads."""
    return cls(p.raw, *[base] * n)


def test_product_statuses():
    lib, p = hinm.library(), _plan(4096, 4096, 64, 0.5, 0.25)
    q = _fake(p)

    def one(st=q, x=4096, n=640, ldx=640, y=4096, ldy=640, ws=1 << 20, size=1 << 40):
        return lib.hinm_spmm_fp8(ctypes.byref(st), x, n, ldx, y, ldy, ws, size, None)

    def many(st=q, e=4, starts=4096, counts=4096, n=640, ws=1 << 20, size=1 << 40):
        return lib.hinm_spmm_experts_fp8(ctypes.byref(st), e, 4096, n, n, starts, counts, 4096, n, ws, size, None)

    need = ctypes.c_size_t()
    assert lib.hinm_spmm_fp8_workspace_bytes(ctypes.byref(p.raw), 640, ctypes.byref(need)) == 0 and need.value > 4096 * 640
    assert one(n=-1) == 2 and one(n=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25) == 2
    assert one(ldx=639) == 2 and one(ldy=639) == 2 and one(ldx=1 << 31) == 2
    assert one(x=None) == 1 and one(y=None) == 1 and one(x=4097) == 5 and one(y=4097) == 5
    assert one(st=_fake(p, base=(1 << 20) + 8)) == 5 and one(st=hinm.Fp8T(p.raw)) == 1
    assert one(ws=None) == 6 and one(size=need.value - 1) == 6 and one(ws=(1 << 20) + 16) == 5
    assert one(n=0, ldx=0, ldy=0, x=None, y=None, ws=None, size=0) == 0
    assert one(st=_fake(_plan(96, 256, 48))) == 2               # tile height
    bad = hinm.PlanT.from_buffer_copy(p.raw)
    bad.n_dense += 1
    assert one(st=hinm.Fp8T(bad, *[1 << 20] * 7)) == 1
    assert lib.hinm_spmm_fp8(None, 4096, 1, 1, 4096, 1, None, 0, None) == 1
    assert many(e=0) == 2 and many(e=1025) == 2 and many(starts=None) == 1 and many(counts=None) == 1
    assert many(starts=4098) == 5 and many(counts=4098) == 5 and many(ws=None) == 6
    full = hinm.PackedT(p.raw, *[1 << 20] * 5)
    assert lib.hinm_fp8_quantize(None, 1, ctypes.byref(q), None) == 1 and lib.hinm_fp8_quantize(ctypes.byref(full), 1, None, None) == 1
    assert lib.hinm_fp8_quantize(ctypes.byref(full), 0, ctypes.byref(q), None) == 1
    assert lib.hinm_fp8_quantize(ctypes.byref(full), 1, ctypes.byref(_fake(p, base=(1 << 20) + 4)), None) == 5
    assert lib.hinm_fp8_quantize(ctypes.byref(full), 1, ctypes.byref(hinm.Fp8T(p.raw)), None) == 1
    assert lib.hinm_fp8_dequantize(ctypes.byref(q), 1, ctypes.byref(hinm.PackedT(p.raw)), None) == 1


def test_workspace_sizes():
    """None for a few tokens, rounded activations for more, never smaller than for fewer."""
    lib, n = hinm.library(), ctypes.c_size_t()
    for p in (_plan(), _plan(4096, 11008), _plan(64, 20000)):
        sizes = []
        for cols in (0, 1, 16, 33, 64, 500, 5000, 1 << 20, 1 << 24):
            assert lib.hinm_spmm_experts_fp8_workspace_bytes(ctypes.byref(p.raw), 1, cols, ctypes.byref(n)) == 0
            sizes.append(n.value)
        assert sizes[0] == 0 and sizes == sorted(sizes) and sizes[-1] < 3 << 30
        assert (sizes[2] == 0) == (p.cin < 18900)
        for cols in (-1, (1 << 24) + 1, 1 << 62):
            assert lib.hinm_spmm_experts_fp8_workspace_bytes(ctypes.byref(p.raw), 1, cols, ctypes.byref(n)) == 2
    assert lib.hinm_spmm_fp8_workspace_bytes(ctypes.byref(p.raw), 1, None) == 1


def test_stored_weights():
    q = _eight(n=2)
    back = hinm.HinmFp8.from_state_dict(q.state_dict())
    assert back.n_experts == 2 and back.plan == q.plan and back.nbytes() == q.nbytes()
    assert hinm.HinmFp8.from_state_dict(_eight().state_dict()).n_experts is None
    sd = q.state_dict()
    for change, message in (({"format_version": 99}, "layout version"), ({"n_experts": -1}, "n_experts >= 0"),
                            ({"val_24": sd["val_24"].view(torch.uint8)}, "val_24"),
                            ({"scale_24": sd["scale_24"][:, 1:]}, "scale_24"), ({"n_experts": 0}, "val_dense"),
                            ({"format": "hinm-mx4"}, "hinm-fp8")):
        with pytest.raises(ValueError, match=message):
            hinm.HinmFp8.from_state_dict(dict(sd, **change))


# --- the mixture-of-experts layer -----------------------------------------------------------------------------------
UP, DOWN = _plan(192, 128), _plan(128, 192)


def _layer(make=_sixteen):
    return make(UP, n=4), make(UP, n=4), make(DOWN, n=4)


def _xl(n=3, e=4, hidden=128, dtype=torch.float32):
    return torch.zeros(hidden, n, dtype=BF16), torch.zeros(e, n, dtype=dtype)


@pytest.mark.parametrize("weights,message", [
    (lambda: (_eight(UP, 4), *_layer()[1:]), "of one kind"), (lambda: (*_layer()[:2], _four(DOWN, 4)), "of one kind"),
    (lambda: (torch.zeros(4), *_layer()[1:]), "of one kind"), (lambda: (_eight(UP), _eight(UP), _eight(DOWN)), "of one kind"),
    (lambda: (*_layer()[:2], _sixteen(DOWN, 3)), "equal numbers of experts"), (lambda: _layer(), "on a GPU"),
    (lambda: _layer(_four), "on a GPU"), (lambda: _layer(_eight), "on a GPU")])
def test_layer_kinds(weights, message):
    with pytest.raises(ValueError, match=message):
        hinm.moe_layer(*_xl(), *weights(), 2)


@pytest.mark.parametrize("x,logits,message", [
    (_xl()[0], torch.zeros(4, 3, dtype=torch.float16), "logits must be bf16 or fp32"), (_xl()[0], torch.zeros(5, 3), r"logits must be .* \[4, tokens\]"),
    (_xl()[0], torch.zeros(3, 4).t(), "unit column stride"), (_xl()[0], torch.zeros(1, 3).expand(4, 3), "rows that do not overlap"),
    (torch.zeros(129, 3, dtype=BF16), torch.zeros(4, 3), r"x must be bf16 \[128, 3\]"), (torch.zeros(128, 4, dtype=BF16), torch.zeros(4, 3), r"x must be bf16 \[128, 3\]")])
def test_layer_inputs(x, logits, message):
    with pytest.raises(ValueError, match=message):
        hinm.moe_layer(x, logits, *_layer(), 2)


def test_layer_workspace():
    need = lambda up=UP, down=DOWN, e=4, n=3, k=2: hinm.moe_layer_workspace_bytes(up, down, e, n, k)
    assert need(n=0) == 0 and 0 < need(n=1) < need(n=32) and need(e=1024, n=32, k=16) > need(e=4, n=32, k=2)
    for kw, message in (({"n": 33}, "33 tokens; 0 to 32"), ({"n": -1}, "0 to 32"), ({"k": 0}, "top_k=0"), ({"k": 5}, "top_k=5"),
                        ({"e": 40, "k": 17}, "top_k=17"), ({"e": 0, "k": 1}, "n_experts=0"), ({"e": 1025}, "n_experts=1025"),
                        ({"down": UP}, r"is needed"), ({"up": _plan(192, 128, 48), "down": DOWN}, "multiples of 64"),
                        ({"up": _plan(16448, 128), "down": _plan(128, 16448)}, "at most 16384")):
        with pytest.raises(hinm.HinmError, match=message):
            need(**kw)


def test_layer_statuses():
    lib = hinm.library()

    def call(**kw):
        v = {"logits": 4096, "type": 1, "ldl": 3, "x": 4096, "n": 3, "ldx": 3, "e": 4, "k": 2, "values": 2, "gate": _fake(UP),
             "up": _fake(UP), "down": _fake(DOWN), "y": 4096, "ldy": 3, "ws": 1 << 20, "size": 1 << 40, **kw}
        ref = lambda s: None if s is None else ctypes.byref(s)
        return lib.hinm_moe_layer(v["logits"], v["type"], v["ldl"], v["x"], v["n"], v["ldx"], v["e"], v["k"], 1, v["values"],
                                  ref(v["gate"]), ref(v["up"]), ref(v["down"]), v["y"], v["ldy"], v["ws"], v["size"], None)

    need = hinm.moe_layer_workspace_bytes(UP, DOWN, 4, 3, 2)
    assert call(values=3) == 1 and call(values=-1) == 1 and call(type=7) == 1
    for name in ("gate", "up", "down", "logits", "x", "y"):
        assert call(**{name: None}) == 1, name
    assert call(ws=None) == 6 and call(size=need - 1) == 6 and call(ws=(1 << 20) + 128) == 5
    assert call(ldl=2) == 2 and call(ldx=2) == 2 and call(ldy=2) == 2 and call(ldx=1 << 31) == 2
    assert call(logits=4098) == 5 and call(x=4097) == 5 and call(y=4097) == 5
    assert call(n=33, ldl=33, ldx=33, ldy=33) == 2 and call(k=5) == 2 and call(e=0) == 2
    assert call(gate=_fake(_plan(128, 128))) == 2               # another shape than up's
    assert call(gate=_fake(_plan(192, 128, 192))) == 2          # another tile height than up's
    assert call(up=_fake(UP, base=(1 << 20) + 8)) == 5 and call(down=hinm.Fp8T(DOWN.raw)) == 1
    assert call(values=0, gate=hinm.PackedT(UP.raw), up=_fake(UP, hinm.PackedT, n=5), down=_fake(DOWN, hinm.PackedT, n=5)) == 1
    empty = _plan(192, 128, 64, 0.999, 0.999)                   # keeps nothing
    assert empty.n_dense + empty.n_24 == 0
    assert call(gate=_fake(empty)) == 2 and call(up=_fake(empty)) == 2
    assert call(n=0, ldl=0, ldx=0, ldy=0, logits=None, x=None, y=None, ws=None, size=0) == 0
