"""Each refusal of the mixture-of-experts calls for its own reason, told from the message (CPU only: tensors in host
memory are refused last, so every other check is reached)."""
import ctypes

import pytest
import torch

import structured_sparse_gemm_amd as hinm

BF16 = torch.bfloat16


def _routing(n=6, k=2, e=4, cols=40, **kw):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)
    r = hinm.Routing(z(n, k), torch.zeros(n, k), z(n, k), z(e + 1), z(e), z(cols))
    for name, v in kw.items():
        setattr(r, name, v)
    return r


def _stack(e=4, four_bit=False):
    p = hinm.plan(128, 256, 64, 0.75, 0.55)
    if four_bit:
        return hinm.HinmMx4(p, **{k: torch.zeros((e, *s), dtype=t) for k, (s, t) in hinm._mx4_shapes(p).items()},
                            n_experts=e)
    return hinm.Experts.stack([hinm.alloc_packed(p, "cpu") for _ in range(e)])


@pytest.mark.parametrize("x,message", [
    (torch.zeros(16, 6), r"x must be bf16 \[channels, 6\]"), (torch.zeros(16, 5, dtype=BF16), r"x must be bf16 \[channels, 6\]"),
    (torch.zeros(6, 16, dtype=BF16).t(), "x must have unit column stride"),
    (torch.zeros(1, 6, dtype=BF16).expand(16, 6), "x must have a row stride of at least its 6 columns"),
    (torch.zeros(16, 6, dtype=BF16), "on a GPU")])
def test_dispatch(x, message):
    with pytest.raises(ValueError, match=message):
        hinm.dispatch(x, _routing())


def test_dispatch_sources():
    with pytest.raises(ValueError, match="routing.src must be a contiguous int32"):
        hinm.dispatch(torch.zeros(16, 6, dtype=BF16), _routing(src=torch.zeros(40, dtype=torch.int64)))


@pytest.mark.parametrize("kw,cols,message", [
    ({}, 39, r"y must be bf16 \[channels, 40\]"),
    ({"weights": torch.zeros(6, 2, dtype=torch.float64)}, 40, "routing.weights must be a contiguous float32"),
    ({"slots": torch.zeros(6, 4, dtype=torch.int32)[:, ::2]}, 40, "routing.slots must be a contiguous int32"),
    ({}, 40, "on a GPU")])
def test_combine(kw, cols, message):
    with pytest.raises(ValueError, match=message):
        hinm.combine(torch.zeros(16, cols, dtype=BF16), _routing(**kw))


@pytest.mark.parametrize("four_bit", [False, True])
@pytest.mark.parametrize("kw,x,message", [
    ({}, torch.zeros(255, 40, dtype=BF16), r"x must be bf16 \[256, "), ({"e": 3}, torch.zeros(256, 40, dtype=BF16), "3 experts"),
    ({"starts": torch.zeros(4, dtype=torch.int32)}, torch.zeros(256, 40, dtype=BF16), "routing.starts must be"),
    ({"counts": torch.zeros(4)}, torch.zeros(256, 40, dtype=BF16), "routing.counts must be"),
    ({}, torch.zeros(256, 40, dtype=BF16), "on a GPU")])
def test_spmm_experts(kw, x, message, four_bit):
    with pytest.raises(ValueError, match=message):
        hinm.spmm_experts(_stack(four_bit=four_bit), x, _routing(**kw))


@pytest.mark.parametrize("x,message", [(torch.zeros(255, 3, dtype=BF16), r"x must be bf16 \[256, columns\]"),
                                       (torch.zeros(256, 3), r"x must be bf16 \[256, columns\]"),
                                       (torch.zeros(256, 3, dtype=BF16), "on a GPU")])
def test_spmm_of_a_four_bit_weight(x, message):
    p = hinm.plan(128, 256, 64, 0.75, 0.55)
    q = hinm.HinmMx4(p, **{k: torch.zeros(s, dtype=t) for k, (s, t) in hinm._mx4_shapes(p).items()})
    with pytest.raises(ValueError, match=message):
        hinm.spmm(q, x)


@pytest.mark.parametrize("four_bit", [False, True])
@pytest.mark.parametrize("cols", [0, 6, 39, 41])
def test_spmm_experts_of_another_routing(cols, four_bit):
    """X before dispatch (6 tokens) or in the order of another routing: its ranges would be cut silently."""
    with pytest.raises(ValueError, match=f"x has {cols} columns, the routing 40"):
        hinm.spmm_experts(_stack(four_bit=four_bit), torch.zeros(256, cols, dtype=BF16), _routing())


@pytest.mark.parametrize("cols", [(1 << 24) + 1, 1 << 62])
def test_workspace_queries_refuse_what_the_products_refuse(cols):
    """More than 2^24 columns: the bytes of a copy of X would pass 63 bits."""
    p = hinm.plan(128, 256, 64, 0.75, 0.55)
    for aligned in (True, False):
        assert hinm.spmm_experts_workspace_bytes(p, 4, 1 << 24, aligned) >= 0
        with pytest.raises(hinm.HinmError, match="exceed 2"):
            hinm.spmm_experts_workspace_bytes(p, 4, cols, aligned)
        n = ctypes.c_size_t()
        assert hinm.library().hinm_spmm_mx4_workspace_bytes(ctypes.byref(p.raw), cols, int(aligned), ctypes.byref(n)) == 2
