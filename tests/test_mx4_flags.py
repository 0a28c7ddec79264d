"""The flags of a packed weight (block-diagonal orders get a schedule of their own) through 4-bit values and back."""
import pytest
import torch

import structured_sparse_gemm_amd as hinm
import synth


def test_stored_four_bit_weights_keep_their_flags():
    p = hinm.plan(128, 256, 64, 0.75, 0.55)
    q = hinm.HinmMx4(p, **{k: torch.zeros(s, dtype=t) for k, (s, t) in hinm._mx4_shapes(p).items()},
                     flags=hinm.HINM_PACKED_WINDOWED)
    sd = q.state_dict()
    assert hinm.HinmMx4.from_state_dict(sd).flags == hinm.HINM_PACKED_WINDOWED
    del sd["flags"]                                          # stored before the flags were kept
    assert hinm.HinmMx4.from_state_dict(sd).flags == 0


@pytest.mark.gpu
@pytest.mark.parametrize("ordered", [True, False])
def test_dequantised_weights_keep_their_flags(ordered):
    """Identity orders are block-diagonal, random ones are not; the product of the dequantised weight runs under its
    flags and agrees with one that ignores them (another order of the same fp32 sums, each rounded once to bf16)."""
    dev = torch.device("cuda:0")
    w = synth.small(256, 512, 64, 0.5, 0.25, 1, seed=11)
    pk = hinm.pack(w.w_bf16.to(dev), w.importance.to(dev), 64, 0.5, 0.25, None if ordered else w.perm.to(dev))
    assert bool(pk.flags & hinm.HINM_PACKED_WINDOWED) == ordered
    back = hinm.quantize_mx4(pk).dequantize()
    assert back.flags == pk.flags and back.struct().flags == pk.flags
    plain = hinm.HinmPacked(back.plan, *[getattr(back, b) for b in hinm._BUFFERS])
    x = torch.randn(512, 300, generator=torch.Generator().manual_seed(1)).bfloat16().to(dev)
    a, b = hinm.spmm(back, x).double(), hinm.spmm(plain, x).double()
    # two sums of at most 256 kept terms, a whole fp32 step each, then half a bf16 step on both sides
    wmax = max(float(back.val_dense.view(torch.bfloat16).abs().max()), float(back.val_24.view(torch.bfloat16).abs().max()))
    sums = 2 * 256 * 2.0 ** -23 * wmax * x.double().abs().sum(0)
    assert bool(((a - b).abs() <= sums + 2.0 ** -8 * (a.abs() + b.abs() + sums)).all())
    st = hinm.quantize_mx4(hinm.Experts.stack([pk, pk]))
    assert st.flags == 0 and isinstance(st.dequantize(), hinm.Experts)
