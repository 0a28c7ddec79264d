"""Calls that read a weight's buffers as those of one uniform bf16 weight refuse every other kind (CPU only: nothing
here reaches a launch)."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as hinm

P = dict(cout=128, cin=256, tile_rows=64, t_s=0.75, v_s=0.55)


def _plan():
    return hinm.plan(*P.values())


def _stack():
    return hinm.Experts.stack([hinm.alloc_packed(_plan(), "cpu") for _ in range(2)])


def _four_bit(n=None):
    lead = () if n is None else (n,)
    return hinm.HinmMx4(_plan(), **{k: torch.zeros((*lead, *s), dtype=t) for k, (s, t) in hinm._mx4_shapes(_plan()).items()},
                        n_experts=n)


def _per_tile():
    p = hinm.plan_tiles(P["cout"], P["cin"], 64, P["t_s"], [0.55, 0.5])
    z = lambda shape, t: torch.zeros(shape, dtype=t)
    return hinm.HinmTPacked(p, torch.from_numpy(np.array(p.tiles)), z((p.dense_blocks, 64, 32), torch.int16),
                            z((p.dense_blocks * 32,), torch.int32), z((p.blocks_24, 64, 32), torch.int16),
                            z((p.blocks_24, 64), torch.int64), z((p.blocks_24 * 64,), torch.int32))


OTHERS = [(_stack, "stack of experts"), (_four_bit, "bf16 values"), (lambda: _four_bit(2), "stack of experts"),
          (_per_tile, "uniform packed weights"), (lambda: torch.zeros(4), "not a Tensor")]


@pytest.mark.parametrize("make,message", OTHERS)
def test_groups_take_bf16_weights(make, message):
    one = hinm.alloc_packed(_plan(), "cpu")
    assert hinm.Group([one, one]).workspace_bytes(16) >= 0
    for members in ([make()], [one, make()]):
        with pytest.raises(ValueError, match=message):
            hinm.Group(members)


@pytest.mark.parametrize("make,message", OTHERS)
def test_products_without_allocation_take_bf16_weights(make, message):
    x, y = torch.zeros(256, 4, dtype=torch.bfloat16), torch.zeros(128, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=message):
        hinm.spmm_noalloc(make(), x, y)


@pytest.mark.parametrize("make,message", OTHERS)
def test_translation_takes_bf16_weights(make, message):
    with pytest.raises(ValueError, match=message):
        hinm.translate_indices(make(), torch.arange(256, dtype=torch.int32))


@pytest.mark.parametrize("make,message", [(_stack, "stack of experts"), (lambda: _four_bit(2), "spmm_experts"),
                                          (lambda: torch.zeros(4), "not a Tensor")])
def test_products_take_one_weight(make, message):
    with pytest.raises(ValueError, match=message):
        hinm.spmm(make(), torch.zeros(256, 4, dtype=torch.bfloat16))
