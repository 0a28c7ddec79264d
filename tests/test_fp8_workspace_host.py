"""Workspaces of 8-bit products (host only): one that is large enough for some columns is so for fewer."""
import ctypes

import pytest

import structured_sparse_gemm_amd as hinm


def _sizes(p, experts, cols):
    lib, n = hinm.library(), ctypes.c_size_t()
    out = []
    for c in cols:
        assert lib.hinm_spmm_experts_fp8_workspace_bytes(ctypes.byref(p.raw), experts, c, ctypes.byref(n)) == 0
        out.append(n.value)
    return out


# 64, 172, 256, 257 row blocks of one weight: up to 256 the smallest batches of the many-token kernel may split; channels
# of which LDS holds sixteen columns, eight and none
@pytest.mark.parametrize("cout,cin", [(4096, 11008), (4096, 4096), (11008, 4096), (16384, 512), (16448, 512), (64, 20000), (128, 256)])
@pytest.mark.parametrize("experts", [1, 2, 8, 300])
def test_never_smaller_than_for_fewer_columns(cout, cin, experts):
    p = hinm.plan(cout, cin, 64, 0.75, 0.55)
    cols = sorted({c for b in (1, 16, 32, 96, 112 * experts, 256 * experts, 512, 1024, 4096, 1 << 16, 1 << 20, 1 << 23)
                   for c in range(max(b - 3, 0), b + 4)} | set(range(0, 3000, 37)) | {1 << 24})
    sizes = _sizes(p, experts, cols)
    fell = [(a, b) for a, b, s, t in zip(cols, cols[1:], sizes, sizes[1:]) if t < s]
    assert not fell, fell[:5]


def test_sizes_are_asked_for_in_any_order():
    """Remembering sizes needs nothing that another call on the weight has set up (another thread may be half-way)."""
    import torch
    p = hinm.plan(128, 256, 64, 0.75, 0.55)
    q = hinm.HinmFp8(p, **{k: torch.zeros(s, dtype=t) for k, (s, t) in hinm._fp8_shapes(p).items()})
    assert hinm._fp8_need(q, 640) == hinm._fp8_need(q, 640) == _sizes(p, 1, [640])[0]
