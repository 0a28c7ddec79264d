"""The router where its blocks of 64 tokens are many: 16 waves sum a run of blocks each, 8 loads at a time, so that
over 8192 tokens a run takes more than one turn and the last wave's may be short or empty."""
import numpy as np
import pytest
import torch

import moe_helpers as mh

pytestmark = pytest.mark.gpu
hinm = pytest.importorskip("structured_sparse_gemm_amd")


@pytest.mark.parametrize("n,e,k", [(8192, 3, 1), (8193, 65, 2), (9217, 4, 3), (16385, 6, 2)])
def test_long_routes(n, e, k):
    logits = torch.randn(e, n, generator=torch.Generator().manual_seed(n)).bfloat16()
    logits[:, ::37] = float("-inf")
    print(f"[route] n={n} e={e} k={k}", flush=True)
    r = hinm.route(logits.to("cuda:0"), k, renormalize=False)
    torch.cuda.synchronize()
    want = mh.route(logits.double().numpy(), k, False, 8, hinm.route_columns(n, e, k))
    for f in ("ids", "counts", "starts", "slots", "src"):
        assert np.array_equal(getattr(r, f).cpu().numpy(), want[f]), f
    # an exponential of a difference below 16, rounded once (16 2^-24) and off by two steps (2^-23 each); the sum's
    # terms the same; division and the last rounding half a step each
    assert np.all(np.abs(r.weights.double().cpu().numpy() - want["weights"]) <= 42 * 2.0 ** -24 * want["weights"])
