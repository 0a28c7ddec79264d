"""Host threads that call on one stream share its default workspace: every call's kernels are enqueued together, so each
gets its own results (calls of several kernels: rounding of X and product, the layer's two kernels, copy of X and
product)."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
hinm = pytest.importorskip("structured_sparse_gemm_amd")
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def _packed(cout, cin, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(cout, cin, generator=g) * cin ** -0.5).bfloat16().to(DEV)
    perm = torch.stack([torch.randperm(cin, generator=g) for _ in range(cout // 64)]).int().to(DEV)
    return hinm.pack(w, w.float().abs(), 64, 0.75, 0.55, perm)


def _x(rows, n, seed):
    return torch.randn(rows, n, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)


def _stack(cout, cin, seed):
    return hinm.Experts.stack([_packed(cout, cin, seed + e) for e in range(4)])


def _layer(i):
    w = [_stack(128, 192, 1), _stack(128, 192, 11), _stack(192, 128, 21)]
    x, logits = _x(192, 5 + i, i), torch.randn(4, 5 + i, generator=torch.Generator().manual_seed(i)).to(DEV)
    return lambda: hinm.moe_layer(x, logits, *w, 2)


def _product(i):
    q, x = hinm.quantize_fp8(_packed(128, 256, 5)), _x(256, 130 + 7 * i, i)
    return lambda: hinm.spmm(q, x)


def _routed(i):
    w = hinm.quantize_fp8(_stack(128, 256, 1))
    x, logits = _x(256, 300 + i, i), torch.randn(4, 300 + i, generator=torch.Generator().manual_seed(i)).to(DEV)

    def call():
        r = hinm.route(logits, 2)
        return hinm.combine(hinm.spmm_experts(w, hinm.dispatch(x, r), r), r)
    return call


@pytest.mark.parametrize("kind", [_layer, _product, _routed], ids=["layer", "product8", "routed"])
def test_threads_on_one_stream(kind):
    calls = [kind(i) for i in range(4)]
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    got, failed, ready = [[] for _ in calls], [], threading.Barrier(len(calls))

    def work(i):
        try:
            ready.wait(30)
            for _ in range(200):
                got[i].append(calls[i]())
        except BaseException as e:                       # the main thread reports it
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    print(f"[threads] {kind.__name__}", flush=True)
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for ys, y in zip(got, want):
        assert len(ys) == 200 and all(torch.equal(z, y) for z in ys)
