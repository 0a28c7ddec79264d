"""Expert and 4-bit products at sizes where the launch's token block, K split and copy of X change, against 64-bit
products on the GPU.

What a call splits into is not visible from outside, but its workspace is: with room for splits it holds 64 KiB of
arrival counters and the sums of 512 workgroups of 64 rows x `block` tokens, and without it neither.  The tests read
the block they mean from that size.

Tolerance, per output: every fp32 addition of the matrix instructions is granted a whole step, 2^-23 of the largest
running sum, sum |w||x|, for each kept term and 64 more for the joins; one rounding to bf16, 2^-8 of the value; the
64-bit product itself is off by less than 2^-40 of that sum.
"""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
hinm = pytest.importorskip("structured_sparse_gemm_amd")
DEV = torch.device("cuda:0")


def _pack(cout, cin, t, v, seed):
    w = synth.small(cout, cin, 64, t, v, 1, seed=seed)
    return hinm.pack(w.w_bf16.to(DEV), w.importance.to(DEV), 64, t, v, w.perm.to(DEV))


def _weight(pk) -> torch.Tensor:
    """float64 [cout, cin] of a packed weight, from its buffers."""
    p = pk.plan
    T, R = p.n_tiles, p.tile_rows
    out = torch.zeros(T, R, p.cin, dtype=torch.float64, device=DEV)

    def put(cols, vals):                                     # [T, R, n] each; a pad's column is negative
        out.scatter_add_(2, cols.clamp(min=0), torch.where(cols >= 0, vals, 0.0))

    if p.n_dense_pad:
        vals = pk.val_dense.view(torch.bfloat16).double().transpose(1, 2).reshape(T, R, -1)
        put(pk.idx_dense.long()[:, None, :].expand(T, R, p.n_dense_pad), vals)
    if p.n_24_pad:
        vals = pk.val_24.view(torch.bfloat16).double().transpose(1, 2).reshape(T, R, -1)     # two of every four
        place = (pk.meta_24[..., None] >> (2 * torch.arange(32, device=DEV))) & 3            # [T, blocks, R, 32]
        place = place.transpose(1, 2).reshape(T, R, -1) + 4 * (torch.arange(p.n_24_pad // 2, device=DEV) // 2)
        put(pk.idx_24.long()[:, None, :].expand(T, R, p.n_24_pad).gather(2, place), vals)
    return out.view(p.cout, p.cin)


def _check(y, w, x, kept, what):
    x = x.double()
    ref, mag = w @ x, w.abs() @ x.abs()
    acc = (kept + 64) * 2.0 ** -23 * mag
    bad = ~((y.double() - ref).abs() <= acc + 2.0 ** -8 * (ref.abs() + acc) + 2.0 ** -133)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} outputs off, the first at {bad.nonzero()[0].tolist()}"


def _stack(cout, cin, t, v, n, mx4, seed=0):
    """A stack of n experts and their weights in float64."""
    pk = [_pack(cout, cin, t, v, seed + i) for i in range(n)]
    st = hinm.Experts.stack(pk)
    if not mx4:
        return st, [_weight(p) for p in pk]
    return hinm.quantize_mx4(st), [_weight(hinm.quantize_mx4(p).dequantize()) for p in pk]


def _routing(starts, counts, cols):
    i32 = lambda q: torch.tensor(q, dtype=torch.int32, device=DEV)
    return hinm.Routing(i32([[0]]), torch.ones(1, 1, device=DEV), i32([[0]]), i32(list(starts) + [cols]), i32(counts),
                        i32([0] * cols))


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("cout,cin,t,v,cols,start,count", [
    (4096, 4096, 0.5, 0.25, 72, 0, 64),          # 64 tokens of one expert, aligned to 8: 3 blocks of 32 by the columns, 2 in use
    (2048, 4096, 0.5, 0.25, 136, 0, 128), (4096, 11008, 0.75, 0.55, 72, 8, 64), (4096, 2052, 0.5, 0.25, 384, 1, 1),
    (4096, 1028, 0.5, 0.25, 1024, 8, 100),       # 128-token blocks
    (4096, 1028, 0.5, 0.25, 4096, 24, 10),       # 256-token blocks
    (4096, 1028, 0.5, 0.25, 4096, 3, 0)])
def test_one_expert_with_fewer_columns_than_the_buffer(cout, cin, t, v, cols, start, count, mx4):
    """A stack of one expert whose range leaves workgroups idle that all columns would fill: no workspace is asked
    for, and the product runs without one."""
    print(f"[experts] one of {cout}x{cin}, {count} of {cols} columns, mx4={mx4}", flush=True)
    st, (w,) = _stack(cout, cin, t, v, 1, mx4)
    assert hinm.spmm_experts_workspace_bytes(st.plan, 1, cols) == 0
    x = torch.randn(cin, cols, generator=torch.Generator().manual_seed(count)).bfloat16().to(DEV)
    y = torch.full((cout, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    hinm.spmm_experts(st, x, _routing([start], [count], cols), out=y)
    torch.cuda.synchronize()
    _check(y[:, start:start + count], w, x[:, start:start + count], cin - st.plan.z, "one expert")
    assert bool((y[:, :start] == 7).all()) and bool((y[:, start + count:] == 7).all())


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("cout,block,counts", [(4096, 128, [150, 100, 147]), (4096, 256, [300, 211, 401])])
def test_last_column_of_a_copied_x(cout, block, counts, mx4):
    """X rows that are not aligned are copied.  With a multiple of 8 columns the copy's rows have no pad, and a range
    that starts at an odd column and ends with the buffer has the last element of X in a word that crosses its end:
    the last column takes it all the same."""
    cin, t, v = 516, 0.5, 0.25
    st, ws = _stack(cout, cin, t, v, 3, mx4)
    cols = -(-(sum(counts) + 3) // 8) * 8                     # leading columns that belong to nobody
    starts = [cols - sum(counts[i:]) for i in range(3)]
    assert starts[2] % 2 == 1
    room = hinm.spmm_experts_workspace_bytes(st.plan, 3, cols)
    assert room == 65536 + 512 * 64 * block * 4
    assert hinm.spmm_experts_workspace_bytes(st.plan, 3, cols, x_aligned=False) == room + -(-cin * cols * 2 // 256) * 256
    x = torch.randn(cin, cols + 1, generator=torch.Generator().manual_seed(block)).bfloat16().to(DEV)[:, 1:]
    x[-1] = 64.0                                              # a lost element shows in every row that keeps it
    y = torch.full((cout, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    print(f"[experts] copied X, {cout} rows, {cols} columns from {starts[2]}, mx4={mx4}", flush=True)
    hinm.spmm_experts(st, x, _routing(starts, counts, cols), out=y)
    torch.cuda.synchronize()
    assert any(bool(w[:, -1].any()) for w in ws)
    for w, s, c in zip(ws, starts, counts):
        _check(y[:, s:s + c], w, x[:, s:s + c], cin - st.plan.z, f"columns from {s}")
    assert bool((y[:, :starts[0]] == 7).all())
