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


# --------------------------------------------------------------------------- blocks of 128 and 256 tokens

def _block_of(plan, e, cols):
    """Tokens a workgroup takes, read from the room for the sums of split items; None without such room."""
    n = hinm.spmm_experts_workspace_bytes(plan, e, cols)
    return (n - 65536) // (512 * 64 * 4) if n else None


def _layout(counts, how):
    """Starts and columns of ranges: "aligned" as the router makes them; "gaps" at odd columns with others' between
    them; "end" one behind another from column 1, the last one ending with the buffer."""
    if how == "end":
        return [1 + sum(counts[:i]) for i in range(len(counts))], 1 + sum(counts)
    starts, at = [], 0 if how == "aligned" else 1
    for c in counts:
        starts.append(at)
        at += -(-c // 8) * 8 if how == "aligned" else c + 3
    return starts, at


def _matrices(cin, cout, cols, how, seed):
    """X and Y: rows of whole 16 bytes, or (with "gaps") both an odd number of elements apart from an odd place."""
    off, ld = (1, cols + 1 + cols % 2) if how == "gaps" else (0, -(-cols // 8) * 8)
    x = torch.randn(off + cin * ld, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)
    y = torch.full((off + cout * ld,), 7.0, dtype=torch.bfloat16, device=DEV)
    return x[off:].view(cin, ld)[:, :cols], y, y[off:].view(cout, ld)[:, :cols]


def _run(st, ws, counts, how, seed):
    """Two calls against the 64-bit products; other columns' X is NaN, and their Y has to stay."""
    starts, cols = _layout(counts, how)
    p = st.plan
    x, store, y = _matrices(p.cin, p.cout, cols, how, seed)
    mine = torch.zeros(cols, dtype=torch.bool)
    for s, c in zip(starts, counts):
        mine[s:s + c] = True
    x[:, ~mine.to(DEV)] = float("nan")
    r = _routing(starts, counts, cols)
    hinm.spmm_experts(st, x, r, out=y)
    first = store.clone()
    hinm.spmm_experts(st, x, r, out=y)
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), store.view(torch.int16))   # the same bits on every call
    for e, (s, c) in enumerate(zip(starts, counts)):
        if c:
            _check(y[:, s:s + c], ws[e], x[:, s:s + c], p.cin - p.z, f"expert {e}")
    y[:, mine.to(DEV)] = 7.0
    assert bool((store == 7).all())                                        # everything else as it was


@pytest.mark.parametrize("how", ["aligned", "gaps", "end"])
@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("cout,cin,t,v,block,counts", [
    (4096, 516, 0.5, 0.25, 128, [130, 128, 129]),            # items enough: no split
    (4096, 516, 0.75, 0.55, 128, [1, 385, 7]),
    (4096, 260, 0.0, 0.0, 256, [257, 300, 511]),             # dense blocks alone
    (4096, 516, 0.5, 0.25, 256, [700, 0, 255]),
    (1536, 1028, 0.5, 0.25, 128, [0] * 5 + [461, 0, 300, 0, 0, 155] + [0] * 4 + [1]),   # 16 experts: split in two
    (1024, 1028, 0.5, 0.25, 256, [555, 1, 777, 299]),        # split in two
    (1024, 2052, 0.5, 0.25, 256, [0, 1509, 0, 1]),           # split in four
    (512, 2052, 0.5, 0.25, 256, [5, 3001, 0, 129]),          # few tiles, split in four
])
def test_long_ranges(cout, cin, t, v, block, counts, mx4, how):
    st, ws = _stack(cout, cin, t, v, len(counts), mx4, seed=cin)
    cols = _layout(counts, how)[1]
    if len(counts) == 16:                                    # 49 to 64 columns an expert on average
        assert 16 * 48 < cols <= 16 * 64
    print(f"[experts] {cout}x{cin} counts={counts} mx4={mx4} {how}", flush=True)
    assert _block_of(st.plan, len(counts), cols) == block
    _run(st, ws, counts, how, seed=cout + cols)


@pytest.mark.parametrize("mx4", [False, True])
def test_long_ranges_of_large_weights(mx4):
    """Two experts of 11008x4096 over 2047 tokens."""
    g = torch.Generator(device=DEV).manual_seed(2)
    pk = []
    for _ in range(2):
        w = torch.randn(11008, 4096, generator=g, device=DEV).bfloat16()
        perm = torch.rand(172, 4096, generator=g, device=DEV).argsort(1).int()
        pk.append(hinm.pack(w, w.float().abs(), 64, 0.75, 0.55, perm))
    st = hinm.Experts.stack(pk)
    if mx4:
        st = hinm.quantize_mx4(st)
        pk = [hinm.quantize_mx4(p).dequantize() for p in pk]
    ws = [_weight(p) for p in pk]
    for how in ("aligned", "end"):
        print(f"[experts] 11008x4096, mx4={mx4} {how}", flush=True)
        assert _block_of(st.plan, 2, _layout([1500, 547], how)[1]) == 256
        _run(st, ws, [1500, 547], how, seed=5)


@pytest.mark.parametrize("cout,cin,batch,room", [
    (4096, 516, 1000, 0), (4096, 516, 999, 0),               # 128 tokens, 512 items
    (2048, 1028, 1000, 128), (2048, 1028, 1001, 128),        # 128 tokens, split in two
    (4096, 516, 1100, 0), (4096, 516, 1101, 0), (4096, 516, 1281, 0)])   # 256 tokens
@pytest.mark.parametrize("aligned", [True, False])
def test_long_four_bit_products(cout, cin, batch, room, aligned):
    pk = _pack(cout, cin, 0.5, 0.25, seed=batch)
    q = hinm.quantize_mx4(pk)
    w = _weight(q.dequantize())
    split = 65536 + 512 * 64 * 4 * room if room else 0
    ld = -(-batch // 8) * 8 if aligned else batch + 1 + batch % 2
    x = torch.randn(cin, ld, generator=torch.Generator().manual_seed(batch)).bfloat16().to(DEV)[:, ld - batch if not aligned else 0:]
    x = x[:, :batch]
    print(f"[mx4 spmm] {cout}x{cin} batch={batch} aligned={aligned}", flush=True)
    assert hinm.spmm_experts_workspace_bytes(q.plan, 1, batch) == split
    copy = -(-cin * -(-batch // 8) * 8 * 2 // 256) * 256     # more than 32 tokens a workgroup: unaligned rows are copied
    assert hinm.spmm_experts_workspace_bytes(q.plan, 1, batch, x_aligned=False) == max(split, 65536) + copy
    y = hinm.spmm(q, x)
    again = hinm.spmm(q, x)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    _check(y, w, x, cin - q.plan.z, f"batch {batch}")


# --------------------------------------------------------------------------- blocks of 16 and 32 tokens

@pytest.mark.parametrize("cin", [992, 1024, 1056, 2016, 2048, 2080])
@pytest.mark.parametrize("batch", [1, 16, 17, 32, 33])
def test_splits_of_short_products(cin, batch):
    """31, 32, 33, 63, 64 and 65 K-blocks of dense values, at which the number of splits steps, and the token counts
    around blocks of 16 and 32."""
    pk = _pack(128, cin, 0.0, 0.0, seed=cin)
    assert pk.plan.n_dense_pad // 32 == cin // 32
    q = hinm.quantize_mx4(pk)
    x = torch.randn(cin, batch, generator=torch.Generator().manual_seed(batch)).bfloat16().to(DEV)
    print(f"[mx4 spmm] 128x{cin} batch={batch}", flush=True)
    assert _block_of(q.plan, 1, batch) == (16 if batch <= 16 else 32)
    _check(hinm.spmm(q, x), _weight(q.dequantize()), x, cin, f"batch {batch}")
    st = hinm.Experts.stack([pk, pk])
    counts = [batch, 3]
    _run(st, [_weight(pk)] * 2, counts, "gaps", seed=cin + batch)


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("counts,block", [([16, 17, 3], 16), ([20, 20, 20], 16), ([21, 20, 23], 32), ([48, 32, 33], 32),
                                          ([1, 0, 140], 32)])
def test_short_ranges(counts, block, mx4):
    st, ws = _stack(192, 516, 0.75, 0.55, 3, mx4, seed=9)
    assert _block_of(st.plan, 3, sum(counts)) == block
    for how in ("aligned", "gaps", "end"):
        print(f"[experts] counts={counts} mx4={mx4} {how}", flush=True)
        _run(st, ws, counts, how, seed=sum(counts))
