"""Why 8-bit codes become bf16 on their way to the matrix instructions: gfx950's E4M3 instructions add products with
some 13 bits below the largest of eight, the bf16 ones keep what fp32 sums keep (tests/probe/e4m3_sums_probe.hip, built
by __graft_entry__.build())."""
import ctypes
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
LIB = os.path.join(os.path.dirname(os.path.abspath(__file__)), "probe", "libe4m3_sums_probe.so")
DEV = torch.device("cuda:0")


def _sum(a, b, e4m3):
    """The sum of 32 products of E4M3 values, by one instruction."""
    if not os.path.exists(LIB):
        raise FileNotFoundError(f"{LIB} is not built; run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB)
    lib.e4m3_sums_probe.argtypes, lib.e4m3_sums_probe.restype = [ctypes.c_int] + [ctypes.c_void_p] * 3, ctypes.c_int
    t = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    da, db = a.to(t).to(DEV), b.to(t).to(DEV)
    assert torch.equal(da.cpu().float(), a) and torch.equal(db.cpu().float(), b)
    d = torch.full((64,), float("nan"), device=DEV)
    torch.cuda.synchronize()
    rc = lib.e4m3_sums_probe(int(e4m3), da.data_ptr(), db.data_ptr(), d.data_ptr())
    assert rc == 0, f"HIP error {rc}"
    assert bool((d == d[0]).all())
    return float(d[0])


def _case(power):
    """2^16 - 2^16 + 2^power."""
    a, b = torch.zeros(32), torch.zeros(32)
    a[0], a[1], a[2] = 256.0, -256.0, 2.0 ** (power // 2)
    b[0], b[1], b[2] = 256.0, 256.0, 2.0 ** (power - power // 2)
    return a, b


def test_layouts():
    """Small whole numbers in every slot: exact in both."""
    g = torch.Generator().manual_seed(0)
    for _ in range(4):
        a, b = (torch.randint(-8, 9, (32,), generator=g).float() for _ in range(2))
        print("[probe] layouts", flush=True)
        assert _sum(a, b, True) == _sum(a, b, False) == float((a * b).sum())


@pytest.mark.parametrize("power", [8, 4, 2, 0, -4])
def test_small_products_beside_large_ones(power):
    print(f"[probe] 2^16 - 2^16 + 2^{power}", flush=True)
    assert _sum(*_case(power), False) == 2.0 ** power
    assert _sum(*_case(power), True) == (2.0 ** power if power >= 4 else 0.0)
