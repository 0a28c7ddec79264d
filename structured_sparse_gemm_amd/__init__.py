"""Python binding of libhinm: hierarchical N:M sparse weight x dense activation on MI355X.

Argument marshalling only.  Every step of the pack and of the product runs in
the HIP kernels of ``libhinm.so``; PyTorch supplies device memory and the
current HIP stream.  If the library is not built, every call raises: there is
no fallback path.

    packed = pack(w_bf16, importance, tile_rows, t_s, v_s, perm=None)
    y = spmm(packed, x_bf16)          # y = (W (.) M) x, bf16 [cout, batch]
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import os
from typing import Optional, Tuple

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhinm.so")

HINM_ABI_VERSION = 2
HINM_PACKED_WINDOWED = 1     # flags bit: block-diagonal perms (blocks of 64), see include/hinm.h
HINM_FORMAT_VERSION = 1       # packed-buffer layout version (include/hinm.h)
HINM_MX4_FORMAT_VERSION = 1   # layout version of 4-bit microscaled values (include/hinm.h)
HINM_BF16, HINM_FP32 = 0, 1   # element types of the router's logits
HINM_NOALLOC_SCRATCH_BYTES = 65536 + (32 << 20)   # hinm_spmm_noalloc's device array (include/hinm.h)
STATUS = {0: "HINM_OK", 1: "HINM_EINVAL", 2: "HINM_ESHAPE", 3: "HINM_EPERM", 4: "HINM_EIMPORTANCE",
          5: "HINM_EALIGN", 6: "HINM_EWORKSPACE", 7: "HINM_EHIP", 8: "HINM_EDEVICE"}

# Every symbol the C ABI exports (include/hinm.h).
EXPORTS = ("hinm_abi_version", "hinm_plan", "hinm_pack_workspace_bytes", "hinm_pack",
           "hinm_spmm_workspace_bytes", "hinm_spmm", "hinm_spmm_rows", "hinm_translate_indices",
           "hinm_boundary_workspace_bytes", "hinm_boundary_search", "hinm_plan_tiles",
           "hinm_pack_tiles_workspace_bytes", "hinm_pack_tiles", "hinm_spmm_tiles_workspace_bytes",
           "hinm_spmm_tiles", "hinm_boundary_search_tiles", "hinm_gyro_workspace_bytes", "hinm_gyro_permute",
           "hinm_set_option", "hinm_get_option", "hinm_spmm_noalloc", "hinm_spmm_group_workspace_bytes",
           "hinm_spmm_group", "hinm_route_columns", "hinm_route_workspace_bytes", "hinm_route", "hinm_dispatch",
           "hinm_combine", "hinm_spmm_experts_workspace_bytes", "hinm_spmm_experts", "hinm_mx4_quantize",
           "hinm_mx4_dequantize", "hinm_spmm_mx4_workspace_bytes", "hinm_spmm_mx4", "hinm_spmm_experts_mx4",
           "hinm_status_str", "hinm_last_error")

# Launch-shape options (hinm_set_option): name -> HINM_OPT_* key.
OPTIONS = {"decode_path": 1, "decode_wgs": 2, "prefill_nt": 3, "prefill_splits": 4, "prefill_path": 5,
           "prefill_per_xcd": 6, "prefill_tb_group": 7, "prefill_stagger": 8}


class HinmError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status
        self.name = STATUS.get(status, str(status))


class PlanT(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_int32), ("cout", ctypes.c_int32), ("cin", ctypes.c_int32),
                ("tile_rows", ctypes.c_int32), ("n_tiles", ctypes.c_int32), ("z", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("n_dense", ctypes.c_int32), ("n_24", ctypes.c_int32),
                ("n_pruned", ctypes.c_int32), ("n_dense_pad", ctypes.c_int32), ("n_24_pad", ctypes.c_int32),
                ("kb_dense", ctypes.c_int32), ("kb_24", ctypes.c_int32),
                ("t_s", ctypes.c_double), ("v_s", ctypes.c_double), ("p_s", ctypes.c_double),
                ("bytes_val_dense", ctypes.c_int64), ("bytes_idx_dense", ctypes.c_int64),
                ("bytes_val_24", ctypes.c_int64), ("bytes_meta_24", ctypes.c_int64),
                ("bytes_idx_24", ctypes.c_int64)]


class PackedT(ctypes.Structure):
    _fields_ = [("plan", PlanT), ("val_dense", ctypes.c_void_p), ("idx_dense", ctypes.c_void_p),
                ("val_24", ctypes.c_void_p), ("meta_24", ctypes.c_void_p), ("idx_24", ctypes.c_void_p),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class Mx4T(ctypes.Structure):
    _fields_ = [("plan", PlanT), ("val_dense", ctypes.c_void_p), ("scale_dense", ctypes.c_void_p),
                ("idx_dense", ctypes.c_void_p), ("val_24", ctypes.c_void_p), ("scale_24", ctypes.c_void_p),
                ("meta_24", ctypes.c_void_p), ("idx_24", ctypes.c_void_p)]


class TPlanT(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_int32), ("cout", ctypes.c_int32), ("cin", ctypes.c_int32),
                ("tile_rows", ctypes.c_int32), ("n_tiles", ctypes.c_int32), ("z", ctypes.c_int32),
                ("max_n_dense_pad", ctypes.c_int32), ("max_n_24_pad", ctypes.c_int32),
                ("dense_blocks", ctypes.c_int32), ("blocks_24", ctypes.c_int32), ("t_s", ctypes.c_double),
                ("bytes_val_dense", ctypes.c_int64), ("bytes_idx_dense", ctypes.c_int64),
                ("bytes_val_24", ctypes.c_int64), ("bytes_meta_24", ctypes.c_int64),
                ("bytes_idx_24", ctypes.c_int64), ("bytes_tiles", ctypes.c_int64)]


class TPackedT(ctypes.Structure):
    _fields_ = [("plan", TPlanT), ("tiles", ctypes.c_void_p), ("val_dense", ctypes.c_void_p),
                ("idx_dense", ctypes.c_void_p), ("val_24", ctypes.c_void_p), ("meta_24", ctypes.c_void_p),
                ("idx_24", ctypes.c_void_p)]


_lib = None


def library() -> ctypes.CDLL:
    """Loads libhinm.so (built in-tree); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                              "python structured_sparse_gemm_amd/build.py")
        lib = ctypes.CDLL(LIB_PATH)
        P, S, I64, I32, D, VP = (ctypes.POINTER(PlanT), ctypes.c_size_t, ctypes.c_int64, ctypes.c_int32,
                                 ctypes.c_double, ctypes.c_void_p)
        sig = {
            "hinm_abi_version": ([], ctypes.c_int),
            "hinm_plan": ([I64, I64, I32, D, D, P], ctypes.c_int),
            "hinm_pack_workspace_bytes": ([P, ctypes.POINTER(S)], ctypes.c_int),
            "hinm_pack": ([P, VP, I64, VP, I64, VP, ctypes.POINTER(PackedT), VP, S, VP], ctypes.c_int),
            "hinm_spmm_workspace_bytes": ([P, I64, ctypes.POINTER(S)], ctypes.c_int),
            "hinm_spmm": ([ctypes.POINTER(PackedT), VP, I64, I64, VP, I64, VP, S, VP], ctypes.c_int),
            "hinm_spmm_rows": ([ctypes.POINTER(PackedT), VP, I64, I64, VP, I64, VP, VP, S, VP], ctypes.c_int),
            "hinm_translate_indices": ([ctypes.POINTER(PackedT), VP, VP, S, VP], ctypes.c_int),
            "hinm_boundary_workspace_bytes": ([I64, I64, I32, ctypes.POINTER(S)], ctypes.c_int),
            "hinm_plan_tiles": ([I64, I64, I32, D, ctypes.POINTER(D), ctypes.POINTER(TPlanT), ctypes.POINTER(I32)],
                                ctypes.c_int),
            "hinm_pack_tiles_workspace_bytes": ([ctypes.POINTER(TPlanT), ctypes.POINTER(S)], ctypes.c_int),
            "hinm_pack_tiles": ([ctypes.POINTER(TPlanT), VP, I64, VP, I64, VP, ctypes.POINTER(TPackedT), VP, S, VP],
                                ctypes.c_int),
            "hinm_spmm_tiles_workspace_bytes": ([ctypes.POINTER(TPlanT), I64, ctypes.POINTER(S)], ctypes.c_int),
            "hinm_spmm_tiles": ([ctypes.POINTER(TPackedT), VP, I64, I64, VP, I64, VP, S, VP], ctypes.c_int),
            "hinm_boundary_search_tiles": ([I64, I64, I32, D, D, VP, I64, VP, VP, S, ctypes.POINTER(D),
                                            ctypes.POINTER(I32), VP], ctypes.c_int),
            "hinm_boundary_search": ([I64, I64, I32, D, D, VP, I64, VP, VP, S, ctypes.POINTER(D),
                                      ctypes.POINTER(D), ctypes.POINTER(D), I32, ctypes.POINTER(I32), VP],
                                     ctypes.c_int),
            "hinm_gyro_workspace_bytes": ([P, I32, ctypes.POINTER(S)], ctypes.c_int),
            "hinm_gyro_permute": ([P, VP, I64, VP, I32, I32, I32, VP, VP, ctypes.POINTER(D), VP, S, VP],
                                  ctypes.c_int),
            "hinm_set_option": ([ctypes.c_int, I64], ctypes.c_int),
            "hinm_spmm_noalloc": ([ctypes.POINTER(PackedT), VP, I64, I64, VP, I64, VP], ctypes.c_int),
            "hinm_spmm_group_workspace_bytes": ([ctypes.c_int, VP, I64, ctypes.POINTER(S)], ctypes.c_int),
            "hinm_spmm_group": ([ctypes.c_int, VP, VP, I64, I64, VP, VP, VP, S, VP], ctypes.c_int),
            "hinm_route_columns": ([I64, I32, I32, I32, ctypes.POINTER(I64)], ctypes.c_int),
            "hinm_route_workspace_bytes": ([I64, I32, ctypes.POINTER(S)], ctypes.c_int),
            "hinm_route": ([VP, I32, I64, I64, I32, I32, I32, I32, VP, VP, VP, VP, VP, VP, I64, VP, S, VP],
                           ctypes.c_int),
            "hinm_dispatch": ([VP, I64, I64, I64, VP, I64, VP, I64, VP], ctypes.c_int),
            "hinm_combine": ([VP, I64, I64, I64, VP, VP, I64, I32, VP, I64, VP], ctypes.c_int),
            "hinm_spmm_experts_workspace_bytes": ([P, I32, I64, I32, ctypes.POINTER(S)], ctypes.c_int),
            "hinm_spmm_experts": ([ctypes.POINTER(PackedT), I32, VP, I64, I64, VP, VP, VP, I64, VP, S, VP],
                                  ctypes.c_int),
            "hinm_spmm_experts_mx4": ([ctypes.POINTER(Mx4T), I32, VP, I64, I64, VP, VP, VP, I64, VP, S, VP],
                                      ctypes.c_int),
            "hinm_mx4_quantize": ([ctypes.POINTER(PackedT), I32, ctypes.POINTER(Mx4T), VP], ctypes.c_int),
            "hinm_mx4_dequantize": ([ctypes.POINTER(Mx4T), I32, ctypes.POINTER(PackedT), VP], ctypes.c_int),
            "hinm_spmm_mx4_workspace_bytes": ([P, I64, I32, ctypes.POINTER(S)], ctypes.c_int),
            "hinm_spmm_mx4": ([ctypes.POINTER(Mx4T), VP, I64, I64, VP, I64, VP, S, VP], ctypes.c_int),
            "hinm_get_option": ([ctypes.c_int, ctypes.POINTER(I64)], ctypes.c_int),
            "hinm_status_str": ([ctypes.c_int], ctypes.c_char_p),
            "hinm_last_error": ([], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, res
        if lib.hinm_abi_version() != HINM_ABI_VERSION:
            raise ImportError("libhinm ABI version mismatch")
        _lib = lib
    return _lib


def _check(status: int) -> None:
    if status != 0:
        raise HinmError(status, library().hinm_last_error().decode())


@dataclasses.dataclass(frozen=True)
class Plan:
    cout: int
    cin: int
    tile_rows: int
    n_tiles: int
    z: int
    groups: int
    n_dense: int
    n_24: int
    n_pruned: int
    n_dense_pad: int
    n_24_pad: int
    t_s: float
    v_s: float
    p_s: float
    bytes_val_dense: int
    bytes_idx_dense: int
    bytes_val_24: int
    bytes_meta_24: int
    bytes_idx_24: int
    raw: PlanT = dataclasses.field(repr=False, compare=False)

    @property
    def packed_bytes(self) -> int:
        return (self.bytes_val_dense + self.bytes_idx_dense + self.bytes_val_24 + self.bytes_meta_24
                + self.bytes_idx_24)


def plan(cout: int, cin: int, tile_rows: int, t_s: float, v_s: float) -> Plan:
    """Region counts (host only, needs no GPU)."""
    raw = PlanT()
    _check(library().hinm_plan(cout, cin, tile_rows, float(t_s), float(v_s), ctypes.byref(raw)))
    kw = {f.name: getattr(raw, f.name) for f in dataclasses.fields(Plan) if f.name != "raw"}
    return Plan(raw=raw, **kw)


@dataclasses.dataclass
class HinmPacked:
    """A packed weight: the plan and its five device buffers (torch tensors)."""

    plan: Plan
    val_dense: torch.Tensor   # int16 bits of bf16 [T, n_dense_pad/32, R, 32]
    idx_dense: torch.Tensor   # int32 [T, n_dense_pad]
    val_24: torch.Tensor      # int16 bits of bf16 [T, n_24_pad/64, R, 32]
    meta_24: torch.Tensor     # int64 bits of uint64 [T, n_24_pad/64, R]
    idx_24: torch.Tensor      # int32 [T, n_24_pad]
    flags: int = 0            # HINM_PACKED_* bits (set by pack)

    def struct(self) -> PackedT:
        """The C view of this weight (built once; the tensors must not be replaced afterwards)."""
        st = self.__dict__.get("_struct")
        if st is None:
            def ptr(t):
                return t.data_ptr() if t.numel() else None
            st = PackedT(self.plan.raw, ptr(self.val_dense), ptr(self.idx_dense), ptr(self.val_24),
                         ptr(self.meta_24), ptr(self.idx_24), self.flags, 0)
            self.__dict__["_struct"] = st
            self.__dict__["_ws_need"] = {}
        return st

    @property
    def device(self) -> torch.device:
        return self.idx_24.device

    def nbytes(self) -> int:
        return self.plan.packed_bytes

    def state_dict(self) -> dict:
        """Plain tensors and numbers (torch.save / torch.load(weights_only=True) round-trip them): the
        layout version, the plan's arguments and the five buffers."""
        p = self.plan
        return {"format": "hinm-packed", "format_version": HINM_FORMAT_VERSION, "cout": p.cout, "cin": p.cin,
                "tile_rows": p.tile_rows, "t_s": p.t_s, "v_s": p.v_s, "flags": int(self.flags),
                **{k: getattr(self, k) for k in _BUFFERS}}

    @classmethod
    def from_state_dict(cls, sd: dict, device=None) -> "HinmPacked":
        """Rebuilds a packed weight from state_dict() output: checks the layout version, recomputes the
        plan from its arguments and checks every buffer's dtype and shape against it."""
        _check_format(sd, "hinm-packed")
        p = plan(int(sd["cout"]), int(sd["cin"]), int(sd["tile_rows"]), float(sd["t_s"]), float(sd["v_s"]))
        T, R = p.n_tiles, p.tile_rows
        want = {"val_dense": ((T, p.n_dense_pad // 32, R, 32), torch.int16),
                "idx_dense": ((T, p.n_dense_pad), torch.int32),
                "val_24": ((T, p.n_24_pad // 64, R, 32), torch.int16),
                "meta_24": ((T, p.n_24_pad // 64, R), torch.int64),
                "idx_24": ((T, p.n_24_pad), torch.int32)}
        return cls(p, **_checked_buffers(sd, want, device), flags=int(sd.get("flags", 0)))


_BUFFERS = ("val_dense", "idx_dense", "val_24", "meta_24", "idx_24")


def _check_format(sd: dict, kind: str, version: int = HINM_FORMAT_VERSION) -> None:
    if not isinstance(sd, dict) or sd.get("format") != kind:
        raise ValueError(f"not a stored {kind} weight")
    if sd.get("format_version") != version:
        raise ValueError(f"stored layout version {sd.get('format_version')!r}, this library reads "
                         f"{version}: pack the weight again")


def _checked_buffers(sd: dict, want: dict, device) -> dict:
    out = {}
    for k, (shape, dtype) in want.items():
        t = sd.get(k)
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != tuple(shape):
            got = (None if not isinstance(t, torch.Tensor) else (t.dtype, tuple(t.shape)))
            raise ValueError(f"stored buffer {k}: expected {dtype} {tuple(shape)}, found {got}")
        t = t.contiguous()
        out[k] = t.to(device) if device is not None else t
    return out


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(device: torch.device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index if device.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(device).cuda_stream


def _empty(shape, dtype, device):
    # 256-byte aligned by the caching allocator; zero-size buffers stay empty.
    return torch.empty(shape, dtype=dtype, device=device)


def pack_workspace_bytes(p: Plan) -> int:
    n = ctypes.c_size_t()
    _check(library().hinm_pack_workspace_bytes(ctypes.byref(p.raw), ctypes.byref(n)))
    return n.value


def alloc_packed(p: Plan, device) -> HinmPacked:
    T, R = p.n_tiles, p.tile_rows
    return HinmPacked(
        p,
        _empty((T, p.n_dense_pad // 32, R, 32), torch.int16, device),
        _empty((T, p.n_dense_pad), torch.int32, device),
        _empty((T, p.n_24_pad // 64, R, 32), torch.int16, device),
        _empty((T, p.n_24_pad // 64, R), torch.int64, device),
        _empty((T, p.n_24_pad), torch.int32, device))


def pack(w: torch.Tensor, importance: torch.Tensor, tile_rows: int, t_s: float, v_s: float,
         perm: Optional[torch.Tensor] = None) -> HinmPacked:
    """Packs a bf16 weight [cout, cin] on its device (synchronous).

    importance: fp32 [cout, cin] (finite, >= 0); perm: int32 [cout/tile_rows, cin]
    or None for the identity, perm[t][j] = original column at position j of tile t.
    """
    if w.dtype != torch.bfloat16 or w.dim() != 2 or not w.is_cuda:
        raise ValueError("w must be a 2-D bf16 CUDA tensor")
    if importance.dtype != torch.float32 or importance.shape != w.shape or importance.device != w.device:
        raise ValueError("importance must be fp32 with the shape and device of w")
    if w.stride(1) != 1 or importance.stride(1) != 1:
        raise ValueError("w and importance must have unit column stride")
    cout, cin = w.shape
    p = plan(cout, cin, tile_rows, t_s, v_s)
    if perm is not None:
        if perm.dtype != torch.int32 or perm.shape != (p.n_tiles, cin) or perm.device != w.device:
            raise ValueError(f"perm must be int32 [{p.n_tiles}, {cin}] on the device of w")
        perm = perm.contiguous()
    out = alloc_packed(p, w.device)
    ws = torch.empty(pack_workspace_bytes(p), dtype=torch.uint8, device=w.device)
    st = out.struct()
    with torch.cuda.device(w.device):
        _check(library().hinm_pack(ctypes.byref(p.raw), w.data_ptr(), w.stride(0), importance.data_ptr(),
                                   importance.stride(0), perm.data_ptr() if perm is not None else None,
                                   ctypes.byref(st), ws.data_ptr(), ws.numel(), _stream_ptr(w.device)))
    out.flags = int(st.flags)
    return out


@dataclasses.dataclass
class TilePlan:
    """Per-tile region counts (hinm_plan_tiles): shared fields, buffer sizes and the tile table."""

    raw: TPlanT = dataclasses.field(repr=False)
    tiles: "np.ndarray"          # int32 [n_tiles, 4]: first dense block, n_dense, first 2:4 block, n_24
    v_s: tuple

    def __getattr__(self, name):
        raw = self.__dict__.get("raw")
        if raw is not None and name in dict(TPlanT._fields_):
            return getattr(raw, name)
        raise AttributeError(name)

    @property
    def packed_bytes(self) -> int:
        r = self.raw
        return r.bytes_val_dense + r.bytes_idx_dense + r.bytes_val_24 + r.bytes_meta_24 + r.bytes_idx_24


def plan_tiles(cout: int, cin: int, tile_rows: int, t_s: float, v_s) -> TilePlan:
    """Per-tile plan (host only): tile t uses v_s[t]."""
    import numpy as np
    v = [float(x) for x in v_s]
    raw = TPlanT()
    n_tiles = cout // tile_rows if tile_rows > 0 else 0
    if len(v) != n_tiles:
        raise ValueError(f"{n_tiles} per-tile v_s values are needed, got {len(v)}")
    arr = (ctypes.c_double * max(1, len(v)))(*v)
    tiles = (ctypes.c_int32 * max(1, 4 * n_tiles))()
    _check(library().hinm_plan_tiles(cout, cin, tile_rows, float(t_s), arr, ctypes.byref(raw), tiles))
    return TilePlan(raw=raw, tiles=np.ctypeslib.as_array(tiles)[:4 * n_tiles].reshape(n_tiles, 4).copy(),
                    v_s=tuple(v))


@dataclasses.dataclass
class HinmTPacked:
    """A packed weight with per-tile counts: the plan, the device tile table and five device buffers."""

    plan: TilePlan
    tiles: torch.Tensor       # int32 [T, 4] on the device
    val_dense: torch.Tensor   # int16 bits of bf16 [dense_blocks, R, 32]
    idx_dense: torch.Tensor   # int32 [dense_blocks * 32]
    val_24: torch.Tensor      # int16 bits of bf16 [blocks_24, R, 32]
    meta_24: torch.Tensor     # int64 bits of uint64 [blocks_24, R]
    idx_24: torch.Tensor      # int32 [blocks_24 * 64]

    def struct(self) -> TPackedT:
        st = self.__dict__.get("_struct")
        if st is None:
            def ptr(t):
                return t.data_ptr() if t.numel() else None
            st = TPackedT(self.plan.raw, ptr(self.tiles), ptr(self.val_dense), ptr(self.idx_dense),
                          ptr(self.val_24), ptr(self.meta_24), ptr(self.idx_24))
            self.__dict__["_struct"] = st
            self.__dict__["_ws_need"] = {}
        return st

    @property
    def device(self) -> torch.device:
        return self.tiles.device

    def nbytes(self) -> int:
        return self.plan.packed_bytes

    def state_dict(self) -> dict:
        """As HinmPacked.state_dict, with the per-tile v_s and the tile table."""
        p = self.plan
        return {"format": "hinm-packed-tiles", "format_version": HINM_FORMAT_VERSION, "cout": p.cout,
                "cin": p.cin, "tile_rows": p.tile_rows, "t_s": p.t_s,
                "v_s": torch.tensor(p.v_s, dtype=torch.float64), "tiles": self.tiles,
                **{k: getattr(self, k) for k in _BUFFERS}}

    @classmethod
    def from_state_dict(cls, sd: dict, device=None) -> "HinmTPacked":
        _check_format(sd, "hinm-packed-tiles")
        v = sd.get("v_s")
        if not isinstance(v, torch.Tensor):
            raise ValueError("stored per-tile v_s missing")
        p = plan_tiles(int(sd["cout"]), int(sd["cin"]), int(sd["tile_rows"]), float(sd["t_s"]), v.tolist())
        R = p.tile_rows
        want = {"tiles": ((p.n_tiles, 4), torch.int32),
                "val_dense": ((p.dense_blocks, R, 32), torch.int16),
                "idx_dense": ((p.dense_blocks * 32,), torch.int32),
                "val_24": ((p.blocks_24, R, 32), torch.int16),
                "meta_24": ((p.blocks_24, R), torch.int64),
                "idx_24": ((p.blocks_24 * 64,), torch.int32)}
        bufs = _checked_buffers(sd, want, device)
        if not np.array_equal(bufs["tiles"].cpu().numpy(), p.tiles):
            raise ValueError("stored tile table does not match the per-tile plan")
        return cls(p, **bufs)


def pack_tiles(w: torch.Tensor, importance: torch.Tensor, tile_rows: int, t_s: float, v_s,
               perm: Optional[torch.Tensor] = None) -> HinmTPacked:
    """Packs a bf16 weight with one v_s per tile (hinm_pack_tiles, synchronous)."""
    if w.dtype != torch.bfloat16 or w.dim() != 2 or not w.is_cuda:
        raise ValueError("w must be a 2-D bf16 CUDA tensor")
    if importance.dtype != torch.float32 or importance.shape != w.shape or importance.device != w.device:
        raise ValueError("importance must be fp32 with the shape and device of w")
    if w.stride(1) != 1 or importance.stride(1) != 1:
        raise ValueError("w and importance must have unit column stride")
    cout, cin = w.shape
    p = plan_tiles(cout, cin, tile_rows, t_s, v_s)
    if perm is not None:
        if perm.dtype != torch.int32 or perm.shape != (p.n_tiles, cin) or perm.device != w.device:
            raise ValueError(f"perm must be int32 [{p.n_tiles}, {cin}] on the device of w")
        perm = perm.contiguous()
    dev, R = w.device, tile_rows
    out = HinmTPacked(p, torch.from_numpy(p.tiles).to(dev),
                      _empty((p.dense_blocks, R, 32), torch.int16, dev), _empty((p.dense_blocks * 32,), torch.int32, dev),
                      _empty((p.blocks_24, R, 32), torch.int16, dev), _empty((p.blocks_24, R), torch.int64, dev),
                      _empty((p.blocks_24 * 64,), torch.int32, dev))
    n = ctypes.c_size_t()
    _check(library().hinm_pack_tiles_workspace_bytes(ctypes.byref(p.raw), ctypes.byref(n)))
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    st = out.struct()
    with torch.cuda.device(dev):
        _check(library().hinm_pack_tiles(ctypes.byref(p.raw), w.data_ptr(), w.stride(0), importance.data_ptr(),
                                         importance.stride(0), perm.data_ptr() if perm is not None else None,
                                         ctypes.byref(st), ws.data_ptr(), ws.numel(), _stream_ptr(dev)))
    return out


def spmm_tiles_workspace_bytes(p: TilePlan, batch: int) -> int:
    n = ctypes.c_size_t()
    _check(library().hinm_spmm_tiles_workspace_bytes(ctypes.byref(p.raw), batch, ctypes.byref(n)))
    return n.value


def spmm_workspace_bytes(p: Plan, batch: int) -> int:
    n = ctypes.c_size_t()
    _check(library().hinm_spmm_workspace_bytes(ctypes.byref(p.raw), batch, ctypes.byref(n)))
    return n.value


def _one_weight(packed, what: str) -> None:
    """Refuses what is not a single uniform bf16 weight: the C calls read its buffers as such."""
    if isinstance(packed, HinmPacked):
        return
    if isinstance(packed, Experts) or (isinstance(packed, HinmMx4) and packed.n_experts is not None):
        raise ValueError(f"{what} takes one weight; a stack of experts is multiplied by spmm_experts")
    if isinstance(packed, HinmMx4):
        raise ValueError(f"{what} takes bf16 values; 4-bit weights are multiplied one at a time by spmm")
    if isinstance(packed, HinmTPacked):
        raise ValueError(f"{what} takes uniform packed weights (pack, not pack_tiles)")
    raise ValueError(f"{what} takes a packed weight, not a {type(packed).__name__}")


_ws_cache = {}
_ws_retired = []
_opt_gen = 0


def get_option(name: str) -> int:
    """Current value of a launch-shape option (see OPTIONS and hinm_set_option)."""
    v = ctypes.c_int64()
    _check(library().hinm_get_option(OPTIONS[name], ctypes.byref(v)))
    return v.value


def set_option(name: str, value: int) -> None:
    """Sets a process-wide launch-shape option (hinm_set_option)."""
    global _opt_gen
    _check(library().hinm_set_option(OPTIONS[name], int(value)))
    _opt_gen += 1          # workspace sizes remembered per weight depend on the options


class options:
    """Context manager: ``with options(prefill_splits=2): ...`` sets options and restores them on exit."""

    def __init__(self, **kw):
        for k in kw:
            if k not in OPTIONS:
                raise KeyError(f"unknown option {k!r}; known: {sorted(OPTIONS)}")
        self.kw = kw
        self.saved = {}

    def __enter__(self):
        for k, v in self.kw.items():
            self.saved[k] = get_option(k)
            set_option(k, v)
        return self

    def __exit__(self, *exc):
        for k, v in self.saved.items():
            set_option(k, v)
        return False


def _workspace(device: torch.device, stream: int, nbytes: int) -> Optional[torch.Tensor]:
    """The default workspace of (device, stream): zero-filled when made, at least nbytes.

    One per stream, because a workspace holds the split reduction's arrival
    counters and partial sums, so products that may overlap (different
    streams) must not share one.  A buffer that is outgrown is kept alive, not
    freed: HIP graphs captured earlier, or work still queued, may name it.
    """
    if nbytes == 0:
        return None
    key = (device.index, stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        if buf is not None:
            _ws_retired.append(buf)
        buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def spmm(packed: HinmPacked, x: torch.Tensor, out: Optional[torch.Tensor] = None,
         workspace: Optional[torch.Tensor] = None, out_rows: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = (W (.) M) X: x bf16 [cin, batch] (row stride >= batch), returns bf16 [cout, batch].

    With ``out_rows`` (int32 [cout] on the device, a permutation), row r of the
    product is written to row out_rows[r] of Y (hinm_spmm_rows).
    Asynchronous on the current stream.  ``workspace`` (uint8, device, zero-filled before its first use) may
    be given; otherwise each stream has its own default workspace, so products on different streams may
    overlap.  The per-call host work is kept to argument checks and one C call, so that small products are
    not bound by Python.  A weight with 4-bit microscaled values (quantize_mx4) runs hinm_spmm_mx4; it takes no
    ``out_rows``.
    """
    if isinstance(packed, HinmMx4):
        if out_rows is not None:
            raise ValueError("out_rows is not supported with 4-bit values")
        return _spmm_mx4(packed, x, out, workspace)
    tiled = isinstance(packed, HinmTPacked)
    if not tiled and not isinstance(packed, HinmPacked):
        _one_weight(packed, "spmm")
    p = packed.plan
    dev = x.device
    if tiled and out_rows is not None:
        raise ValueError("out_rows is not supported with per-tile counts")
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[0] != p.cin or dev != packed.idx_24.device:
        raise ValueError(f"x must be bf16 [{p.cin}, batch] on {packed.device}")
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    batch = x.shape[1]
    if out is None:
        out = torch.empty((p.cout, batch), dtype=torch.bfloat16, device=dev)
    elif out.dtype != torch.bfloat16 or out.shape != (p.cout, batch) or out.stride(1) != 1 or out.device != dev:
        raise ValueError(f"out must be bf16 [{p.cout}, {batch}] with unit column stride on {dev}")
    if out_rows is not None and (out_rows.dtype != torch.int32 or out_rows.shape != (p.cout,)
                                 or not out_rows.is_contiguous() or out_rows.device != dev):
        raise ValueError(f"out_rows must be a contiguous int32 [{p.cout}] tensor on {dev}")
    st = packed.struct()
    need_cache = packed.__dict__["_ws_need"]
    need = need_cache.get((batch, _opt_gen))
    if need is None:
        need = need_cache[(batch, _opt_gen)] = (spmm_tiles_workspace_bytes(p, batch) if tiled else
                                                spmm_workspace_bytes(p, batch))
    stream = _stream_ptr(dev)
    if workspace is None:
        workspace = _workspace(dev, stream, need)
    lib = library()
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_n = workspace.numel() if workspace is not None else 0
    ldx = max(x.stride(0), batch) if batch else 0
    ldy = max(out.stride(0), batch) if batch else 0
    if tiled:
        call, args = lib.hinm_spmm_tiles, (ctypes.byref(st), x.data_ptr(), batch, ldx, out.data_ptr(), ldy, ws_ptr,
                                           ws_n, stream)
    elif out_rows is None:
        call, args = lib.hinm_spmm, (ctypes.byref(st), x.data_ptr(), batch, ldx, out.data_ptr(), ldy, ws_ptr, ws_n,
                                     stream)
    else:
        call, args = lib.hinm_spmm_rows, (ctypes.byref(st), x.data_ptr(), batch, ldx, out.data_ptr(), ldy,
                                          out_rows.data_ptr(), ws_ptr, ws_n, stream)
    if dev.index is None or dev.index == torch.cuda.current_device():
        _check(call(*args))
    else:
        with torch.cuda.device(dev):
            _check(call(*args))
    return out


class Group:
    """Several packed weights that multiply the same activations (hinm_spmm_group), e.g. the q, k and v
    projections of a layer.  Takes bf16 weights from pack.  Holds the C array of weight pointers; the weights must
    stay alive."""

    def __init__(self, packed):
        self.packed = list(packed)
        if not 1 <= len(self.packed) <= 8:
            raise ValueError("a group holds 1 to 8 packed weights")
        for p in self.packed:
            _one_weight(p, "a group")
        self.structs = [p.struct() for p in self.packed]
        self.ptrs = (ctypes.c_void_p * len(self.structs))(*[ctypes.addressof(st) for st in self.structs])
        self._need = {}

    def workspace_bytes(self, batch: int) -> int:
        key = (batch, _opt_gen)
        if key not in self._need:
            n = ctypes.c_size_t()
            _check(library().hinm_spmm_group_workspace_bytes(len(self.packed), self.ptrs, batch, ctypes.byref(n)))
            self._need[key] = n.value
        return self._need[key]


def spmm_group(group: Group, x: torch.Tensor, outs=None, workspace: Optional[torch.Tensor] = None):
    """[(W_g (.) M_g) X for g in the group]: x bf16 [cin, batch]; returns (or fills) one bf16 [cout_g, batch]
    output per weight.  Asynchronous on the current stream; workspace as in spmm."""
    ws0 = group.packed[0]
    p0 = ws0.plan
    dev = x.device
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[0] != p0.cin or dev != ws0.device or x.stride(1) != 1:
        raise ValueError(f"x must be bf16 [{p0.cin}, batch] with unit column stride on {ws0.device}")
    batch = x.shape[1]
    if outs is None:
        outs = [torch.empty((pk.plan.cout, batch), dtype=torch.bfloat16, device=dev) for pk in group.packed]
    for pk, o in zip(group.packed, outs):
        if o.dtype != torch.bfloat16 or o.shape != (pk.plan.cout, batch) or o.stride(1) != 1 or o.device != dev:
            raise ValueError(f"each output must be bf16 [cout, {batch}] with unit column stride on {dev}")
    if len(outs) != len(group.packed):
        raise ValueError("one output per weight")
    need = group.workspace_bytes(batch)
    stream = _stream_ptr(dev)
    if workspace is None:
        workspace = _workspace(dev, stream, need)
    ys = (ctypes.c_void_p * len(outs))(*[o.data_ptr() for o in outs])
    ldys = (ctypes.c_int64 * len(outs))(*[max(o.stride(0), batch) if batch else 0 for o in outs])
    ldx = max(x.stride(0), batch) if batch else 0
    with torch.cuda.device(dev):
        _check(library().hinm_spmm_group(len(outs), group.ptrs, x.data_ptr(), batch, ldx, ys, ldys,
                                         workspace.data_ptr() if workspace is not None else None,
                                         workspace.numel() if workspace is not None else 0, stream))
    return outs


def spmm_noalloc(packed: HinmPacked, x: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
    """Y = (W (.) M) X into ``out`` through hinm_spmm_noalloc: no workspace, no device allocation (the
    scratch is the library's own device array, shared by every call on the device, so calls on different
    streams of one device must not overlap).  x bf16 [cin, batch], out bf16 [cout, batch], both with unit
    column stride.  Asynchronous on the current stream."""
    _one_weight(packed, "spmm_noalloc")
    p = packed.plan
    dev = x.device
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[0] != p.cin or dev != packed.device or x.stride(1) != 1:
        raise ValueError(f"x must be bf16 [{p.cin}, batch] with unit column stride on {packed.device}")
    batch = x.shape[1]
    if out.dtype != torch.bfloat16 or out.shape != (p.cout, batch) or out.stride(1) != 1 or out.device != dev:
        raise ValueError(f"out must be bf16 [{p.cout}, {batch}] with unit column stride on {dev}")
    ldx = max(x.stride(0), batch) if batch else 0
    ldy = max(out.stride(0), batch) if batch else 0
    with torch.cuda.device(dev):
        _check(library().hinm_spmm_noalloc(ctypes.byref(packed.struct()), x.data_ptr(), batch, ldx, out.data_ptr(),
                                           ldy, _stream_ptr(dev)))
    return out


def translate_indices(packed: HinmPacked, mapping: torch.Tensor) -> HinmPacked:
    """Rewrites the packed index lists in place through ``mapping`` (int32 [cin] permutation on the device):
    index i becomes mapping[i], pads stay -1 (hinm_translate_indices).  Synchronous; returns ``packed``."""
    _one_weight(packed, "translate_indices")
    p = packed.plan
    dev = packed.idx_24.device
    if mapping.dtype != torch.int32 or mapping.shape != (p.cin,) or not mapping.is_contiguous() or mapping.device != dev:
        raise ValueError(f"mapping must be a contiguous int32 [{p.cin}] tensor on {dev}")
    ws = torch.empty(256, dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = packed.struct()
        _check(library().hinm_translate_indices(ctypes.byref(st), mapping.data_ptr(), ws.data_ptr(),
                                                ws.numel(), _stream_ptr(dev)))
    packed.flags = int(st.flags)
    return packed


def boundary_search(importance: torch.Tensor, perm: Optional[torch.Tensor], tile_rows: int, t_s: float,
                    step: float = 0.01, trace_cap: int = 256):
    """Device boundary search for v_s (hinm_boundary_search).  importance fp32 [cout, cin] and perm int32
    [n_tiles, cin] (or None) on the device.  Returns (v_s, [(v, R_total), ...] of the grid points visited)."""
    if importance.dtype != torch.float32 or importance.dim() != 2 or importance.stride(1) != 1:
        raise ValueError("importance must be float32 [cout, cin] with unit column stride")
    cout, cin = importance.shape
    dev = importance.device
    if perm is not None and (perm.dtype != torch.int32 or not perm.is_contiguous() or perm.device != dev):
        raise ValueError("perm must be a contiguous int32 tensor on the importance's device")
    lib = library()
    n = ctypes.c_size_t()
    _check(lib.hinm_boundary_workspace_bytes(cout, cin, tile_rows, ctypes.byref(n)))
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    v = ctypes.c_double()
    tv = (ctypes.c_double * trace_cap)()
    tr = (ctypes.c_double * trace_cap)()
    tl = ctypes.c_int32()
    with torch.cuda.device(dev):
        _check(lib.hinm_boundary_search(cout, cin, tile_rows, float(t_s), float(step), importance.data_ptr(),
                                        importance.stride(0), perm.data_ptr() if perm is not None else None,
                                        ws.data_ptr(), ws.numel(), ctypes.byref(v), tv, tr, trace_cap,
                                        ctypes.byref(tl), _stream_ptr(dev)))
    k = min(tl.value, trace_cap)
    return v.value, [(tv[i], tr[i]) for i in range(k)]


def gyro_permute(importance: torch.Tensor, perm: torch.Tensor, tile_rows: int, t_s: float, v_s: float,
                 rounds: int, cluster_size: int, kmeans_iters: int, sample, init):
    """In-tile input-channel gyro permutation (hinm_gyro_permute), synchronous.

    importance fp32 [cout, cin] and perm int32 [n_tiles, cin] on the device; sample uint8
    [rounds, n_tiles, groups] and init int32 [rounds, n_tiles, n_clusters] (numpy, host).
    Returns (new perm tensor, cost trace float64 numpy [rounds + 1, n_tiles]); perm is not modified.
    """
    if importance.dtype != torch.float32 or importance.dim() != 2 or importance.stride(1) != 1:
        raise ValueError("importance must be float32 [cout, cin] with unit column stride")
    cout, cin = importance.shape
    dev = importance.device
    p = plan(cout, cin, tile_rows, t_s, v_s)
    if perm.dtype != torch.int32 or perm.shape != (p.n_tiles, cin) or perm.device != dev:
        raise ValueError(f"perm must be int32 [{p.n_tiles}, {cin}] on the importance's device")
    out = perm.clone().contiguous()
    sample = np.ascontiguousarray(sample, dtype=np.uint8)
    init = np.ascontiguousarray(init, dtype=np.int32)
    lib = library()
    n = ctypes.c_size_t()
    _check(lib.hinm_gyro_workspace_bytes(ctypes.byref(p.raw), int(cluster_size), ctypes.byref(n)))
    ws = torch.empty(max(1, n.value), dtype=torch.uint8, device=dev)
    trace = np.zeros((rounds + 1, p.n_tiles), dtype=np.float64)
    with torch.cuda.device(dev):
        _check(lib.hinm_gyro_permute(ctypes.byref(p.raw), importance.data_ptr(), importance.stride(0),
                                     out.data_ptr(), int(rounds), int(cluster_size), int(kmeans_iters),
                                     sample.ctypes.data if sample.size else None,
                                     init.ctypes.data if init.size else None,
                                     trace.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), ws.data_ptr(),
                                     ws.numel(), _stream_ptr(dev)))
    return out, trace


def boundary_search_tiles(importance: torch.Tensor, perm: Optional[torch.Tensor], tile_rows: int, t_s: float,
                          step: float = 0.01):
    """Per-tile device boundary search (hinm_boundary_search_tiles).  Returns (v_s per tile, grid points per tile)."""
    if importance.dtype != torch.float32 or importance.dim() != 2 or importance.stride(1) != 1:
        raise ValueError("importance must be float32 [cout, cin] with unit column stride")
    cout, cin = importance.shape
    dev = importance.device
    if perm is not None and (perm.dtype != torch.int32 or not perm.is_contiguous() or perm.device != dev):
        raise ValueError("perm must be a contiguous int32 tensor on the importance's device")
    lib = library()
    n = ctypes.c_size_t()
    _check(lib.hinm_boundary_workspace_bytes(cout, cin, tile_rows, ctypes.byref(n)))
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    T = cout // tile_rows
    v = (ctypes.c_double * max(1, T))()
    pts = (ctypes.c_int32 * max(1, T))()
    with torch.cuda.device(dev):
        _check(lib.hinm_boundary_search_tiles(cout, cin, tile_rows, float(t_s), float(step), importance.data_ptr(),
                                              importance.stride(0), perm.data_ptr() if perm is not None else None,
                                              ws.data_ptr(), ws.numel(), v, pts, _stream_ptr(dev)))
    return [v[i] for i in range(T)], [pts[i] for i in range(T)]


# ---------------------------------------------------------------------------
# Mixture-of-experts layers and 4-bit microscaled values.
# ---------------------------------------------------------------------------

def _on_gpu(dev: torch.device) -> None:
    if dev.type != "cuda":
        raise ValueError(f"the weights and the routing must be on a GPU, not on {dev}")


def _matrix(t: torch.Tensor, rows: Optional[int], cols: Optional[int], dev: torch.device, what: str) -> int:
    """Checks a bf16 matrix and returns its row stride in elements."""
    if (t.dtype != torch.bfloat16 or t.dim() != 2 or t.device != dev or (rows is not None and t.shape[0] != rows)
            or (cols is not None and t.shape[1] != cols)):
        raise ValueError(f"{what} must be bf16 [{'channels' if rows is None else rows}, "
                         f"{'columns' if cols is None else cols}] on {dev}")
    n = t.shape[1]
    if n > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have unit column stride")
    ld = t.stride(0)
    if t.shape[0] > 1 and ld < n:
        raise ValueError(f"{what} must have a row stride of at least its {n} columns")
    return ld if ld > n else n


def _index(t: torch.Tensor, shape, dev: torch.device, what: str, dtype=torch.int32) -> None:
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {str(dtype).split('.')[1]} {list(shape)} tensor on {dev}")


def _call(dev: torch.device, fn, *args) -> None:
    """One C call with ``dev`` current."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        _check(fn(*args))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args))


def _split_workspace(dev: torch.device, stream: int, need: Tuple[int, int]) -> Optional[torch.Tensor]:
    """The default workspace of an expert or 4-bit product that needs (bytes, bytes without the copy of X).

    The stream's own, as for spmm.  A new one where the workspace holds a copy of X, so that no stream keeps the
    largest X it has seen, and while a graph is captured, out of the graph's memory, so that graphs captured on one
    stream and replayed on several never share one; its arrival counters are cleared on the stream (by a node of the
    graph) where the product may split."""
    total, split = need
    if total and (total > split or torch.cuda.is_current_stream_capturing()):
        ws = torch.empty(total, dtype=torch.uint8, device=dev)
        if split:
            ws[:65536].zero_()
        return ws
    return _workspace(dev, stream, total)


def _split_need(p: Plan, n_experts: int, n_cols: int, x_aligned: bool) -> Tuple[int, int]:
    total = spmm_experts_workspace_bytes(p, n_experts, n_cols, x_aligned)
    return total, total if x_aligned else spmm_experts_workspace_bytes(p, n_experts, n_cols)


@dataclasses.dataclass
class Routing:
    """Where every token goes (hinm_route): its experts, their weights, and the column order by expert."""

    ids: torch.Tensor       # int32 [tokens, top_k]: experts, best first; -1: none
    weights: torch.Tensor   # fp32 [tokens, top_k]
    slots: torch.Tensor     # int32 [tokens, top_k]: column of each (token, choice); -1: none
    starts: torch.Tensor    # int32 [experts + 1]: first column of every expert
    counts: torch.Tensor    # int32 [experts]
    src: torch.Tensor       # int32 [columns]: token of every column; -1: none

    @property
    def n_tokens(self) -> int:
        return self.slots.shape[0]

    @property
    def top_k(self) -> int:
        return self.slots.shape[1]

    @property
    def n_experts(self) -> int:
        return self.counts.shape[0]

    @property
    def n_cols(self) -> int:
        return self.src.shape[0]


def route_columns(n_tokens: int, n_experts: int, top_k: int, align: int = 8) -> int:
    """Columns any such routing fits into (hinm_route_columns, host only)."""
    n = ctypes.c_int64()
    _check(library().hinm_route_columns(n_tokens, n_experts, top_k, align, ctypes.byref(n)))
    return n.value


def route(logits: torch.Tensor, top_k: int, renormalize: bool = True, align: int = 8) -> Routing:
    """Router (hinm_route): logits bf16 or fp32 [experts, tokens] (unit column stride) -> Routing.

    Experts with NaN or -inf logits are not eligible; weights are softmax over the chosen experts
    (``renormalize``) or over all eligible ones.  Every expert's columns start at a multiple of ``align``.
    Asynchronous on the current stream; the column count depends on the sizes alone."""
    if logits.dtype not in (torch.bfloat16, torch.float32) or logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be a 2-D bf16 or fp32 CUDA tensor [experts, tokens]")
    e, n = logits.shape
    ld = logits.stride(0)
    if (n > 1 and logits.stride(1) != 1) or (e > 1 and ld < n):
        raise ValueError("logits must have unit column stride and rows that do not overlap")
    dev, lib = logits.device, library()
    cols, need = _route_sizes(n, e, top_k, align)
    nk = n * top_k
    ids, slots, starts, counts, src = torch.empty(2 * nk + 2 * e + 1 + cols, dtype=torch.int32, device=dev).split(
        (nk, nk, e + 1, e, cols))
    r = Routing(ids.view(n, top_k), torch.empty((n, top_k), dtype=torch.float32, device=dev), slots.view(n, top_k),
                starts, counts, src)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(dev, lib.hinm_route, logits.data_ptr(), HINM_BF16 if logits.dtype == torch.bfloat16 else HINM_FP32, n,
          max(ld, n), e, top_k, int(renormalize), align, ids.data_ptr(), r.weights.data_ptr(), slots.data_ptr(),
          starts.data_ptr(), counts.data_ptr(), src.data_ptr(), cols, ws.data_ptr() if need else None, need,
          _stream_ptr(dev))
    return r


@functools.lru_cache(maxsize=1024)
def _route_sizes(n_tokens: int, n_experts: int, top_k: int, align: int):
    need = ctypes.c_size_t()
    _check(library().hinm_route_workspace_bytes(n_tokens, n_experts, ctypes.byref(need)))
    return route_columns(n_tokens, n_experts, top_k, align), need.value


def dispatch(x: torch.Tensor, routing: Routing, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Token columns in the experts' order (hinm_dispatch): x bf16 [channels, tokens] -> bf16 [channels, columns],
    zeros in columns without a token.  Asynchronous on the current stream."""
    dev = routing.src.device
    ldx = _matrix(x, None, routing.n_tokens, dev, "x")
    _index(routing.src, (routing.n_cols,), dev, "routing.src")
    _on_gpu(dev)
    c, cols = x.shape[0], routing.n_cols
    if out is None:
        out = torch.empty((c, cols), dtype=torch.bfloat16, device=dev)
    ldo = _matrix(out, c, cols, dev, "out")
    _call(dev, library().hinm_dispatch, x.data_ptr(), c, routing.n_tokens, ldx, routing.src.data_ptr(), cols,
          out.data_ptr(), ldo, _stream_ptr(dev))
    return out


def combine(y: torch.Tensor, routing: Routing, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Weighted sum of every token's expert columns (hinm_combine): y bf16 [channels, columns] -> bf16
    [channels, tokens].  Asynchronous on the current stream."""
    dev = routing.slots.device
    ldy = _matrix(y, None, routing.n_cols, dev, "y")
    n, k, c = routing.n_tokens, routing.top_k, y.shape[0]
    _index(routing.slots, (n, k), dev, "routing.slots")
    _index(routing.weights, (n, k), dev, "routing.weights", torch.float32)
    _on_gpu(dev)
    if out is None:
        out = torch.empty((c, n), dtype=torch.bfloat16, device=dev)
    ldo = _matrix(out, c, n, dev, "out")
    _call(dev, library().hinm_combine, y.data_ptr(), c, routing.n_cols, ldy, routing.slots.data_ptr(),
          routing.weights.data_ptr(), n, k, out.data_ptr(), ldo, _stream_ptr(dev))
    return out


def _ptr(t: torch.Tensor) -> Optional[int]:
    return t.data_ptr() if t.numel() else None


@dataclasses.dataclass
class Experts:
    """Packed weights of one plan laid end to end, one per expert: HinmPacked's buffers with a leading expert
    axis (all contiguous; the tensors must not be replaced afterwards)."""

    plan: Plan
    val_dense: torch.Tensor
    idx_dense: torch.Tensor
    val_24: torch.Tensor
    meta_24: torch.Tensor
    idx_24: torch.Tensor

    @classmethod
    def stack(cls, packed) -> "Experts":
        """Copies packed weights (HinmPacked of equal plans on one device) into one stack."""
        packed = list(packed)
        if not packed or any(not isinstance(p, HinmPacked) for p in packed):
            raise ValueError("a stack takes one or more uniform packed weights (pack, not pack_tiles)")
        p0 = packed[0]
        for p in packed:
            if p.plan != p0.plan or p.device != p0.device:
                raise ValueError("stacked weights must have equal plans and be on one device")
        return cls(p0.plan, *[torch.stack([getattr(p, k) for p in packed]) for k in _BUFFERS])

    @property
    def n_experts(self) -> int:
        return self.idx_24.shape[0]

    @property
    def device(self) -> torch.device:
        return self.idx_24.device

    def nbytes(self) -> int:
        return self.n_experts * self.plan.packed_bytes

    def struct(self) -> PackedT:
        st = self.__dict__.get("_struct")
        if st is None:
            st = self.__dict__["_struct"] = PackedT(self.plan.raw, *[_ptr(getattr(self, k)) for k in _BUFFERS], 0, 0)
        return st

    def state_dict(self) -> dict:
        """As HinmPacked.state_dict, every buffer with its expert axis."""
        p = self.plan
        return {"format": "hinm-experts", "format_version": HINM_FORMAT_VERSION, "n_experts": self.n_experts,
                "cout": p.cout, "cin": p.cin, "tile_rows": p.tile_rows, "t_s": p.t_s, "v_s": p.v_s,
                **{k: getattr(self, k) for k in _BUFFERS}}

    @classmethod
    def from_state_dict(cls, sd: dict, device=None) -> "Experts":
        _check_format(sd, "hinm-experts")
        p = plan(int(sd["cout"]), int(sd["cin"]), int(sd["tile_rows"]), float(sd["t_s"]), float(sd["v_s"]))
        n = int(sd["n_experts"])
        if n < 1:
            raise ValueError("a stored stack needs at least one expert")
        return cls(p, **_checked_buffers(sd, {k: ((n, *s), t) for k, (s, t) in _packed_shapes(p).items()}, device))


def _packed_shapes(p: Plan) -> dict:
    T, R, D, S = p.n_tiles, p.tile_rows, p.n_dense_pad, p.n_24_pad
    return {"val_dense": ((T, D // 32, R, 32), torch.int16), "idx_dense": ((T, D), torch.int32),
            "val_24": ((T, S // 64, R, 32), torch.int16), "meta_24": ((T, S // 64, R), torch.int64),
            "idx_24": ((T, S), torch.int32)}


def _mx4_shapes(p: Plan) -> dict:
    T, G, D, S = p.n_tiles, p.tile_rows // 64, p.n_dense_pad, p.n_24_pad
    return {"val_dense": ((T, D // 32, G, 4, 16, 4), torch.int32), "scale_dense": ((T, D // 32, G, 16, 4), torch.uint8),
            "idx_dense": ((T, D), torch.int32), "val_24": ((T, S // 64, G, 4, 16, 4), torch.int32),
            "scale_24": ((T, S // 64, G, 16, 4), torch.uint8), "meta_24": ((T, S // 64, G, 4, 16, 4), torch.int16),
            "idx_24": ((T, S), torch.int32)}


_MX4_BUFFERS = ("val_dense", "scale_dense", "idx_dense", "val_24", "scale_24", "meta_24", "idx_24")


@dataclasses.dataclass
class HinmMx4:
    """A packed weight, or a stack of them, with 4-bit microscaled values (hinm_mx4_t; buffers of a stack have a
    leading expert axis).  Made by quantize_mx4; the tensors must not be replaced afterwards."""

    plan: Plan
    val_dense: torch.Tensor    # int32 bits of 8 codes
    scale_dense: torch.Tensor  # uint8
    idx_dense: torch.Tensor    # int32
    val_24: torch.Tensor
    scale_24: torch.Tensor
    meta_24: torch.Tensor      # int16 bits of uint16
    idx_24: torch.Tensor
    n_experts: Optional[int] = None   # None: one weight
    flags: int = 0                    # of the one weight it was made from, for dequantize

    @property
    def device(self) -> torch.device:
        return self.idx_24.device

    def nbytes(self) -> int:
        return sum(getattr(self, k).numel() * getattr(self, k).element_size() for k in _MX4_BUFFERS)

    def struct(self) -> Mx4T:
        st = self.__dict__.get("_struct")
        if st is None:
            st = self.__dict__["_struct"] = Mx4T(self.plan.raw, *[_ptr(getattr(self, k)) for k in _MX4_BUFFERS])
            self.__dict__["_ws_need"] = {}
        return st

    def dequantize(self):
        """The bf16 packed weight (or Experts stack) of the same values, exact (hinm_mx4_dequantize).  One weight
        keeps the flags of the weight it was made from: they describe the index lists, which are copied."""
        _on_gpu(self.device)
        lead = () if self.n_experts is None else (self.n_experts,)
        bufs = {k: _empty((*lead, *s), t, self.device) for k, (s, t) in _packed_shapes(self.plan).items()}
        out = (HinmPacked if self.n_experts is None else Experts)(self.plan, **bufs)
        _call(self.device, library().hinm_mx4_dequantize, ctypes.byref(self.struct()), self.n_experts or 1,
              ctypes.byref(out.struct()), _stream_ptr(self.device))
        if self.n_experts is None:
            out.flags = out.struct().flags = int(self.flags)
        return out

    def state_dict(self) -> dict:
        """As HinmPacked.state_dict; n_experts 0 marks a single weight."""
        p = self.plan
        return {"format": "hinm-mx4", "format_version": HINM_MX4_FORMAT_VERSION, "n_experts": self.n_experts or 0,
                "cout": p.cout, "cin": p.cin, "tile_rows": p.tile_rows, "t_s": p.t_s, "v_s": p.v_s,
                "flags": int(self.flags), **{k: getattr(self, k) for k in _MX4_BUFFERS}}

    @classmethod
    def from_state_dict(cls, sd: dict, device=None) -> "HinmMx4":
        _check_format(sd, "hinm-mx4", HINM_MX4_FORMAT_VERSION)
        p = plan(int(sd["cout"]), int(sd["cin"]), int(sd["tile_rows"]), float(sd["t_s"]), float(sd["v_s"]))
        n = int(sd["n_experts"])
        if n < 0 or p.tile_rows % 64:
            raise ValueError("a stored 4-bit weight needs tile_rows % 64 == 0 and n_experts >= 0")
        lead = (n,) if n else ()
        want = {k: ((*lead, *s), t) for k, (s, t) in _mx4_shapes(p).items()}
        return cls(p, **_checked_buffers(sd, want, device), n_experts=n or None, flags=int(sd.get("flags", 0)))


def quantize_mx4(packed) -> HinmMx4:
    """Rounds the values of a packed weight or an Experts stack to 4-bit microscaled values
    (hinm_mx4_quantize): blocks of 32 kept values of a row, E2M1 codes, one E8M0 scale.  Needs tile_rows a multiple
    of 64.  Asynchronous on the current stream."""
    if not isinstance(packed, (HinmPacked, Experts)):
        raise ValueError("quantize_mx4 takes a HinmPacked weight or an Experts stack")
    p, n = packed.plan, packed.n_experts if isinstance(packed, Experts) else None
    lead = () if n is None else (n,)
    dev = packed.device
    _on_gpu(dev)
    out = HinmMx4(p, **{k: _empty((*lead, *s), t, dev) for k, (s, t) in _mx4_shapes(p).items()}, n_experts=n,
                  flags=packed.flags if n is None else 0)
    _call(dev, library().hinm_mx4_quantize, ctypes.byref(packed.struct()), n or 1, ctypes.byref(out.struct()),
          _stream_ptr(dev))
    return out


def _spmm_mx4(packed: HinmMx4, x: torch.Tensor, out, workspace) -> torch.Tensor:
    if packed.n_experts is not None:
        raise ValueError("spmm takes one weight; multiply a stack with spmm_experts")
    p, dev = packed.plan, packed.idx_24.device
    ldx = _matrix(x, p.cin, None, dev, "x")
    _on_gpu(dev)
    batch = x.shape[1]
    if out is None:
        out = torch.empty((p.cout, batch), dtype=torch.bfloat16, device=dev)
    ldy = _matrix(out, p.cout, batch, dev, "out")
    st, lib = packed.struct(), library()
    needs = packed.__dict__["_ws_need"]
    key = (batch, ldx % 8 == 0 and x.data_ptr() % 16 == 0)
    need = needs.get(key)
    if need is None:
        need = needs[key] = _split_need(p, 1, *key)
    stream = _stream_ptr(dev)
    if workspace is None:
        workspace = _split_workspace(dev, stream, need)
    elif workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    _call(dev, lib.hinm_spmm_mx4, ctypes.byref(st), x.data_ptr(), batch, ldx, out.data_ptr(), ldy,
          workspace.data_ptr() if workspace is not None else None, workspace.numel() if workspace is not None else 0,
          stream)
    return out


def spmm_experts_workspace_bytes(p: Plan, n_experts: int, n_cols: int, x_aligned: bool = True) -> int:
    n = ctypes.c_size_t()
    _check(library().hinm_spmm_experts_workspace_bytes(ctypes.byref(p.raw), n_experts, n_cols, int(x_aligned),
                                                       ctypes.byref(n)))
    return n.value


def spmm_experts(experts, x: torch.Tensor, routing: Routing, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Every expert's product over its own columns (hinm_spmm_experts, or hinm_spmm_experts_mx4 for a quantised
    stack): x bf16 [cin, columns] in the routing's order, as many as it has -> bf16 [cout, columns].

    Columns that belong to no expert are left as they were in ``out`` (unspecified in a new one), which must not
    overlap x.  The ranges are
    read on the device: no host synchronisation.  Asynchronous on the current stream; workspace as in spmm, but
    while a graph is captured each call has its own."""
    mx4 = isinstance(experts, HinmMx4)
    if not (mx4 and experts.n_experts is not None) and not isinstance(experts, Experts):
        raise ValueError("spmm_experts takes an Experts stack or a quantised one")
    p, dev, e = experts.plan, experts.idx_24.device, experts.n_experts
    ldx = _matrix(x, p.cin, None, dev, "x")
    cols = x.shape[1]
    if routing.counts.shape[0] != e:
        raise ValueError(f"the routing has {routing.counts.shape[0]} experts, the stack {e}")
    if cols != routing.n_cols:
        raise ValueError(f"x has {cols} columns, the routing {routing.n_cols}")
    _index(routing.starts, (e + 1,), dev, "routing.starts")
    _index(routing.counts, (e,), dev, "routing.counts")
    _on_gpu(dev)
    if out is None:
        out = torch.empty((p.cout, cols), dtype=torch.bfloat16, device=dev)
    ldy = _matrix(out, p.cout, cols, dev, "out")
    needs = experts.__dict__.setdefault("_expert_need", {})
    key = (cols, ldx % 8 == 0 and x.data_ptr() % 16 == 0)
    need = needs.get(key)
    if need is None:
        need = needs[key] = _split_need(p, e, *key)
    stream = _stream_ptr(dev)
    if workspace is None:
        workspace = _split_workspace(dev, stream, need)
    elif workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    lib = library()
    _call(dev, lib.hinm_spmm_experts_mx4 if mx4 else lib.hinm_spmm_experts, ctypes.byref(experts.struct()), e,
          x.data_ptr(), cols, ldx, routing.starts.data_ptr(), routing.counts.data_ptr(), out.data_ptr(), ldy,
          workspace.data_ptr() if workspace is not None else None, workspace.numel() if workspace is not None else 0,
          stream)
    return out


__all__ = ["HinmError", "HinmPacked", "Plan", "plan", "pack", "spmm", "spmm_noalloc", "Group", "spmm_group", "set_option", "get_option", "options",
           "OPTIONS", "translate_indices", "boundary_search", "plan_tiles", "pack_tiles", "boundary_search_tiles",
           "HinmTPacked", "TilePlan", "spmm_tiles_workspace_bytes", "alloc_packed",
           "pack_workspace_bytes",
           "spmm_workspace_bytes", "Routing", "route", "route_columns", "dispatch", "combine", "Experts",
           "spmm_experts", "spmm_experts_workspace_bytes", "HinmMx4", "quantize_mx4",
           "library", "LIB_PATH", "EXPORTS"]
