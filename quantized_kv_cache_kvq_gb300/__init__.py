"""Python binding of libkvq (argument marshalling only).

Every step of the decode path runs in the CUDA library: this module allocates
device memory with torch, packs the C structs of ``include/kvq.h`` and calls
the C ABI with the current torch stream.  There is no CPU fallback: importing
works without a GPU (so the library can be inspected), but every compute call
needs the built ``libkvq.so`` and a CUDA device, and raises otherwise.

Entry points mirror the C names: ``append``, ``decode_attn``, ``meter``,
``decode_workspace_size``, ``debug_dither``, ``debug_encode``, those of the
runs (``map_runs``, ``append_runs``, ``attn_runs`` and
``attn_runs_workspace_size``) and of trees of drafted tokens (``tree_runs``,
``rope_runs``, ``attn_tree``, ``attn_tree_workspace_size``, ``verify_runs``,
``keep_runs``), plus the ``PagedCache`` helper that owns one layer's planes.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
from ctypes import POINTER, c_double, c_float, c_int32, c_int64, c_size_t, c_uint32, c_uint64, c_void_p

import torch

__all__ = [
    "FMT",
    "KvqError",
    "lib",
    "load",
    "PagedCache",
    "MeterParams",
    "append",
    "decode_attn",
    "decode_attn_noalloc",
    "decode_workspace_size",
    "append_rope",
    "meter",
    "debug_dither",
    "debug_encode",
    "tile_bytes",
    "status_string",
    "read_err",
    "map_runs",
    "append_runs",
    "attn_runs",
    "attn_runs_workspace_size",
    "tree_runs",
    "rope_runs",
    "attn_tree",
    "attn_tree_workspace_size",
    "verify_runs",
    "keep_runs",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("KVQ_LIB") or os.path.join(_HERE, "libkvq.so")

FMT = {"bf16": 0, "e4m3": 1, "e4m3s": 2, "int8": 3, "int8g32": 4, "e4m3p": 16, "int8p": 17}
PAGE_SCALED = ("e4m3p", "int8p")  # 8-bit codes with one power-of-two scale per (page, kv head)
SCALE_TILE_BYTES = {"e4m3s": 32, "int8": 32, "int8g32": 128}  # fp16 scales of a page's 16 tokens
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
TIER_A, TIER_B, TIER_V, TIER_S = 1, 2, 4, 8
METER_STATE_FLOATS = 8  # floats per (sequence, query head) cell of meter_state
HEAD_DIM, PAGE, N_BANDS = 128, 16, 16
MAX_TREE = 1024  # tokens of a run that is a tree
_SM_SCALE = 1.0 / math.sqrt(HEAD_DIM)
_INT32 = torch.int32

STATUS = {
    0: "KVQ_OK",
    1: "KVQ_ERR_INVALID_ARG",
    2: "KVQ_ERR_UNSUPPORTED_LAYOUT",
    3: "KVQ_ERR_WORKSPACE_TOO_SMALL",
    4: "KVQ_ERR_CUDA",
    5: "KVQ_ERR_DEVICE_BOUNDS",
    6: "KVQ_ERR_NONFINITE_INPUT",
    7: "KVQ_ERR_RANGE",
    8: "KVQ_ERR_TIMEOUT",
    9: "KVQ_ERR_NO_PAGES",
}


class KvqError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}")
        self.status = status


class _Cache(ctypes.Structure):
    _fields_ = [
        ("k_fmt", c_int32),
        ("v_fmt", c_int32),
        ("num_kv_heads", c_int32),
        ("num_pages", c_int32),
        ("layer", c_int32),
        ("reserved", c_int32),
        ("dither_seed", c_uint64),
        ("k_data", c_void_p),
        ("v_data", c_void_p),
        ("k_scale", c_void_p),
        ("v_scale", c_void_p),
        ("witness", c_void_p),
        ("v_witness", c_void_p),
        ("outlier_pairs", c_void_p),
        ("n_outlier_pairs", c_int32),
        ("reserved2", c_int32),
        ("k_outlier", c_void_p),
    ]


class DecodeExtras(ctypes.Structure):
    _fields_ = [("page_log_contrib", c_void_p), ("contrib_stride", c_int32), ("reserved", c_int32)]


class MeterParams(ctypes.Structure):
    _fields_ = [
        ("tiers", c_uint32),
        ("n_layers", c_int32),
        ("n_q_heads", c_int32),
        ("n_steps", c_int32),
        ("delta_req", c_double),
        ("tau", c_float),
        ("reserved", c_int32),
    ]


_lib = None


def load(path: str = LIB_PATH):
    """Load libkvq.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libkvq.so not built ({path}); run __graft_entry__.build()")
    L = ctypes.CDLL(path)
    L.kvq_tile_bytes.restype = c_size_t
    L.kvq_tile_bytes.argtypes = [c_int32, c_int32]
    L.kvq_append.restype = c_int32
    L.kvq_append.argtypes = [POINTER(_Cache), c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p]
    L.kvq_append_rope.restype = c_int32
    L.kvq_append_rope.argtypes = [POINTER(_Cache), c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_void_p,
                                  c_int32, c_void_p, c_void_p]
    L.kvq_decode_workspace_size.restype = c_size_t
    L.kvq_decode_workspace_size.argtypes = [c_int32, c_int32, c_int32]
    L.kvq_decode_attn.restype = c_int32
    L.kvq_decode_attn.argtypes = [
        POINTER(_Cache), POINTER(_Cache), c_int32, c_void_p, c_int32, c_int32, c_int32, c_void_p, c_int32,
        c_void_p, c_float, POINTER(MeterParams), c_void_p, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p,
    ]
    L.kvq_decode_attn_append.restype = c_int32
    L.kvq_decode_attn_append.argtypes = [
        POINTER(_Cache), c_void_p, c_void_p, c_int32, POINTER(_Cache), c_int32, c_void_p, c_int32, c_int32, c_int32,
        c_void_p, c_int32, c_void_p, c_float, POINTER(MeterParams), c_void_p, c_void_p, c_void_p, c_size_t, c_void_p,
        c_void_p,
    ]
    L.kvq_decode_attn_ex.restype = c_int32
    L.kvq_decode_attn_ex.argtypes = [
        POINTER(_Cache), c_void_p, c_void_p, c_int32, POINTER(_Cache), c_int32, c_void_p, c_int32, c_int32, c_int32,
        c_void_p, c_int32, c_void_p, c_float, POINTER(MeterParams), POINTER(DecodeExtras), c_void_p, c_void_p,
        c_void_p, c_size_t, c_void_p, c_void_p,
    ]
    L.kvq_gate.restype = c_int32
    L.kvq_gate.argtypes = [c_void_p, c_int32, c_void_p, c_int32, c_int32, c_void_p, c_int32, c_float, c_void_p,
                           c_void_p, c_int32, c_void_p]
    L.kvq_zero_witness.restype = c_int32
    L.kvq_zero_witness.argtypes = [POINTER(_Cache), c_void_p, c_int32, c_void_p, c_void_p]
    L.kvq_decode_attn_noalloc.restype = c_int32
    L.kvq_decode_attn_noalloc.argtypes = [
        POINTER(_Cache), POINTER(_Cache), c_int32, c_void_p, c_int32, c_int32, c_int32, c_void_p, c_int32,
        c_void_p, c_float, POINTER(MeterParams), c_void_p, c_void_p, c_void_p, c_void_p,
    ]
    L.kvq_meter.restype = c_int32
    L.kvq_meter.argtypes = [c_void_p, c_int32, c_int32, c_int32, POINTER(MeterParams), c_void_p, c_void_p,
                            c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    L.kvq_map_runs.restype = c_int32
    L.kvq_map_runs.argtypes = [c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_void_p,
                               c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p]
    L.kvq_map_runs_ex.restype = c_int32
    L.kvq_map_runs_ex.argtypes = L.kvq_map_runs.argtypes[:14] + [c_void_p, c_void_p, c_void_p, c_void_p]
    L.kvq_append_runs.restype = c_int32
    L.kvq_append_runs.argtypes = [POINTER(_Cache), c_void_p, c_int64, c_void_p, c_int64, c_int32, c_void_p, c_int32,
                                  c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p]
    L.kvq_attn_runs_workspace_size.restype = c_size_t
    L.kvq_attn_runs_workspace_size.argtypes = [c_int32] * 6
    L.kvq_attn_runs.restype = c_int32
    L.kvq_attn_runs.argtypes = [POINTER(_Cache), c_void_p, c_int64, c_int32, c_int32, c_void_p, c_int32, c_int32, c_int32,
                                c_void_p, c_int32, c_void_p, c_float, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p,
                                c_void_p]
    L.kvq_tree_runs.restype = c_int32
    L.kvq_tree_runs.argtypes = [c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_void_p]
    L.kvq_rope_runs.restype = c_int32
    L.kvq_rope_runs.argtypes = [c_void_p, c_int64, c_int32, c_void_p, c_int64, c_int32, c_int32, c_void_p, c_void_p, c_float,
                                c_void_p, c_void_p, c_int32, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int32, c_int32,
                                c_void_p, c_void_p]
    L.kvq_attn_tree_workspace_size.restype = c_size_t
    L.kvq_attn_tree_workspace_size.argtypes = [c_int32] * 6
    L.kvq_attn_tree.restype = c_int32
    L.kvq_attn_tree.argtypes = [POINTER(_Cache), c_void_p, c_int64, c_int32, c_int32, c_void_p, c_int32, c_int32, c_int32,
                                c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_float, c_void_p, c_void_p, c_void_p, c_size_t,
                                c_void_p, c_void_p]
    L.kvq_verify_runs.restype = c_int32
    L.kvq_verify_runs.argtypes = [c_void_p, c_int64, c_void_p, c_int64, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    L.kvq_keep_runs.restype = c_int32
    L.kvq_keep_runs.argtypes = [c_void_p, c_int32, c_void_p, c_int32, c_int32, c_void_p, c_int32, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_void_p]
    L.kvq_sizeof.restype = c_size_t
    L.kvq_sizeof.argtypes = [c_int32]
    L.kvq_debug_dither.restype = c_int32
    L.kvq_debug_dither.argtypes = [c_uint64, c_int32, c_int32, c_void_p, c_int32, c_void_p, c_void_p]
    L.kvq_debug_encode.restype = c_int32
    L.kvq_debug_encode.argtypes = [c_int32, c_void_p, c_int64, c_void_p, c_void_p]
    L.kvq_debug_time_decode.restype = c_int32
    L.kvq_debug_time_decode.argtypes = [c_void_p, c_void_p]
    L.kvq_debug_wait_timeout.restype = c_int32
    L.kvq_debug_wait_timeout.argtypes = [c_uint64, c_void_p, c_void_p]
    L.kvq_status_string.restype = ctypes.c_char_p
    L.kvq_status_string.argtypes = [c_int32]
    L.kvq_version.restype = c_int32
    L.kvq_version.argtypes = []
    _lib = L
    return L


def lib():
    return load()


def _check(status: int, where: str):
    if status != 0:
        raise KvqError(status, where)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def tile_bytes(fmt: str, plane: int) -> int:
    return int(lib().kvq_tile_bytes(FMT[fmt], plane))


def status_string(status: int) -> str:
    return lib().kvq_status_string(status).decode()


def _plane(name: str):
    """A plane of PagedCache.  Those of a page-scaled cache may be exchanged (the kernels take their sizes from the cache's heads and
    pages, so each is looked at when it is put in)."""
    slot = "_" + name

    def put(self, t):
        if self.k_fmt in PAGE_SCALED:
            n = self.num_pages * self.num_kv_heads
            dtype, n = (torch.float16, n) if name.endswith("scale") else (torch.uint8, 2048 * n)
            assert t.dtype is dtype and t.numel() == n and t.is_contiguous(), f"{name}: {n} elements of {dtype}, contiguous"
        setattr(self, slot, t)

    return property(operator.attrgetter(slot), put)


class PagedCache:
    """One layer's paged planes (device memory owned by torch tensors).

    The page-scaled formats ("e4m3p", "int8p") have fp16 scale planes [num_kv_heads, num_pages] and no witness."""

    k, v, k_scale, v_scale = _plane("k"), _plane("v"), _plane("k_scale"), _plane("v_scale")

    def __init__(self, k_fmt: str, v_fmt: str, num_kv_heads: int, num_pages: int, layer: int = 0,
                 seed: int = 0, device="cuda", witness: bool = True, value_witness: bool = False,
                 outlier_pairs: torch.Tensor | None = None):
        self.k_fmt, self.v_fmt = k_fmt, v_fmt
        self.num_kv_heads, self.num_pages, self.layer, self.seed = num_kv_heads, num_pages, layer, seed
        n = num_pages * num_kv_heads
        kb = 4096 if k_fmt == "bf16" else 2048
        vb = 4096 if v_fmt == "bf16" else 2048
        z = dict(dtype=torch.uint8, device=device)
        if k_fmt in PAGE_SCALED or v_fmt in PAGE_SCALED:
            assert k_fmt == v_fmt and not value_witness and outlier_pairs is None
            sc = dict(dtype=torch.float16, device=device)
            self._page_scaled(torch.zeros((n, kb), **z), torch.zeros((n, vb), **z),
                              torch.zeros((num_kv_heads, num_pages), **sc), torch.zeros((num_kv_heads, num_pages), **sc))
            return
        self.k = torch.zeros((n, kb), **z)
        self.v = torch.zeros((n, vb), **z)
        self.k_scale = torch.zeros((n, SCALE_TILE_BYTES[k_fmt]), **z) if k_fmt in SCALE_TILE_BYTES else None
        self.v_scale = torch.zeros((n, SCALE_TILE_BYTES[v_fmt]), **z) if v_fmt in SCALE_TILE_BYTES else None
        self.witness = torch.zeros((n, 512), **z) if witness else None
        self.v_witness = torch.zeros((n, 64), **z) if value_witness else None
        # fixed-channel key outlier bypass: [num_kv_heads, m] int32 RoPE pairs (INT8-dithered keys)
        self.n_out = 0 if outlier_pairs is None else int(outlier_pairs.shape[1])
        self.outlier_pairs = None
        self.k_outlier = None
        if self.n_out:
            assert outlier_pairs.shape[0] == num_kv_heads and outlier_pairs.dtype == torch.int32
            self.outlier_pairs = outlier_pairs.to(device).contiguous()
            self.k_outlier = torch.zeros((n, 256 if self.n_out <= 4 else 512), **z)

    def _page_scaled(self, k, v, k_scale, v_scale):
        _on(k.get_device(), v, k_scale, v_scale)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.witness = self.v_witness = self.outlier_pairs = self.k_outlier = None
        self.n_out = 0

    @classmethod
    def over(cls, k_fmt: str, v_fmt: str, num_kv_heads: int, num_pages: int, *, k: torch.Tensor, v: torch.Tensor,
             k_scale: torch.Tensor, v_scale: torch.Tensor, layer: int = 0) -> "PagedCache":
        """A page-scaled cache over planes that the caller has: k, v uint8 [num_pages * num_kv_heads, 2048], k_scale,
        v_scale fp16 [num_kv_heads, num_pages]."""
        assert k_fmt in PAGE_SCALED and v_fmt == k_fmt
        n = num_pages * num_kv_heads
        for t in (k, v):
            assert t.dtype == torch.uint8 and t.shape == (n, 2048) and t.is_contiguous()
        for t in (k_scale, v_scale):
            assert t.dtype == torch.float16 and t.shape == (num_kv_heads, num_pages) and t.is_contiguous()
        c = cls.__new__(cls)
        c.k_fmt, c.v_fmt = k_fmt, v_fmt
        c.num_kv_heads, c.num_pages, c.layer, c.seed = num_kv_heads, num_pages, layer, 0
        c._page_scaled(k, v, k_scale, v_scale)
        return c

    def _check_device(self, device: int):
        _on(device, self._k, self._v, self._k_scale, self._v_scale)

    def desc(self) -> _Cache:
        if self.k_fmt in PAGE_SCALED:
            f = FMT[self.k_fmt]
            return _Cache(f, f, self.num_kv_heads, self.num_pages, self.layer, 0, 0, self._k.data_ptr(), self._v.data_ptr(),
                          self._k_scale.data_ptr(), self._v_scale.data_ptr())
        return _Cache(FMT[self.k_fmt], FMT[self.v_fmt], self.num_kv_heads, self.num_pages, self.layer, 0,
                      self.seed & 0xFFFFFFFFFFFFFFFF, _ptr(self.k), _ptr(self.v), _ptr(self.k_scale),
                      _ptr(self.v_scale), _ptr(self.witness), _ptr(self.v_witness), _ptr(self.outlier_pairs),
                      self.n_out, 0, _ptr(self.k_outlier))

    def _packed(self, device: int) -> bytes:
        """desc() as bytes, checked to be on ``device``.  The cache holds them, as a caller of the C function holds its descriptors; every call
        compares them with the planes as they are now, and makes them anew where a plane, a size or the device is another one (a step's
        keep_runs takes those of all layers: of host work, 36 made anew are 65 us and 36 held ones 16)."""
        if self.k_fmt not in PAGE_SCALED:
            return bytes(self.desc())  # the library's to refuse
        at = (self._k.data_ptr(), self._v.data_ptr(), self._k_scale.data_ptr(), self._v_scale.data_ptr(), device, self.layer, self.num_kv_heads,
              self.num_pages, self.k_fmt)
        if self.__dict__.get("_packed_at") != at:
            self._check_device(device)
            self._packed_desc, self._packed_at = bytes(self.desc()), at
        return self._packed_desc

    def nbytes(self) -> int:
        return sum(t.nbytes for t in (self.k, self.v, self.k_scale, self.v_scale, self.witness, self.v_witness,
                                      self.k_outlier) if t is not None)


def read_err(err: torch.Tensor) -> int:
    return int(err.item())


def append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
           err: torch.Tensor | None = None, stream=None):
    """kvq_append: quantize k, v [n, Hkv, 128] (fp32 or bf16) into the slots of ``cache``."""
    assert k.is_contiguous() and v.is_contiguous() and k.dtype == v.dtype and k.shape == v.shape
    assert slot_mapping.dtype == torch.int32 and slot_mapping.is_contiguous()
    d = cache.desc()
    _check(lib().kvq_append(ctypes.byref(d), k.data_ptr(), v.data_ptr(), DTYPE[k.dtype], slot_mapping.data_ptr(),
                            int(k.shape[0]), _ptr(err), _stream(stream)), "kvq_append")


def append_rope(cache: PagedCache, k_pre: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                cos_sin: torch.Tensor, slot_mapping: torch.Tensor, err: torch.Tensor | None = None, stream=None):
    """kvq_append_rope: rotate the pre-RoPE keys k_pre [n, Hkv, 128] at ``positions`` [n] with the fp32 table
    ``cos_sin`` [max_position, 128] (cos of the 64 pair angles, then their sin), then quantize as kvq_append."""
    assert k_pre.is_contiguous() and v.is_contiguous() and k_pre.dtype == v.dtype and k_pre.shape == v.shape
    assert slot_mapping.dtype == torch.int32 and slot_mapping.is_contiguous()
    assert positions.dtype == torch.int32 and positions.is_contiguous() and positions.numel() == k_pre.shape[0]
    assert cos_sin.dtype == torch.float32 and cos_sin.is_contiguous() and cos_sin.dim() == 2 and cos_sin.shape[1] == HEAD_DIM
    d = cache.desc()
    _check(lib().kvq_append_rope(ctypes.byref(d), k_pre.data_ptr(), v.data_ptr(), DTYPE[k_pre.dtype],
                                 positions.data_ptr(), cos_sin.data_ptr(), int(cos_sin.shape[0]),
                                 slot_mapping.data_ptr(), int(k_pre.shape[0]), _ptr(err), _stream(stream)),
           "kvq_append_rope")


def decode_workspace_size(batch: int, num_kv_heads: int, num_q_heads: int) -> int:
    return int(lib().kvq_decode_workspace_size(batch, num_kv_heads, num_q_heads))


def meter_params(tiers: int = TIER_A, n_layers: int = 1, n_q_heads: int = 1, n_steps: int = 256,
                 delta_req: float = 1e-2, tau: float = 0.2) -> MeterParams:
    return MeterParams(tiers, n_layers, n_q_heads, n_steps, delta_req, tau, 0)


def decode_attn(cache: PagedCache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                out: torch.Tensor, workspace: torch.Tensor, *, prefix: PagedCache | None = None,
                prefix_len: int = 0, sm_scale: float | None = None, meter: MeterParams | None = None,
                meter_state: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None):
    """kvq_decode_attn for one layer: q [B, Hq, 128] -> out [B, Hq, 128] (+ meter_state [B, Hq, 8])."""
    B, Hq, D = q.shape
    assert D == HEAD_DIM and q.is_contiguous() and out.is_contiguous()
    assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    d = cache.desc()
    pd = prefix.desc() if prefix is not None else None
    _check(lib().kvq_decode_attn(
        ctypes.byref(d), ctypes.byref(pd) if pd is not None else None, int(prefix_len), q.data_ptr(), DTYPE[q.dtype],
        B, Hq, block_table.data_ptr(), int(block_table.shape[1]) if block_table.dim() == 2 else 0,
        seq_lens.data_ptr(), float(sm_scale), ctypes.byref(meter) if meter is not None else None,
        out.data_ptr(), _ptr(meter_state), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _ptr(err), _stream(stream)), "kvq_decode_attn")


def decode_attn_append(cache: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                       block_table: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, *,
                       prefix: PagedCache | None = None, prefix_len: int = 0, sm_scale: float | None = None,
                       meter: MeterParams | None = None, meter_state: torch.Tensor | None = None,
                       err: torch.Tensor | None = None, stream=None):
    """kvq_decode_attn_append: append each sequence's newest token (k_new, v_new [B, Hkv, 128]) and decode."""
    B, Hq, D = q.shape
    assert D == HEAD_DIM and q.is_contiguous() and out.is_contiguous()
    assert k_new.is_contiguous() and v_new.is_contiguous() and k_new.dtype == v_new.dtype and k_new.shape == v_new.shape
    assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    d = cache.desc()
    pd = prefix.desc() if prefix is not None else None
    _check(lib().kvq_decode_attn_append(
        ctypes.byref(d), k_new.data_ptr(), v_new.data_ptr(), DTYPE[k_new.dtype],
        ctypes.byref(pd) if pd is not None else None, int(prefix_len), q.data_ptr(), DTYPE[q.dtype],
        B, Hq, block_table.data_ptr(), int(block_table.shape[1]) if block_table.dim() == 2 else 0,
        seq_lens.data_ptr(), float(sm_scale), ctypes.byref(meter) if meter is not None else None,
        out.data_ptr(), _ptr(meter_state), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _ptr(err), _stream(stream)), "kvq_decode_attn_append")


def decode_attn_ex(cache: PagedCache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                   out: torch.Tensor, workspace: torch.Tensor, *, k_new: torch.Tensor | None = None,
                   v_new: torch.Tensor | None = None, prefix: PagedCache | None = None, prefix_len: int = 0,
                   sm_scale: float | None = None, meter: MeterParams | None = None,
                   meter_state: torch.Tensor | None = None, page_log_contrib: torch.Tensor | None = None,
                   err: torch.Tensor | None = None, stream=None):
    """kvq_decode_attn_ex: decode (with the optional newest-token append) and the optional per-page
    log contributions page_log_contrib [B, Hq, stride] (fp32) for kvq_gate."""
    B, Hq, D = q.shape
    assert D == HEAD_DIM and q.is_contiguous() and out.is_contiguous()
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    d = cache.desc()
    pd = prefix.desc() if prefix is not None else None
    ex = None
    if page_log_contrib is not None:
        assert page_log_contrib.dtype == torch.float32 and page_log_contrib.is_contiguous()
        ex = DecodeExtras(page_log_contrib.data_ptr(), int(page_log_contrib.shape[-1]), 0)
    _check(lib().kvq_decode_attn_ex(
        ctypes.byref(d), _ptr(k_new), _ptr(v_new), DTYPE[k_new.dtype] if k_new is not None else 0,
        ctypes.byref(pd) if pd is not None else None, int(prefix_len), q.data_ptr(), DTYPE[q.dtype], B, Hq,
        block_table.data_ptr(), int(block_table.shape[1]) if block_table.dim() == 2 else 0, seq_lens.data_ptr(),
        float(sm_scale), ctypes.byref(meter) if meter is not None else None, ctypes.byref(ex) if ex is not None else None,
        out.data_ptr(), _ptr(meter_state), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _ptr(err), _stream(stream)), "kvq_decode_attn_ex")


def gate(page_log_contrib: torch.Tensor, meter_state: torch.Tensor, seq_lens: torch.Tensor, prefix_len: int,
         tau: float, n_page_in: torch.Tensor, page_list: torch.Tensor | None = None, stream=None):
    """kvq_gate: greedy page-in plan per (sequence, query head)."""
    B, Hq, stride = page_log_contrib.shape
    _check(lib().kvq_gate(page_log_contrib.data_ptr(), stride, meter_state.data_ptr(), B, Hq, seq_lens.data_ptr(),
                          int(prefix_len), float(tau), n_page_in.data_ptr(), _ptr(page_list),
                          int(page_list.shape[-1]) if page_list is not None else 0, _stream(stream)), "kvq_gate")


def zero_witness(cache: PagedCache, slots: torch.Tensor, err: torch.Tensor | None = None, stream=None):
    """kvq_zero_witness: zero the witness (and value witness) of repaired slots."""
    d = cache.desc()
    _check(lib().kvq_zero_witness(ctypes.byref(d), slots.data_ptr(), int(slots.numel()), _ptr(err), _stream(stream)),
           "kvq_zero_witness")


def decode_attn_noalloc(cache: PagedCache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                        out: torch.Tensor, *, prefix: PagedCache | None = None, prefix_len: int = 0,
                        sm_scale: float | None = None, meter: MeterParams | None = None,
                        meter_state: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None):
    """kvq_decode_attn_noalloc: decode_attn with the library's own static scratch (no workspace argument).

    For callers that cannot allocate device scratch; calls share the library's scratch array, so
    calls must not overlap on the GPU."""
    B, Hq, D = q.shape
    assert D == HEAD_DIM and q.is_contiguous() and out.is_contiguous()
    assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    d = cache.desc()
    pd = prefix.desc() if prefix is not None else None
    _check(lib().kvq_decode_attn_noalloc(
        ctypes.byref(d), ctypes.byref(pd) if pd is not None else None, int(prefix_len), q.data_ptr(), DTYPE[q.dtype],
        B, Hq, block_table.data_ptr(), int(block_table.shape[1]) if block_table.dim() == 2 else 0,
        seq_lens.data_ptr(), float(sm_scale), ctypes.byref(meter) if meter is not None else None,
        out.data_ptr(), _ptr(meter_state), _ptr(err), _stream(stream)), "kvq_decode_attn_noalloc")


def meter(meter_state: torch.Tensor, n_layers: int, batch: int, num_q_heads: int, params: MeterParams,
          meter_a: torch.Tensor, raw_a: torch.Tensor, counts: torch.Tensor, cert_b: torch.Tensor | None = None,
          ranking: torch.Tensor | None = None, out_bound: torch.Tensor | None = None,
          two_sided: torch.Tensor | None = None, det_tanh: torch.Tensor | None = None, stream=None):
    """kvq_meter over meter_state [L, B, Hq, 8]."""
    _check(lib().kvq_meter(meter_state.data_ptr(), n_layers, batch, num_q_heads, ctypes.byref(params),
                           meter_a.data_ptr(), raw_a.data_ptr(), _ptr(cert_b), _ptr(out_bound), _ptr(two_sided),
                           _ptr(det_tanh), counts.data_ptr(), _ptr(ranking), _stream(stream)), "kvq_meter")


def _rows(x: torch.Tensor, rows: int, heads: int) -> int:
    """Row stride of a [rows, heads, 128] tensor whose rows are dense: a slice of a fused projection is taken as it is."""
    if x.is_contiguous():
        return heads * HEAD_DIM
    s0, s1, s2 = x.stride()
    assert s2 == 1 and (heads == 1 or s1 == HEAD_DIM)
    return s0 if rows > 1 else heads * HEAD_DIM


def _on(device: int, *tensors):
    for t in tensors:
        assert t is None or t.get_device() == device, "one CUDA device"


def _i32(device: int, *tensors):
    for t in tensors:
        assert t is None or (t.dtype is _INT32 and t.get_device() == device and t.is_contiguous()), \
            "int32, contiguous and on one CUDA device"


def _launch(name: str, fn, device: int, stream, *args):
    """The call fn(*args, stream) with ``device`` current, on ``stream`` or that device's current stream."""
    assert device >= 0, "CUDA tensors"
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _launch(name, fn, device, stream, *args)
    status = fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream)
    if status:
        raise KvqError(status, name)


def map_runs(new_lens: torch.Tensor, seq_lens: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor,
             block_table: torch.Tensor, run_starts: torch.Tensor, seq_lens_out: torch.Tensor, free_count_out: torch.Tensor,
             *, slot_mapping: torch.Tensor | None = None, positions: torch.Tensor | None = None,
             kept_pages: torch.Tensor | None = None, held_pages: torch.Tensor | None = None, max_rows: int | None = None,
             err: torch.Tensor | None = None, stream=None):
    """kvq_map_runs_ex: pages, slots and positions of a step from new_lens [B] (negative: finished) and seq_lens [B].

    free_pages [capacity] is the stack of free pages with free_count [1] in use, block_table [B, max_pages]; run_starts
    [B + 1], seq_lens_out [B] and free_count_out [1] are written (the latter two may be the inputs), and slot_mapping and
    positions [max_rows] where given.  A step of more than max_rows tokens is not taken: give the rows of the step's tensors
    where there is no slot_mapping to tell them, or the lengths of a larger step move on and its tokens are missed.  kept_pages [B]: the first pages of a finished request that do not go back, others hold
    them too; held_pages [B], in and out: the pages that a request has, those behind a length that was set back among them.
    All int32 and contiguous."""
    device = run_starts.get_device()
    _i32(device, new_lens, seq_lens, free_pages, free_count, block_table, run_starts, seq_lens_out, free_count_out,
         slot_mapping, positions, kept_pages, held_pages, err)
    B, width = block_table.shape
    assert new_lens.numel() == B and seq_lens.numel() == B and seq_lens_out.numel() == B and run_starts.numel() == B + 1
    assert free_count.numel() == 1 and free_count_out.numel() == 1 and (kept_pages is None or kept_pages.numel() == B)
    assert held_pages is None or held_pages.numel() == B
    rows = 0x7FFFFFFF if max_rows is None else max_rows
    for t in (slot_mapping, positions):
        if t is not None:
            assert max_rows is None or t.numel() == max_rows
            max_rows = rows = t.numel()
    _launch("kvq_map_runs_ex", lib().kvq_map_runs_ex, device, stream, new_lens.data_ptr(), seq_lens.data_ptr(), B,
            free_pages.data_ptr(), free_pages.numel(), free_count.data_ptr(), block_table.data_ptr(), width,
            run_starts.data_ptr(), seq_lens_out.data_ptr(), free_count_out.data_ptr(), _ptr(slot_mapping), _ptr(positions),
            rows, _ptr(kept_pages), _ptr(held_pages), _ptr(err))


def append_runs(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor,
                *, run_starts: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None):
    """kvq_append_runs: quantize the runs' keys and values k, v [rows, Hkv, 128] (fp32 or bf16; rows may be strided) into
    a page-scaled cache.  run_starts [B + 1]; None: one new token for each request."""
    rows, heads, d = k.shape
    assert k.dtype == v.dtype and k.shape == v.shape and heads == cache.num_kv_heads and d == HEAD_DIM
    device = k.get_device()
    _on(device, v)
    cache._check_device(device)
    _i32(device, seq_lens, block_table, run_starts, err)
    B, width = block_table.shape
    assert seq_lens.numel() == B and (run_starts is None or run_starts.numel() == B + 1)
    _launch("kvq_append_runs", lib().kvq_append_runs, device, stream, ctypes.byref(cache.desc()), k.data_ptr(), _rows(k, rows, heads),
            v.data_ptr(), _rows(v, rows, heads), DTYPE[k.dtype], _ptr(run_starts), B, rows, block_table.data_ptr(), width,
            seq_lens.data_ptr(), _ptr(err))


def attn_runs_workspace_size(batch: int, num_rows: int, max_run: int, num_kv_heads: int, num_q_heads: int,
                             q_dtype: torch.dtype) -> int:
    return int(lib().kvq_attn_runs_workspace_size(batch, num_rows, max_run, num_kv_heads, num_q_heads, DTYPE[q_dtype]))


def attn_runs(cache: PagedCache, q: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor, out: torch.Tensor,
              workspace: torch.Tensor, *, run_starts: torch.Tensor | None = None, max_run: int | None = None,
              lse: torch.Tensor | None = None, sm_scale: float | None = None, err: torch.Tensor | None = None, stream=None):
    """kvq_attn_runs: causal attention of the runs' queries q [rows, Hq, 128] (fp32 or bf16; rows may be strided) over a
    page-scaled cache -> out [rows, Hq, 128] in q's type (+ lse [rows, Hq] fp32).  No run is longer than max_run
    (None: one token without run_starts, else as many as there are rows; the workspace goes by the same number); run_starts
    None: one query token for each request."""
    rows, Hq, d = q.shape
    assert d == HEAD_DIM and out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous()
    device = q.get_device()
    assert workspace.is_contiguous(), "workspace: one piece of memory"
    _on(device, out, workspace, lse)
    cache._check_device(device)
    _i32(device, seq_lens, block_table, run_starts, err)
    B, width = block_table.shape
    assert seq_lens.numel() == B and (run_starts is None or run_starts.numel() == B + 1)
    if max_run is None:
        max_run = 1 if run_starts is None else rows
    assert lse is None or (lse.dtype is torch.float32 and lse.is_contiguous() and lse.numel() == rows * Hq)
    _launch("kvq_attn_runs", lib().kvq_attn_runs, device, stream, ctypes.byref(cache.desc()), q.data_ptr(), _rows(q, rows, Hq),
            DTYPE[q.dtype], Hq, _ptr(run_starts), B, rows, max_run, block_table.data_ptr(), width, seq_lens.data_ptr(),
            _SM_SCALE if sm_scale is None else sm_scale, out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.nbytes,
            _ptr(err))


def _tree(batch: int, rows: int, run_starts, *per_row):
    assert run_starts is None and rows == batch or run_starts is not None and run_starts.numel() == batch + 1
    for t in per_row:
        assert t is None or t.numel() == rows, "one for each row"


def tree_runs(parents: torch.Tensor, seq_lens: torch.Tensor, mask: torch.Tensor, *, positions: torch.Tensor | None = None,
              run_starts: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None):
    """kvq_tree_runs: parents [rows] (of a run's row i: an earlier row of the run, or -1) -> mask [rows, words], bit j of row i for
    j = i and i's ancestors, and positions [rows].  seq_lens [B] count the runs' tokens; words: for 32 tokens of a run each.  All int32
    and contiguous.  run_starts None: one token for each request."""
    device = parents.get_device()
    _i32(device, parents, seq_lens, mask, positions, run_starts, err)
    rows, words = mask.shape
    _tree(seq_lens.numel(), rows, run_starts, parents, positions)
    _launch("kvq_tree_runs", lib().kvq_tree_runs, device, stream, parents.data_ptr(), _ptr(run_starts), seq_lens.numel(), rows,
            seq_lens.data_ptr(), mask.data_ptr(), words, _ptr(positions), _ptr(err))


def _f32(device: int, n: int, t):
    assert t is None or (t.dtype is torch.float32 and t.is_contiguous() and t.numel() == n and t.get_device() == device), \
        f"{n} fp32, contiguous and on one CUDA device"


def rope_runs(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor, cos_sin: torch.Tensor, *,
              q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
              q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, run_starts: torch.Tensor | None = None,
              err: torch.Tensor | None = None, stream=None):
    """kvq_rope_runs: q [rows, Hq, 128] and k [rows, Hkv, 128] (fp32 or bf16; rows may be strided; either may be None) normed per head
    where q_weight / k_weight [128] (fp32) are given, and rotated to positions [rows] with the table ``cos_sin`` of append_rope.  In place
    unless q_out / k_out are given.  run_starts [B + 1]: rows behind the last run are left as they are."""
    one = q if q is not None else k
    assert one is not None, "queries, keys, or both"
    device, rows, dtype = one.get_device(), one.shape[0], one.dtype
    args = []
    for x, y in ((q, q_out), (k, k_out)):
        if x is None:
            assert y is None
            args.append((None, 0, 0, None, 0))
            continue
        n, heads, d = x.shape
        assert n == rows and d == HEAD_DIM and x.dtype is dtype and x.get_device() == device
        stride = _rows(x, n, heads)
        if y is None:
            args.append((x.data_ptr(), stride, heads, x.data_ptr(), stride))
        else:
            assert y.shape == x.shape and y.dtype is dtype and y.get_device() == device
            args.append((x.data_ptr(), stride, heads, y.data_ptr(), _rows(y, n, heads)))
    (qp, qs, hq, qo, qos), (kp, ks, hk, ko, kos) = args
    _i32(device, positions, run_starts, err)
    table = cos_sin.shape
    assert positions.numel() == rows and len(table) == 2 and table[1] == HEAD_DIM
    _f32(device, table[0] * HEAD_DIM, cos_sin)
    _f32(device, HEAD_DIM, q_weight)
    _f32(device, HEAD_DIM, k_weight)
    _launch("kvq_rope_runs", lib().kvq_rope_runs, device, stream, qp, qs, hq, kp, ks, hk, DTYPE[dtype], _ptr(q_weight),
            _ptr(k_weight), eps, positions.data_ptr(), cos_sin.data_ptr(), table[0], qo, qos, ko, kos, _ptr(run_starts),
            0 if run_starts is None else run_starts.numel() - 1, rows, _ptr(err))


def attn_tree_workspace_size(batch: int, num_rows: int, max_run: int, num_kv_heads: int, num_q_heads: int, q_dtype: torch.dtype) -> int:
    return int(lib().kvq_attn_tree_workspace_size(batch, num_rows, max_run, num_kv_heads, num_q_heads, DTYPE[q_dtype]))


def attn_tree(cache: PagedCache, q: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor, mask: torch.Tensor,
              out: torch.Tensor, workspace: torch.Tensor, *, run_starts: torch.Tensor | None = None, max_run: int | None = None,
              lse: torch.Tensor | None = None, sm_scale: float | None = None, err: torch.Tensor | None = None, stream=None):
    """kvq_attn_tree: attn_runs where a row sees all tokens before its run, and of its run those whose bits its mask [rows, words] has (int32,
    as tree_runs writes them).  max_run None: one token without run_starts, else as many as the mask has bits for or as there are rows."""
    rows, Hq, d = q.shape
    assert d == HEAD_DIM and out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous()
    device = q.get_device()
    assert workspace.is_contiguous(), "workspace: one piece of memory"
    _on(device, out, workspace, lse)
    cache._check_device(device)
    _i32(device, seq_lens, block_table, mask, run_starts, err)
    B, width = block_table.shape
    assert seq_lens.numel() == B and (run_starts is None or run_starts.numel() == B + 1) and mask.shape[0] == rows
    words = mask.shape[1]
    if max_run is None:
        max_run = 1 if run_starts is None else min(rows, 32 * words, MAX_TREE)
    assert lse is None or (lse.dtype is torch.float32 and lse.is_contiguous() and lse.numel() == rows * Hq)
    _launch("kvq_attn_tree", lib().kvq_attn_tree, device, stream, ctypes.byref(cache.desc()), q.data_ptr(), _rows(q, rows, Hq),
            DTYPE[q.dtype], Hq, _ptr(run_starts), B, rows, max_run, block_table.data_ptr(), width, seq_lens.data_ptr(),
            mask.data_ptr(), words, _SM_SCALE if sm_scale is None else sm_scale, out.data_ptr(), _ptr(lse), workspace.data_ptr(),
            workspace.nbytes, _ptr(err))


def _vocab_rows(x: torch.Tensor) -> int:
    rows, vocab = x.shape
    assert vocab == 1 or x.stride(1) == 1, "a row's elements side by side"
    return x.stride(0) if rows > 1 else vocab


def verify_runs(target: torch.Tensor, tokens: torch.Tensor, parents: torch.Tensor, uniform: torch.Tensor | None, keep: torch.Tensor,
                kept_lens: torch.Tensor, next_tokens: torch.Tensor, *, draft: torch.Tensor | None = None,
                seq_lens: torch.Tensor | None = None, seq_lens_out: torch.Tensor | None = None,
                run_starts: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None):
    """kvq_verify_runs: the path of every tree that the target accepts -> keep [rows] (the path's rows, -1 behind them), kept_lens [B]
    and next_tokens [B].

    target [rows, vocab] (fp32 or bf16; rows may be strided): probabilities of the token after each row, or any scores where
    uniform is None (greedy).  uniform [rows, 2] fp32 in [0, 1): for accepting the row's token, for drawing after it.  draft: probabilities
    that the rows' children were drawn from independently; None: children are no draws.  tokens, parents [rows] int32.  seq_lens [B] (with
    the runs' tokens) -> seq_lens_out [B] (with the kept ones), which may be the same tensor."""
    device = target.get_device()
    rows, vocab = target.shape
    assert draft is None or (draft.shape == target.shape and draft.dtype == target.dtype)
    _on(device, draft)
    _i32(device, tokens, parents, keep, kept_lens, next_tokens, seq_lens, seq_lens_out, run_starts, err)
    _f32(device, 2 * rows, uniform)
    B = kept_lens.numel()
    _tree(B, rows, run_starts, tokens, parents, keep)
    for t in (next_tokens, seq_lens, seq_lens_out):
        assert t is None or t.numel() == B
    _launch("kvq_verify_runs", lib().kvq_verify_runs, device, stream, target.data_ptr(), _vocab_rows(target), _ptr(draft),
            0 if draft is None else _vocab_rows(draft), DTYPE[target.dtype], vocab, tokens.data_ptr(), parents.data_ptr(), _ptr(uniform),
            _ptr(run_starts), B, rows, keep.data_ptr(), kept_lens.data_ptr(), next_tokens.data_ptr(), _ptr(seq_lens),
            _ptr(seq_lens_out), _ptr(err))


def keep_runs(caches, seq_lens: torch.Tensor, block_table: torch.Tensor, keep: torch.Tensor, kept_lens: torch.Tensor, *,
              run_starts: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None):
    """kvq_keep_runs: after verify_runs, the kept tokens' keys and values to the front of their runs, in ``caches`` (a page-scaled PagedCache, or a
    list of them, one for each layer, all alike).  seq_lens [B] count the kept tokens already (verify_runs's seq_lens_out)."""
    caches = [caches] if isinstance(caches, PagedCache) else list(caches)
    device = seq_lens.get_device()
    descs = b"".join([c._packed(device) for c in caches])
    _i32(device, seq_lens, block_table, keep, kept_lens, run_starts, err)
    B, width = block_table.shape
    assert seq_lens.numel() == B and kept_lens.numel() == B
    _tree(B, keep.numel(), run_starts)
    _launch("kvq_keep_runs", lib().kvq_keep_runs, device, stream, descs, len(caches), _ptr(run_starts), B, keep.numel(),
            block_table.data_ptr(), width, seq_lens.data_ptr(), keep.data_ptr(), kept_lens.data_ptr(), _ptr(err))


def debug_dither(seed: int, layer: int, kv_head: int, slots: torch.Tensor, out: torch.Tensor, stream=None):
    _check(lib().kvq_debug_dither(seed & 0xFFFFFFFFFFFFFFFF, layer, kv_head, slots.data_ptr(), int(slots.numel()),
                                  out.data_ptr(), _stream(stream)), "kvq_debug_dither")


def debug_time_decode(start: "torch.cuda.Event | None", stop: "torch.cuda.Event | None"):
    """kvq_debug_time_decode: record these events around every decode kernel launch (None, None clears)."""
    if start is None or stop is None:
        _check(lib().kvq_debug_time_decode(None, None), "kvq_debug_time_decode")
        return
    _check(lib().kvq_debug_time_decode(start.cuda_event, stop.cuda_event), "kvq_debug_time_decode")


def debug_wait_timeout(limit_ns: int, err: torch.Tensor, stream=None):
    """kvq_debug_wait_timeout: a bounded wait that runs out; err receives KVQ_ERR_TIMEOUT."""
    _check(lib().kvq_debug_wait_timeout(int(limit_ns), err.data_ptr(), _stream(stream)), "kvq_debug_wait_timeout")


def debug_encode(kind: int, x: torch.Tensor, out: torch.Tensor, stream=None):
    _check(lib().kvq_debug_encode(kind, x.data_ptr(), int(x.numel()), out.data_ptr(), _stream(stream)),
           "kvq_debug_encode")
