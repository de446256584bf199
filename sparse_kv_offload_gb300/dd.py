"""Thin Python binding of libdd (include/dd.h, include/dd_synth.h).

Argument marshalling only: every function checks the tensors it is given
(device, dtype, size, contiguity), passes their addresses and the current CUDA
stream to the C ABI, and raises ``DDError`` on a non-OK status.  All compute
runs in the library's CUDA kernels; there is no fallback -- importing this
module without a built ``libdd.so`` raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libdd.so")

DD_OK, DD_ERR_INVALID_ARG, DD_ERR_CUDA, DD_ERR_CAPACITY, DD_ERR_TIMEOUT, DD_ERR_DEVICE_CHECK = range(6)
GATHER_ZEROCOPY, GATHER_MEMCPY, GATHER_KERNEL, GATHER_AUTO = 0, 1, 2, 3
TRACE_SLOTS = 256          # per-SM slots of a step's timing words (DD_TRACE_SLOTS)
LM_MEAN, LM_MINMAX = 0, 1
D_HEAD = 128               # head dimension of the library
KV_BF16, KV_4BIT = 0, 1
KV4_ROW_BYTES = 72         # bytes of a 4-bit row of 128 values (DD_KV4_ROW_BYTES)
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_BY_PARTS, ROPE_BY_WAVELENGTH = range(5)
ROPE_TABLE_BYTES = 8704

EXPORTED = (
    "dd_create", "dd_destroy", "dd_build_landmarks", "dd_score_landmarks", "dd_select_topk",
    "dd_resolve_union", "dd_gather_kv", "dd_sparse_attn_decode", "dd_step", "dd_get_status",
    "dd_launch_count", "dd_status_str", "dd_last_cuda_error", "dd_synth_kv", "dd_synth_queries", "dd_sparse_attn_decode_noalloc",
    "dd_build_landmarks_minmax", "dd_score_landmarks_minmax", "dd_update_residency",
    "dd_prefetch_kv", "dd_select_topk_mass", "dd_selftest_bounded_wait", "dd_step_folds_scoring",
    "dd_rope_table", "dd_rope_rows", "dd_append_kv", "dd_gather_kv4", "dd_sparse_attn_decode_kv4",
)


class DDError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = ""
        if status == DD_ERR_CUDA:
            detail = " [" + _lib.dd_last_cuda_error().decode() + "]"
        super().__init__(f"{what}: {status_str(status)} ({status}){detail}")


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "d", "L", "cs", "k", "n_q")]


_vp = ctypes.c_void_p


class StepArgs(ctypes.Structure):
    _fields_ = [
        ("layer", ctypes.c_int32), ("q", _vp), ("lm", _vp), ("Kh", _vp), ("Vh", _vp),
        ("resident_slot", _vp), ("Khot", _vp), ("Vhot", _vp), ("Kst", _vp * 2), ("Vst", _vp * 2),
        ("mode", ctypes.c_int), ("softmax_scale", ctypes.c_float), ("out", _vp),
        ("scores", _vp), ("sel", _vp), ("union_idx", _vp), ("union_slot", _vp), ("union_cnt", _vp),
        ("miss_list", _vp), ("miss_count", _vp), ("attn_slot", _vp), ("union_qmask", _vp),
        ("stage_events", _vp * 6),
        ("lm_kind", ctypes.c_int),
        ("K_tail", _vp),
        ("V_tail", _vp),
        ("mass_gamma", ctypes.c_float),
        ("mass_k_min", ctypes.c_int32),
        ("sel_cnt", _vp),
        ("trace", _vp),
    ]


class RopeParams(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("scaling", ctypes.c_int), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("orig_len", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("gain", ctypes.c_double)]


class RopeRef(ctypes.Structure):
    _fields_ = [("table", _vp), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int)]


# dd_append_args: k, v; their strides; T, format; start_pos, new_len, rope, Kh, Vh, Khot,
# Vhot, resident_slot, k_exp, v_exp
_append_args = struct.Struct("@2P6q2i10P")
_strides = struct.Struct("@3q")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libdd.so is not built ({LIB_PATH}); run sparse_kv_offload_gb300.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    i32, i64, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    sig = {
        "dd_create": (i32, [ctypes.POINTER(Dims), i64, i64, ctypes.POINTER(_vp)]),
        "dd_destroy": (i32, [_vp]),
        "dd_build_landmarks": (i32, [_vp, _vp, _vp, _vp]),
        "dd_score_landmarks": (i32, [_vp, _vp, _vp, _vp, _vp]),
        "dd_build_landmarks_minmax": (i32, [_vp, _vp, _vp, _vp]),
        "dd_score_landmarks_minmax": (i32, [_vp, _vp, _vp, _vp, _vp]),
        "dd_select_topk": (i32, [_vp, _vp, _vp, _vp]),
        "dd_resolve_union": (i32, [_vp] * 11),
        "dd_gather_kv": (i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp]),
        "dd_sparse_attn_decode": (i32, [_vp] * 12 + [f32, _vp, _vp]),
        "dd_step": (i32, [_vp, ctypes.POINTER(StepArgs), _vp]),
        "dd_update_residency": (i32, [_vp, i32, i32, i32] + [_vp] * 13),
        "dd_selftest_bounded_wait": (i32, [_vp, i32, _vp]),
        "dd_select_topk_mass": (i32, [_vp, _vp, _vp, _vp, f32, i32, f32, _vp]),
        "dd_prefetch_kv": (i32, [_vp, _vp, i32, i32, i32, _vp, _vp, _vp, _vp, _vp, _vp, i32, _vp]),
        "dd_rope_table": (i32, [ctypes.POINTER(RopeParams), _vp]),
        "dd_rope_rows": (i32, [_vp, _vp, _vp, ctypes.c_char_p, _vp, ctypes.c_char_p, i32, i32, _vp, _vp, _vp]),
        "dd_append_kv": (i32, [_vp, ctypes.c_char_p, _vp]),
        "dd_gather_kv4": (i32, [_vp] * 7 + [i32] + [_vp] * 3),
        "dd_sparse_attn_decode_kv4": (i32, [_vp] * 16 + [f32, _vp, _vp]),
        "dd_get_status": (i32, [_vp, ctypes.POINTER(i32)]),
        "dd_launch_count": (i64, [_vp]),
        "dd_step_folds_scoring": (i32, [ctypes.POINTER(Dims), i32, ctypes.c_int, f32]),
        "dd_status_str": (ctypes.c_char_p, [i32]),
        "dd_last_cuda_error": (ctypes.c_char_p, []),
        "dd_synth_kv": (i32, [ctypes.POINTER(Dims), ctypes.c_uint64, i32, _vp, _vp, _vp, i64, _vp, _vp]),
        "dd_synth_queries": (i32, [ctypes.POINTER(Dims), ctypes.c_uint64, i32, ctypes.POINTER(f32), _vp, _vp]),
        "dd_sparse_attn_decode_noalloc": (i32, [ctypes.POINTER(Dims), i64, i64] + [_vp] * 9 + [f32, _vp, _vp, _vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def status_str(s: int) -> str:
    return _lib.dd_status_str(int(s)).decode()


def _chk(status: int, what: str):
    if status != DD_OK:
        raise DDError(status, what)


def _stream(stream) -> int:
    # the current stream's raw handle without building a torch.cuda.Stream
    # object (a tenth of the host time of torch.cuda.current_stream())
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t, dtype=None, numel=None, device=True, name="tensor", allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not device and (t.is_cuda or not t.is_pinned()):
        raise ValueError(f"{name} must be a pinned host tensor")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def _rows(t, shape, name, writable=False):
    """Address and (request, token, head) strides of bf16 rows [B, T, H, 128]: any strides
    that are multiples of 8 elements (16 bytes), the last dimension dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {shape}")
    B, T, H, _ = shape
    if t.is_contiguous():      # dense rows: nothing more to look at
        return t.data_ptr(), T * H * D_HEAD, H * D_HEAD, D_HEAD
    st = t.stride()
    if t.numel() and st[3] != 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    st = tuple(s if n > 1 else 0 for s, n in zip(st[:3], shape[:3]))   # a dimension of one has no stride
    if any(s % 8 for s in st):
        raise ValueError(f"{name}: strides must be multiples of 8 elements")
    if writable:
        extent = D_HEAD
        for s, n in sorted((s, n) for s, n in zip(st, shape[:3]) if n > 1):
            if s < extent:
                raise ValueError(f"{name}: rows overlap")
            extent += s * (n - 1)
    return t.data_ptr(), *st


def _dev(t, dtype, numel, name):
    """_ptr of a device tensor, None allowed: one test when all is well (a step's calls
    take a dozen tensors each, and the host runs just ahead of the GPU)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() >= numel:
            return t.data_ptr()
    except AttributeError:
        pass
    return _ptr(t, dtype, numel, name=name)


def _i32(t, numel, name, allow_none=False):
    if t is None and not allow_none:
        raise ValueError(f"{name} is required")
    return _dev(t, torch.int32, numel, name)


def _either(t, dtype, numel, name, allow_none=False):
    """Address of a tensor in device or in pinned host memory."""
    if isinstance(t, torch.Tensor):
        return _dev(t, dtype, numel, name) if t.is_cuda else _ptr(t, dtype, numel, device=False, name=name)
    return _ptr(t, dtype, numel, name=name, allow_none=allow_none)


class Rope:
    """Rotary positions: dd_rope_table's table on the device and the pairs' layout."""

    def __init__(self, table, rot_dim, layout):
        self.table = table
        self.rot_dim = int(rot_dim)
        self.layout = int(layout)
        self._ref = RopeRef(_ptr(table, torch.uint8, ROPE_TABLE_BYTES, name="table"), self.rot_dim, self.layout)
        self._addr = ctypes.addressof(self._ref)


def rope_host_table(rot_dim, base=10000.0, scaling=0, factor=1.0, orig_len=0.0, beta_fast=32.0, beta_slow=1.0,
                    gain=0.0) -> torch.Tensor:
    """dd_rope_table's output as a uint8 host tensor (no GPU needed; see dd.h)."""
    t = torch.zeros(ROPE_TABLE_BYTES, dtype=torch.uint8)
    p = RopeParams(int(rot_dim), int(scaling), float(base), float(factor), float(orig_len), float(beta_fast),
                   float(beta_slow), float(gain))
    _chk(_lib.dd_rope_table(ctypes.byref(p), t.data_ptr()), "dd_rope_table")
    return t


def rope_table(rot_dim, base=10000.0, layout=0, scaling=0, device="cuda", **scaling_params) -> Rope:
    """Rotary positions for Context.rope and Context.append_kv, made once: ``layout``
    ROPE_HALF or ROPE_INTERLEAVED, ``scaling`` one of ROPE_PLAIN .. ROPE_BY_WAVELENGTH
    with its factor, orig_len, beta_fast, beta_slow and gain (see dd.h)."""
    if layout not in (ROPE_HALF, ROPE_INTERLEAVED):
        raise ValueError(f"layout must be ROPE_HALF or ROPE_INTERLEAVED, got {layout}")
    return Rope(rope_host_table(rot_dim, base=base, scaling=scaling, **scaling_params).to(device), rot_dim, layout)


@dataclass(frozen=True)
class Shape:
    B: int
    Hq: int
    Hkv: int
    d: int
    L: int
    cs: int
    k: int
    n_q: int

    @property
    def C(self):
        return self.L // self.cs

    @property
    def G(self):
        return self.Hq // self.Hkv

    @property
    def umax(self):
        return min(self.C, self.n_q * self.k)

    def dims(self) -> Dims:
        return Dims(self.B, self.Hq, self.Hkv, self.d, self.L, self.cs, self.k, self.n_q)


def step_folds_scoring(shape: "Shape", sm_count: int, lm_kind: int = 0, mass_gamma: float = 0.0) -> int:
    """Ring depth of the selection kernel that scores its own unit inside dd_step
    (0: the step runs the scoring kernel first); host only."""
    d = shape.dims()
    return int(_lib.dd_step_folds_scoring(ctypes.byref(d), int(sm_count), int(lm_kind), float(mass_gamma)))


class Context:
    """One libdd context (workspace, status word, events, copy stream) on the current device."""

    def __init__(self, shape: Shape, max_misses: int, hot_slots: int = 0):
        self.shape = shape
        self.max_misses = int(max_misses)
        self.hot_slots = int(hot_slots)
        self._dims = shape.dims()
        h = _vp()
        _chk(_lib.dd_create(ctypes.byref(self._dims), self.max_misses, self.hot_slots, ctypes.byref(h)), "dd_create")
        self._h = h

    def close(self):
        if self._h:
            _lib.dd_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    # ------------------------------------------------------------------ stages
    def build_landmarks(self, K, lm, stream=None):
        s = self.shape
        n = s.B * s.Hkv * s.L * s.d
        kp = _ptr(K, torch.bfloat16, n, device=K.is_cuda, name="K")
        _chk(_lib.dd_build_landmarks(self._h, kp, _ptr(lm, torch.bfloat16, s.B * s.Hkv * s.C * s.d, name="lm"),
                                     _stream(stream)), "dd_build_landmarks")

    def score_landmarks(self, q, lm, scores, stream=None):
        s = self.shape
        _chk(_lib.dd_score_landmarks(
            self._h, _ptr(q, torch.bfloat16, s.B * s.n_q * s.Hq * s.d, name="q"),
            _ptr(lm, torch.bfloat16, s.B * s.Hkv * s.C * s.d, name="lm"),
            _ptr(scores, torch.float32, s.B * s.n_q * s.Hkv * s.C, name="scores"), _stream(stream)),
            "dd_score_landmarks")

    def build_landmarks_minmax(self, K, lm2, stream=None):
        s = self.shape
        n = s.B * s.Hkv * s.L * s.d
        kp = _ptr(K, torch.bfloat16, n, device=K.is_cuda, name="K")
        _chk(_lib.dd_build_landmarks_minmax(
            self._h, kp, _ptr(lm2, torch.bfloat16, s.B * s.Hkv * s.C * 2 * s.d, name="lm2"), _stream(stream)),
            "dd_build_landmarks_minmax")

    def score_landmarks_minmax(self, q, lm2, scores, stream=None):
        s = self.shape
        _chk(_lib.dd_score_landmarks_minmax(
            self._h, _ptr(q, torch.bfloat16, s.B * s.n_q * s.Hq * s.d, name="q"),
            _ptr(lm2, torch.bfloat16, s.B * s.Hkv * s.C * 2 * s.d, name="lm2"),
            _ptr(scores, torch.float32, s.B * s.n_q * s.Hkv * s.C, name="scores"), _stream(stream)),
            "dd_score_landmarks_minmax")

    def select_topk(self, scores, sel, stream=None):
        s = self.shape
        _chk(_lib.dd_select_topk(self._h, _ptr(scores, torch.float32, s.B * s.n_q * s.Hkv * s.C, name="scores"),
                                 _ptr(sel, torch.int32, s.B * s.n_q * s.Hkv * s.k, name="sel"), _stream(stream)),
             "dd_select_topk")

    def resolve_union(self, sel, resident_slot, union_idx, union_slot, union_qmask, union_cnt, miss_list,
                      miss_count, attn_slot=None, stream=None):
        s = self.shape
        nu = s.B * s.Hkv * s.umax
        _chk(_lib.dd_resolve_union(
            self._h, _ptr(sel, torch.int32, s.B * s.n_q * s.Hkv * s.k, name="sel"),
            _ptr(resident_slot, torch.int32, s.B * s.Hkv * s.C, name="resident_slot"),
            _ptr(union_idx, torch.int32, nu, name="union_idx"), _ptr(union_slot, torch.int32, nu, name="union_slot"),
            _ptr(union_qmask, torch.uint8, nu, name="union_qmask"),
            _ptr(union_cnt, torch.int32, s.B * s.Hkv, name="union_cnt"),
            _ptr(miss_list, torch.int32, max(1, self.max_misses), name="miss_list"),
            _ptr(miss_count, torch.int32, 1, name="miss_count"),
            _ptr(attn_slot, torch.int32, s.B * s.n_q * s.Hkv * s.k, name="attn_slot", allow_none=True),
            _stream(stream)), "dd_resolve_union")

    def gather_kv(self, Kh, Vh, miss_list, miss_count, Kst, Vst, mode=GATHER_ZEROCOPY, stream=None):
        s = self.shape
        n = s.B * s.Hkv * s.L * s.d
        ns = self.max_misses * s.cs * s.d
        _chk(_lib.dd_gather_kv(
            self._h, _ptr(Kh, torch.bfloat16, n, device=False, name="Kh"),
            _ptr(Vh, torch.bfloat16, n, device=False, name="Vh"),
            _ptr(miss_list, torch.int32, 1, name="miss_list"), _ptr(miss_count, torch.int32, 1, name="miss_count"),
            _ptr(Kst, torch.bfloat16, ns, name="Kst"), _ptr(Vst, torch.bfloat16, ns, name="Vst"), int(mode),
            _stream(stream)), "dd_gather_kv")

    def sparse_attn_decode(self, q, Khot, Vhot, Kst, Vst, union_slot, union_qmask, union_cnt, miss_count, out,
                           softmax_scale=0.0, stream=None, K_tail=None, V_tail=None):
        s = self.shape
        nh = self.hot_slots * s.cs * s.d
        ns = self.max_misses * s.cs * s.d
        nu = s.B * s.Hkv * s.umax
        nt = s.B * s.n_q * s.Hkv * s.d
        _chk(_lib.dd_sparse_attn_decode(
            self._h, _ptr(q, torch.bfloat16, s.B * s.n_q * s.Hq * s.d, name="q"),
            _ptr(Khot, torch.bfloat16, nh, name="Khot", allow_none=True),
            _ptr(Vhot, torch.bfloat16, nh, name="Vhot", allow_none=True),
            _ptr(Kst, torch.bfloat16, ns, name="Kst", allow_none=True),
            _ptr(Vst, torch.bfloat16, ns, name="Vst", allow_none=True),
            _ptr(K_tail, torch.bfloat16, nt, name="K_tail", allow_none=True),
            _ptr(V_tail, torch.bfloat16, nt, name="V_tail", allow_none=True),
            _ptr(union_slot, torch.int32, nu, name="union_slot"), _ptr(union_qmask, torch.uint8, nu, name="union_qmask"),
            _ptr(union_cnt, torch.int32, s.B * s.Hkv, name="union_cnt"),
            _ptr(miss_count, torch.int32, 1, name="miss_count"), float(softmax_scale),
            _ptr(out, torch.float32, s.B * s.n_q * s.Hq * s.d, name="out"), _stream(stream)),
            "dd_sparse_attn_decode")

    # ------------------------------------------- rotary positions, appends, 4-bit cache
    def rope(self, rope, x, out, start_pos, new_len=None, stream=None):
        """Rotate rows x bf16 [B, T, H, 128] into ``out`` (may be x): row t of request b at
        position start_pos[b] + t, rows t >= new_len[b] left out (see dd.h)."""
        if x.dim() != 4:
            raise ValueError("x must be [B, T, H, 128]")
        B = self.shape.B
        _, T, H, _ = x.shape
        shape = (B, T, H, D_HEAD)
        xp, *xs = _rows(x, shape, "x")
        op, *os_ = _rows(out, shape, "out", writable=True)
        _chk(_lib.dd_rope_rows(self._h, rope._addr, xp, _strides.pack(*xs), op, _strides.pack(*os_), T, H,
                               _i32(start_pos, B, "start_pos"), _dev(new_len, torch.int32, B, "new_len"),
                               _stream(stream)), "dd_rope_rows")

    def append_kv(self, k, v, start_pos, new_len=None, rope=None, Kh=None, Vh=None, Khot=None, Vhot=None,
                  resident_slot=None, kv_format=KV_BF16, k_exp=None, v_exp=None, stream=None):
        """Append rows k, v bf16 [B, T, Hkv, 128] to the home cache Kh/Vh (pinned host or
        device) and to the resident copies in Khot/Vhot, keys rotated by ``rope`` on the
        way; kv_format KV_BF16 or KV_4BIT (see dd.h)."""
        s = self.shape
        if k.dim() != 4:
            raise ValueError("k must be [B, T, Hkv, 128]")
        T = k.shape[1]
        four = kv_format == KV_4BIT
        dt, row = (torch.uint8, KV4_ROW_BYTES) if four else (torch.bfloat16, s.d)
        nh, nr = s.B * s.Hkv * s.L * row, self.hot_slots * s.cs * row
        shape = (s.B, T, s.Hkv, D_HEAD)
        kp, *ks = _rows(k, shape, "k")
        vp, *vs = _rows(v, shape, "v")
        i32 = torch.int32
        a = _append_args.pack(
            kp, vp, *ks, *vs, T, int(kv_format), _i32(start_pos, s.B, "start_pos"),
            _dev(new_len, i32, s.B, "new_len") or 0, rope._addr if rope is not None else 0,
            _either(Kh, dt, nh, "Kh", True) or 0, _either(Vh, dt, nh, "Vh", True) or 0, _dev(Khot, dt, nr, "Khot") or 0,
            _dev(Vhot, dt, nr, "Vhot") or 0, _dev(resident_slot, i32, s.B * s.Hkv * s.C, "resident_slot") or 0,
            _dev(k_exp, i32, s.Hkv, "k_exp") or 0, _dev(v_exp, i32, s.Hkv, "v_exp") or 0)
        _chk(_lib.dd_append_kv(self._h, a, _stream(stream)), "dd_append_kv")

    def gather_kv4(self, Kh, Vh, miss_list, miss_count, Kst, Vst, expand=False, k_exp=None, v_exp=None, stream=None):
        """Missing chunks of a 4-bit home cache (pinned host or device) into staging, as they
        are or, with ``expand``, as bf16 values (see dd.h)."""
        s = self.shape
        n = s.B * s.Hkv * s.L * KV4_ROW_BYTES
        dt, row = (torch.bfloat16, s.d) if expand else (torch.uint8, KV4_ROW_BYTES)
        ns = self.max_misses * s.cs * row
        _chk(_lib.dd_gather_kv4(
            self._h, _either(Kh, torch.uint8, n, "Kh"), _either(Vh, torch.uint8, n, "Vh"),
            _i32(miss_list, 1, "miss_list"), _i32(miss_count, 1, "miss_count"), _dev(Kst, dt, ns, "Kst"),
            _dev(Vst, dt, ns, "Vst"), 1 if expand else 0, _i32(k_exp, s.Hkv, "k_exp", True),
            _i32(v_exp, s.Hkv, "v_exp", True), _stream(stream)), "dd_gather_kv4")

    def sparse_attn_decode_kv4(self, q, Khot, Vhot, Kst, Vst, union_slot, union_cnt, out, union_qmask=None,
                               union_idx=None, kv_len=None, miss_count=None, k_exp=None, v_exp=None, K_tail=None,
                               V_tail=None, softmax_scale=0.0, stream=None):
        """sparse_attn_decode over 4-bit pages (uint8 [slots, cs*72]); rows at positions >=
        kv_len[b] are left out (see dd.h)."""
        s = self.shape
        page = s.cs * KV4_ROW_BYTES
        nh, ns = self.hot_slots * page, self.max_misses * page
        units = s.B * s.Hkv
        nu, nt = units * s.umax, s.B * s.n_q * s.Hkv * s.d
        nq = s.B * s.n_q * s.Hq * s.d
        u8, bf, i32 = torch.uint8, torch.bfloat16, torch.int32
        if q is None or out is None:
            raise ValueError("q and out are required")
        _chk(_lib.dd_sparse_attn_decode_kv4(
            self._h, _dev(q, bf, nq, "q"), _dev(Khot, u8, nh, "Khot"), _dev(Vhot, u8, nh, "Vhot"),
            _dev(Kst, u8, ns, "Kst"), _dev(Vst, u8, ns, "Vst"), _dev(k_exp, i32, s.Hkv, "k_exp"),
            _dev(v_exp, i32, s.Hkv, "v_exp"), _dev(K_tail, bf, nt, "K_tail"), _dev(V_tail, bf, nt, "V_tail"),
            _dev(union_idx, i32, nu, "union_idx"), _i32(union_slot, nu, "union_slot"),
            _dev(union_qmask, u8, nu, "union_qmask"), _i32(union_cnt, units, "union_cnt"),
            _dev(miss_count, i32, 1, "miss_count"), _dev(kv_len, i32, s.B, "kv_len"), float(softmax_scale),
            _dev(out, torch.float32, nq, "out"), _stream(stream)), "dd_sparse_attn_decode_kv4")

    def selftest_bounded_wait(self, kind, stream=None):
        """Run a bounded device wait that nothing signals (see dd.h); the status
        word then holds DD_ERR_TIMEOUT."""
        _chk(_lib.dd_selftest_bounded_wait(self._h, int(kind), _stream(stream)), "dd_selftest_bounded_wait")

    def select_topk_mass(self, scores, sel, gamma, k_min=1, sel_cnt=None, softmax_scale=0.0, stream=None):
        """Coverage-budget top-k (see dd.h): rows padded with -1, lengths in sel_cnt."""
        s = self.shape
        rows = s.B * s.n_q * s.Hkv
        _chk(_lib.dd_select_topk_mass(
            self._h, _ptr(scores, torch.float32, rows * s.C, name="scores"),
            _ptr(sel, torch.int32, rows * s.k, name="sel"),
            _ptr(sel_cnt, torch.int32, rows, name="sel_cnt", allow_none=True), float(gamma), int(k_min),
            float(softmax_scale), _stream(stream)), "dd_select_topk_mass")

    def prefetch_kv(self, sel, n_pred, Kh, Vh, Kpf, Vpf, pf_map, pf_count=None, ctas_per_sm=8, stream=None,
                    sel_rows=None, first_row=0):
        """Predictive prefetch of rows first_row .. first_row+n_pred-1 of ``sel``
        [B, sel_rows, Hkv, k] (sel_rows defaults to n_pred; see dd.h)."""
        s = self.shape
        n = s.B * s.Hkv * s.L * s.d
        ns = self.max_misses * s.cs * s.d
        rows = n_pred if sel_rows is None else sel_rows
        _chk(_lib.dd_prefetch_kv(
            self._h, _ptr(sel, torch.int32, s.B * max(rows, 0) * s.Hkv * s.k, name="sel"), int(rows),
            int(first_row), int(n_pred),
            _ptr(Kh, torch.bfloat16, n, device=False, name="Kh"), _ptr(Vh, torch.bfloat16, n, device=False, name="Vh"),
            _ptr(Kpf, torch.bfloat16, ns, name="Kpf", allow_none=True),
            _ptr(Vpf, torch.bfloat16, ns, name="Vpf", allow_none=True),
            _ptr(pf_map, torch.int32, s.B * s.Hkv * s.C, name="pf_map"),
            _ptr(pf_count, torch.int32, 1, name="pf_count", allow_none=True), int(ctas_per_sm), _stream(stream)),
            "dd_prefetch_kv")

    def update_residency(self, step, cap, slots_per_unit, Kst, Vst, resident_slot, slot_chunk, last_used, Khot,
                         Vhot, admitted=None, union_idx=None, union_slot=None, union_cnt=None, miss_count=None,
                         stream=None):
        """Capped LRU residency update after a step (see dd.h); the union arrays default
        to the context's workspace (the last step that used it)."""
        s = self.shape
        units = s.B * s.Hkv
        nu = units * s.umax
        nh = self.hot_slots * s.cs * s.d
        ns = self.max_misses * s.cs * s.d
        _chk(_lib.dd_update_residency(
            self._h, int(step), int(cap), int(slots_per_unit),
            _ptr(union_idx, torch.int32, nu, name="union_idx", allow_none=True),
            _ptr(union_slot, torch.int32, nu, name="union_slot", allow_none=True),
            _ptr(union_cnt, torch.int32, units, name="union_cnt", allow_none=True),
            _ptr(miss_count, torch.int32, 1, name="miss_count", allow_none=True),
            _ptr(Kst, torch.bfloat16, ns, name="Kst", allow_none=True),
            _ptr(Vst, torch.bfloat16, ns, name="Vst", allow_none=True),
            _ptr(resident_slot, torch.int32, units * s.C, name="resident_slot"),
            _ptr(slot_chunk, torch.int32, units * slots_per_unit, name="slot_chunk"),
            _ptr(last_used, torch.int32, units * slots_per_unit, name="last_used"),
            _ptr(Khot, torch.bfloat16, nh, name="Khot"), _ptr(Vhot, torch.bfloat16, nh, name="Vhot"),
            _ptr(admitted, torch.int32, units, name="admitted", allow_none=True), _stream(stream)),
            "dd_update_residency")

    def step(self, layer, q, lm, Kh, Vh, resident_slot, Khot, Vhot, Kst_pair, Vst_pair, out,
             mode=GATHER_ZEROCOPY, softmax_scale=0.0, intermediates=None, stage_events=None, stream=None,
             lm_kind=LM_MEAN, K_tail=None, V_tail=None, mass_gamma=0.0, mass_k_min=1, sel_cnt=None, trace=None):
        """One layer; ``intermediates`` optionally maps names of dd_step_args' optional
        outputs (scores, sel, union_idx, union_slot, union_qmask, union_cnt, miss_list,
        miss_count, attn_slot) to caller tensors; ``stage_events`` optionally gives six
        torch.cuda.Event objects recorded at the stage boundaries; ``lm_kind`` says
        whether ``lm`` holds mean landmarks or min/max landmarks (twice the size)."""
        s = self.shape
        a = StepArgs()
        a.layer = int(layer)
        a.q = _ptr(q, torch.bfloat16, s.B * s.n_q * s.Hq * s.d, name="q")
        a.lm_kind = int(lm_kind)
        a.mass_gamma = float(mass_gamma)
        a.mass_k_min = int(mass_k_min)
        a.sel_cnt = _ptr(sel_cnt, torch.int32, s.B * s.n_q * s.Hkv, name="sel_cnt", allow_none=True)
        # int64 tensor of 3 * 2 * TRACE_SLOTS (uint64 bits): see dd_step_args.trace
        a.trace = _ptr(trace, torch.int64, 6 * TRACE_SLOTS, name="trace", allow_none=True)
        a.K_tail = _ptr(K_tail, torch.bfloat16, s.B * s.n_q * s.Hkv * s.d, name="K_tail", allow_none=True)
        a.V_tail = _ptr(V_tail, torch.bfloat16, s.B * s.n_q * s.Hkv * s.d, name="V_tail", allow_none=True)
        a.lm = _ptr(lm, torch.bfloat16, s.B * s.Hkv * s.C * s.d * (2 if lm_kind == LM_MINMAX else 1), name="lm")
        n = s.B * s.Hkv * s.L * s.d
        a.Kh = _ptr(Kh, torch.bfloat16, n, device=False, name="Kh")
        a.Vh = _ptr(Vh, torch.bfloat16, n, device=False, name="Vh")
        a.resident_slot = _ptr(resident_slot, torch.int32, s.B * s.Hkv * s.C, name="resident_slot")
        nh = self.hot_slots * s.cs * s.d
        a.Khot = _ptr(Khot, torch.bfloat16, nh, name="Khot", allow_none=True)
        a.Vhot = _ptr(Vhot, torch.bfloat16, nh, name="Vhot", allow_none=True)
        ns = self.max_misses * s.cs * s.d
        for p in range(2):
            a.Kst[p] = _ptr(Kst_pair[p], torch.bfloat16, ns, name="Kst", allow_none=True)
            a.Vst[p] = _ptr(Vst_pair[p], torch.bfloat16, ns, name="Vst", allow_none=True)
        a.mode = int(mode)
        a.softmax_scale = float(softmax_scale)
        a.out = _ptr(out, torch.float32, s.B * s.n_q * s.Hq * s.d, name="out")
        for name, t in (intermediates or {}).items():
            dt = {"scores": torch.float32, "union_qmask": torch.uint8}.get(name, torch.int32)
            setattr(a, name, _ptr(t, dt, 1, name=name))
        for i, ev in enumerate(stage_events or ()):
            if ev is not None:
                a.stage_events[i] = ev.cuda_event
        self._last_args = a
        _chk(_lib.dd_step(self._h, ctypes.byref(a), _stream(stream)), "dd_step")

    def status(self) -> int:
        """Wait for the device, return and clear the device status word."""
        v = ctypes.c_int32(0)
        _chk(_lib.dd_get_status(self._h, ctypes.byref(v)), "dd_get_status")
        return int(v.value)

    def launch_count(self) -> int:
        return int(_lib.dd_launch_count(self._h))


# ---------------------------------------------------------------- allocation-free attention
def sparse_attn_decode_noalloc(shape: Shape, hot_slots, max_misses, q, Khot, Vhot, Kst, Vst, union_slot,
                               union_qmask, union_cnt, miss_count, out, device_status, softmax_scale=0.0,
                               stream=None):
    """dd_sparse_attn_decode without a context, for callers that cannot
    allocate device memory: its split-K partials sit in the library's fixed
    16 MiB device array.  ``device_status`` is a zeroed device int32 tensor that
    receives a device-detected dd_status code.  Calls that overlap on the GPU
    share that array and race; serialise them."""
    s = shape
    dims = s.dims()
    nh = int(hot_slots) * s.cs * s.d
    ns = int(max_misses) * s.cs * s.d
    nu = s.B * s.Hkv * s.umax
    _chk(_lib.dd_sparse_attn_decode_noalloc(
        ctypes.byref(dims), int(hot_slots), int(max_misses),
        _ptr(q, torch.bfloat16, s.B * s.n_q * s.Hq * s.d, name="q"),
        _ptr(Khot, torch.bfloat16, nh, name="Khot", allow_none=True),
        _ptr(Vhot, torch.bfloat16, nh, name="Vhot", allow_none=True),
        _ptr(Kst, torch.bfloat16, ns, name="Kst", allow_none=True),
        _ptr(Vst, torch.bfloat16, ns, name="Vst", allow_none=True),
        _ptr(union_slot, torch.int32, nu, name="union_slot"), _ptr(union_qmask, torch.uint8, nu, name="union_qmask"),
        _ptr(union_cnt, torch.int32, s.B * s.Hkv, name="union_cnt"), _ptr(miss_count, torch.int32, 1, name="miss_count"),
        float(softmax_scale), _ptr(out, torch.float32, s.B * s.n_q * s.Hq * s.d, name="out"),
        _ptr(device_status, torch.int32, 1, name="device_status"), _stream(stream)),
        "dd_sparse_attn_decode_noalloc")


# ---------------------------------------------------------------- generator
def synth_kv(shape: Shape, seed: int, tensor_id: int, dst, bias=None, u_hat=None, chunk_map=None, stream=None):
    dims = shape.dims()
    n_slots = 0 if chunk_map is None else int(chunk_map.numel())
    numel = n_slots * shape.cs * shape.d if chunk_map is not None else shape.B * shape.Hkv * shape.L * shape.d
    dp = _ptr(dst, torch.bfloat16, numel, device=dst.is_cuda, name="dst")
    _chk(_lib.dd_synth_kv(ctypes.byref(dims), int(seed), int(tensor_id),
                          _ptr(bias, torch.float32, shape.B * shape.Hkv * shape.C, name="bias", allow_none=True),
                          _ptr(u_hat, torch.float32, shape.B * shape.Hkv * shape.d, name="u_hat", allow_none=True),
                          _ptr(chunk_map, torch.int32, n_slots, name="chunk_map", allow_none=True), n_slots, dp,
                          _stream(stream)), "dd_synth_kv")


def synth_queries(shape: Shape, seed: int, layer: int, spec_scale, dst, stream=None):
    dims = shape.dims()
    sc = (ctypes.c_float * max(1, shape.n_q))(*[float(x) for x in list(spec_scale)[:shape.n_q]])
    _chk(_lib.dd_synth_queries(ctypes.byref(dims), int(seed), int(layer), sc,
                               _ptr(dst, torch.bfloat16, shape.B * shape.n_q * shape.Hq * shape.d, name="q"),
                               _stream(stream)), "dd_synth_queries")


def default_scale(d: int = 128) -> float:
    return 1.0 / math.sqrt(d)
