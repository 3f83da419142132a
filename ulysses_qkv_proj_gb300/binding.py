"""ctypes binding of libqnre (include/qnre.h).  Argument marshalling only.

The names follow the C ABI: `qnre_forward`, `qnre_forward_noalloc`,
`ulysses_pack_head_chunk`, `ulysses_merge_output_head_chunk`,
`ulysses_scatter_heads`, `ulysses_gather_heads`,
`ulysses_pack_output_sequence_chunk`, `ulysses_gather_output_head_chunk`,
`ulysses_scatter_qkv_head_chunk`, plus the `Plan` wrapper around
`qnre_plan_create` / `qnre_plan_destroy`, and the speculative-decoding calls
over a `PagedCache` (`qnre_qk_norm_rope` and its gradient,
`qnre_qkv_norm_rope_append`, `qnre_cache_*`, `qnre_tree_masks`,
`qnre_tree_attention`, `qnre_verify_tree`) and the calls for many answers from one
prompt (`qnre_rope_table`, `qnre_cache_shared_prefix`, `qnre_prefix_attention`,
`qnre_sample`, `qnre_filter_probs`).  Tensors are torch CUDA tensors;
torch supplies device memory and the current stream, nothing else.  Every
failure status raises `QnreError`; a missing library raises at first use.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import struct
from typing import Dict, List, Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqnre.so")
DEBUG_LIB_PATH = os.path.join(HERE, "libqnre_debug.so")  # QNRE_LIB=<this path> selects it
HEADER = os.path.join(os.path.dirname(HERE), "include", "qnre.h")

QNRE_OK = 0
STATUS_NAMES = {
    0: "QNRE_OK", 1: "QNRE_ERR_INVALID_ARG", 2: "QNRE_ERR_UNSUPPORTED", 3: "QNRE_ERR_ALIGNMENT",
    4: "QNRE_ERR_ALIAS", 5: "QNRE_ERR_CAPACITY", 6: "QNRE_ERR_CUDA", 7: "QNRE_ERR_DEVICE",
}
LAYOUTS = {"bshd": 0, "fused": 1}
ROPE_STYLES = {"rotate_half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "yarn": 3, "wavelength": 4}
FLAG_EPILOGUE_OFF = 0x1
FLAG_W_MULTICAST = 0x2
FLAG_ONE_PAIR = 0x4
DEVICE_BAD_POSITION = 0x1
DEVICE_WAIT_TIMEOUT = 0x2
DEVICE_READY_TIMEOUT = 0x4
DEVICE_BOUNDS = 0x8
HEAD_DIM = 128


class QnreError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class _Out(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("fused", ctypes.c_void_p)]


class _PlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("device", "pairs_per_cluster", "clusters", "sms", "row_tiles",
                                            "col_tiles", "work_items", "half_items", "launches")]


class _Tensor4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("shape", ctypes.c_int64 * 4),
                ("stride", ctypes.c_int64 * 4), ("dtype", ctypes.c_int32)]


_pack_tensor4 = struct.Struct("P4q4qi4x").pack  # the layout of _Tensor4


class _Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "block_table", "seq_lens", "page_refs", "status", "scratch")] + \
        [(n, ctypes.c_int32) for n in ("layers", "pages", "heads", "page_size", "head_dim", "rows", "max_blocks",
                                       "dtype")]


class _RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32)] + \
        [(n, ctypes.c_double) for n in ("factor", "original", "low", "high", "magnitude")]


_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libqnre.so (built by ulysses_qkv_proj_gb300.build), or the library the
    QNRE_LIB environment variable names (the debug build); raises if it is missing."""
    global _lib, _native
    if _lib is not None:
        return _lib
    try:
        import torch  # noqa: F401  (its libraries, before the module that links to them)
        from . import _marshal as _native
    except ImportError:
        _native = None
    path = path or os.environ.get("QNRE_LIB") or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libqnre.so not built ({path}); run `python -m ulysses_qkv_proj_gb300.build`")
    lib = ctypes.CDLL(path)
    c_int, c_i64, c_vp, c_uint = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_uint
    lib.qnre_status_string.restype = ctypes.c_char_p
    lib.qnre_status_string.argtypes = [c_int]
    lib.qnre_plan_create.restype = c_int
    lib.qnre_plan_create.argtypes = [ctypes.POINTER(c_vp), c_int, c_int, c_int, c_int, c_int, c_i64, c_int, c_uint]
    lib.qnre_plan_destroy.restype = c_int
    lib.qnre_plan_destroy.argtypes = [c_vp]
    lib.qnre_plan_reserve_sms.restype = c_int
    lib.qnre_plan_reserve_sms.argtypes = [c_vp, c_int]
    lib.qnre_plan_describe.restype = c_int
    lib.qnre_plan_describe.argtypes = [c_vp, c_int, c_int, ctypes.POINTER(_PlanInfo)]
    lib.qnre_forward.restype = c_int
    lib.qnre_forward.argtypes = [c_vp, c_int, c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp,
                                 ctypes.POINTER(_Out), c_vp]
    lib.qnre_plan_device_status.restype = c_int
    lib.qnre_plan_device_status.argtypes = [c_vp, c_vp, ctypes.POINTER(c_uint), c_int]
    lib.qnre_debug_bounds.restype = c_int
    lib.qnre_debug_bounds.argtypes = [ctypes.POINTER(ctypes.c_ulonglong), c_int]
    lib.ulysses_pack_head_chunk.restype = c_int
    lib.ulysses_pack_head_chunk.argtypes = [ctypes.POINTER(_Tensor4)] * 3 + [c_int, c_int, c_int, c_vp, c_vp]
    lib.ulysses_merge_output_head_chunk.restype = c_int
    lib.ulysses_merge_output_head_chunk.argtypes = [ctypes.POINTER(_Tensor4), c_int, c_int, c_int, c_vp, c_vp]
    lib.ulysses_pack_head_chunk_schedule.restype = c_int
    lib.ulysses_pack_head_chunk_schedule.argtypes = [ctypes.POINTER(_Tensor4)] * 3 + [
        c_int, c_int, ctypes.POINTER(c_int), ctypes.POINTER(c_int), ctypes.POINTER(c_vp), c_vp]
    lib.ulysses_merge_output_head_chunk_schedule.restype = c_int
    lib.ulysses_merge_output_head_chunk_schedule.argtypes = [ctypes.POINTER(ctypes.POINTER(_Tensor4)), c_int, c_int,
                                                            c_int, ctypes.POINTER(c_int), c_vp, c_vp]
    lib.qnre_forward_noalloc.restype = c_int
    lib.qnre_forward_noalloc.argtypes = [c_int, c_int, c_int, c_int, c_int, c_uint, c_int, c_int,
                                         c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp, ctypes.POINTER(_Out), c_vp, c_vp]
    i32 = ctypes.c_int32
    lib.ulysses_scatter_heads.restype = c_int
    lib.ulysses_scatter_heads.argtypes = [c_vp, c_int, c_int, c_int, c_int, c_int, i32, c_vp, c_vp]
    lib.ulysses_gather_heads.restype = c_int
    lib.ulysses_gather_heads.argtypes = [c_vp, c_int, c_int, c_int, c_int, c_int, i32, c_vp, c_vp]
    lib.ulysses_pack_output_sequence_chunk.restype = c_int
    lib.ulysses_pack_output_sequence_chunk.argtypes = [ctypes.POINTER(_Tensor4), c_int, c_vp, c_vp]
    lib.ulysses_gather_output_head_chunk.restype = c_int
    lib.ulysses_gather_output_head_chunk.argtypes = [c_vp, c_int, c_int, c_int, c_int, c_int, i32, c_int, c_int,
                                                     c_vp, c_vp]
    lib.ulysses_scatter_qkv_head_chunk.restype = c_int
    lib.ulysses_scatter_qkv_head_chunk.argtypes = [ctypes.POINTER(_Tensor4)] * 3 + [c_int, c_int, c_int, c_vp, c_vp]
    lib.qnre_forward_publish.restype = c_int
    lib.qnre_forward_publish.argtypes = [c_vp, c_int, c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp,
                                         ctypes.POINTER(_Out), c_vp, c_vp]
    lib.qnre_ready_target.restype = c_int
    lib.qnre_ready_target.argtypes = [c_vp, c_int, c_int, ctypes.POINTER(c_uint)]
    lib.qnre_wait_ready.restype = c_int
    lib.qnre_wait_ready.argtypes = [c_vp, c_vp, c_uint, ctypes.c_uint64, c_vp]
    lib.ulysses_sage2_workspace_bytes.restype = c_int
    lib.ulysses_sage2_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int, ctypes.POINTER(ctypes.c_uint64)]
    lib.ulysses_sage2_scatter_qkv.restype = c_int
    lib.ulysses_sage2_scatter_qkv.argtypes = [ctypes.POINTER(_Tensor4)] * 3 + [c_int, c_int] + [c_vp] * 7 + \
        [ctypes.c_uint64, c_vp]
    t4, cache = c_vp, ctypes.POINTER(_Cache)  # views go over as packed bytes (_view4)
    for name in ("truncate", "fork", "reserve", "copy_pages"):
        fn = getattr(lib, "qnre_cache_" + name)
        fn.restype = c_int
        fn.argtypes = [cache, c_vp, c_vp, c_int, c_vp]
    lib.qnre_cache_compact.restype = c_int
    lib.qnre_cache_compact.argtypes = [cache, c_vp, c_vp, c_vp, c_int, c_int, c_vp]
    table = [c_vp, c_vp, c_vp, c_i64, c_int, c_int, c_vp]  # norm weights, cos_sin, n_pos, rot, style, positions
    lib.qnre_qk_norm_rope.restype = c_int
    lib.qnre_qk_norm_rope.argtypes = [t4, t4, *table, t4, t4, c_vp]
    lib.qnre_qk_norm_rope_workspace_bytes.restype = c_int
    lib.qnre_qk_norm_rope_workspace_bytes.argtypes = [c_int, ctypes.POINTER(ctypes.c_uint64)]
    lib.qnre_qk_norm_rope_backward.restype = c_int
    lib.qnre_qk_norm_rope_backward.argtypes = [t4, t4, t4, t4, *table, t4, t4, c_vp, c_vp, c_vp, ctypes.c_uint64, c_vp]
    lib.qnre_qkv_norm_rope_append.restype = c_int
    lib.qnre_qkv_norm_rope_append.argtypes = [t4, t4, t4, *table, t4, cache, c_int, c_vp, c_vp, c_vp]
    lib.qnre_tree_attention_workspace_bytes.restype = c_int
    lib.qnre_tree_attention_workspace_bytes.argtypes = [c_int, ctypes.POINTER(ctypes.c_uint64)]
    lib.qnre_tree_attention.restype = c_int
    lib.qnre_tree_attention.argtypes = [t4, cache, c_int, c_vp, c_vp, c_vp, ctypes.c_float, c_vp, c_vp, c_vp,
                                        ctypes.c_uint64, c_vp]
    lib.qnre_verify_tree.restype = c_int
    lib.qnre_verify_tree.argtypes = [c_vp, c_i64, c_i64, c_vp, c_i64, c_i64, c_int, c_int, c_i64] + [c_vp] * 9
    lib.qnre_tree_masks.restype = c_int
    lib.qnre_tree_masks.argtypes = [c_vp, c_int, c_int, c_vp, c_vp, c_vp]
    lib.qnre_rope_table.restype = c_int
    lib.qnre_rope_table.argtypes = [c_vp, c_i64, c_int, c_i64, ctypes.c_double, ctypes.POINTER(_RopeScaling), c_vp]
    lib.qnre_cache_shared_prefix.restype = c_int
    lib.qnre_cache_shared_prefix.argtypes = [cache, c_vp, c_int, c_vp, c_int, c_vp, c_vp]
    lib.qnre_prefix_attention_workspace_bytes.restype = c_int
    lib.qnre_prefix_attention_workspace_bytes.argtypes = [c_int] * 6 + [ctypes.POINTER(ctypes.c_uint64)]
    lib.qnre_prefix_attention.restype = c_int
    lib.qnre_prefix_attention.argtypes = [t4, cache, c_int, c_vp, c_vp, c_int, c_vp, c_vp, c_vp, c_vp, ctypes.c_float,
                                          ctypes.c_float, c_vp, c_vp, c_vp, c_vp, ctypes.c_uint64, c_vp]
    lib.qnre_sample.restype = c_int
    lib.qnre_sample.argtypes = [c_vp, c_i64, i32, c_int, c_i64] + [c_vp] * 7
    lib.qnre_filter_probs.restype = c_int
    lib.qnre_filter_probs.argtypes = [c_vp, c_i64, c_i64, i32, c_int, c_int, c_i64] + [c_vp] * 6
    for name in ("qnre_qk_norm_rope", "qnre_qk_norm_rope_backward", "qnre_qkv_norm_rope_append", "qnre_tree_attention",
                 "qnre_verify_tree", "qnre_cache_truncate", "qnre_cache_fork", "qnre_cache_reserve",
                 "qnre_cache_compact", "qnre_cache_copy_pages", "qnre_sample", "qnre_filter_probs",
                 "qnre_cache_shared_prefix", "qnre_prefix_attention", "qnre_rope_table"):
        _entry[name] = ctypes.cast(getattr(lib, name), c_vp).value
    _lib = lib
    return lib


def header_functions(path: str = HEADER) -> List[str]:
    """Names of the functions include/qnre.h declares."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*([A-Za-z_][A-Za-z0-9_]*)\s*\(",
                      text, flags=re.M)


def _check(status: int, where: str) -> None:
    if status != QNRE_OK:
        raise QnreError(status, where)


_dtype_codes: Dict[object, int] = {}


def _dtype_code(t) -> int:
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise QnreError(2, f"dtype {t.dtype}")
    return code


# A decode step's kernels run for a few microseconds, so the calls' own cost counts: the current
# stream is read as a raw handle (0.4 us on a Grace core; building the Stream object takes 2.9), a view
# is packed in one go (1.0 us; field by field 2.4), and the decoding calls are read and made natively (_marshal)
# where that module was built: None from it means that a check failed, and the Python checks then say which.
def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _tensor4(t) -> _Tensor4:
    if t.dim() != 4:
        raise QnreError(1, "expected a rank-4 view")
    return _Tensor4.from_buffer_copy(_pack_tensor4(t.data_ptr(), *t.shape, *t.stride(), _dtype_code(t)))


class Plan:
    """qnre_plan_create / qnre_plan_destroy."""

    def __init__(self, hidden: int, num_heads: int, P: int, layout: str = "bshd",
                 max_tokens: int = 1, rope_style: str = "rotate_half", head_dim: int = HEAD_DIM,
                 flags: int = 0):
        lib = load_library()
        self._handle = ctypes.c_void_p()
        self.hidden, self.num_heads, self.P = hidden, num_heads, P
        self.layout, self.rope_style, self.max_tokens, self.flags = layout, rope_style, max_tokens, flags
        _check(lib.qnre_plan_create(ctypes.byref(self._handle), hidden, num_heads, head_dim, P,
                                    LAYOUTS.get(layout, -1), max_tokens, ROPE_STYLES.get(rope_style, -1),
                                    flags), "qnre_plan_create")

    @property
    def handle(self):
        return self._handle

    def destroy(self) -> None:
        if self._handle:
            _check(load_library().qnre_plan_destroy(self._handle), "qnre_plan_destroy")
            self._handle = ctypes.c_void_p()

    def __del__(self):
        try:
            if self._handle:
                load_library().qnre_plan_destroy(self._handle)
        except Exception:
            pass

    def reserve_sms(self, sms: int) -> None:
        """qnre_plan_reserve_sms: leave `sms` SMs free of the fused kernel (0 = use all)."""
        _check(load_library().qnre_plan_reserve_sms(self._handle, sms), "qnre_plan_reserve_sms")

    def describe(self, B: int, S_local: int) -> Dict[str, int]:
        """qnre_plan_describe: how a forward of (B, S_local) runs (clusters, SMs, work list)."""
        info = _PlanInfo()
        _check(load_library().qnre_plan_describe(self._handle, B, S_local, ctypes.byref(info)),
               "qnre_plan_describe")
        return {name: getattr(info, name) for name, _ in _PlanInfo._fields_}

    def device_status(self, clear: bool = True, stream=None) -> int:
        bits = ctypes.c_uint(0)
        st = load_library().qnre_plan_device_status(self._handle, _stream_ptr(stream), ctypes.byref(bits),
                                                    1 if clear else 0)
        if st not in (QNRE_OK, 7):
            raise QnreError(st, "qnre_plan_device_status")
        return bits.value


def debug_bounds(reset: bool = True) -> int:
    """Accesses the debug build's layout and Sage2 kernels skipped (qnre_debug_bounds);
    raises QnreError(QNRE_ERR_UNSUPPORTED) on the release build."""
    n = ctypes.c_ulonglong(0)
    st = load_library().qnre_debug_bounds(ctypes.byref(n), 1 if reset else 0)
    if st != QNRE_OK:
        raise QnreError(st, "qnre_debug_bounds")
    return n.value


def qnre_forward(plan: Plan, x, w_qkv, q_norm_w, k_norm_w, cos_sin, positions, out: Dict[str, object],
                 stream=None) -> None:
    """x: bf16 [P, B, S_local, hidden]; out: {"q","k","v"} (bshd) or {"fused"} (fused)."""
    if x.dim() != 4 or x.shape[0] != plan.P:
        raise QnreError(1, "qnre_forward: x must be [P, B, S_local, hidden]")
    o = _Out(_ptr(out.get("q")), _ptr(out.get("k")), _ptr(out.get("v")), _ptr(out.get("fused")))
    _check(load_library().qnre_forward(plan.handle, x.shape[1], x.shape[2], x.data_ptr(), w_qkv.data_ptr(),
                                       q_norm_w.data_ptr(), k_norm_w.data_ptr(), cos_sin.data_ptr(),
                                       cos_sin.shape[0], _ptr(positions), ctypes.byref(o),
                                       _stream_ptr(stream)), "qnre_forward")


def ulysses_pack_head_chunk(q, k, v, world_size: int, head_offset: int, head_count: int, out,
                            stream=None):
    """Pack one head band of strided q/k/v [B, S, H, D] into contiguous out [B, S, W*cnt, 3D]."""
    tq, tk, tv = _tensor4(q), _tensor4(k), _tensor4(v)
    _check(load_library().ulysses_pack_head_chunk(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                                  world_size, head_offset, head_count, out.data_ptr(),
                                                  _stream_ptr(stream)), "ulysses_pack_head_chunk")
    return out


def ulysses_merge_output_head_chunk(received, world_size: int, local_heads: int, head_offset: int, out,
                                    stream=None):
    """Merge received [B, S, W*cnt, D] into band head_offset of contiguous out [B, S, W*L, D]."""
    tr = _tensor4(received)
    _check(load_library().ulysses_merge_output_head_chunk(ctypes.byref(tr), world_size, local_heads,
                                                          head_offset, out.data_ptr(), _stream_ptr(stream)),
           "ulysses_merge_output_head_chunk")
    return out


def ulysses_pack_head_chunk_schedule(q, k, v, world_size: int, schedule, outs, stream=None):
    """Every (head_offset, head_count) chunk of `schedule` packed into outs[i] in one launch."""
    n = len(schedule)
    tq, tk, tv = _tensor4(q), _tensor4(k), _tensor4(v)
    offs = (ctypes.c_int * n)(*[int(o) for o, _ in schedule])
    cnts = (ctypes.c_int * n)(*[int(c) for _, c in schedule])
    ptrs = (ctypes.c_void_p * n)(*[_contig(o, "pack_head_chunk_schedule") for o in outs])
    _check(load_library().ulysses_pack_head_chunk_schedule(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                                           world_size, n, offs, cnts, ptrs, _stream_ptr(stream)),
           "ulysses_pack_head_chunk_schedule")
    return outs


def ulysses_merge_output_head_chunk_schedule(received, world_size: int, local_heads: int, head_offsets, out,
                                             stream=None):
    """Every received[i] merged at band head_offsets[i] of `out` in one launch."""
    n = len(received)
    views = [_tensor4(r) for r in received]
    arr = (ctypes.POINTER(_Tensor4) * n)(*[ctypes.pointer(t) for t in views])
    offs = (ctypes.c_int * n)(*[int(o) for o in head_offsets])
    _check(load_library().ulysses_merge_output_head_chunk_schedule(arr, world_size, local_heads, n, offs,
                                                                   _contig(out, "merge_output_head_chunk_schedule"),
                                                                   _stream_ptr(stream)),
           "ulysses_merge_output_head_chunk_schedule")
    return out


def qnre_forward_publish(plan: Plan, x, w_qkv, q_norm_w, k_norm_w, cos_sin, positions, out: Dict[str, object],
                         ready, stream=None) -> None:
    """qnre_forward that also publishes per-destination readiness counts into ready (int32 CUDA [P])."""
    if x.dim() != 4 or x.shape[0] != plan.P:
        raise QnreError(1, "qnre_forward_publish: x must be [P, B, S_local, hidden]")
    o = _Out(_ptr(out.get("q")), _ptr(out.get("k")), _ptr(out.get("v")), _ptr(out.get("fused")))
    _check(load_library().qnre_forward_publish(plan.handle, x.shape[1], x.shape[2], x.data_ptr(), w_qkv.data_ptr(),
                                               q_norm_w.data_ptr(), k_norm_w.data_ptr(), cos_sin.data_ptr(),
                                               cos_sin.shape[0], _ptr(positions), ctypes.byref(o), ready.data_ptr(),
                                               _stream_ptr(stream)), "qnre_forward_publish")


def qnre_ready_target(plan: Plan, B: int, S_local: int) -> int:
    t = ctypes.c_uint(0)
    _check(load_library().qnre_ready_target(plan.handle, B, S_local, ctypes.byref(t)), "qnre_ready_target")
    return t.value


def qnre_wait_ready(plan: Plan, ready, target: int, timeout_ns: int, stream=None) -> None:
    """Enqueue the bounded one-CTA wait for every ready[r] >= target; expiry sets DEVICE_READY_TIMEOUT."""
    _check(load_library().qnre_wait_ready(plan.handle, ready.data_ptr(), target, timeout_ns, _stream_ptr(stream)),
           "qnre_wait_ready")


def qnre_forward_noalloc(hidden: int, num_heads: int, P: int, x, w_qkv, q_norm_w, k_norm_w, cos_sin, positions,
                         out: Dict[str, object], layout: str = "bshd", rope_style: str = "rotate_half",
                         flags: int = 0, device_status=None, stream=None) -> None:
    """qnre_forward without a plan: for callers that cannot allocate device memory when they
    project.  device_status: optional int32 CUDA tensor of one element that receives the
    call's QNRE_DEVICE_* bits."""
    if x.dim() != 4 or x.shape[0] != P:
        raise QnreError(1, "qnre_forward_noalloc: x must be [P, B, S_local, hidden]")
    o = _Out(_ptr(out.get("q")), _ptr(out.get("k")), _ptr(out.get("v")), _ptr(out.get("fused")))
    _check(load_library().qnre_forward_noalloc(hidden, num_heads, P, LAYOUTS.get(layout, -1),
                                               ROPE_STYLES.get(rope_style, -1), flags, x.shape[1], x.shape[2],
                                               x.data_ptr(), w_qkv.data_ptr(), q_norm_w.data_ptr(),
                                               k_norm_w.data_ptr(), cos_sin.data_ptr(), cos_sin.shape[0],
                                               _ptr(positions), ctypes.byref(o), _ptr(device_status),
                                               _stream_ptr(stream)), "qnre_forward_noalloc")


def _contig(t, where: str):
    if not t.is_contiguous():
        raise QnreError(1, f"{where}: tensor must be contiguous")
    return t.data_ptr()


def ulysses_scatter_heads(x, out, stream=None):
    """x [P, B, S_local, H, D] -> out [P, B, P*S_local, H/P, D] (both contiguous)."""
    P, B, S, H, D = x.shape
    _check(load_library().ulysses_scatter_heads(_contig(x, "scatter_heads"), P, B, S, H, D, _dtype_code(x),
                                                _contig(out, "scatter_heads"), _stream_ptr(stream)),
           "ulysses_scatter_heads")
    return out


def ulysses_gather_heads(y, out, stream=None):
    """y [P, B, S_global, H_local, D] -> out [P, B, S_global/P, P*H_local, D] (both contiguous)."""
    P, B, S_g, H_l, D = y.shape
    _check(load_library().ulysses_gather_heads(_contig(y, "gather_heads"), P, B, S_g, H_l, D, _dtype_code(y),
                                               _contig(out, "gather_heads"), _stream_ptr(stream)),
           "ulysses_gather_heads")
    return out


def ulysses_pack_output_sequence_chunk(x, world_size: int, out, stream=None):
    """x view [B, S_global, head_count, D] -> out [world_size, B, S_global/world_size, head_count, D]."""
    tx = _tensor4(x)
    _check(load_library().ulysses_pack_output_sequence_chunk(ctypes.byref(tx), world_size,
                                                             _contig(out, "pack_output_sequence_chunk"),
                                                             _stream_ptr(stream)),
           "ulysses_pack_output_sequence_chunk")
    return out


def ulysses_gather_output_head_chunk(x, local_heads: int, head_offset: int, out, stream=None):
    """x [P, B, S_global, head_count, D] -> band head_offset of out [P, B, S_global/P, P*local_heads, D]."""
    P, B, S_g, cnt, D = x.shape
    _check(load_library().ulysses_gather_output_head_chunk(_contig(x, "gather_output_head_chunk"), P, B, S_g, cnt, D,
                                                           _dtype_code(x), local_heads, head_offset,
                                                           _contig(out, "gather_output_head_chunk"),
                                                           _stream_ptr(stream)),
           "ulysses_gather_output_head_chunk")
    return out


def ulysses_scatter_qkv_head_chunk(q, k, v, P: int, head_offset: int, head_count: int, out, stream=None):
    """q/k/v views [P*B, S_local, H, D] -> out [P, B, P*S_local, head_count, 3*D] (contiguous)."""
    tq, tk, tv = _tensor4(q), _tensor4(k), _tensor4(v)
    _check(load_library().ulysses_scatter_qkv_head_chunk(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv), P,
                                                         head_offset, head_count,
                                                         _contig(out, "scatter_qkv_head_chunk"),
                                                         _stream_ptr(stream)),
           "ulysses_scatter_qkv_head_chunk")
    return out


def alloc_outputs(plan: Plan, B: int, S_local: int, device="cuda") -> Dict[str, object]:
    """Output buffers for qnre_forward (uninitialised bf16)."""
    import torch
    H_local = plan.num_heads // plan.P
    S_g = plan.P * S_local
    if plan.layout == "bshd":
        return {g: torch.empty((plan.P, B, S_g, H_local, HEAD_DIM), dtype=torch.bfloat16, device=device)
                for g in "qkv"}
    return {"fused": torch.empty((plan.P, B, S_g, H_local, 3 * HEAD_DIM), dtype=torch.bfloat16, device=device)}


def ulysses_sage2_workspace_bytes(P: int, B: int, L: int, H: int, D: int) -> int:
    """Scratch bytes ulysses_sage2_scatter_qkv needs for these sizes."""
    n = ctypes.c_uint64()
    _check(load_library().ulysses_sage2_workspace_bytes(P, B, L, H, D, ctypes.byref(n)),
           "ulysses_sage2_workspace_bytes")
    return n.value


def sage2_outputs(P: int, B: int, L: int, H: int, D: int, used_sequence: int, device="cuda") -> Dict[str, object]:
    """Output buffers (uninitialised) and the workspace for ulysses_sage2_scatter_qkv."""
    import torch
    S, H_l = P * L, H // P
    S_pad = -(-S // 64) * 64
    U = used_sequence
    ws = ulysses_sage2_workspace_bytes(P, B, L, H, D)
    return {"q": torch.empty((P, B, S, H_l, D), dtype=torch.int8, device=device),
            "k": torch.empty((P, B, S, H_l, D), dtype=torch.int8, device=device),
            "v": torch.empty((P, B, D, H_l, S_pad), dtype=torch.uint8, device=device),
            "q_scale": torch.empty((P, B, H_l, -(-U // 32)), dtype=torch.float32, device=device),
            "k_scale": torch.empty((P, B, H_l, -(-U // 64)), dtype=torch.float32, device=device),
            "v_scale": torch.empty((P, B, H_l, D), dtype=torch.float32, device=device),
            "workspace": torch.empty((ws,), dtype=torch.uint8, device=device)}


def ulysses_sage2_scatter_qkv(q, k, v, P: int, used_sequence: int, out: Dict[str, object], stream=None):
    """q/k/v views [P*B, L, H, D] (bf16 or fp16) -> the Sage2 codes and scales of every
    destination rank in `out` (see sage2_outputs)."""
    tq, tk, tv = _tensor4(q), _tensor4(k), _tensor4(v)
    names = ("q", "k", "v", "q_scale", "k_scale", "v_scale")
    ptrs = [_contig(out[n], "sage2_scatter_qkv") for n in names]
    ws = out["workspace"]
    _check(load_library().ulysses_sage2_scatter_qkv(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv), P,
                                                    used_sequence, *ptrs, _contig(ws, "sage2_scatter_qkv"),
                                                    ws.numel() * ws.element_size(), _stream_ptr(stream)),
           "ulysses_sage2_scatter_qkv")
    return out


# ---------------------------------------------------------------------------
# Speculative decoding over a paged cache
# ---------------------------------------------------------------------------
MAX_NODES = 64
CACHE_NO_PAGES = 0x1
CACHE_BAD_ROW = 0x2
CACHE_BAD_PAGE = 0x4
CACHE_BAD_REFS = 0x8
CACHE_WAIT_TIMEOUT = 0x10


class PagedCache:
    """A paged K/V cache over tensors the caller owns, all on one device (qnre_cache_t).

    k, v         bf16 or fp16 [layers, pages, heads, page_size, head_dim]
    block_table  int32 [rows, max_blocks], -1 where a row holds no page
    seq_lens     int32 [rows];  page_refs  int32 [pages], 0 = free
    """

    def __init__(self, k, v, block_table, seq_lens, page_refs):
        import torch
        if k.dim() != 5 or v.shape != k.shape or v.dtype != k.dtype:
            raise QnreError(1, "PagedCache: k and v must be [layers, pages, heads, page_size, head_dim] alike")
        layers, pages, heads, page_size, head_dim = k.shape
        rows = seq_lens.numel()
        if block_table.dim() != 2 or block_table.shape[0] != rows or page_refs.numel() != pages:
            raise QnreError(1, "PagedCache: block_table [rows, max_blocks], seq_lens [rows], page_refs [pages]")
        if any(t.device != k.device for t in (v, block_table, seq_lens, page_refs)):
            raise QnreError(1, "PagedCache: every tensor must lie on one device")
        self.k, self.v = k, v
        self.block_table, self.seq_lens, self.page_refs = block_table, seq_lens, page_refs
        self.status_word = torch.zeros(1, dtype=torch.int32, device=k.device)
        self.scratch = torch.empty(4 * pages + 4, dtype=torch.int32, device=k.device)
        self._struct = _Cache(_contig(k, "PagedCache"), _contig(v, "PagedCache"),
                              _i32("PagedCache", block_table), _i32("PagedCache", seq_lens),
                              _i32("PagedCache", page_refs), self.status_word.data_ptr(), self.scratch.data_ptr(),
                              layers, pages, heads, page_size, head_dim, rows, block_table.shape[1], _dtype_code(k))
        self.handle, self.address = ctypes.byref(self._struct), ctypes.addressof(self._struct)

    def status(self, clear: bool = True) -> int:
        """The CACHE_* bits kernels have set (waits for the current stream)."""
        bits = int(self.status_word.item())
        if clear and bits:
            self.status_word.zero_()
        return bits


def alloc_paged_cache(layers: int, pages: int, heads: int, page_size: int, head_dim: int, rows: int, max_blocks: int,
                      dtype=None, device="cuda") -> PagedCache:
    """An empty cache (pools uninitialised, every page free)."""
    import torch
    shape = (layers, pages, heads, page_size, head_dim)
    pools = [torch.empty(shape, dtype=dtype or torch.bfloat16, device=device) for _ in range(2)]
    return PagedCache(*pools, torch.full((rows, max_blocks), -1, dtype=torch.int32, device=device),
                      torch.zeros(rows, dtype=torch.int32, device=device),
                      torch.zeros(pages, dtype=torch.int32, device=device))


_int32 = _int64 = _float32 = None


def _load_dtypes():
    global _int32, _int64, _float32
    import torch
    _int32, _int64, _float32 = torch.int32, torch.int64, torch.float32


_native = None  # the _marshal module once load_library has found it
_entry: Dict[str, int] = {}  # addresses of the entry points that it calls itself


def _sizes(t):
    return t.shape if _native is None else _native.sizes(t)


def _i32(where: str, t, *shape):
    """Pointer of a contiguous int32 tensor (None passes), its shape checked where given."""
    if t is None:
        return None
    if _native is not None:
        p = _native.pointer(t, 3, *shape)
        if p is not None:
            return p
    if _int32 is None:
        _load_dtypes()
    if t.dtype is not _int32:
        raise QnreError(1, f"{where}: expected int32")
    if shape and t.shape != shape:
        raise QnreError(1, f"{where}: expected shape {list(shape)}")
    if not t.is_contiguous():
        raise QnreError(1, f"{where}: tensor must be contiguous")
    return t.data_ptr()


def _f32(where: str, t, *shape):
    if _native is not None:
        p = _native.pointer(t, 2, *shape)
        if p is not None:
            return p
    if _int32 is None:
        _load_dtypes()
    if t.dtype is not _float32:
        raise QnreError(1, f"{where}: expected float32")
    if shape and t.shape != shape:
        raise QnreError(1, f"{where}: expected shape {list(shape)}")
    if not t.is_contiguous():
        raise QnreError(1, f"{where}: tensor must be contiguous")
    return t.data_ptr()


def _view4(t) -> bytes:
    """A rank-4 view as the bytes of a qnre_tensor4_t."""
    if _native is not None:
        b = _native.view4(t)
        if b is not None:
            return b
    if t.dim() != 4:
        raise QnreError(1, "expected a rank-4 view")
    return _pack_tensor4(t.data_ptr(), *t.shape, *t.stride(), _dtype_codes.get(t.dtype) or _dtype_code(t))


def _weight(where: str, w, dim: int, like) -> int:
    if _native is not None:
        p = _native.pointer(w, _native.type_code(like), dim)
        if p is not None:
            return p
    dtype = like.dtype
    if w.dtype is not dtype or w.shape != (dim,) or not w.is_contiguous():
        raise QnreError(1, f"{where}: norm weights are contiguous [{dim}] of the input's dtype")
    return w.data_ptr()


def _on_device(where: str, *tensors) -> None:
    """Every tensor given (None passes) lies on one device, and that is the current CUDA device, where the kernels run.
    (Where there is no CUDA at all tensors of the CPU pass: the entry points check them and launch nothing.)"""
    import torch
    devices = {t.device for t in tensors if t is not None}
    if len(devices) == 1:
        d = devices.pop()
        if d.type == "cuda" and d.index == torch.cuda.current_device():
            return
        if d.type == "cpu" and not torch.cuda.is_available():
            return
    raise QnreError(1, f"{where}: every tensor must lie on the current CUDA device")


def qnre_cache_truncate(cache: PagedCache, rows, lens, stream=None) -> None:
    """Row rows[i] keeps its first lens[i] tokens; the blocks past them are released (0 frees the row)."""
    where, lib = "qnre_cache_truncate", load_library()
    if _native is not None:
        st = _native.cache_rows(_entry[where], cache.address, cache.k, rows, lens, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    n = rows.numel()
    args = _i32(where, rows, n), _i32(where, lens, n), n
    _on_device(where, cache.k, rows, lens)
    _check(lib.qnre_cache_truncate(cache.handle, *args, _stream_ptr(stream)), where)


def qnre_cache_fork(cache: PagedCache, src, dst, stream=None) -> None:
    """Empty row dst[i] becomes a copy of row src[i] that shares its pages."""
    where, lib = "qnre_cache_fork", load_library()
    if _native is not None:
        st = _native.cache_rows(_entry[where], cache.address, cache.k, src, dst, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    n = src.numel()
    args = _i32(where, src, n), _i32(where, dst, n), n
    _on_device(where, cache.k, src, dst)
    _check(lib.qnre_cache_fork(cache.handle, *args, _stream_ptr(stream)), where)


def qnre_cache_reserve(cache: PagedCache, rows, counts, stream=None) -> None:
    """Pages of its own for the next counts[i] tokens of row rows[i] (lowest free pages, copy on write)."""
    where, lib = "qnre_cache_reserve", load_library()
    if _native is not None:
        st = _native.cache_rows(_entry[where], cache.address, cache.k, rows, counts, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    n = rows.numel()
    args = _i32(where, rows, n), _i32(where, counts, n), n
    _on_device(where, cache.k, rows, counts)
    _check(lib.qnre_cache_reserve(cache.handle, *args, _stream_ptr(stream)), where)


def qnre_cache_compact(cache: PagedCache, rows, path, counts, stream=None) -> None:
    """Keep the accepted nodes path[i][:counts[i]] of row rows[i]'s drafts; its length grows by counts[i]."""
    where, lib = "qnre_cache_compact", load_library()
    if _native is not None:
        st = _native.compact(_entry[where], cache.address, cache.k, rows, path, counts, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    n = rows.numel()
    shape = _sizes(path)
    if len(shape) != 2:
        raise QnreError(1, f"{where}: path must be [n, nodes]")
    args = _i32(where, rows, n), _i32(where, path, n, shape[1]), _i32(where, counts, n), n, shape[1]
    _on_device(where, cache.k, rows, path, counts)
    _check(lib.qnre_cache_compact(cache.handle, *args, _stream_ptr(stream)), where)


def qnre_cache_copy_pages(cache: PagedCache, src, dst, stream=None) -> None:
    """Page src[i] to page dst[i] in every layer."""
    where, lib = "qnre_cache_copy_pages", load_library()
    if _native is not None:
        st = _native.cache_rows(_entry[where], cache.address, cache.k, src, dst, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    n = src.numel()
    args = _i32(where, src, n), _i32(where, dst, n), n
    _on_device(where, cache.k, src, dst)
    _check(lib.qnre_cache_copy_pages(cache.handle, *args, _stream_ptr(stream)), where)


def _norm_inputs(where: str, q, k, q_norm_w, k_norm_w, cos_sin, positions):
    table = _sizes(cos_sin)
    if len(table) != 2:
        raise QnreError(1, f"{where}: cos_sin must be [n_pos, rot]")
    vq, vk = _view4(q), _view4(k)
    B, S, _, dim = _sizes(q)
    head = (vq, vk, _weight(where, q_norm_w, dim, q), _weight(where, k_norm_w, dim, k), _f32(where, cos_sin), *table)
    return head, _i32(where, positions, B, S)


def qnre_qk_norm_rope(q, k, q_norm_w, k_norm_w, cos_sin, positions, q_out, k_out, rope_style: str = "rotate_half",
                      stream=None) -> None:
    """Per-head RMSNorm and rotation of q [B, S, Hq, D] and k [B, S, Hk, D] (views; in place allowed)."""
    where = "qnre_qk_norm_rope"
    lib, style = load_library(), ROPE_STYLES.get(rope_style, -1)
    if _native is not None:
        st = _native.norm(_entry[where], q, k, q_norm_w, k_norm_w, cos_sin, positions, q_out, k_out, style, _stream_ptr,
                          stream)
        if st is not None:
            return _check(st, where)
    head, pos = _norm_inputs(where, q, k, q_norm_w, k_norm_w, cos_sin, positions)
    args = *head, style, pos, _view4(q_out), _view4(k_out)
    _on_device(where, q, k, q_norm_w, k_norm_w, cos_sin, positions, q_out, k_out)
    _check(lib.qnre_qk_norm_rope(*args, _stream_ptr(stream)), where)


def qk_norm_rope_workspace(q, k=None):
    """The scratch tensor qnre_qk_norm_rope_backward needs for heads like q's."""
    import torch
    n = ctypes.c_uint64()
    _check(load_library().qnre_qk_norm_rope_workspace_bytes(q.shape[-1], ctypes.byref(n)),
           "qnre_qk_norm_rope_workspace_bytes")
    return torch.empty(n.value, dtype=torch.uint8, device=q.device)


def qnre_qk_norm_rope_backward(gq, gk, q, k, q_norm_w, k_norm_w, cos_sin, positions, dq, dk, dq_norm_w, dk_norm_w,
                               workspace, rope_style: str = "rotate_half", stream=None) -> None:
    """Gradient of qnre_qk_norm_rope: dq, dk (input dtype) and the fp32 weight gradients."""
    where = "qnre_qk_norm_rope_backward"
    lib, style = load_library(), ROPE_STYLES.get(rope_style, -1)
    if _native is not None:
        st = _native.norm_backward(_entry[where], gq, gk, q, k, q_norm_w, k_norm_w, cos_sin, positions, dq, dk, dq_norm_w,
                                   dk_norm_w, workspace, style, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    head, pos = _norm_inputs(where, q, k, q_norm_w, k_norm_w, cos_sin, positions)
    D = q.shape[-1]
    args = (_view4(gq), _view4(gk), *head, style, pos, _view4(dq), _view4(dk), _f32(where, dq_norm_w, D),
            _f32(where, dk_norm_w, D), _contig(workspace, where), workspace.numel() * workspace.element_size())
    _on_device(where, gq, gk, q, k, q_norm_w, k_norm_w, cos_sin, positions, dq, dk, dq_norm_w, dk_norm_w, workspace)
    _check(lib.qnre_qk_norm_rope_backward(*args, _stream_ptr(stream)), where)


def qnre_qkv_norm_rope_append(q, k, v, q_norm_w, k_norm_w, cos_sin, positions, q_out, cache: PagedCache, layer: int,
                              rows, counts=None, rope_style: str = "rotate_half", stream=None) -> None:
    """qnre_qk_norm_rope of the rows' new tokens [n, S, ...]; k and v go into the cache behind seq_lens."""
    where = "qnre_qkv_norm_rope_append"
    lib, style = load_library(), ROPE_STYLES.get(rope_style, -1)
    if _native is not None:
        st = _native.append(_entry[where], q, k, v, q_norm_w, k_norm_w, cos_sin, positions, q_out, cache.address, cache.k,
                            layer, rows, counts, style, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    head, pos = _norm_inputs(where, q, k, q_norm_w, k_norm_w, cos_sin, positions)
    n = q.shape[0]
    args = (head[0], head[1], _view4(v), *head[2:], style, pos, _view4(q_out), cache.handle, layer, _i32(where, rows, n),
            _i32(where, counts, n))
    _on_device(where, q, k, v, q_norm_w, k_norm_w, cos_sin, positions, q_out, cache.k, rows, counts)
    _check(lib.qnre_qkv_norm_rope_append(*args, _stream_ptr(stream)), where)


def qnre_tree_masks(parents, masks=None, depths=None, stream=None) -> None:
    """Ancestor masks (int64 [n, nodes], bit j: node j) and depths (int32) of trees given by parents int32 [n, nodes]."""
    where = "qnre_tree_masks"
    if parents.dim() != 2:
        raise QnreError(1, f"{where}: parents must be [n, nodes]")
    n, nodes = _sizes(parents)
    args = _i32(where, parents), n, nodes, _i64(where, masks, n, nodes), _i32(where, depths, n, nodes)
    _on_device(where, parents, masks, depths)
    _check(load_library().qnre_tree_masks(*args, _stream_ptr(stream)), where)


def tree_attention_workspace(q, cache: PagedCache):
    """The scratch tensor qnre_tree_attention needs on this cache (any batch)."""
    import torch
    n = ctypes.c_uint64()
    _check(load_library().qnre_tree_attention_workspace_bytes(cache.k.shape[-1], ctypes.byref(n)),
           "qnre_tree_attention_workspace_bytes")
    return torch.empty(n.value, dtype=torch.uint8, device=q.device)


def _same(where: str, t, like):
    """Pointer of a contiguous tensor of like's shape and type."""
    if _native is not None:
        p = _native.pointer(t, _native.type_code(like), *_native.sizes(like))
        if p is not None:
            return p
    if t.shape != like.shape or t.dtype != like.dtype:
        raise QnreError(1, f"{where}: the output must be contiguous, of the input's shape and dtype")
    return _contig(t, where)


def _i64(where: str, t, *shape):
    """Pointer of a contiguous int64 tensor of that shape (None passes)."""
    if t is None:
        return None
    if _native is not None:
        p = _native.pointer(t, 4, *shape)
        if p is not None:
            return p
    if _int64 is None:
        _load_dtypes()
    if t.dtype is not _int64 or t.shape != shape:
        raise QnreError(1, f"{where}: expected int64 {list(shape)}")
    return _contig(t, where)


def qnre_tree_attention(q, cache: PagedCache, layer: int, rows, mask, out, lse=None, counts=None, scale=None,
                        workspace=None, stream=None) -> None:
    """Attention of drafted nodes q [n, nodes, Hq, D] over their rows' tokens and the nodes of mask (int64 [n, nodes];
    None: a chain) into out (contiguous); scale defaults to 1/sqrt(D)."""
    where, lib = "qnre_tree_attention", load_library()
    if _native is not None:
        st = _native.attention(_entry[where], q, cache.address, cache.k, layer, rows, mask, out, lse, counts, scale,
                               workspace, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    tq = _view4(q)
    n, nodes, heads, dim = _sizes(q)
    to = _same(where, out, q)
    tm = _i64(where, mask, n, nodes)
    if workspace is None:
        raise QnreError(1, f"{where}: workspace is missing (tree_attention_workspace)")
    args = (tq, cache.handle, layer, _i32(where, rows, n), tm, _i32(where, counts, n),
            dim ** -0.5 if scale is None else scale, to, None if lse is None else _f32(where, lse, n, nodes, heads),
            _contig(workspace, where), workspace.numel() * workspace.element_size())
    _on_device(where, q, cache.k, rows, mask, out, lse, counts, workspace)
    _check(lib.qnre_tree_attention(*args, _stream_ptr(stream)), where)


def qnre_verify_tree(target_probs, draft_probs, tokens, parents, accept_u, sample_u, path, counts, next_token,
                     node_counts=None, stream=None) -> None:
    """Walk drafted trees against target_probs [n, nodes, V] (fp32; draft_probs alike or None) with given random
    numbers; fills path [n, nodes], counts [n] and next_token [n] (int32)."""
    where, lib = "qnre_verify_tree", load_library()
    if _native is not None:
        st = _native.verify(_entry[where], target_probs, draft_probs, tokens, parents, accept_u, sample_u, path, counts,
                            next_token, node_counts, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    shape = _sizes(target_probs)
    if len(shape) != 3:
        raise QnreError(1, f"{where}: target_probs must be [n, nodes, vocab]")
    n, nodes, vocab = shape
    rows = []
    for t in (target_probs, draft_probs):
        p = None if t is None or _native is None else _native.pointer(t, 2, n, nodes, vocab)
        if t is None:
            rows += [None, 0, 0]
        elif p is not None:
            rows += [p, nodes * vocab, vocab]
        else:
            if _float32 is None:
                _load_dtypes()
            if t.dtype is not _float32 or t.shape != shape or (t.stride(2) != 1 and vocab > 1):
                raise QnreError(1, f"{where}: probabilities are float32 [n, nodes, vocab], each row contiguous")
            rows += [t.data_ptr(), t.stride(0), t.stride(1)]
    args = (*rows, n, nodes, vocab, _i32(where, tokens, n, nodes), _i32(where, parents, n, nodes),
            _i32(where, node_counts, n), _f32(where, accept_u, n, nodes), _f32(where, sample_u, n),
            _i32(where, path, n, nodes), _i32(where, counts, n), _i32(where, next_token, n))
    _on_device(where, target_probs, draft_probs, tokens, parents, accept_u, sample_u, path, counts, next_token, node_counts)
    _check(lib.qnre_verify_tree(*args, _stream_ptr(stream)), where)


# ---------------------------------------------------------------------------
# Many answers from one prompt
# ---------------------------------------------------------------------------
MAX_VOCAB = 1048576


def qnre_rope_table(cos_sin, theta: float = 1e4, first: int = 0, scaling: str = "none", factor: float = 1.0,
                    original: float = 0.0, low: float = 1.0, high: Optional[float] = None,
                    magnitude: Optional[float] = None, stream=None) -> None:
    """Fill cos_sin (fp32 [n_pos, rot]) with rows [cos | sin] of positions first.., frequencies scaled as `scaling` says
    (none, linear, base, yarn, wavelength).  high defaults to 32 turns (yarn) or 4 (wavelength), magnitude to
    0.1 ln(factor) + 1 for yarn with a factor above 1, and to 1 otherwise."""
    where = "qnre_rope_table"
    lib = load_library()
    kind = ROPE_SCALINGS.get(scaling, -1)
    if high is None:
        high = 32.0 if kind == 3 else 4.0
    if magnitude is None:
        magnitude = 0.1 * math.log(factor) + 1.0 if kind == 3 and factor > 1 else 1.0
    if _native is not None:
        st = _native.rope_table(_entry[where], cos_sin, theta, first, kind, factor, original, low, high, magnitude, _stream_ptr,
                                stream)
        if st is not None:
            return _check(st, where)
    shape = _sizes(cos_sin)
    if len(shape) != 2:
        raise QnreError(1, f"{where}: cos_sin must be [n_pos, rot]")
    args = _f32(where, cos_sin), *shape, first, theta, ctypes.byref(_RopeScaling(kind, factor, original, low, high, magnitude))
    _on_device(where, cos_sin)
    _check(lib.qnre_rope_table(*args, _stream_ptr(stream)), where)


def qnre_cache_shared_prefix(cache: PagedCache, rows, groups, shared, stream=None) -> None:
    """shared[g] = tokens that rows[groups[g]:groups[g + 1]] all hold in the same pages (whole pages; int32 lists)."""
    where, lib = "qnre_cache_shared_prefix", load_library()
    if _native is not None:
        st = _native.shared_prefix(_entry[where], cache.address, cache.k, rows, groups, shared, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    n, n_groups = rows.numel(), shared.numel()
    args = _i32(where, rows, n), n, _i32(where, groups, n_groups + 1), n_groups, _i32(where, shared, n_groups)
    _on_device(where, cache.k, rows, groups, shared)
    _check(lib.qnre_cache_shared_prefix(cache.handle, *args, _stream_ptr(stream)), where)


def prefix_attention_workspace(q, cache: PagedCache, groups: bool = True):
    """The scratch tensor qnre_prefix_attention needs for queries like q on this cache (without groups less)."""
    import torch
    n = ctypes.c_uint64()
    _check(load_library().qnre_prefix_attention_workspace_bytes(q.shape[0], q.shape[1], q.shape[2], cache.k.shape[2],
                                                                q.shape[3], 1 if groups else 0, ctypes.byref(n)),
           "qnre_prefix_attention_workspace_bytes")
    return torch.empty(n.value, dtype=torch.uint8, device=q.device)


def qnre_prefix_attention(q, cache: PagedCache, layer: int, rows, groups, shared, mask, out, lse=None, counts=None,
                          depths=None, scale=None, softcap=0.0, slopes=None, workspace=None, stream=None) -> None:
    """qnre_tree_attention whose groups of rows (groups and shared as qnre_cache_shared_prefix takes and gives them, or None)
    read their common tokens once; scores capped by softcap tanh(s / softcap) where softcap > 0, and biased by
    slopes[h] (pos_key - pos_query) where slopes (fp32 [Hq]) are given (depths: int32 [n, nodes], None for a chain)."""
    where, lib = "qnre_prefix_attention", load_library()
    if _native is not None:
        st = _native.prefix_attention(_entry[where], q, cache.address, cache.k, layer, rows, groups, shared, mask, out, lse,
                                      counts, depths, scale, softcap, slopes, workspace, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    tq = _view4(q)
    n, nodes, heads, dim = _sizes(q)
    to = _same(where, out, q)
    tm = _i64(where, mask, n, nodes)
    if workspace is None:
        raise QnreError(1, f"{where}: workspace is missing (prefix_attention_workspace)")
    if (groups is None) != (shared is None):
        raise QnreError(1, f"{where}: groups and shared go together")
    n_groups = 0 if shared is None else shared.numel()
    args = (tq, cache.handle, layer, _i32(where, rows, n), _i32(where, groups, n_groups + 1), n_groups,
            _i32(where, shared, n_groups), tm, _i32(where, depths, n, nodes), _i32(where, counts, n),
            dim ** -0.5 if scale is None else scale, softcap, None if slopes is None else _f32(where, slopes, heads), to,
            None if lse is None else _f32(where, lse, n, nodes, heads), _contig(workspace, where),
            workspace.numel() * workspace.element_size())
    _on_device(where, q, cache.k, rows, groups, shared, mask, out, lse, counts, depths, slopes, workspace)
    _check(lib.qnre_prefix_attention(*args, _stream_ptr(stream)), where)


def _settings(where: str, n: int, temperature, top_k, top_p, min_p):
    return [None if temperature is None else _f32(where, temperature, n), _i32(where, top_k, n),
            *(None if t is None else _f32(where, t, n) for t in (top_p, min_p))]


def qnre_sample(logits, u, tokens, temperature=None, top_k=None, top_p=None, min_p=None, stream=None) -> None:
    """Draw tokens (int32 [n]) from logits [n, vocab] (bf16, fp16 or fp32, each row contiguous) by the random numbers u
    (fp32 [n]); temperature, top_p and min_p are fp32 [n], top_k int32 [n], None where not used."""
    where, lib = "qnre_sample", load_library()
    if _native is not None:
        st = _native.sample(_entry[where], logits, u, tokens, temperature, top_k, top_p, min_p, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise QnreError(1, f"{where}: logits must be [n, vocab], each row contiguous")
    n, vocab = logits.shape
    code = _dtype_code(logits)
    args = (logits.data_ptr(), logits.stride(0), code, n, vocab, *_settings(where, n, temperature, top_k, top_p, min_p),
            _f32(where, u, n), _i32(where, tokens, n))
    _on_device(where, logits, u, tokens, temperature, top_k, top_p, min_p)
    _check(lib.qnre_sample(*args, _stream_ptr(stream)), where)


def qnre_filter_probs(logits, probs, temperature=None, top_k=None, top_p=None, min_p=None, stream=None) -> None:
    """Probabilities (fp32 [n, nodes, vocab], as qnre_verify_tree takes them) of logits [n, nodes, vocab] under the settings
    of qnre_sample, one set a request."""
    where, lib = "qnre_filter_probs", load_library()
    if _native is not None:
        st = _native.filter(_entry[where], logits, probs, temperature, top_k, top_p, min_p, _stream_ptr, stream)
        if st is not None:
            return _check(st, where)
    if logits.dim() != 3 or (logits.stride(2) != 1 and logits.shape[2] > 1):
        raise QnreError(1, f"{where}: logits must be [n, nodes, vocab], each row contiguous")
    n, nodes, vocab = logits.shape
    code = _dtype_code(logits)
    args = (logits.data_ptr(), logits.stride(0), logits.stride(1), code, n, nodes, vocab,
            *_settings(where, n, temperature, top_k, top_p, min_p), _f32(where, probs, n, nodes, vocab))
    _on_device(where, logits, probs, temperature, top_k, top_p, min_p)
    _check(lib.qnre_filter_probs(*args, _stream_ptr(stream)), where)
