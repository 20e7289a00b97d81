"""Thin ctypes binding of libkvq.so (argument marshalling only).

Every function here forwards to the C entry point of the same name in
``include/kvq.h``; torch tensors are used only to own device memory and to
name the current CUDA stream.  There is no fallback: if ``libkvq.so`` is
missing or the GPU call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import (POINTER, byref, c_double, c_float, c_int, c_int32, c_int64, c_size_t, c_uint8,
                    c_void_p)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

KVQ_OK = 0
KVQ_STATUS_OUTLIER_OVERFLOW = 1
KVQ_STATUS_LEN_OVERFLOW = 2
KVQ_STATUS_NOT_EMPTY = 4
KVQ_STATUS_WAIT_TIMEOUT = 8
KVQ_STATUS_NO_PAGES = 64
KVQ_STATUS_BAD_PAGE = 128
CHUNK = 64
NOALLOC_SCRATCH_BYTES = 1 << 20  # KVQ_NOALLOC_SCRATCH_BYTES

EXPORTS = (
    "kvq_abi_version", "kvq_strerror", "kvq_validate_cfg", "kvq_layout", "kvq_cache_reset",
    "kvq_quantize_workspace", "kvq_quantize_append", "kvq_decode_qk", "kvq_decode_qk_workspace",
    "kvq_decode_splits",
    "kvq_softmax_merge", "kvq_decode_pv", "kvq_decode_workspace", "kvq_decode_attention",
    "kvq_dequantize", "kvq_fp16_decode_attention", "kvq_fit_workspace", "kvq_fit_codebook",
    "kvq_get_status", "kvq_quantize_append_noalloc", "kvq_decode_partial", "kvq_merge_partials",
    "kvq_decode_attention_fused", "kvq_decode_fused_workspace",
    "kvq_step_input_bytes", "kvq_step_workspace", "kvq_step_create", "kvq_step_launch",
    "kvq_step_destroy",
    "kvq_paged_validate_cfg", "kvq_paged_layout", "kvq_paged_reset", "kvq_paged_get_status",
    "kvq_page_plan", "kvq_page_plan_list", "kvq_page_release", "kvq_paged_append",
    "kvq_paged_dequantize", "kvq_paged_attention", "kvq_paged_attention_workspace", "kvq_rope",
)


class KvqError(RuntimeError):
    def __init__(self, code: int, where: str):
        msg = load().kvq_strerror(code).decode()
        super().__init__(f"{where}: {msg} ({code})")
        self.code = code


class Cfg(ctypes.Structure):
    _fields_ = [("B", c_int32), ("Hq", c_int32), ("Hkv", c_int32), ("D", c_int32),
                ("bits", c_int32), ("T_max", c_int32), ("out_cap_k", c_int32),
                ("out_cap_v", c_int32), ("outlier_frac", c_double), ("rope_theta", c_double)]


_CACHE_FIELDS = ("kcodes", "vcodes", "kthr", "kparams", "vparams", "kout", "vout", "kchunk",
                 "vchunk", "kcount", "vcount", "len", "status")


class CacheStruct(ctypes.Structure):
    _fields_ = [(f, c_void_p) for f in _CACHE_FIELDS]


class CodebookStruct(ctypes.Structure):
    _fields_ = [("levels", c_void_p), ("bounds", c_void_p)]


class Sizes(ctypes.Structure):
    _fields_ = [(f, c_size_t) for f in _CACHE_FIELDS]


class StepDesc(ctypes.Structure):
    _fields_ = [("layers", c_int32), ("caches", POINTER(CacheStruct)),
                ("cbK", POINTER(CodebookStruct)), ("cbV", POINTER(CodebookStruct)),
                ("n_new", c_int32), ("max_len", c_int32), ("splits", c_int32), ("fused", c_int32),
                ("inputs", c_void_p), ("out", c_void_p), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t)]


class PagedCfg(ctypes.Structure):
    _fields_ = [(f, c_int32) for f in ("Hq", "Hkv", "D", "page_tokens", "num_pages", "max_pages",
                                       "dtype", "k_exp", "v_exp")]


class PagedStruct(ctypes.Structure):
    _fields_ = [("pool", c_void_p), ("status", c_void_p)]


class RopeCfg(ctypes.Structure):
    _fields_ = [(f, c_int32) for f in ("Hq", "Hkv", "D", "rot_dim", "dtype", "adjacent", "axes")]
    _fields_ += [("pair_axis", c_uint8 * 128)]
    py = None  # kept by make_rope_cfg


_lib = None


def load():
    """Load libkvq.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with "
                          "`python -m long_context_decode_nuq_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = c_void_p
    sig = {
        "kvq_abi_version": ([], c_int),
        "kvq_strerror": ([c_int], ctypes.c_char_p),
        "kvq_validate_cfg": ([POINTER(Cfg)], c_int),
        "kvq_layout": ([POINTER(Cfg), POINTER(Sizes)], c_int),
        "kvq_cache_reset": ([POINTER(Cfg), POINTER(CacheStruct), P], c_int),
        "kvq_quantize_workspace": ([POINTER(Cfg), c_int32, c_int32, POINTER(c_size_t)], c_int),
        "kvq_quantize_append": ([POINTER(Cfg), POINTER(CacheStruct), POINTER(CodebookStruct),
                                 POINTER(CodebookStruct), P, P, c_int32, P, c_int32, P, c_size_t,
                                 P], c_int),
        "kvq_decode_qk": ([POINTER(Cfg), POINTER(CacheStruct), POINTER(CodebookStruct), P, P,
                           c_int32, P, P, c_int32, P, c_size_t, P], c_int),
        "kvq_decode_qk_workspace": ([POINTER(Cfg), c_int32, POINTER(c_size_t)], c_int),
        "kvq_decode_splits": ([POINTER(Cfg), c_int32], c_int),
        "kvq_softmax_merge": ([POINTER(Cfg), P, c_int32, P, P], c_int),
        "kvq_decode_pv": ([POINTER(Cfg), POINTER(CacheStruct), POINTER(CodebookStruct), P, P,
                           c_int32, P, P, c_int32, P], c_int),
        "kvq_decode_workspace": ([POINTER(Cfg), c_int32, c_int32, POINTER(c_size_t)], c_int),
        "kvq_decode_attention": ([POINTER(Cfg), POINTER(CacheStruct), POINTER(CodebookStruct),
                                  POINTER(CodebookStruct), P, P, c_int32, P, P, c_size_t,
                                  c_int32, P], c_int),
        "kvq_dequantize": ([POINTER(Cfg), POINTER(CacheStruct), POINTER(CodebookStruct),
                            POINTER(CodebookStruct), c_int32, c_int32, P, P, P], c_int),
        "kvq_fp16_decode_attention": ([POINTER(Cfg), P, P, c_int32, P, P, P, c_int32, P, P,
                                       c_size_t, c_int32, P], c_int),
        "kvq_fit_workspace": ([c_int32, c_int32, POINTER(c_size_t)], c_int),
        "kvq_fit_codebook": ([P, c_int32, c_int32, c_double, P, c_int32, c_int32, P, P, P,
                              c_size_t, P], c_int),
        "kvq_get_status": ([POINTER(CacheStruct), POINTER(c_int32), P], c_int),
        "kvq_decode_partial": ([POINTER(Cfg), POINTER(CacheStruct), POINTER(CodebookStruct),
                                POINTER(CodebookStruct), P, P, c_int32, c_int32, P, P, P,
                                c_size_t, c_int32, P], c_int),
        "kvq_merge_partials": ([POINTER(Cfg), c_int32, P, P, P, P], c_int),
        "kvq_decode_attention_fused": ([POINTER(Cfg), POINTER(CacheStruct),
                                        POINTER(CodebookStruct), POINTER(CodebookStruct), P, P,
                                        c_int32, P, P, c_size_t, c_int32, P], c_int),
        "kvq_decode_fused_workspace": ([POINTER(Cfg), c_int32, c_int32, POINTER(c_size_t)],
                                       c_int),
        "kvq_quantize_append_noalloc": ([POINTER(Cfg), POINTER(CacheStruct),
                                         POINTER(CodebookStruct), POINTER(CodebookStruct), P, P,
                                         c_int32, P, P], c_int),
        "kvq_step_input_bytes": ([POINTER(Cfg), c_int32, c_int32, POINTER(c_size_t)], c_int),
        "kvq_step_workspace": ([POINTER(Cfg), c_int32, c_int32, c_int32, c_int32,
                                POINTER(c_size_t)], c_int),
        "kvq_step_create": ([POINTER(Cfg), POINTER(StepDesc), POINTER(c_void_p)], c_int),
        "kvq_step_launch": ([P, P, P], c_int),
        "kvq_step_destroy": ([P], c_int),
        "kvq_paged_validate_cfg": ([P], c_int),
        "kvq_paged_layout": ([P, POINTER(c_size_t)], c_int),
        "kvq_paged_reset": ([P, P], c_int),
        "kvq_paged_get_status": ([P, POINTER(c_int32), P], c_int),
        "kvq_page_plan": ([P, P, c_int32, P, P, P, P, P, c_int32, P, P, P, P, P, P], c_int),
        "kvq_page_plan_list": ([P, P, c_int32, P, P, P, P, c_int32, P, c_int32, P, P, P, P, P, P],
                               c_int),
        "kvq_page_release": ([P, P, c_int32, P, P, P, P, P, P], c_int),
        "kvq_paged_append": ([P, P, P, c_int64, P, c_int64, P, c_int32, P], c_int),
        "kvq_paged_dequantize": ([P, P, P, c_int32, P, P, P], c_int),
        "kvq_paged_attention": ([P, P, P, c_int64, P, c_int32, c_int32, P, P, c_int32, c_int32,
                                 c_float, c_int32, P, P, P, c_size_t, c_int32, P], c_int),
        "kvq_paged_attention_workspace": ([P, c_int32, c_int32, c_int32, c_int32, c_int32,
                                           POINTER(c_size_t)], c_int),
        "kvq_rope": ([P, P, c_int64, P, c_int64, P, P, c_int32, c_int32, P, c_int64, P, c_int64,
                      P], c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(code: int, where: str) -> None:
    if code != KVQ_OK:
        raise KvqError(code, where)


def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return c_void_p(s.cuda_stream)


def make_cfg(B, Hq, Hkv, bits, T_max, outlier_frac, rope_theta, out_cap_k, out_cap_v, D=128):
    return Cfg(B, Hq, Hkv, D, bits, T_max, out_cap_k, out_cap_v, float(outlier_frac),
               float(rope_theta))


def kvq_abi_version() -> int:
    return load().kvq_abi_version()


def kvq_validate_cfg(cfg: Cfg) -> int:
    return load().kvq_validate_cfg(ctypes.byref(cfg))


def kvq_layout(cfg: Cfg) -> dict:
    s = Sizes()
    _check(load().kvq_layout(ctypes.byref(cfg), ctypes.byref(s)), "kvq_layout")
    return {f: getattr(s, f) for f in _CACHE_FIELDS}


class Cache:
    """Device arrays of one layer's cache, allocated with torch per kvq_layout."""

    def __init__(self, cfg: Cfg, device="cuda"):
        import torch
        self.cfg = cfg
        sz = kvq_layout(cfg)
        n = cfg.Hkv * cfg.D
        BW = 16 * cfg.bits                      # words of a 4-token code block
        nq = (cfg.T_max + 3) // 4
        nch = (cfg.T_max + CHUNK - 1) // CHUNK + 1
        dev = torch.device(device)
        i32, f32, f16 = torch.int32, torch.float32, torch.float16
        self.kcodes = torch.zeros((cfg.B, cfg.Hkv, nq, BW), dtype=i32, device=dev)
        self.vcodes = torch.zeros((cfg.B, cfg.Hkv, nq, BW), dtype=i32, device=dev)
        self.kthr = torch.zeros((cfg.B, n, 2), dtype=f16, device=dev)
        self.kparams = torch.zeros((cfg.B, n, 2), dtype=f32, device=dev)
        self.vparams = torch.zeros((cfg.B, cfg.T_max, 2), dtype=f32, device=dev)
        H = cfg.Hkv  # one outlier list per (sequence, kv head)
        self.kout = torch.zeros((cfg.B, H, max(cfg.out_cap_k, 8)), dtype=i32, device=dev)
        self.vout = torch.zeros((cfg.B, H, max(cfg.out_cap_v, 8)), dtype=i32, device=dev)
        self.kchunk = torch.zeros((cfg.B, H, nch), dtype=i32, device=dev)
        self.vchunk = torch.zeros((cfg.B, H, nch), dtype=i32, device=dev)
        self.kcount = torch.zeros((cfg.B, H), dtype=i32, device=dev)
        self.vcount = torch.zeros((cfg.B, H), dtype=i32, device=dev)
        self.len = torch.zeros((cfg.B,), dtype=i32, device=dev)
        self.status = torch.zeros((4,), dtype=i32, device=dev)
        for f in _CACHE_FIELDS:
            assert getattr(self, f).numel() * getattr(self, f).element_size() >= sz[f], f
        self.struct = CacheStruct(*[getattr(self, f).data_ptr() for f in _CACHE_FIELDS])

    def nbytes(self) -> int:
        return sum(getattr(self, f).numel() * getattr(self, f).element_size()
                   for f in _CACHE_FIELDS)


class Codebook:
    """A per-layer NUQ datatype on the device (levels, bounds as float32 tensors)."""

    def __init__(self, levels, bounds):
        self.levels = levels
        self.bounds = bounds
        self.struct = CodebookStruct(levels.data_ptr(), bounds.data_ptr())


def kvq_cache_reset(cache: Cache, stream=None) -> None:
    _check(load().kvq_cache_reset(ctypes.byref(cache.cfg), ctypes.byref(cache.struct),
                                  _stream(stream)), "kvq_cache_reset")


def kvq_quantize_workspace(cfg: Cfg, n_new: int, calibrate: int) -> int:
    b = c_size_t()
    _check(load().kvq_quantize_workspace(ctypes.byref(cfg), n_new, calibrate, ctypes.byref(b)),
           "kvq_quantize_workspace")
    return b.value


def kvq_quantize_append(cache: Cache, cbK: Codebook, cbV: Codebook, k, v, n_new: int, plen,
                        calibrate: int, workspace, stream=None) -> None:
    _check(load().kvq_quantize_append(
        ctypes.byref(cache.cfg), ctypes.byref(cache.struct), ctypes.byref(cbK.struct),
        ctypes.byref(cbV.struct), _ptr(k), _ptr(v), n_new, _ptr(plen), calibrate,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
        "kvq_quantize_append")


def kvq_decode_splits(cfg: Cfg, max_len: int) -> int:
    return load().kvq_decode_splits(ctypes.byref(cfg), max_len)


def kvq_decode_qk_workspace(cfg: Cfg, max_len: int) -> int:
    n = c_size_t()
    _check(load().kvq_decode_qk_workspace(ctypes.byref(cfg), max_len, ctypes.byref(n)),
           "kvq_decode_qk_workspace")
    return n.value


def kvq_decode_qk(cache: Cache, cbK: Codebook, q, qpos, max_len: int, logits, stats, splits: int,
                  workspace, stream=None) -> None:
    _check(load().kvq_decode_qk(ctypes.byref(cache.cfg), ctypes.byref(cache.struct),
                                ctypes.byref(cbK.struct), _ptr(q), _ptr(qpos), max_len,
                                _ptr(logits), _ptr(stats), splits, _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)),
           "kvq_decode_qk")


def kvq_softmax_merge(cfg: Cfg, stats, splits: int, ml, stream=None) -> None:
    _check(load().kvq_softmax_merge(ctypes.byref(cfg), _ptr(stats), splits, _ptr(ml),
                                    _stream(stream)), "kvq_softmax_merge")


def kvq_decode_pv(cache: Cache, cbV: Codebook, logits, ml, max_len: int, out, part, splits: int,
                  stream=None) -> None:
    _check(load().kvq_decode_pv(ctypes.byref(cache.cfg), ctypes.byref(cache.struct),
                                ctypes.byref(cbV.struct), _ptr(logits), _ptr(ml), max_len,
                                _ptr(out), _ptr(part), splits, _stream(stream)), "kvq_decode_pv")


def kvq_decode_workspace(cfg: Cfg, max_len: int, splits: int) -> int:
    b = c_size_t()
    _check(load().kvq_decode_workspace(ctypes.byref(cfg), max_len, splits, ctypes.byref(b)),
           "kvq_decode_workspace")
    return b.value


def kvq_decode_attention(cache: Cache, cbK: Codebook, cbV: Codebook, q, qpos, max_len: int, out,
                         workspace, splits: int = 0, stream=None) -> None:
    _check(load().kvq_decode_attention(
        ctypes.byref(cache.cfg), ctypes.byref(cache.struct), ctypes.byref(cbK.struct),
        ctypes.byref(cbV.struct), _ptr(q), _ptr(qpos), max_len, _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), splits, _stream(stream)),
        "kvq_decode_attention")


def kvq_decode_fused_workspace(cfg: Cfg, max_len: int, splits: int) -> int:
    b = c_size_t()
    _check(load().kvq_decode_fused_workspace(ctypes.byref(cfg), max_len, splits, ctypes.byref(b)),
           "kvq_decode_fused_workspace")
    return b.value


def kvq_decode_attention_fused(cache: Cache, cbK: Codebook, cbV: Codebook, q, qpos, max_len: int,
                               out, workspace, splits: int = 0, stream=None) -> None:
    _check(load().kvq_decode_attention_fused(
        ctypes.byref(cache.cfg), ctypes.byref(cache.struct), ctypes.byref(cbK.struct),
        ctypes.byref(cbV.struct), _ptr(q), _ptr(qpos), max_len, _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), splits, _stream(stream)),
        "kvq_decode_attention_fused")


def kvq_decode_partial(cache: Cache, cbK: Codebook, cbV: Codebook, q, qpos, max_len: int,
                       pos_offset: int, ml, o, workspace, splits: int = 0, stream=None) -> None:
    _check(load().kvq_decode_partial(
        ctypes.byref(cache.cfg), ctypes.byref(cache.struct), ctypes.byref(cbK.struct),
        ctypes.byref(cbV.struct), _ptr(q), _ptr(qpos), max_len, pos_offset, _ptr(ml), _ptr(o),
        _ptr(workspace), workspace.numel() * workspace.element_size(), splits, _stream(stream)),
        "kvq_decode_partial")


def kvq_merge_partials(cfg: Cfg, parts: int, ml, o, out, stream=None) -> None:
    _check(load().kvq_merge_partials(ctypes.byref(cfg), parts, _ptr(ml), _ptr(o), _ptr(out),
                                     _stream(stream)), "kvq_merge_partials")


def kvq_dequantize(cache: Cache, cbK: Codebook, cbV: Codebook, t0: int, nt: int, khat, vhat,
                   stream=None) -> None:
    _check(load().kvq_dequantize(ctypes.byref(cache.cfg), ctypes.byref(cache.struct),
                                 ctypes.byref(cbK.struct), ctypes.byref(cbV.struct), t0, nt,
                                 _ptr(khat), _ptr(vhat), _stream(stream)), "kvq_dequantize")


def kvq_fp16_decode_attention(cfg: Cfg, K, V, T_stride: int, lens, q, qpos, max_len: int, out,
                              workspace, splits: int = 0, stream=None) -> None:
    _check(load().kvq_fp16_decode_attention(
        ctypes.byref(cfg), _ptr(K), _ptr(V), T_stride, _ptr(lens), _ptr(q), _ptr(qpos), max_len,
        _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(), splits,
        _stream(stream)), "kvq_fp16_decode_attention")


def kvq_fit_workspace(n_vec: int, vec_len: int) -> int:
    b = c_size_t()
    _check(load().kvq_fit_workspace(n_vec, vec_len, ctypes.byref(b)), "kvq_fit_workspace")
    return b.value


def kvq_fit_codebook(samples, f: float, bits: int, levels, bounds, workspace, weights=None,
                     max_iter: int = 100, stream=None) -> None:
    n_vec, vec_len = samples.shape
    _check(load().kvq_fit_codebook(_ptr(samples), n_vec, vec_len, float(f), _ptr(weights), bits,
                                   max_iter, _ptr(levels), _ptr(bounds), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
           "kvq_fit_codebook")


def kvq_quantize_append_noalloc(cache: Cache, cbK: Codebook, cbV: Codebook, k, v, n_new: int,
                                plen=None, stream=None) -> None:
    """Append without a workspace: the library's own fixed device scratch is used instead."""
    _check(load().kvq_quantize_append_noalloc(
        ctypes.byref(cache.cfg), ctypes.byref(cache.struct), ctypes.byref(cbK.struct),
        ctypes.byref(cbV.struct), _ptr(k), _ptr(v), n_new, _ptr(plen), _stream(stream)),
        "kvq_quantize_append_noalloc")


def kvq_step_input_bytes(cfg: Cfg, layers: int, n_new: int) -> int:
    b = c_size_t()
    _check(load().kvq_step_input_bytes(ctypes.byref(cfg), layers, n_new, ctypes.byref(b)),
           "kvq_step_input_bytes")
    return b.value


def kvq_step_workspace(cfg: Cfg, n_new: int, max_len: int, splits: int = 0,
                       fused: int = 0) -> int:
    b = c_size_t()
    _check(load().kvq_step_workspace(ctypes.byref(cfg), n_new, max_len, splits, fused,
                                     ctypes.byref(b)), "kvq_step_workspace")
    return b.value


class Step:
    """Handle of a recorded whole-model step (kvq_step_create); keeps its buffers alive."""

    def __init__(self, handle, keep):
        self.handle = handle
        self._keep = keep

    def destroy(self) -> None:
        if self.handle:
            _check(load().kvq_step_destroy(self.handle), "kvq_step_destroy")
            self.handle = None


def kvq_step_create(cfg: Cfg, caches, cbK, cbV, n_new: int, max_len: int, inputs, out,
                    workspace, splits: int = 0, fused: int = 0) -> Step:
    """caches, cbK, cbV: one Cache / Codebook per layer, in layer order."""
    L = len(caches)
    if len(cbK) != L or len(cbV) != L:
        raise ValueError(f"kvq_step_create: {L} caches but {len(cbK)} key and {len(cbV)} value "
                         "codebooks")
    carr = (CacheStruct * L)(*[c.struct for c in caches])
    karr = (CodebookStruct * L)(*[c.struct for c in cbK])
    varr = (CodebookStruct * L)(*[c.struct for c in cbV])
    desc = StepDesc(L, carr, karr, varr, n_new, max_len, splits, fused, inputs.data_ptr(),
                    out.data_ptr(), workspace.data_ptr(),
                    workspace.numel() * workspace.element_size())
    h = c_void_p()
    _check(load().kvq_step_create(ctypes.byref(cfg), ctypes.byref(desc), ctypes.byref(h)),
           "kvq_step_create")
    return Step(h, (inputs, out, workspace, list(caches), list(cbK), list(cbV)))


def kvq_step_launch(step: Step, inputs=None, stream=None) -> None:
    """inputs: a packed input record (host or device tensor), or None if already in place."""
    _check(load().kvq_step_launch(step.handle, _ptr(inputs), _stream(stream)),
           "kvq_step_launch")


def kvq_step_destroy(step: Step) -> None:
    step.destroy()


def kvq_get_status(cache: Cache, stream=None) -> int:
    out = c_int32()
    _check(load().kvq_get_status(ctypes.byref(cache.struct), ctypes.byref(out), _stream(stream)),
           "kvq_get_status")
    return out.value


# ------------------------------------------------------------------------- paged 4-bit cache
# These calls check what a pointer cannot say -- types, shapes, strides, devices -- and raise
# ValueError; they launch on the tensors' device, on `stream` or that device's current stream.

def _dtype_code(dtype) -> int:
    import torch
    code = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}.get(dtype)
    if code is None:
        raise ValueError(f"dtype {dtype} is not float16, bfloat16 or float32")
    return code


def _int32(where, *sizes) -> None:
    """ctypes cuts an int to 32 bits without a word."""
    if max(sizes) > 0x7fffffff or min(sizes) < -0x80000000:
        raise ValueError(f"{where}: {sizes} do not fit 32 bits")


def make_paged_cfg(Hq, Hkv, D, page_tokens, num_pages, max_pages, dtype, k_exp=0,
                   v_exp=0) -> PagedCfg:
    """dtype: torch.float16 or torch.bfloat16.  Raises KvqError where the library refuses it."""
    _int32("make_paged_cfg", Hq, Hkv, D, page_tokens, num_pages, max_pages, k_exp, v_exp)
    cfg = PagedCfg(Hq, Hkv, D, page_tokens, num_pages, max_pages, _dtype_code(dtype), k_exp, v_exp)
    _check(load().kvq_paged_validate_cfg(byref(cfg)), "kvq_paged_validate_cfg")
    return cfg


def kvq_paged_validate_cfg(cfg: PagedCfg) -> int:
    return load().kvq_paged_validate_cfg(byref(cfg))


def kvq_paged_layout(cfg: PagedCfg) -> int:
    """Bytes of the pool."""
    n = c_size_t()
    _check(load().kvq_paged_layout(byref(cfg), byref(n)), "kvq_paged_layout")
    return n.value


class PagedCache:
    """The pool of a paged 4-bit cache and its status word (one layer; the block tables, free list
    and lengths belong to the requests and are shared by all layers)."""

    def __init__(self, cfg: PagedCfg, device="cuda", pool=None):
        torch = _torch()
        self.cfg = cfg
        n = kvq_paged_layout(cfg)
        if pool is None:
            pool = torch.empty(n, dtype=torch.uint8, device=device)
        elif pool.dtype != torch.uint8 or pool.numel() < n or not pool.is_contiguous():
            raise ValueError(f"PagedCache: the pool is a contiguous uint8 tensor of {n} bytes")
        self.pool = pool
        self.status = torch.zeros(1, dtype=torch.int32, device=pool.device)
        self.device = pool.device
        self.index = pool.get_device()
        self.dtype = torch.bfloat16 if cfg.dtype else torch.float16
        self.struct = PagedStruct(pool.data_ptr(), self.status.data_ptr())
        self.args = byref(cfg), byref(self.struct)
        self.q_row, self.kv_row, self.width = (cfg.Hq, cfg.D), (cfg.Hkv, cfg.D), cfg.max_pages

    def nbytes(self) -> int:
        return self.pool.numel()


_i32 = _f32 = _f64 = _raw_stream = _current = None


def _torch():
    """torch, and the names that the calls below need every time (a call costs a few microseconds
    of host time, as much as the smallest kernels take)."""
    global _i32, _f32, _f64, _raw_stream, _current
    import torch
    if _i32 is None:
        _raw_stream, _current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        _i32, _f32, _f64 = torch.int32, torch.float32, torch.float64
    return torch


def _call(where, fn, i, stream, *args):
    """fn(*args, stream) on the device of number i (-1: host memory)."""
    if i < 0:
        raise ValueError(f"{where}: the tensors are not on a CUDA device")
    s = _raw_stream(i) if stream is None else stream.cuda_stream
    if _current() == i:
        code = fn(*args, s)
    else:
        with _torch().cuda.device(i):
            code = fn(*args, s)
    if code != KVQ_OK:
        raise KvqError(code, where)


def _ints(where, i, *tensors):
    for t in tensors:
        if t.dtype is not _i32 or t.get_device() != i or not t.is_contiguous():
            raise ValueError(f"{where}: {tuple(t.shape)} {t.dtype} on {t.device} is not a contiguous "
                             "int32 tensor on the call's device")


def _rows(where, name, t, shape, dtype, i):
    """A [n, heads, D] tensor whose rows may lie apart; its row stride."""
    if t.dtype is not dtype or t.get_device() != i or t.shape != shape:
        raise ValueError(f"{where}: {name} is {tuple(t.shape)} {t.dtype} on {t.device}, not "
                         f"{shape} {dtype} on the call's device")
    n, heads, d = shape
    if t.is_contiguous():
        return heads * d
    row, head, one = t.stride()
    if (one != 1 and d > 1) or (head != d and heads > 1):
        raise ValueError(f"{where}: {name}'s heads and channels are not contiguous")
    return row if n > 1 else heads * d


def kvq_paged_reset(cache: PagedCache, stream=None) -> None:
    _call("kvq_paged_reset", load().kvq_paged_reset, cache.index, stream, cache.args[1])


def kvq_paged_get_status(cache: PagedCache, stream=None) -> int:
    out = c_int32()

    def read(s):
        return load().kvq_paged_get_status(cache.args[1], byref(out), s)

    _call("kvq_paged_get_status", read, cache.index, stream)
    return out.value


def _table(where, cache, table, B):
    _ints(where, cache.index, table)
    if table.shape != (B, cache.width):
        raise ValueError(f"{where}: block_table is {tuple(table.shape)}, not {(B, cache.width)}")


def kvq_page_plan(cache: PagedCache, lens, n_new, block_table, free_pages, n_free, cu_new, len_out,
                  n_free_out, slots, positions, stream=None) -> None:
    """n_free counts as at most the entries of free_pages (kvq_page_plan_list)."""
    w, B, cap = "kvq_page_plan", lens.numel(), slots.numel()
    _ints(w, cache.index, lens, n_new, free_pages, n_free, cu_new, len_out, n_free_out, slots,
          positions)
    _table(w, cache, block_table, B)
    if (n_new.numel() != B or cu_new.numel() != B + 1 or len_out.numel() != B
            or n_free.numel() != 1 or n_free_out.numel() != 1 or positions.numel() != cap):
        raise ValueError(f"{w}: sizes do not agree with {B} requests and {cap} tokens")
    _call(w, load().kvq_page_plan_list, cache.index, stream, *cache.args, B, lens.data_ptr(),
          n_new.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(), free_pages.numel(),
          n_free.data_ptr(), cap, cu_new.data_ptr(), len_out.data_ptr(), n_free_out.data_ptr(),
          slots.data_ptr(), positions.data_ptr())


def kvq_page_release(cache: PagedCache, lens, done, block_table, free_pages, n_free,
                     stream=None) -> None:
    w, B = "kvq_page_release", lens.numel()
    _ints(w, cache.index, lens, done, free_pages, n_free)
    _table(w, cache, block_table, B)
    if done.numel() != B or n_free.numel() != 1 or free_pages.numel() < cache.cfg.num_pages:
        raise ValueError(f"{w}: sizes do not agree with {B} requests and {cache.cfg.num_pages} pages")
    _call(w, load().kvq_page_release, cache.index, stream, *cache.args, B, lens.data_ptr(),
          done.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(), n_free.data_ptr())


def kvq_paged_append(cache: PagedCache, k, v, slots, stream=None) -> None:
    w, i, n = "kvq_paged_append", cache.index, slots.numel()
    _ints(w, i, slots)
    shape = n, *cache.kv_row
    ks, vs = _rows(w, "k", k, shape, cache.dtype, i), _rows(w, "v", v, shape, cache.dtype, i)
    _call(w, load().kvq_paged_append, i, stream, *cache.args, k.data_ptr(), ks, v.data_ptr(), vs,
          slots.data_ptr(), n)


def kvq_paged_dequantize(cache: PagedCache, slots, khat, vhat, stream=None) -> None:
    w, i, n = "kvq_paged_dequantize", cache.index, slots.numel()
    _ints(w, i, slots)
    shape = n, *cache.kv_row
    _rows(w, "khat", khat, shape, cache.dtype, i)
    _rows(w, "vhat", vhat, shape, cache.dtype, i)
    if not (khat.is_contiguous() and vhat.is_contiguous()):
        raise ValueError(f"{w}: an output is not contiguous")
    _call(w, load().kvq_paged_dequantize, i, stream, *cache.args, slots.data_ptr(), n,
          khat.data_ptr(), vhat.data_ptr())


def kvq_paged_attention_workspace(cfg: PagedCfg, B: int, total_q: int, max_q: int, max_len: int,
                                  splits: int = 0) -> int:
    _int32("kvq_paged_attention_workspace", B, total_q, max_q, max_len, splits)
    n = c_size_t()
    _check(load().kvq_paged_attention_workspace(byref(cfg), B, total_q, max_q, max_len, splits,
                                                byref(n)), "kvq_paged_attention_workspace")
    return n.value


def kvq_paged_attention(cache: PagedCache, q, cu_q, lens, block_table, max_q: int, max_len: int,
                        sm_scale: float, out, workspace=None, window: int = 0, lse=None,
                        splits: int = 0, stream=None) -> None:
    """cu_q: int32 [B + 1], or None for one query per request."""
    w, i, B, n = "kvq_paged_attention", cache.index, lens.numel(), q.shape[0]
    _ints(w, i, lens)
    if (max_q | max_len | window | splits) >> 31:  # one of them negative or past 31 bits
        _int32(w, max_q, max_len, window, splits)
    _table(w, cache, block_table, B)
    shape = n, *cache.q_row
    qs = _rows(w, "q", q, shape, cache.dtype, i)
    _rows(w, "out", out, shape, cache.dtype, i)
    if not out.is_contiguous():
        raise ValueError(f"{w}: out is not contiguous")
    cu = l = ws = None
    wb = 0
    if cu_q is not None:
        _ints(w, i, cu_q)
        if cu_q.numel() != B + 1:
            raise ValueError(f"{w}: cu_q has {cu_q.numel()} entries for {B} requests")
        cu = cu_q.data_ptr()
    if lse is not None:
        if (lse.dtype is not _f32 or lse.get_device() != i or lse.shape != shape[:2]
                or not lse.is_contiguous()):
            raise ValueError(f"{w}: lse is a contiguous float32 tensor {shape[:2]} on q's device")
        l = lse.data_ptr()
    if workspace is not None:
        if workspace.get_device() != i or not workspace.is_contiguous():
            raise ValueError(f"{w}: the workspace is a contiguous tensor on q's device")
        ws, wb = workspace.data_ptr(), workspace.nbytes
    _call(w, load().kvq_paged_attention, i, stream, *cache.args, q.data_ptr(), qs, cu, B, n,
          lens.data_ptr(), block_table.data_ptr(), max_q, max_len, sm_scale, window,
          out.data_ptr(), l, ws, wb, splits)


def make_rope_cfg(Hq, Hkv, D, rot_dim, pair_axis, dtype, adjacent=False) -> RopeCfg:
    """pair_axis: the axis (0, 1, ...) of each of the rot_dim/2 pairs, as a list.  The result is
    not to be changed."""
    axes = [int(x) for x in pair_axis]
    if len(axes) != rot_dim // 2 or len(axes) > 128 or min(axes, default=-1) < 0 or max(axes) > 7:
        raise ValueError(f"make_rope_cfg: pair_axis names an axis (0 .. 7) for each of the "
                         f"{rot_dim // 2} pairs")
    _int32("make_rope_cfg", Hq, Hkv, D, rot_dim)
    cfg = RopeCfg(Hq, Hkv, D, rot_dim, _dtype_code(dtype), int(bool(adjacent)), max(axes) + 1,
                  (c_uint8 * 128)(*axes))
    cfg.py = _rope_shape(cfg)
    return cfg


def _rope_shape(cfg: RopeCfg):
    """What kvq_rope checks the tensors against."""
    torch = _torch()
    dtypes = torch.float16, torch.bfloat16, torch.float32
    if not 0 <= cfg.dtype < len(dtypes):
        raise ValueError(f"RopeCfg: dtype {cfg.dtype} is not float16, bfloat16 or float32's (0 .. 2)")
    return cfg.Hq, cfg.Hkv, cfg.D, cfg.axes, cfg.rot_dim // 2, dtypes[cfg.dtype]


def kvq_rope(cfg: RopeCfg, q, k, positions, freqs, q_out, k_out, inverse=False,
             stream=None) -> None:
    """q, k [n, heads, D] (k may be None when cfg.Hkv is 0), positions int32 [axes, n], freqs
    float64 [rot_dim / 2]; q_out and k_out may be q and k."""
    w, n, i = "kvq_rope", q.shape[0], q.get_device()
    Hq, Hkv, d, axes, half, dtype = cfg.py or _rope_shape(cfg)
    _ints(w, i, positions)
    if positions.shape != (axes, n) and not (axes == 1 and positions.numel() == n):
        raise ValueError(f"{w}: positions is {tuple(positions.shape)}, not {(axes, n)}")
    if (freqs.dtype is not _f64 or freqs.numel() != half or freqs.get_device() != i
            or not freqs.is_contiguous()):
        raise ValueError(f"{w}: freqs is a float64 tensor of {half} on q's device")
    shape = n, Hq, d
    qs, qos = _rows(w, "q", q, shape, dtype, i), _rows(w, "q_out", q_out, shape, dtype, i)
    kp = kop = None
    ks = kos = 0
    if Hkv:
        shape = n, Hkv, d
        ks, kos = _rows(w, "k", k, shape, dtype, i), _rows(w, "k_out", k_out, shape, dtype, i)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    _call(w, load().kvq_rope, i, stream, byref(cfg), q.data_ptr(), qs, kp, ks,
          positions.data_ptr(), freqs.data_ptr(), n, int(inverse), q_out.data_ptr(), qos, kop, kos)
