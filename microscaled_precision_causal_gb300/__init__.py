"""GB300 (sm_103a) FLAMIA attention: thin Python binding of libflamia.

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libflamia.so`` (built in-tree by ``build.py``).  PyTorch supplies device
memory and streams.  If the library is missing, every call raises -- there is
no CPU fallback.

The functions mirror the C ABI in ``include/flamia.h``:
``flamia_plan_bytes``, ``flamia_plan_build``, ``flamia_quantize_tokenblock``,
``flamia_fwd``, ``flamia_bwd_workspace_bytes``, ``flamia_bwd``,
``flamia_get_device_status``; ``FlamiaAttention`` strings them into the
training call (quantize Q/K/V, forward, backward).  ``flamia_scored_fwd``,
``flamia_scored_bwd``, ``flamia_relbias_expand`` and ``flamia_relbias_reduce``
are the bf16 attention calls with changed scores (tanh cap, distance bias,
bucketed relative bias, prefix); ``FlamiaScoredAttention`` strings those.
``flamia_cache_plan_build``, ``flamia_cache_write``, ``flamia_cache_read`` and
``flamia_cached_fwd`` keep keys and values in pages (E4M3 or bf16) and attend to
them; ``FlamiaPagedCache`` holds the pages, ``FlamiaCachedAttention`` a step's calls.
"""
from __future__ import annotations

import ctypes
import operator
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libflamia.so")

FLAMIA_OK = 0
STATUS_NAMES = {0: "ok", -1: "invalid argument", -2: "unsupported", -3: "misaligned", -4: "workspace", -5: "cuda"}
DEV_BAD_CU_SEQLENS, DEV_TIMEOUT, DEV_CAPACITY = 1, 2, 4
DEV_BAD_KV_LENS, DEV_BAD_PAGE, DEV_PLAN_MISMATCH = 8, 16, 32

EXPORTED = (
    "flamia_default_options", "flamia_plan_bytes", "flamia_plan_build", "flamia_quantize_tokenblock",
    "flamia_fwd", "flamia_bwd_workspace_bytes", "flamia_bwd", "flamia_get_device_status",
    "flamia_status_string", "flamia_bwd_static_scratch", "flamia_quantize_nvfp4", "flamia_plan_build_window",
    "flamia_quantize_hadamard", "flamia_quantize_qkv", "flamia_default_score_options", "flamia_scored_fwd",
    "flamia_scored_bwd_workspace_bytes", "flamia_scored_bwd", "flamia_relbias_expand", "flamia_relbias_reduce",
    "flamia_cache_plan_bytes", "flamia_cache_plan_build", "flamia_cache_write", "flamia_cache_read",
    "flamia_cached_fwd_workspace_bytes", "flamia_cached_fwd",
)
STATIC_SCRATCH_BYTES = 64 << 20
REL_MAX = 1024
CACHE_FORMATS = {"bf16": 0, "e4m3": 1}
PAGE_SIZES = (16, 32, 64, 128)


class FlamiaError(RuntimeError):
    pass


class Options(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "p_boost_log2", "bwd_p_boost_log2", "dq_headroom_log2", "strict_per_token", "strict_row_ds",
        "strict_causal_dq", "mixed_nvfp4", "deterministic")] + [("timing_events", ctypes.POINTER(ctypes.c_void_p)),
                                                                 ("mixed", ctypes.c_void_p),
                                                                 ("debug_p_ds", ctypes.c_void_p),
                                                                 ("window_left", ctypes.c_int),
                                                                 ("window_right", ctypes.c_int),
                                                                 ("rotate", ctypes.c_int),
                                                                 ("dynamic_schedule", ctypes.c_int)]


class QTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("stats", ctypes.c_void_p)]


class MixedOperands(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q_codes_e2m1", "q_scales_e4m3", "k_codes_e2m1", "k_scales_e4m3",
                                               "v_tok_codes", "v_tok_scales")]


class ScoreOptions(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("rel_bias", ctypes.c_void_p),
                ("rel_max", ctypes.c_int), ("prefix_lens", ctypes.c_void_p), ("window_left", ctypes.c_int),
                ("window_right", ctypes.c_int)]


class KVCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scales", "v_scales")] + [
        (n, ctypes.c_int) for n in ("num_pages", "page_size", "hkv", "head_dim", "format")]


_lib = None


def lib():
    """Load libflamia.so (raises FlamiaError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FlamiaError(f"{LIB_PATH} is missing: build it with microscaled_precision_causal_gb300.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    f32 = ctypes.c_float
    qp = ctypes.POINTER(QTensor)
    sp = ctypes.POINTER(ScoreOptions)
    op = ctypes.POINTER(Options)
    cp = ctypes.POINTER(KVCache)
    sig = {
        "flamia_default_options": (None, [op]),
        "flamia_plan_bytes": (sz, [i64, i32]),
        "flamia_plan_build": (i32, [vp, i32, i64, vp, sz, vp]),
        "flamia_plan_build_window": (i32, [vp, i32, i64, i32, i32, i32, vp, sz, vp]),
        "flamia_quantize_tokenblock": (i32, [vp, i64, i32, i32, vp, i32, vp, i32, vp, vp, vp, vp]),
        "flamia_fwd": (i32, [qp, qp, qp, vp, i32, i64, i32, i32, i32, i32, f32, op, vp, vp, vp, vp]),
        "flamia_bwd_workspace_bytes": (sz, [i64, i32, i32, i32, i32]),
        "flamia_bwd": (i32, [qp, qp, qp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, f32, op, vp, vp, vp, vp, vp,
                             sz, vp]),
        "flamia_bwd_static_scratch": (i32, [qp, qp, qp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, f32, op, vp,
                                            vp, vp, vp, vp]),
        "flamia_get_device_status": (i32, [vp, ctypes.POINTER(ctypes.c_int), vp]),
        "flamia_status_string": (ctypes.c_char_p, [i32]),
        "flamia_quantize_nvfp4": (i32, [vp, i64, i32, i32, vp, vp, vp]),
        "flamia_quantize_hadamard": (i32, [vp, i64, i32, i32, vp, i32, vp, vp, vp, vp, vp]),
        "flamia_quantize_qkv": (i32, [vp, vp, vp, i64, i32, i32, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                      vp]),
        "flamia_default_score_options": (None, [sp]),
        "flamia_scored_fwd": (i32, [vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, f32, sp, vp, vp, vp, vp]),
        "flamia_scored_bwd_workspace_bytes": (sz, [i64, i32, i32, i32, i32, i32]),
        "flamia_scored_bwd": (i32, [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, f32, sp, vp, vp, vp, vp,
                                    vp, vp, sz, vp]),
        "flamia_relbias_expand": (i32, [vp, i32, i32, i32, i32, vp, i32, vp]),
        "flamia_relbias_reduce": (i32, [vp, i32, i32, i32, i32, i32, vp, vp]),
        "flamia_cache_plan_bytes": (sz, [i64, i32, i32, i32]),
        "flamia_cache_plan_build": (i32, [vp, vp, i32, i64, i32, i32, i32, i64, i32, vp, sz, vp]),
        "flamia_cache_write": (i32, [cp, vp, i32, i32, i64, vp, vp, vp, vp]),
        "flamia_cache_read": (i32, [cp, vp, i32, i32, i64, vp, vp, vp, vp]),
        "flamia_cached_fwd_workspace_bytes": (sz, [i32, i32, i32, i32]),
        "flamia_cached_fwd": (i32, [vp, cp, vp, i32, i32, i64, i32, i32, i32, f32, f32, vp, vp, vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != FLAMIA_OK:
        raise FlamiaError(f"{what}: {lib().flamia_status_string(rc).decode()} ({rc})")


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def default_options() -> Options:
    o = Options()
    lib().flamia_default_options(ctypes.byref(o))
    return o


def qtensor(codes, scales, stats=None) -> QTensor:
    return QTensor(_ptr(codes), _ptr(scales), _ptr(stats))


# ---------------------------------------------------------------- C ABI mirrors

def flamia_plan_bytes(total_tokens: int, num_seqs: int) -> int:
    return int(lib().flamia_plan_bytes(total_tokens, num_seqs))


def flamia_plan_build(cu_seqlens, num_seqs: int, total_tokens: int, plan, stream=None):
    _check(lib().flamia_plan_build(_ptr(cu_seqlens), num_seqs, total_tokens, _ptr(plan), plan.numel() * plan.element_size(),
                                   _stream(stream)), "flamia_plan_build")


def flamia_plan_build_window(cu_seqlens, num_seqs: int, total_tokens: int, causal: int, window_left: int,
                             window_right: int, plan, stream=None):
    _check(lib().flamia_plan_build_window(_ptr(cu_seqlens), num_seqs, total_tokens, int(causal), window_left,
                                          window_right, _ptr(plan), plan.numel() * plan.element_size(),
                                          _stream(stream)), "flamia_plan_build_window")


def flamia_quantize_tokenblock(x, cu_seqlens, num_seqs: int, plan, codes, scales, stats=None, per_token: bool = False,
                               stream=None):
    T, H, d = x.shape
    _check(lib().flamia_quantize_tokenblock(_ptr(x), T, H, d, _ptr(cu_seqlens), num_seqs, _ptr(plan), int(per_token),
                                            _ptr(codes), _ptr(scales), _ptr(stats), _stream(stream)),
           "flamia_quantize_tokenblock")


def flamia_quantize_qkv(q, k, v, cu_seqlens, num_seqs: int, plan, q_codes, q_scales, k_codes, k_scales, k_stats,
                        v_codes, v_scales, v_stats, per_token: bool = False, stream=None):
    T, hq, d = q.shape
    hkv = k.shape[1]
    _check(lib().flamia_quantize_qkv(_ptr(q), _ptr(k), _ptr(v), T, hq, hkv, d, _ptr(cu_seqlens), num_seqs, _ptr(plan),
                                     int(per_token), _ptr(q_codes), _ptr(q_scales), _ptr(k_codes), _ptr(k_scales),
                                     _ptr(k_stats), _ptr(v_codes), _ptr(v_scales), _ptr(v_stats), _stream(stream)),
           "flamia_quantize_qkv")


def flamia_quantize_hadamard(x, cu_seqlens, num_seqs: int, plan, codes, scales, stats=None, stream=None):
    T, H, d = x.shape
    _check(lib().flamia_quantize_hadamard(_ptr(x), T, H, d, _ptr(cu_seqlens), num_seqs, _ptr(plan), _ptr(codes),
                                          _ptr(scales), _ptr(stats), _stream(stream)), "flamia_quantize_hadamard")


def flamia_quantize_nvfp4(x, codes, scales, stream=None):
    T, H, d = x.shape
    _check(lib().flamia_quantize_nvfp4(_ptr(x), T, H, d, _ptr(codes), _ptr(scales), _stream(stream)),
           "flamia_quantize_nvfp4")


def flamia_fwd(q: QTensor, k: QTensor, v: QTensor, cu_seqlens, num_seqs: int, total_tokens: int, hq: int, hkv: int,
               head_dim: int, plan, out, lse, softmax_scale: float = 0.0, opts: Optional[Options] = None,
               causal: int = 1, stream=None):
    _check(lib().flamia_fwd(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), _ptr(cu_seqlens), num_seqs, total_tokens,
                            hq, hkv, head_dim, causal, softmax_scale, ctypes.byref(opts) if opts else None, _ptr(plan),
                            _ptr(out), _ptr(lse), _stream(stream)), "flamia_fwd")


def flamia_bwd_workspace_bytes(total_tokens: int, num_seqs: int, hq: int, hkv: int, head_dim: int) -> int:
    return int(lib().flamia_bwd_workspace_bytes(total_tokens, num_seqs, hq, hkv, head_dim))


def flamia_bwd(q: QTensor, k: QTensor, v: QTensor, out, lse, dout, cu_seqlens, num_seqs: int, total_tokens: int,
               hq: int, hkv: int, head_dim: int, plan, dq, dk, dv, workspace, softmax_scale: float = 0.0,
               opts: Optional[Options] = None, causal: int = 1, stream=None):
    _check(lib().flamia_bwd(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), _ptr(out), _ptr(lse), _ptr(dout),
                            _ptr(cu_seqlens), num_seqs, total_tokens, hq, hkv, head_dim, causal, softmax_scale,
                            ctypes.byref(opts) if opts else None, _ptr(plan), _ptr(dq), _ptr(dk), _ptr(dv),
                            _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
           "flamia_bwd")


def flamia_bwd_static_scratch(q: QTensor, k: QTensor, v: QTensor, out, lse, dout, cu_seqlens, num_seqs: int,
                              total_tokens: int, hq: int, hkv: int, head_dim: int, plan, dq, dk, dv,
                              softmax_scale: float = 0.0, opts: Optional[Options] = None, causal: int = 1,
                              stream=None):
    """flamia_bwd without a workspace argument, for callers that cannot allocate
    device memory: the scratch is the library's static device array
    (STATIC_SCRATCH_BYTES per GPU).  The first call on a device must come before
    any stream capture; calls that overlap on the GPU race on the shared array."""
    _check(lib().flamia_bwd_static_scratch(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), _ptr(out), _ptr(lse),
                                           _ptr(dout), _ptr(cu_seqlens), num_seqs, total_tokens, hq, hkv, head_dim,
                                           causal, softmax_scale, ctypes.byref(opts) if opts else None, _ptr(plan),
                                           _ptr(dq), _ptr(dk), _ptr(dv), _stream(stream)),
           "flamia_bwd_static_scratch")


def default_score_options() -> ScoreOptions:
    o = ScoreOptions()
    lib().flamia_default_score_options(ctypes.byref(o))
    return o


def flamia_scored_fwd(q, k, v, cu_seqlens, num_seqs: int, plan, out, lse, softmax_scale: float = 0.0,
                      opts: Optional[ScoreOptions] = None, causal: int = 1, stream=None):
    T, hq, d = q.shape
    _check(lib().flamia_scored_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), num_seqs, T, hq, k.shape[1], d, causal,
                                   softmax_scale, ctypes.byref(opts) if opts else None, _ptr(plan), _ptr(out), _ptr(lse),
                                   _stream(stream)), "flamia_scored_fwd")


def flamia_scored_bwd_workspace_bytes(total_tokens: int, num_seqs: int, hq: int, hkv: int, head_dim: int,
                                      rel_max: int = 0) -> int:
    return int(lib().flamia_scored_bwd_workspace_bytes(total_tokens, num_seqs, hq, hkv, head_dim, rel_max))


def flamia_scored_bwd(q, k, v, out, lse, dout, cu_seqlens, num_seqs: int, plan, dq, dk, dv, workspace, drel_bias=None,
                      softmax_scale: float = 0.0, opts: Optional[ScoreOptions] = None, causal: int = 1, stream=None):
    T, hq, d = q.shape
    _check(lib().flamia_scored_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(cu_seqlens),
                                   num_seqs, T, hq, k.shape[1], d, causal, softmax_scale,
                                   ctypes.byref(opts) if opts else None, _ptr(plan), _ptr(dq), _ptr(dk), _ptr(dv),
                                   _ptr(drel_bias), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "flamia_scored_bwd")


def _rel_max(rel, table) -> int:
    """The width 2 rel_max + 1 says how far the kernels go, in as many rows as the table has heads."""
    if rel.dim() != 2 or table.dim() != 2 or rel.shape[1] % 2 == 0 or rel.shape[0] != table.shape[1]:
        raise FlamiaError(f"relative bias: want [{table.shape[-1]}, 2 rel_max + 1], got {tuple(rel.shape)}")
    return rel.shape[1] // 2


def flamia_relbias_expand(table, max_distance: int, bidirectional: bool, rel_bias, stream=None):
    """table: float [buckets, hq]; rel_bias: float [hq, 2 rel_max + 1] (written)."""
    _check(lib().flamia_relbias_expand(_ptr(table), table.shape[0], table.shape[1], max_distance, int(bidirectional),
                                       _ptr(rel_bias), _rel_max(rel_bias, table), _stream(stream)),
           "flamia_relbias_expand")


def flamia_relbias_reduce(drel_bias, max_distance: int, bidirectional: bool, dtable, stream=None):
    """drel_bias: float [hq, 2 rel_max + 1]; dtable: float [buckets, hq] (written)."""
    _check(lib().flamia_relbias_reduce(_ptr(drel_bias), _rel_max(drel_bias, dtable), dtable.shape[0], dtable.shape[1],
                                       max_distance, int(bidirectional), _ptr(dtable), _stream(stream)),
           "flamia_relbias_reduce")


def flamia_cache_plan_bytes(total_tokens: int, num_seqs: int, hq: int, hkv: int) -> int:
    return int(lib().flamia_cache_plan_bytes(total_tokens, num_seqs, hq, hkv))


def flamia_cache_plan_build(cu_seqlens, kv_lens, num_seqs: int, total_tokens: int, hq: int, hkv: int, max_chunk: int,
                            max_keys: int, window_left: int, plan, stream=None):
    _check(lib().flamia_cache_plan_build(_ptr(cu_seqlens), _ptr(kv_lens), num_seqs, total_tokens, hq, hkv, max_chunk,
                                         max_keys, window_left, _ptr(plan), plan.numel() * plan.element_size(),
                                         _stream(stream)), "flamia_cache_plan_build")


def flamia_cache_write(cache: KVCache, page_table, num_seqs: int, plan, k, v, stream=None):
    _check(lib().flamia_cache_write(ctypes.byref(cache), _ptr(page_table), page_table.shape[1], num_seqs, k.shape[0],
                                    _ptr(plan), _ptr(k), _ptr(v), _stream(stream)), "flamia_cache_write")


def flamia_cache_read(cache: KVCache, page_table, num_seqs: int, plan, k, v, stream=None):
    """k and v: bf16 [T, hkv, head_dim] (written)."""
    _check(lib().flamia_cache_read(ctypes.byref(cache), _ptr(page_table), page_table.shape[1], num_seqs, k.shape[0],
                                   _ptr(plan), _ptr(k), _ptr(v), _stream(stream)), "flamia_cache_read")


def flamia_cached_fwd_workspace_bytes(hq: int, hkv: int, head_dim: int, max_chunk: int) -> int:
    return int(lib().flamia_cached_fwd_workspace_bytes(hq, hkv, head_dim, max_chunk))


def flamia_cached_fwd(q, cache: KVCache, page_table, num_seqs: int, plan, out, lse, workspace, max_chunk: int,
                      window_left: int = -1, softcap: float = 0.0, softmax_scale: float = 0.0, stream=None):
    _check(lib().flamia_cached_fwd(_ptr(q), ctypes.byref(cache), _ptr(page_table), page_table.shape[1], num_seqs, q.shape[0],
                                   q.shape[1], max_chunk, window_left, softcap, softmax_scale, _ptr(plan), _ptr(out),
                                   _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "flamia_cached_fwd")


def flamia_get_device_status(plan, stream=None) -> int:
    st = ctypes.c_int(0)
    _check(lib().flamia_get_device_status(_ptr(plan), ctypes.byref(st), _stream(stream)), "flamia_get_device_status")
    return st.value


# ---------------------------------------------------------------- training call

class FlamiaAttention:
    """Buffers and calls for one packed attention layout.

    All tensors live on one CUDA device; the object owns the plan, the
    quantized Q/K/V views and the backward workspace (allocated once through
    torch, reused across calls: nothing is allocated per call).  causal=False
    gives attention over the whole document; window = (left, right) limits the
    visible keys to i - left <= j <= i + right (-1: no limit; causal calls use
    right = 0).  dynamic_schedule=True makes the causal MXFP8 forward acquire
    its work through cluster launch control instead of the static order (same
    results)."""

    def __init__(self, total_tokens: int, num_seqs: int, hq: int, hkv: int, head_dim: int, device="cuda",
                 strict: bool = False, mixed: bool = False, causal: bool = True, window=(-1, -1),
                 rotate: bool = False, dynamic_schedule: bool = False):
        import torch
        self.T, self.N, self.hq, self.hkv, self.d = total_tokens, num_seqs, hq, hkv, head_dim
        self.causal = 1 if causal else 0
        self.window = (int(window[0]), int(window[1]))
        self.device = torch.device(device)
        dev = self.device
        u8 = torch.uint8
        self.plan = torch.empty(flamia_plan_bytes(total_tokens, num_seqs), dtype=u8, device=dev)
        self.q_codes = torch.empty(total_tokens, hq, head_dim, dtype=u8, device=dev)
        self.q_scales = torch.empty(total_tokens, hq, dtype=u8, device=dev)
        self.k_codes = torch.empty(total_tokens, hkv, head_dim, dtype=u8, device=dev)
        self.k_scales = torch.empty(total_tokens, hkv, dtype=u8, device=dev)
        self.k_stats = torch.empty(total_tokens, hkv, 2, dtype=torch.float32, device=dev)
        self.v_codes = torch.empty(total_tokens, hkv, head_dim, dtype=u8, device=dev)
        self.v_scales = torch.empty(total_tokens, hkv, dtype=u8, device=dev)
        self.v_stats = torch.empty(total_tokens, hkv, 2, dtype=torch.float32, device=dev)
        self.out = torch.empty(total_tokens, hq, head_dim, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(hq, total_tokens, dtype=torch.float32, device=dev)
        self.dq = torch.empty(total_tokens, hq, head_dim, dtype=torch.bfloat16, device=dev)
        self.dk = torch.empty(total_tokens, hkv, head_dim, dtype=torch.bfloat16, device=dev)
        self.dv = torch.empty(total_tokens, hkv, head_dim, dtype=torch.bfloat16, device=dev)
        ws = flamia_bwd_workspace_bytes(total_tokens, num_seqs, hq, hkv, head_dim)
        self.workspace = torch.empty(ws, dtype=u8, device=dev)
        self.opts = default_options()
        self.opts.window_left, self.opts.window_right = self.window
        self.rotate = bool(rotate)      # Q and K rotated by the Hadamard map before quantization
        self.opts.rotate = int(self.rotate)
        self.opts.dynamic_schedule = int(bool(dynamic_schedule))
        self.strict = bool(strict)
        if self.strict:   # per-token operand scales, per-query-row dS exponents, causal dQ boost, deterministic dQ
            for f in ("strict_per_token", "strict_row_ds", "strict_causal_dq", "deterministic"):
                setattr(self.opts, f, 1)
        self.mixed = bool(mixed)
        if self.mixed:    # NVFP4 score operands, per-token V copy for the diagonal key tiles
            T = total_tokens
            self.q4_codes = torch.empty(T, hq, head_dim // 2, dtype=u8, device=dev)
            self.q4_scales = torch.empty(T, hq, head_dim // 16, dtype=u8, device=dev)
            self.k4_codes = torch.empty(T, hkv, head_dim // 2, dtype=u8, device=dev)
            self.k4_scales = torch.empty(T, hkv, head_dim // 16, dtype=u8, device=dev)
            self.vt_codes = torch.empty(T, hkv, head_dim, dtype=u8, device=dev)
            self.vt_scales = torch.empty(T, hkv, dtype=u8, device=dev)
            self._mixed_ops = MixedOperands(_ptr(self.q4_codes), _ptr(self.q4_scales), _ptr(self.k4_codes),
                                            _ptr(self.k4_scales), _ptr(self.vt_codes), _ptr(self.vt_scales))
            self.opts.mixed_nvfp4 = 1
            self.opts.mixed = ctypes.cast(ctypes.pointer(self._mixed_ops), ctypes.c_void_p)

    def views(self):
        return (qtensor(self.q_codes, self.q_scales), qtensor(self.k_codes, self.k_scales, self.k_stats),
                qtensor(self.v_codes, self.v_scales, self.v_stats))

    def plan_build(self, cu_seqlens, stream=None):
        if self.causal and self.window[0] < 0:
            flamia_plan_build(cu_seqlens, self.N, self.T, self.plan, stream)
        else:
            flamia_plan_build_window(cu_seqlens, self.N, self.T, self.causal, self.window[0], self.window[1], self.plan,
                                     stream)

    def quantize(self, q, k, v, cu_seqlens, stream=None):
        pt = self.strict
        if self.rotate:
            flamia_quantize_hadamard(q, cu_seqlens, self.N, self.plan, self.q_codes, self.q_scales, None, stream)
            flamia_quantize_hadamard(k, cu_seqlens, self.N, self.plan, self.k_codes, self.k_scales, self.k_stats,
                                     stream)
            flamia_quantize_tokenblock(v, cu_seqlens, self.N, self.plan, self.v_codes, self.v_scales, self.v_stats, pt,
                                       stream)
        else:             # Q, K and V in one launch
            flamia_quantize_qkv(q, k, v, cu_seqlens, self.N, self.plan, self.q_codes, self.q_scales, self.k_codes,
                                self.k_scales, self.k_stats, self.v_codes, self.v_scales, self.v_stats, pt, stream)
        if self.mixed:
            flamia_quantize_nvfp4(q, self.q4_codes, self.q4_scales, stream)
            flamia_quantize_nvfp4(k, self.k4_codes, self.k4_scales, stream)
            flamia_quantize_tokenblock(v, cu_seqlens, self.N, self.plan, self.vt_codes, self.vt_scales, None, True,
                                       stream)

    def forward(self, cu_seqlens, softmax_scale: float = 0.0, stream=None):
        q, k, v = self.views()
        flamia_fwd(q, k, v, cu_seqlens, self.N, self.T, self.hq, self.hkv, self.d, self.plan, self.out, self.lse,
                   softmax_scale, self.opts, causal=self.causal, stream=stream)
        return self.out, self.lse

    def backward(self, dout, cu_seqlens, softmax_scale: float = 0.0, stream=None):
        q, k, v = self.views()
        flamia_bwd(q, k, v, self.out, self.lse, dout, cu_seqlens, self.N, self.T, self.hq, self.hkv, self.d, self.plan,
                   self.dq, self.dk, self.dv, self.workspace, softmax_scale, self.opts, causal=self.causal,
                   stream=stream)
        return self.dq, self.dk, self.dv

    def training_call(self, q, k, v, dout, cu_seqlens, softmax_scale: float = 0.0, stream=None, build_plan=True):
        """Plan (optional), quantize Q/K/V, forward and backward: one pass of the hot path."""
        if build_plan:
            self.plan_build(cu_seqlens, stream)
        self.quantize(q, k, v, cu_seqlens, stream)
        self.forward(cu_seqlens, softmax_scale, stream)
        return self.backward(dout, cu_seqlens, softmax_scale, stream)

    def device_status(self, stream=None) -> int:
        return flamia_get_device_status(self.plan, stream)

    def bwd_dvec(self):
        """View into the backward workspace: D = rowsum(dO^ o O), float [hq, T], of the last backward call."""
        import torch
        T, H, d = self.T, self.hq, self.d
        rnd = lambda x: (x + 255) // 256 * 256
        off = rnd(rnd(rnd(T * H * d) + T * H) + T * H * 8)
        return self.workspace[off:off + T * H * 4].view(torch.float32).view(H, T)

    def bwd_dout_codes(self):
        """Views into the backward workspace: (dO codes, dO scale bytes) of the last backward call."""
        import torch
        T, H, d = self.T, self.hq, self.d
        rnd = lambda x: (x + 255) // 256 * 256
        n_codes = T * H * d
        codes = self.workspace[:n_codes].view(T, H, d)
        off = rnd(n_codes)
        scales = self.workspace[off:off + T * H].view(T, H)
        return codes, scales


class FlamiaScoredAttention:
    """Buffers and calls of attention with changed scores for one packed layout.

    The bf16 counterpart of FlamiaAttention for layers whose scores are capped by
    a tanh (softcap > 0), fall with the distance (slopes, given per call), get a
    learned relative position bias by buckets (buckets = (number of buckets,
    max_distance, bidirectional), the table given per call) or see a prefix of
    their document whatever the mask (prefix_lens, given per call).  causal and
    window as in FlamiaAttention.

    The object owns the plan, the outputs and the backward workspace; each call
    overwrites the tensors that the last one returned.  Nothing is allocated per
    call, so calls can be captured into a CUDA graph.  Tensors are contiguous, on
    the object's device: q [T, hq, d], k and v [T, hkv, d] bf16; cu_seqlens
    [N + 1] and prefix_lens [N] int32; slopes [hq] and table [buckets, hq] fp32.
    Anything else raises FlamiaError.  Calls run on `stream`, by default the
    object's device's current stream.  Calls of one object share its bias table and
    workspace, forwards too: calls on two streams have to be ordered by the caller
    (an object each lets them overlap).

    The documents of a call are those of the last plan_build (which has to come
    first): forward and backward take cu_seqlens as every call here does, but read
    the plan."""

    def __init__(self, total_tokens: int, num_seqs: int, hq: int, hkv: int, head_dim: int, device="cuda",
                 causal: bool = True, window=(-1, -1), softcap: float = 0.0, buckets=None):
        import torch
        if total_tokens < 0 or num_seqs < 0 or hq <= 0 or hkv <= 0 or hq % hkv or head_dim not in (64, 128):
            raise FlamiaError(f"FlamiaScoredAttention: sizes {(total_tokens, num_seqs, hq, hkv, head_dim)} are not supported")
        self.T, self.N, self.hq, self.hkv, self.d = total_tokens, num_seqs, hq, hkv, head_dim
        self.causal = 1 if causal else 0
        self.window = tuple(max(-1, min(int(x), 2**31 - 1)) for x in window)     # (a bound of T or more is none)
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        dev = self.device
        self.opts = default_score_options()
        self.opts.softcap = float(softcap)
        self.opts.window_left, self.opts.window_right = self.window
        self.rel_max = 0
        f32, bf16 = torch.float32, torch.bfloat16
        if buckets is not None:
            self.num_buckets, self.max_distance, both = int(buckets[0]), int(buckets[1]), bool(buckets[2])
            side = self.num_buckets // 2 if both else self.num_buckets
            if side < 2 or (both and self.num_buckets % 2) or not side // 2 < self.max_distance <= REL_MAX:
                raise FlamiaError(f"FlamiaScoredAttention: buckets {tuple(buckets)} are not supported")
            self.bidirectional = both
            self.rel_max = self.max_distance
            self.rel_bias = torch.empty(hq, 2 * self.rel_max + 1, dtype=f32, device=dev)
            self.drel_bias = torch.empty_like(self.rel_bias)
            self.dtable = torch.empty(self.num_buckets, hq, dtype=f32, device=dev)
        # zeros: a plan without documents, should a captured plan_build not have been replayed yet
        self.plan = torch.zeros(flamia_plan_bytes(total_tokens, num_seqs), dtype=torch.uint8, device=dev)
        self._planned = False
        self.out = torch.empty(total_tokens, hq, head_dim, dtype=bf16, device=dev)
        self.lse = torch.empty(hq, total_tokens, dtype=f32, device=dev)
        self.dq = torch.empty_like(self.out)
        self.dk = torch.empty(total_tokens, hkv, head_dim, dtype=bf16, device=dev)
        self.dv = torch.empty_like(self.dk)
        ws = flamia_scored_bwd_workspace_bytes(total_tokens, num_seqs, hq, hkv, head_dim, self.rel_max)
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev)

    def _want(self, name, t, shape, dtype):
        if t.dtype != dtype or t.shape != shape or t.device != self.device or not t.is_contiguous():
            raise FlamiaError(f"{name}: want contiguous {dtype} {shape} on {self.device}, got {t.dtype} {tuple(t.shape)} "
                              f"on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")

    def _options(self, cu_seqlens, slopes, prefix_lens, table):
        import torch
        self._want("cu_seqlens", cu_seqlens, (self.N + 1,), torch.int32)
        o = ScoreOptions.from_buffer_copy(self.opts)
        if slopes is not None:
            self._want("slopes", slopes, (self.hq,), torch.float32)
            o.slopes = slopes.data_ptr()
        if prefix_lens is not None:
            self._want("prefix_lens", prefix_lens, (self.N,), torch.int32)
            o.prefix_lens = prefix_lens.data_ptr()
        if (table is not None) != (self.rel_max > 0):
            raise FlamiaError("table: given to an object without buckets" if self.rel_max == 0 else
                              "table: an object with buckets needs one")
        if table is not None:
            self._want("table", table, (self.num_buckets, self.hq), torch.float32)
            o.rel_bias, o.rel_max = self.rel_bias.data_ptr(), self.rel_max
        return o

    def _inputs(self, q, k, v):
        import torch
        self._want("q", q, (self.T, self.hq, self.d), torch.bfloat16)
        self._want("k", k, (self.T, self.hkv, self.d), torch.bfloat16)
        self._want("v", v, (self.T, self.hkv, self.d), torch.bfloat16)

    def _run(self, call, stream):
        """call(stream handle) with the object's device current, on `stream` or its current stream."""
        import torch
        if self.device.type != "cuda":
            raise FlamiaError(f"{type(self).__name__} runs on a CUDA device, not on {self.device}")
        index = self.device.index
        if torch._C._cuda_getDevice() != index:
            with torch.cuda.device(self.device):
                return call(_stream(stream))
        if stream is None:             # the common case without the Python objects behind it: a small call is host-bound
            stream = torch._C._cuda_getCurrentRawStream(index)
        return call(_stream(stream))

    def plan_build(self, cu_seqlens, stream=None):
        import torch
        self._want("cu_seqlens", cu_seqlens, (self.N + 1,), torch.int32)
        self._run(lambda stm: flamia_plan_build_window(cu_seqlens, self.N, self.T, self.causal, self.window[0],
                                                       self.window[1], self.plan, stm), stream)
        self._planned = True

    def _need_plan(self):
        if not self._planned:
            raise FlamiaError("FlamiaScoredAttention: plan_build has not been called")

    def forward(self, q, k, v, cu_seqlens, softmax_scale: float = 0.0, slopes=None, prefix_lens=None, table=None,
                stream=None):
        """(out bf16 [T, hq, d], lse fp32 [hq, T])."""
        self._inputs(q, k, v)
        o = self._options(cu_seqlens, slopes, prefix_lens, table)

        def call(stm):
            self._need_plan()
            if table is not None:
                flamia_relbias_expand(table, self.max_distance, self.bidirectional, self.rel_bias, stm)
            flamia_scored_fwd(q, k, v, cu_seqlens, self.N, self.plan, self.out, self.lse, softmax_scale, o, self.causal,
                              stm)
            return self.out, self.lse
        return self._run(call, stream)

    def backward(self, q, k, v, out, lse, dout, cu_seqlens, softmax_scale: float = 0.0, slopes=None, prefix_lens=None,
                 table=None, stream=None):
        """(dq, dk, dv) in bf16 and, with a table, its gradient in fp32.  out and lse: what forward returned for
        these inputs."""
        import torch
        self._inputs(q, k, v)
        self._want("out", out, (self.T, self.hq, self.d), torch.bfloat16)
        self._want("dout", dout, (self.T, self.hq, self.d), torch.bfloat16)
        self._want("lse", lse, (self.hq, self.T), torch.float32)
        o = self._options(cu_seqlens, slopes, prefix_lens, table)

        def call(stm):
            self._need_plan()
            if table is not None:
                flamia_relbias_expand(table, self.max_distance, self.bidirectional, self.rel_bias, stm)
            flamia_scored_bwd(q, k, v, out, lse, dout, cu_seqlens, self.N, self.plan, self.dq, self.dk, self.dv,
                              self.workspace, self.drel_bias if table is not None else None, softmax_scale, o,
                              self.causal, stm)
            if table is None:
                return self.dq, self.dk, self.dv
            flamia_relbias_reduce(self.drel_bias, self.max_distance, self.bidirectional, self.dtable, stm)
            return self.dq, self.dk, self.dv, self.dtable
        return self._run(call, stream)

    def device_status(self, stream=None) -> int:
        return self._run(lambda stm: flamia_get_device_status(self.plan, stm), stream)


# ---------------------------------------------------------------- generation

def _cuda_device(device):
    import torch
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def _kept(name: str, align: int = 16):
    """A tensor that an object's calls read or write.  Another one takes its place by assignment, and the calls go there from
    then on: contiguous, of the same type, shape and device, aligned to `align` bytes.  Anything else raises FlamiaError."""
    slot = "_" + name

    def assign(self, t):
        old = getattr(self, slot, t)
        if t is not old:
            if old is None or t is None:
                raise FlamiaError(f"{name}: {'there is none in this format' if old is None else 'want a tensor'}")
            if (t.dtype != old.dtype or t.shape != old.shape or t.device != old.device or not t.is_contiguous()
                    or t.data_ptr() % align):
                raise FlamiaError(f"{name}: want contiguous {old.dtype} {tuple(old.shape)} on {old.device}, aligned to {align} bytes, "
                                  f"got {t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")
        setattr(self, slot, t)
        self._moved(name, t)

    # (read as often as a step has calls: without a Python function)
    return property(operator.attrgetter(slot), assign)


class FlamiaPagedCache:
    """The pages of one layer's keys and values.

    k and v are [num_pages, hkv, page_size, head_dim], uint8 E4M3 codes with
    k_scales and v_scales [num_pages, hkv, page_size] (uint8 UE8M0 exponents, one
    a token and head) for fmt "e4m3", bf16 and no scales for "bf16".  They start
    as zeros.  Which page holds which positions is the caller's page table.

    The calls go to these tensors' memory.  Contents are replaced with copy_, or by
    assigning another tensor of the same kind; a captured graph stays with the one
    that it was captured with.  Changes of a tensor's own memory (set_, resize_,
    .data) are not followed."""

    k, v, k_scales, v_scales = (_kept(name) for name in ("k", "v", "k_scales", "v_scales"))

    def __init__(self, num_pages: int, page_size: int, hkv: int, head_dim: int, fmt: str = "e4m3", device="cuda"):
        import torch
        if num_pages < 1 or page_size not in PAGE_SIZES or hkv < 1 or head_dim not in (64, 128) or fmt not in CACHE_FORMATS:
            raise FlamiaError(f"FlamiaPagedCache: {(num_pages, page_size, hkv, head_dim, fmt)} is not supported")
        self.num_pages, self.page_size, self.hkv, self.d, self.fmt = num_pages, page_size, hkv, head_dim, fmt
        self.device = _cuda_device(device)
        # what the calls get
        self.view = KVCache(None, None, None, None, num_pages, page_size, hkv, head_dim, CACHE_FORMATS[fmt])
        self.ref = ctypes.pointer(self.view)
        shape = (num_pages, hkv, page_size, head_dim)
        if fmt == "e4m3":
            self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=self.device) for _ in range(2))
            self.k_scales, self.v_scales = (torch.zeros(shape[:3], dtype=torch.uint8, device=self.device) for _ in range(2))
        else:
            self.k, self.v = (torch.zeros(shape, dtype=torch.bfloat16, device=self.device) for _ in range(2))
            self.k_scales = self.v_scales = None
        self.kind = (page_size, hkv, head_dim, self.device)

    def _moved(self, name, t):
        setattr(self.view, name, _ptr(t))


class FlamiaCachedAttention:
    """A step of generation over paged caches: its plan, its writes and its attention.

    A step serves num_seqs sequences with up to total_tokens new tokens, packed;
    sequence n brings cu_seqlens[n + 1] - cu_seqlens[n] <= max_chunk of them (one
    in plain generation, a few that were drafted, a chunk of a prompt, or none)
    and has kv_lens[n] keys with them.  plan_build(cu_seqlens, kv_lens) comes
    first; one plan serves every layer's cache:

        att.plan_build(cu_seqlens, kv_lens)
        for layer in layers:
            att.write(layer.cache, k, v, page_table)
            out, lse = att.forward(layer.cache, q, page_table)

    window: keys up to so many positions before a token's own are seen (-1: all;
    pages wholly before that may be given back); softcap as in
    FlamiaScoredAttention.  read(cache, page_table, k, v) puts the
    step's tokens back into k and v (with kv_lens the chunks themselves: whole
    sequences).

    Tensors are contiguous, on the object's device: q [T, hq, d], k and v [T,
    hkv, d] bf16; cu_seqlens [N + 1], kv_lens [N] and page_table [N, max_pages]
    int32.  Anything else raises FlamiaError.  Errors that the device finds (bad
    lengths, a page outside the cache) show in device_status().  forward returns
    the object's own out and lse, overwritten by its next call.  Nothing is
    allocated per call, so calls can be captured into a CUDA graph: a replay reads
    what the tensors hold by then.  Calls run on `stream`, by default the object's
    device's current stream; calls of one object share its plan, outputs and
    workspace, so calls on two streams have to be ordered by the caller.  plan, out,
    lse and workspace may be assigned as a cache's tensors may."""

    plan, out, lse, workspace = _kept("plan"), _kept("out"), _kept("lse", 4), _kept("workspace", 256)

    def __init__(self, total_tokens: int, num_seqs: int, hq: int, hkv: int, head_dim: int, max_chunk: int,
                 max_pages: int, page_size: int, device="cuda", window: int = -1, softcap: float = 0.0):
        import torch
        if (total_tokens < 0 or num_seqs < 0 or hq <= 0 or hkv <= 0 or hq % hkv or head_dim not in (64, 128) or max_chunk < 1
                or max_pages < 1 or page_size not in PAGE_SIZES or max_pages * page_size > 1 << 30):
            raise FlamiaError("FlamiaCachedAttention: sizes "
                              f"{(total_tokens, num_seqs, hq, hkv, head_dim, max_chunk, max_pages, page_size)} are not supported")
        self.T, self.N, self.hq, self.hkv, self.d = total_tokens, num_seqs, hq, hkv, head_dim
        self.max_chunk, self.max_pages, self.page_size = int(max_chunk), int(max_pages), page_size
        self.window = max(-1, min(int(window), 2**31 - 1))
        self.softcap = float(softcap)
        self.device = _cuda_device(device)
        dev = self.device
        # zeros: a plan of no call, should a captured plan_build not have been replayed yet
        self.plan = torch.zeros(flamia_cache_plan_bytes(total_tokens, num_seqs, hq, hkv), dtype=torch.uint8, device=dev)
        self._planned = False
        self.out = torch.empty(total_tokens, hq, head_dim, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(hq, total_tokens, dtype=torch.float32, device=dev)
        self._ws_bytes = flamia_cached_fwd_workspace_bytes(hq, hkv, head_dim, self.max_chunk)
        self.workspace = torch.empty(self._ws_bytes, dtype=torch.uint8, device=dev)
        # a step's calls are many and small: what does not change is worked out once
        self._lib, self._bf16, self._i32 = lib(), torch.bfloat16, torch.int32
        self._index = dev.index if dev.type == "cuda" else None
        self._device_now, self._stream_now = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self._kind = (page_size, hkv, head_dim, dev)
        self._q_shape, self._kv_shape = (total_tokens, hq, head_dim), (total_tokens, hkv, head_dim)
        self._table_shape = (num_seqs, self.max_pages)

    _want = FlamiaScoredAttention._want
    _run = FlamiaScoredAttention._run

    def _moved(self, name, t):
        pass                           # (the calls ask the tensors)

    def _places(self, cache, page_table):
        if cache.kind != self._kind:
            raise FlamiaError(f"cache: want pages of {self.page_size}, {self.hkv} heads of {self.d} on {self.device}, got "
                              f"{cache.page_size}, {cache.hkv}, {cache.d} on {cache.device}")
        self._want("page_table", page_table, self._table_shape, self._i32)
        if not self._planned:
            raise FlamiaError("FlamiaCachedAttention: plan_build has not been called")

    def plan_build(self, cu_seqlens, kv_lens, stream=None):
        self._want("cu_seqlens", cu_seqlens, (self.N + 1,), self._i32)
        self._want("kv_lens", kv_lens, (self.N,), self._i32)
        self._run(lambda stm: flamia_cache_plan_build(cu_seqlens, kv_lens, self.N, self.T, self.hq, self.hkv, self.max_chunk,
                                                      self.max_pages * self.page_size, self.window, self.plan, stm), stream)
        self._planned = True

    def _call(self, what, f, stream, *args):
        """f(*args, stream handle) with the object's device current, on `stream` or its current stream."""
        if stream is None and self._index is not None and self._device_now() == self._index:
            rc = f(*args, self._stream_now(self._index))
        else:
            rc = self._run(lambda stm: f(*args, stm), stream)
        if rc:
            _check(rc, what)

    def write(self, cache: FlamiaPagedCache, k, v, page_table, stream=None):
        """The new tokens' keys and values into the cache."""
        self._places(cache, page_table)
        self._want("k", k, self._kv_shape, self._bf16)
        self._want("v", v, self._kv_shape, self._bf16)
        self._call("flamia_cache_write", self._lib.flamia_cache_write, stream, cache.ref, page_table.data_ptr(), self.max_pages,
                   self.N, self.T, self._plan.data_ptr(), k.data_ptr(), v.data_ptr())

    def read(self, cache: FlamiaPagedCache, page_table, k, v, stream=None):
        """The new tokens' keys and values from the cache into k and v, which are returned."""
        self._places(cache, page_table)
        self._want("k", k, self._kv_shape, self._bf16)
        self._want("v", v, self._kv_shape, self._bf16)
        self._call("flamia_cache_read", self._lib.flamia_cache_read, stream, cache.ref, page_table.data_ptr(), self.max_pages,
                   self.N, self.T, self._plan.data_ptr(), k.data_ptr(), v.data_ptr())
        return k, v

    def forward(self, cache: FlamiaPagedCache, q, page_table, softmax_scale: float = 0.0, stream=None):
        """(out bf16 [T, hq, d], lse fp32 [hq, T]) of the new tokens, whose keys and values have been written."""
        self._places(cache, page_table)
        self._want("q", q, self._q_shape, self._bf16)
        out, lse = self._out, self._lse
        self._call("flamia_cached_fwd", self._lib.flamia_cached_fwd, stream, q.data_ptr(), cache.ref, page_table.data_ptr(),
                   self.max_pages, self.N, self.T, self.hq, self.max_chunk, self.window, self.softcap, softmax_scale,
                   self._plan.data_ptr(), out.data_ptr(), lse.data_ptr(), self._workspace.data_ptr(), self._ws_bytes)
        return out, lse

    def device_status(self, stream=None) -> int:
        return self._run(lambda stm: flamia_get_device_status(self.plan, stm), stream)
