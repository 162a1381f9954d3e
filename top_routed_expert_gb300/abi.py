"""ctypes binding of the C ABI in include/moe_gb300.h (argument marshalling only).

Every function here has the name of the C entry point it calls and takes
torch tensors that already live on the current CUDA device; it passes their
data pointers and the current torch stream straight to the library and turns
a non-OK status into MoEError.  No arithmetic of the layer happens here, and
there is no fallback: if libmoe_gb300.so is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .build import LIB

MOE_F32, MOE_BF16, MOE_E4M3, MOE_NVFP4 = 0, 1, 2, 3
MOE_FLAG_SIMT_FFN = 0x1
MOE_FLAG_SIMT_ROUTER = 0x2
MOE_FLAG_BF16_EXPERT_OUT = 0x4
MOE_FLAG_ACT_E4M3 = 0x8
MOE_FLAG_ACT_NVFP4 = 0x10
MOE_FLAG_NVFP4_F16 = 0x20
MOE_FLAG_NO_OVERLAP = 0x40
MOE_FLAG_INJECT_TIMEOUT = 0x100
MOE_NOALLOC_MAX_PAIRS = 65536

STATUS = {
    0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
    4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_TIMEOUT", 6: "MOE_ERR_DEVICE_BOUNDS", 7: "MOE_ERR_ARCH",
    8: "MOE_ERR_DEVICE_NONFINITE",
}

MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_ROPE_HALF, MOE_ROPE_INTERLEAVED = 0, 1

# Every symbol the headers under include/ declare.
EXPORTS = ("moe_abi_version", "moe_status_str", "moe_workspace_bytes", "moe_route", "moe_permute",
           "moe_permute_noalloc", "moe_expert_ffn", "moe_combine", "moe_layer_forward", "moe_launch_count",
           "moe_get_device_status", "moe_qk_norm_rope", "moe_route_scores", "moe_kv_append",
           "moe_paged_attention", "moe_paged_attention_ws_bytes", "moe_blockkv_append", "moe_blockkv_attention",
           "moe_blockkv_attention_ws_bytes", "moe_blockkv_read", "moe_add_rms_norm")


class MoEError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


class moe_config_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("d_ff_shared", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class moe_qk_rope_config_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_pos", ctypes.c_int32), ("eps", ctypes.c_float)]


class moe_route_scores_config_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "n_experts", "top_k", "n_groups", "top_groups", "group_rank",
                                              "score", "logit_dtype", "renormalise")]
    _fields_ += [("scale", ctypes.c_float), ("logit_stride", ctypes.c_int64)]


class moe_kv_cache_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "page_table")]
    _fields_ += [(n, ctypes.c_int32) for n in ("n_pages", "page_size", "n_kv_heads", "head_dim", "max_pages")]
    _fields_ += [(n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride")]
    # of make_kv_cache's tensors: device, rows of the page table, (n_kv_heads, head_dim)
    device, batch, heads = None, 1 << 30, None


class moe_kv_append_config_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "batch", "n_q_heads", "rot_dim", "rope_layout", "n_pos")]
    _fields_ += [("eps", ctypes.c_float)]
    _fields_ += [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride", "q_out_stride")]
    # of make_kv_append_config's tensors: elements of a row of q and of k, (n_kv_heads, head_dim), whether rows follow each other
    # the layouts that they have, their rows
    q_row, k_row, heads, dense, like, rows = 0, 0, None, False, None, 0


class moe_paged_attention_config_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "batch", "n_q_heads", "max_q_len", "window", "n_sink")]
    _fields_ += [("sm_scale", ctypes.c_float), ("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]
    # of make_paged_attention_config's tensors: elements of a row of q, head_dim, whether rows follow each other
    # and the layouts that they have
    q_row, head_dim, dense, like = 0, None, False, None


class moe_blockkv_cache_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "page_table")]
    _fields_ += [(n, ctypes.c_int32) for n in ("n_pages", "page_size", "n_kv_heads", "head_dim", "max_pages")]
    _fields_ += [(n, ctypes.c_float) for n in ("k_gscale", "v_gscale")]
    _fields_ += [(n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride", "scale_page_stride",
                                               "scale_head_stride", "scale_token_stride")]
    # of make_blockkv_cache's tensors: device, rows of the page table, (n_kv_heads, head_dim)
    device, batch, heads = None, 1 << 30, None


class moe_blockkv_read_config_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "batch", "out_dtype")]
    _fields_ += [(n, ctypes.c_int64) for n in ("k_stride", "v_stride")]
    # of make_blockkv_read_config's tensors: (n_kv_heads, head_dim), type, elements of a row, whether rows follow each other
    heads, dtype, row, dense = None, None, None, False


class moe_add_norm_config_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "d", "x_dtype", "res_dtype", "out_dtype", "group")]
    _fields_ += [("eps", ctypes.c_float)]
    _fields_ += [(n, ctypes.c_int64) for n in ("x_stride", "res_stride", "sum_stride", "out_stride")]
    # of make_add_rms_norm_config's tensors: types of x, residual, out and sum, whether rows follow each other
    types, dense = None, False


class moe_weights_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w13", "w13_scale", "w13_gscale", "w2", "w2_scale", "w2_gscale",
        "s13", "s13_scale", "s13_gscale", "s2", "s2_scale", "s2_gscale")]


_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB) -> ctypes.CDLL:
    """Load libmoe_gb300.so (built by top_routed_expert_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m top_routed_expert_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    cfgp = ctypes.POINTER(moe_config_t)
    wp = ctypes.POINTER(moe_weights_t)
    sig = {
        "moe_abi_version": (i32, []),
        "moe_status_str": (ctypes.c_char_p, [i32]),
        "moe_workspace_bytes": (sz, [cfgp]),
        "moe_route": (i32, [cfgp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_permute": (i32, [cfgp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_permute_noalloc": (i32, [cfgp, vp, vp, vp, vp, vp]),
        "moe_expert_ffn": (i32, [cfgp, vp, vp, vp, vp, wp, vp, vp, vp, sz, vp]),
        "moe_combine": (i32, [cfgp, vp, vp, vp, vp, vp]),
        "moe_layer_forward": (i32, [cfgp, vp, vp, vp, wp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_launch_count": (ctypes.c_uint64, []),
        "moe_get_device_status": (i32, [vp]),
        "moe_qk_norm_rope": (i32, [ctypes.POINTER(moe_qk_rope_config_t), vp, vp, vp, vp, vp, vp, vp]),
        "moe_route_scores": (i32, [ctypes.POINTER(moe_route_scores_config_t), vp, vp, vp, vp, vp]),
        "moe_kv_append": (i32, [ctypes.POINTER(moe_kv_append_config_t), ctypes.POINTER(moe_kv_cache_t)] + [vp] * 11),
        "moe_paged_attention": (i32, [ctypes.POINTER(moe_paged_attention_config_t), ctypes.POINTER(moe_kv_cache_t)]
                                + [vp] * 6 + [sz, vp]),
        "moe_paged_attention_ws_bytes": (sz, [ctypes.POINTER(moe_paged_attention_config_t),
                                              ctypes.POINTER(moe_kv_cache_t)]),
        "moe_blockkv_append": (i32, [ctypes.POINTER(moe_kv_append_config_t), ctypes.POINTER(moe_blockkv_cache_t)] + [vp] * 11),
        "moe_blockkv_attention": (i32, [ctypes.POINTER(moe_paged_attention_config_t), ctypes.POINTER(moe_blockkv_cache_t)]
                                  + [vp] * 6 + [sz, vp]),
        "moe_blockkv_attention_ws_bytes": (sz, [ctypes.POINTER(moe_paged_attention_config_t),
                                                ctypes.POINTER(moe_blockkv_cache_t)]),
        "moe_blockkv_read": (i32, [ctypes.POINTER(moe_blockkv_read_config_t), ctypes.POINTER(moe_blockkv_cache_t)] + [vp] * 5),
        "moe_add_rms_norm": (i32, [ctypes.POINTER(moe_add_norm_config_t)] + [vp] * 8),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(code: int, where: str):
    if code != 0:
        raise MoEError(code, where)


def make_config(T, d_model, n_experts, top_k, d_ff, d_ff_shared, x_dtype=MOE_BF16, w_dtype=MOE_E4M3,
                y_dtype=MOE_F32, flags=0) -> moe_config_t:
    return moe_config_t(T, d_model, n_experts, top_k, d_ff, d_ff_shared, x_dtype, w_dtype, y_dtype, flags)


def make_weights(w13, w13_scale, w13_gscale, w2, w2_scale, w2_gscale,
                 s13, s13_scale, s13_gscale, s2, s2_scale, s2_gscale) -> moe_weights_t:
    vals = [w13, w13_scale, w13_gscale, w2, w2_scale, w2_gscale, s13, s13_scale, s13_gscale, s2, s2_scale,
            s2_gscale]
    return moe_weights_t(*[None if v is None else v.data_ptr() for v in vals])


def moe_abi_version() -> int:
    return load().moe_abi_version()


def moe_status_str(code: int) -> str:
    return load().moe_status_str(code).decode()


def moe_workspace_bytes(cfg: moe_config_t) -> int:
    return load().moe_workspace_bytes(ctypes.byref(cfg))


def moe_route(cfg, x, w_router, expert_bias, topk_ids, topk_w, ws=None, stream=None):
    _check(load().moe_route(ctypes.byref(cfg), _ptr(x), _ptr(w_router), _ptr(expert_bias), _ptr(topk_ids),
                            _ptr(topk_w), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                            _stream(stream)), "moe_route")


def moe_permute(cfg, topk_ids, expert_offsets, sorted_pair, row_of, ws, stream=None):
    _check(load().moe_permute(ctypes.byref(cfg), _ptr(topk_ids), _ptr(expert_offsets), _ptr(sorted_pair),
                              _ptr(row_of), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                              _stream(stream)), "moe_permute")


def moe_permute_noalloc(cfg, topk_ids, expert_offsets, sorted_pair, row_of, stream=None):
    """moe_permute without a workspace: its scratch is a fixed array inside the
    library (at most MOE_NOALLOC_MAX_PAIRS = 65536 pairs; calls that overlap on
    the GPU race on it)."""
    _check(load().moe_permute_noalloc(ctypes.byref(cfg), _ptr(topk_ids), _ptr(expert_offsets),
                                      _ptr(sorted_pair), _ptr(row_of), _stream(stream)), "moe_permute_noalloc")


def moe_expert_ffn(cfg, x, topk_w, expert_offsets, sorted_pair, weights: moe_weights_t, out_perm, shared_out, ws,
                   stream=None):
    _check(load().moe_expert_ffn(ctypes.byref(cfg), _ptr(x), _ptr(topk_w), _ptr(expert_offsets),
                                 _ptr(sorted_pair), ctypes.byref(weights), _ptr(out_perm), _ptr(shared_out),
                                 _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                 _stream(stream)), "moe_expert_ffn")


def moe_combine(cfg, out_perm, row_of, shared_out, y, stream=None):
    _check(load().moe_combine(ctypes.byref(cfg), _ptr(out_perm), _ptr(row_of), _ptr(shared_out), _ptr(y),
                              _stream(stream)), "moe_combine")


def moe_layer_forward(cfg, x, w_router, expert_bias, weights: moe_weights_t, y, topk_ids=None, topk_w=None,
                      expert_offsets=None, ws=None, stream=None):
    _check(load().moe_layer_forward(ctypes.byref(cfg), _ptr(x), _ptr(w_router), _ptr(expert_bias),
                                    ctypes.byref(weights), _ptr(y), _ptr(topk_ids), _ptr(topk_w),
                                    _ptr(expert_offsets), _ptr(ws),
                                    0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "moe_layer_forward")


def moe_qk_norm_rope(cfg, q, k, gamma_q, gamma_k, cos_sin, positions, stream=None):
    """Fused QK-norm + RoPE, in place on q [T, Hq, D] and k [T, Hkv, D] (bf16)."""
    _check(load().moe_qk_norm_rope(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(gamma_q), _ptr(gamma_k),
                                   _ptr(cos_sin), _ptr(positions), _stream(stream)), "moe_qk_norm_rope")


def _need(cond: bool, what: str):
    if not cond:
        raise ValueError(what)


# The calling thread's current CUDA device, the one that the library launches
# on, and the address of its current stream (a torch without CUDA has neither).
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

# The calls below are a few microseconds long and so is what they cost here: each
# looks at types, sizes and devices alone, written out in it.  Rows' layouts are
# looked at by the make_ functions, which leave what no field of the C structures
# says beside those (a structure made by hand lacks that part of the checks); a
# call's own rows have to lie as its configuration says.
_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_ELSEWHERE = "every tensor has to be on the current CUDA device"


def _rows_at(t: torch.Tensor, T: int, row: int, step: int) -> bool:
    """Whether t has T rows of `row` contiguous elements, `step` apart, whatever shape it gives them."""
    if row == step and t.is_contiguous():
        return t.numel() >= T * row
    shape, strides = t.shape, t.stride()
    if len(shape) < 2 or shape[0] < T or (T > 1 and strides[0] != step):
        return False
    n = 1
    for size, stride in zip(shape[:0:-1], strides[:0:-1]):
        if size > 1 and stride != n:
            return False
        n *= size
    return n >= row


def _stream_of(stream, device: int) -> int:
    """Address of a stream that was given."""
    _need(stream.device_index == device, "the stream has to be one of the current CUDA device")
    return stream.cuda_stream


_RAGGED = "cu: int32 [batch + 1], kv_len: int32 [batch], both contiguous, batch: at most the rows of the page table"


def make_route_scores_config(T, n_experts, top_k, n_groups=1, top_groups=1, group_rank=1, score=MOE_SCORE_SOFTMAX,
                             logit_dtype=MOE_F32, renormalise=True, scale=1.0,
                             logit_stride=None) -> moe_route_scores_config_t:
    return moe_route_scores_config_t(T, n_experts, top_k, n_groups, top_groups, group_rank, score, logit_dtype,
                                     int(renormalise), scale, n_experts if logit_stride is None else logit_stride)


def moe_route_scores(cfg, logits, bias, topk_ids, topk_w, stream=None):
    """Experts and weights from given logits (include/route_scores.h)."""
    dev = _current_device()
    if not (dev == logits.get_device() == topk_ids.get_device() == topk_w.get_device()
            and (bias is None or bias.get_device() == dev)):
        raise ValueError(_ELSEWHERE)
    T, E = cfg.T, cfg.n_experts
    if not (topk_ids.dtype is _I32 and topk_w.dtype is _F32 and topk_ids.numel() >= T * cfg.top_k <= topk_w.numel()
            and logits.dtype is (_BF16 if cfg.logit_dtype == MOE_BF16 else _F32)
            and topk_ids.is_contiguous() and topk_w.is_contiguous()
            and (bias is None or bias.dtype is _F32 and bias.numel() >= E and bias.is_contiguous())):
        raise ValueError("logits: of the configuration's type, bias: float32 [E], topk_ids: int32 [T, k], topk_w: "
                         "float32 [T, k], these three contiguous")
    if logits.numel() < (T - 1) * cfg.logit_stride + E:   # a view, or too short
        _need(T < 1 or (logits.dim() == 2 and logits.shape[0] >= T and logits.shape[1] >= E
                        and logits.stride(0) == cfg.logit_stride),
              "logits: rows of E elements with the configuration's distance between them")
    code = load().moe_route_scores(cfg, logits.data_ptr(), None if bias is None else bias.data_ptr(), topk_ids.data_ptr(),
                                   topk_w.data_ptr(), _current_stream(dev) if stream is None else _stream_of(stream, dev))
    if code:
        raise MoEError(code, "moe_route_scores")


def make_kv_cache(k, v, k_scale, v_scale, page_table) -> moe_kv_cache_t:
    """A paged cache from its tensors: k, v [n_pages, n_kv_heads, page_size, D] of torch.float8_e4m3fn (or their
    bytes) in any stride order with contiguous D, the scales [n_pages, n_kv_heads] float32, page_table
    [batch, max_pages] int32.  The tensors stay alive with the returned object."""
    _need(k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride(), "k and v: one 4-d shape, the same strides")
    codes = (torch.float8_e4m3fn, torch.uint8, torch.int8)
    _need(k.dtype in codes and v.dtype in codes and k.stride(3) == 1,
          "k and v: E4M3 codes (torch.float8_e4m3fn, or bytes), contiguous heads")
    n_pages, heads, page, D = k.shape
    for s in (k_scale, v_scale):
        _need(s.shape == (n_pages, heads) and s.dtype == torch.float32 and s.is_contiguous(),
              "scales: contiguous float32 [n_pages, n_kv_heads]")
    _need(page_table.dim() == 2 and page_table.dtype == torch.int32 and page_table.is_contiguous(),
          "page_table: contiguous int32 [batch, max_pages]")
    # a dimension of size 1 may carry any stride: give it one that the library takes
    strides = [st if n > 1 else D for n, st in zip(k.shape[:3], k.stride()[:3])]
    c = moe_kv_cache_t(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(),
                       n_pages, page, heads, D, page_table.shape[1], *strides)
    c.tensors = (k, v, k_scale, v_scale, page_table)
    c.device, c.batch, c.heads = k.get_device(), page_table.shape[0], (heads, D)
    _need(all(t.get_device() == c.device for t in c.tensors), "the cache's tensors: one device")
    return c


def _row_stride(t: torch.Tensor, dtype=torch.bfloat16) -> int:
    """Row stride of [T, heads, D] with contiguous heads."""
    _need(t.dim() == 3 and t.stride(2) == 1 and (t.shape[1] == 1 or t.stride(1) == t.shape[2]),
          "rows of [T, heads, D] with contiguous heads")
    _need(t.dtype == dtype, f"{'bf16' if dtype == torch.bfloat16 else dtype} rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def make_kv_append_config(q, k, v, q_out, batch, rot_dim=0, n_pos=0, rope_layout=MOE_ROPE_HALF,
                          eps=1e-6) -> moe_kv_append_config_t:
    """Sizes and strides of an append from its tensors (q and q_out may be None)."""
    _need(k.shape == v.shape and (q is None or (q.shape[0] == k.shape[0] and q.shape == q_out.shape)),
          "q, k, v and q_out: the same rows")
    _need(q is None or q.shape[2] == k.shape[2], "q and k: one head size")
    c = moe_kv_append_config_t(k.shape[0], batch, 0 if q is None else q.shape[1], rot_dim, rope_layout, n_pos, eps,
                               0 if q is None else _row_stride(q), _row_stride(k), _row_stride(v),
                               0 if q is None else _row_stride(q_out))
    c.heads = heads, D = tuple(k.shape[1:])
    c.q_row, c.k_row = c.n_q_heads * D, heads * D
    c.dense = c.k_stride == c.v_stride == c.k_row and c.q_stride == c.q_out_stride == c.q_row
    c.like, c.rows = _append_layouts(q, k, v, q_out), k.shape[0]
    return c


def _append_layouts(q, k, v, q_out):
    if q is None:
        return k.shape, k.stride(), v.shape, v.stride()
    return k.shape, k.stride(), v.shape, v.stride(), q.shape, q.stride(), q_out.shape, q_out.stride()


def _append_rows(cfg, T: int, q, k, v, q_out) -> bool:
    """An append's rows, where they are not simply dense."""
    return cfg.k_row == 0 or (_rows_at(k, T, cfg.k_row, cfg.k_stride) and _rows_at(v, T, cfg.k_row, cfg.v_stride) and
                              (q is None or _rows_at(q, T, cfg.q_row, cfg.q_stride)
                               and _rows_at(q_out, T, cfg.q_row, cfg.q_out_stride)))


def _appending(where: str, doc: str):
    """An append's call, to either cache."""
    def call(cfg, cache, q, k, v, gamma_q, gamma_k, cos_sin, positions, cu, kv_len, q_out, stream=None):
        dev = _current_device()
        if not (dev == k.get_device() == v.get_device() == cu.get_device() == kv_len.get_device()
                and (q is None or q.get_device() == q_out.get_device() == dev)
                and (gamma_q is None or gamma_q.get_device() == dev) and (gamma_k is None or gamma_k.get_device() == dev)
                and (cos_sin is None or cos_sin.get_device() == dev) and (positions is None or positions.get_device() == dev)
                and (cache.device is None or cache.device == dev)):
            raise ValueError(_ELSEWHERE)
        B = cfg.batch
        if not (cu.dtype is kv_len.dtype is _I32 and cu.numel() > B <= kv_len.numel() and B <= cache.batch
                and cu.is_contiguous() and kv_len.is_contiguous()):
            raise ValueError(_RAGGED)
        T = cfg.T
        if not (k.dtype is v.dtype is _BF16 and (q is None or q.dtype is q_out.dtype is _BF16)
                and (cfg.heads == cache.heads or cfg.heads is None or cache.heads is None)
                and (cfg.dense and k.is_contiguous() and v.is_contiguous() and k.numel() >= T * cfg.k_row <= v.numel()
                     and (q is None or q.is_contiguous() and q_out.is_contiguous() and q.numel() >= T * cfg.q_row <= q_out.numel())
                     or _append_layouts(q, k, v, q_out) == cfg.like and T <= cfg.rows or _append_rows(cfg, T, q, k, v, q_out))):
            raise ValueError("q, k, v and q_out: bf16 rows of the configuration's shape and distance and the cache's heads")
        D = cache.head_dim
        if not ((gamma_k is None or gamma_k.dtype is _F32 and gamma_k.numel() >= D and gamma_k.is_contiguous())
                and (gamma_q is None or gamma_q.dtype is _F32 and gamma_q.numel() >= D and gamma_q.is_contiguous())
                and (cos_sin is None or cos_sin.dtype is _F32 and cos_sin.numel() >= cfg.n_pos * cfg.rot_dim
                     and cos_sin.is_contiguous())
                and (positions is None or positions.dtype is _I32 and positions.numel() >= T and positions.is_contiguous())):
            raise ValueError("gamma_q, gamma_k: float32 [D], cos_sin: float32 [n_pos, rot_dim / 2, 2], positions: int32 [T], "
                             "all contiguous")
        code = getattr(load(), where)(
            cfg, cache, None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
            None if gamma_q is None else gamma_q.data_ptr(), None if gamma_k is None else gamma_k.data_ptr(),
            None if cos_sin is None else cos_sin.data_ptr(), None if positions is None else positions.data_ptr(),
            cu.data_ptr(), kv_len.data_ptr(), None if q is None else q_out.data_ptr(),
            _current_stream(dev) if stream is None else _stream_of(stream, dev))
        if code:
            raise MoEError(code, where)
    call.__name__ = call.__qualname__ = where
    call.__doc__ = doc
    return call


moe_kv_append = _appending("moe_kv_append", "Norm, rotation and append to the paged cache (include/paged_kv.h).")
moe_blockkv_append = _appending("moe_blockkv_append",
                                "Norm, rotation and append to the paged cache in 4 bits (include/block_kv.h).")


def make_paged_attention_config(q, out, batch, max_q_len=0, window=0, n_sink=0,
                                sm_scale=None) -> moe_paged_attention_config_t:
    """Sizes and strides of an attention call from its tensors; sm_scale defaults to 1/sqrt(D)."""
    _need(q.shape == out.shape, "q and out: the same shape")
    c = moe_paged_attention_config_t(q.shape[0], batch, q.shape[1], max_q_len, window, n_sink,
                                     q.shape[2] ** -0.5 if sm_scale is None else sm_scale, _row_stride(q), _row_stride(out))
    c.q_row, c.head_dim = q.shape[1] * q.shape[2], q.shape[2]
    c.dense = c.q_stride == c.out_stride == c.q_row
    c.like = q.shape, q.stride(), out.shape, out.stride()
    return c


def _attention_rows(cfg, T: int, q, out) -> bool:
    """An attention's rows, where they are not simply dense."""
    if (q.shape, q.stride(), out.shape, out.stride()) == cfg.like and T <= q.shape[0]:
        return True
    return cfg.q_row == 0 or (_rows_at(q, T, cfg.q_row, cfg.q_stride) and _rows_at(out, T, cfg.q_row, cfg.out_stride))


def moe_paged_attention_ws_bytes(cfg, cache) -> int:
    return load().moe_paged_attention_ws_bytes(cfg, cache)


def _attending(where: str, doc: str):
    """An attention's call, over either cache."""
    def call(cfg, cache, q, cu, kv_len, out, lse=None, ws=None, stream=None):
        dev = _current_device()
        if not (dev == q.get_device() == cu.get_device() == kv_len.get_device() == out.get_device()
                and (lse is None or lse.get_device() == dev) and (ws is None or ws.get_device() == dev)
                and (cache.device is None or cache.device == dev)):
            raise ValueError(_ELSEWHERE)
        B = cfg.batch
        if not (cu.dtype is kv_len.dtype is _I32 and cu.numel() > B <= kv_len.numel() and B <= cache.batch
                and cu.is_contiguous() and kv_len.is_contiguous()):
            raise ValueError(_RAGGED)
        T = cfg.T
        if not (q.dtype is out.dtype is _BF16 and (cfg.head_dim is None or cfg.head_dim == cache.head_dim)
                and (cfg.dense and q.is_contiguous() and out.is_contiguous() and q.numel() >= T * cfg.q_row <= out.numel()
                     or _attention_rows(cfg, T, q, out))
                and (lse is None or lse.dtype is _F32 and lse.numel() >= T * cfg.n_q_heads and lse.is_contiguous())
                and (ws is None or ws.is_contiguous())):
            raise ValueError("q and out: bf16 rows of the configuration's shape and distance and the cache's head size, lse: "
                             "contiguous float32 [T, n_q_heads], ws: contiguous")
        code = getattr(load(), where)(
            cfg, cache, q.data_ptr(), cu.data_ptr(), kv_len.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
            None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes,
            _current_stream(dev) if stream is None else _stream_of(stream, dev))
        if code:
            raise MoEError(code, where)
    call.__name__ = call.__qualname__ = where
    call.__doc__ = doc
    return call


moe_paged_attention = _attending("moe_paged_attention",
                                 "Attention of the new tokens over the paged cache (include/paged_kv.h).")
moe_blockkv_attention = _attending("moe_blockkv_attention",
                                   "Attention of the new tokens over the paged cache in 4 bits (include/block_kv.h).")


def make_blockkv_cache(k, v, k_scale, v_scale, page_table, k_gscale=1.0, v_gscale=1.0) -> moe_blockkv_cache_t:
    """A paged cache in 4 bits from its tensors: k, v [n_pages, n_kv_heads, page_size, D / 2] bytes of two E2M1 codes
    each, the scales [n_pages, n_kv_heads, page_size, D / 16] of torch.float8_e4m3fn (or their bytes), both in any
    stride order with a contiguous last dimension; page_table [batch, max_pages] int32; the factors powers of two.
    The tensors stay alive with the returned object."""
    _need(k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride(), "k and v: one 4-d shape, the same strides")
    _need(k_scale.dim() == 4 and k_scale.shape == v_scale.shape and k_scale.stride() == v_scale.stride(),
          "scales: one 4-d shape, the same strides")
    n_pages, heads, page, D = *k.shape[:3], 2 * k.shape[3]
    _need(k_scale.shape == (n_pages, heads, page, D // 16) and D % 16 == 0, "scales: [n_pages, n_kv_heads, page_size, D / 16]")
    byte = (torch.uint8, torch.int8)
    _need(all(t.dtype in byte and t.stride(3) == 1 for t in (k, v)), "k and v: bytes of two codes, contiguous heads")
    _need(all(t.dtype in (torch.float8_e4m3fn, *byte) and t.stride(3) == 1 for t in (k_scale, v_scale)),
          "scales: E4M3 codes (torch.float8_e4m3fn, or bytes), contiguous heads")
    _need(page_table.dim() == 2 and page_table.dtype == torch.int32 and page_table.is_contiguous(),
          "page_table: contiguous int32 [batch, max_pages]")
    # a dimension of size 1 may carry any stride: give it one that the library takes
    strides = [st if n > 1 else D // 2 for n, st in zip(k.shape[:3], k.stride()[:3])]
    strides += [st if n > 1 else D // 16 for n, st in zip(k_scale.shape[:3], k_scale.stride()[:3])]
    c = moe_blockkv_cache_t(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(),
                            n_pages, page, heads, D, page_table.shape[1], k_gscale, v_gscale, *strides)
    c.tensors = (k, v, k_scale, v_scale, page_table)
    c.device, c.batch, c.heads = k.get_device(), page_table.shape[0], (heads, D)
    _need(all(t.get_device() == c.device for t in c.tensors), "the cache's tensors: one device")
    return c


def moe_blockkv_attention_ws_bytes(cfg, cache) -> int:
    return load().moe_blockkv_attention_ws_bytes(cfg, cache)


def _float_type(t: torch.Tensor) -> int:
    _need(t.dtype is _BF16 or t.dtype is _F32, "bf16 or float32")
    return MOE_BF16 if t.dtype is _BF16 else MOE_F32


def make_blockkv_read_config(k_out, v_out, batch) -> moe_blockkv_read_config_t:
    """Sizes, type and strides of a read from its outputs [T, n_kv_heads, D], bf16 or float32 (one may be None)."""
    like = k_out if k_out is not None else v_out
    _need(like is not None and all(t is None or (t.shape == like.shape and t.dtype == like.dtype) for t in (k_out, v_out)),
          "k_out and v_out: one shape and type")
    rows = [0 if t is None else _row_stride(t, like.dtype) for t in (k_out, v_out)]
    c = moe_blockkv_read_config_t(like.shape[0], batch, _float_type(like), *rows)
    c.heads, c.dtype = tuple(like.shape[1:]), like.dtype
    c.row = like.shape[1] * like.shape[2]
    c.dense = all(t is None or step == c.row for t, step in zip((k_out, v_out), rows))
    return c


def _read_rows(cfg, T: int, k_out, v_out) -> bool:
    """moe_blockkv_read's outputs, where they are not simply dense."""
    return cfg.row is None or ((k_out is None or _rows_at(k_out, T, cfg.row, cfg.k_stride))
                               and (v_out is None or _rows_at(v_out, T, cfg.row, cfg.v_stride)))


def moe_blockkv_read(cfg, cache, cu, kv_len, k_out, v_out, stream=None):
    """Rows of the paged cache in 4 bits as bf16 or float32 (include/block_kv.h)."""
    dev = _current_device()
    if not (dev == cu.get_device() == kv_len.get_device() and (k_out is None or k_out.get_device() == dev)
            and (v_out is None or v_out.get_device() == dev) and (cache.device is None or cache.device == dev)):
        raise ValueError(_ELSEWHERE)
    B = cfg.batch
    if not (cu.dtype is kv_len.dtype is _I32 and cu.numel() > B <= kv_len.numel() and B <= cache.batch
            and cu.is_contiguous() and kv_len.is_contiguous()):
        raise ValueError(_RAGGED)
    T, dtype = cfg.T, cfg.dtype
    if not ((cfg.heads == cache.heads or cfg.heads is None or cache.heads is None)
            and (k_out is None or k_out.dtype is dtype or dtype is None) and (v_out is None or v_out.dtype is dtype or dtype is None)
            and (cfg.dense and (k_out is None or k_out.is_contiguous() and k_out.numel() >= T * cfg.row)
                 and (v_out is None or v_out.is_contiguous() and v_out.numel() >= T * cfg.row) or _read_rows(cfg, T, k_out, v_out))):
        raise ValueError("k_out and v_out: rows of the configuration's shape, type and distance and the cache's heads")
    code = load().moe_blockkv_read(cfg, cache, cu.data_ptr(), kv_len.data_ptr(), None if k_out is None else k_out.data_ptr(),
                                   None if v_out is None else v_out.data_ptr(),
                                   _current_stream(dev) if stream is None else _stream_of(stream, dev))
    if code:
        raise MoEError(code, "moe_blockkv_read")


def make_add_rms_norm_config(x, residual=None, out=None, out8=None, sum=None, group=0, eps=1e-6) -> moe_add_norm_config_t:
    """Sizes, types and strides of an addition and norm from its tensors [T, d]."""
    _need(x.dim() == 2 and all(t is None or t.shape == x.shape for t in (residual, out, out8, sum)), "one shape [T, d]")
    _need(all(t is None or t.stride(1) == 1 for t in (x, residual, out, out8, sum)), "contiguous rows")
    _need(sum is None or (residual is not None and sum.dtype == residual.dtype), "sum: of the residual's type")
    codes = (torch.float8_e4m3fn, torch.uint8, torch.int8)
    _need(out8 is None or (out8.dtype in codes and out8.is_contiguous()),
          "out8: contiguous E4M3 codes (torch.float8_e4m3fn, or bytes)")
    T, d = x.shape
    stride = lambda t: d if t is None or T <= 1 else t.stride(0)
    c = moe_add_norm_config_t(T, d, _float_type(x), MOE_BF16 if residual is None else _float_type(residual),
                              MOE_BF16 if out is None else _float_type(out), group, eps, stride(x), stride(residual),
                              stride(sum), stride(out))
    c.types = tuple(None if t is None else t.dtype for t in (x, residual, out, sum))
    c.dense = all(stride(t) == d for t in (x, residual, out, sum))
    return c


def _norm_rows(cfg, T: int, x, residual, out, sum) -> bool:
    """The norm's rows, where they are not simply dense."""
    return (_rows_at(x, T, cfg.d, cfg.x_stride) and (residual is None or _rows_at(residual, T, cfg.d, cfg.res_stride))
            and (out is None or _rows_at(out, T, cfg.d, cfg.out_stride)) and (sum is None or _rows_at(sum, T, cfg.d, cfg.sum_stride)))


def moe_add_rms_norm(cfg, x, residual, gamma, out=None, out8=None, out8_scale=None, sum=None, stream=None):
    """Residual's addition and RMS norm, with an E4M3 copy (include/add_rms_norm.h)."""
    dev = _current_device()
    if not (dev == x.get_device() == gamma.get_device() and (residual is None or residual.get_device() == dev)
            and (out is None or out.get_device() == dev) and (sum is None or sum.get_device() == dev)
            and (out8 is None or out8.get_device() == out8_scale.get_device() == dev)):
        raise ValueError(_ELSEWHERE)
    T, d = cfg.T, cfg.d
    n = T * d
    if cfg.types is not None:
        xt, rt, ot, st = cfg.types
        if not (x.dtype is xt and (residual is None or residual.dtype is rt) and (out is None or out.dtype is ot)
                and (sum is None or sum.dtype is st)
                and (cfg.dense and x.is_contiguous() and x.numel() >= n
                     and (residual is None or residual.is_contiguous() and residual.numel() >= n)
                     and (out is None or out.is_contiguous() and out.numel() >= n)
                     and (sum is None or sum.is_contiguous() and sum.numel() >= n) or _norm_rows(cfg, T, x, residual, out, sum))):
            raise ValueError("x, residual, out and sum: [T, d] of the configuration's types and strides")
    if not (gamma.dtype is _F32 and gamma.numel() >= d and gamma.is_contiguous()):
        raise ValueError("gamma: float32 [d]")
    if not (out8 is None or out8.nbytes >= n and out8.is_contiguous() and out8_scale.dtype is _F32
            and out8_scale.is_contiguous() and out8_scale.numel() * max(cfg.group, 1) >= (n if cfg.group > 0 else T)):
        raise ValueError("out8: contiguous [T, d], out8_scale: contiguous float32 [T, d / group]")
    code = load().moe_add_rms_norm(cfg, x.data_ptr(), None if residual is None else residual.data_ptr(), gamma.data_ptr(),
                                   None if out is None else out.data_ptr(), None if out8 is None else out8.data_ptr(),
                                   None if out8 is None else out8_scale.data_ptr(), None if sum is None else sum.data_ptr(),
                                   _current_stream(dev) if stream is None else _stream_of(stream, dev))
    if code:
        raise MoEError(code, "moe_add_rms_norm")


def moe_launch_count() -> int:
    return load().moe_launch_count()


def moe_get_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status code."""
    return load().moe_get_device_status(_stream(stream))
