"""Python binding of libtopoep (GB300, sm_103a): the topology-aware
expert-routing plan of "TopoEP: Topology-Aware Load Balancing for
Expert-Parallel MoE Training" (§4) plus the expert co-selection statistics of
"Expert Coupling in MoE Pretraining".

This module only marshals arguments into the C ABI declared in
``include/topo.h``; every step runs in the library's CUDA kernels.  The
functions carry the C names and take device pointers as Python ints or as
objects with ``data_ptr()`` (torch tensors), and CUDA streams as raw handles
(``torch.cuda.current_stream().cuda_stream``) or objects with ``cuda_stream``.
A nonzero return code raises :class:`TopoError`.  If the shared library has
not been built, every call raises -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libtopoep.so")

TOPO_OK, TOPO_EINVAL, TOPO_ENOSPC, TOPO_ECUDA = 0, -1, -2, -3
TOPO_ERANGE, TOPO_ESTATE, TOPO_EMAP, TOPO_EOFFSETS, TOPO_ETIMEOUT = -4, -5, -6, -7, -8
TOPO_CALL_HIST, TOPO_CALL_PLAN, TOPO_CALL_REROUTE, TOPO_CALL_LAYOUT = 0, 1, 2, 3
TOPO_CALL_COOCCUR, TOPO_CALL_CHAIN, TOPO_CALL_REROUTE_LAYOUT = 4, 5, 6
TOPO_CALL_PACK = 7
TOPO_CALL_DEDUP = 8
TOPO_CALL_GATE = 9
TOPO_DTYPE_F32 = 0
TOPO_DTYPE_BF16 = 1
TOPO_GATE_MAX_E = 1024
TOPO_SCORE_SOFTMAX = 0
TOPO_SCORE_SIGMOID = 1
TOPO_ROUTE_MAX_GROUPS = 32
TOPO_BLOCK = 128
TOPO_FMT_EIGHT, TOPO_FMT_MX, TOPO_FMT_NV = 0, 1, 2
TOPO_FEW_MAX_TOKENS = 32
TOPO_SHUFFLE_STATS = 4
TOPO_SHUFFLE_MAX_RANKS = 256
TOPO_PLACE_STATS = 4
TOPO_DEDUP_STATS = 4
TOPO_STATS = 8
TOPO_LAYOUT_STATS = 8
EXPORTS = ("topo_workspace_bytes", "topo_ws_reset", "topo_hist", "topo_cooccur", "topo_plan",
           "topo_reroute", "topo_dispatch_layout", "topo_reroute_layout", "topo_read_error",
           "topo_strerror", "topo_hist_noalloc", "topo_permute", "topo_combine",
           "topo_dedup_layout", "topo_gate_hist", "topo_shuffle_workspace_bytes",
           "topo_shuffle_targets", "topo_place_experts", "topo_cooccur_workspace_bytes", "topo_route",
           "topo_route_grad", "topo_permute_quantize", "topo_quantize_rows", "topo_quantize_weight",
           "topo_cols_capacity", "topo_quantize_cols", "topo_swiglu_quantize", "topo_swiglu_grad",
           "topo_expert_workspace_bytes", "topo_expert_gemm", "topo_expert_wgrad", "topo_micro_pitch",
           "topo_quantize_rows_micro", "topo_permute_quantize_micro", "topo_swiglu_quantize_micro",
           "topo_dequantize_micro", "topo_expert_gemm_micro", "topo_few_workspace_bytes", "topo_expert_few")
TOPO_HIST_NOALLOC_SCRATCH_BYTES = 16 << 20


class TopoError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {code} ({strerror(code)})")
        self.code = code


class TopoCfg(ctypes.Structure):
    """Mirror of topo_cfg."""
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("R", ctypes.c_int32), ("ranks_per_node", ctypes.c_int32),
                ("n_slot", ctypes.c_int32), ("tok_bytes", ctypes.c_int64),
                ("expert_bytes", ctypes.c_int64), ("c_intra", ctypes.c_int32),
                ("c_inter", ctypes.c_int32), ("max_refine_iters", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("main_rank", ctypes.c_void_p),
                ("rank_offsets", ctypes.c_void_p)]


class TopoPlan(ctypes.Structure):
    """Mirror of topo_plan_t (device pointers)."""
    _fields_ = [("slot_expert", ctypes.c_void_p), ("route_cnt", ctypes.c_void_p),
                ("inst_load", ctypes.c_void_p), ("rank_load", ctypes.c_void_p),
                ("stats", ctypes.c_void_p)]


class TopoRouteOpts(ctypes.Structure):
    """Mirror of topo_route_opts."""
    _fields_ = [("score", ctypes.c_int32), ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


_lock = threading.Lock()
_lib = None


def lib():
    """The loaded shared library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libtopoep.so not built ({LIB_PATH}); run __graft_entry__.build()")
            L = ctypes.CDLL(LIB_PATH)
            vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
            cfgp, planp = ctypes.POINTER(TopoCfg), ctypes.POINTER(TopoPlan)
            L.topo_workspace_bytes.argtypes = [cfgp, i32, i32]
            L.topo_workspace_bytes.restype = sz
            L.topo_ws_reset.argtypes = [vp, sz, vp]
            L.topo_hist.argtypes = [cfgp, i32, vp, vp, vp, sz, vp]
            L.topo_cooccur.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
            L.topo_plan.argtypes = [cfgp, i32, vp, planp, vp, sz, vp]
            L.topo_reroute.argtypes = [cfgp, i32, vp, planp, vp, vp, sz, vp]
            L.topo_dispatch_layout.argtypes = [cfgp, i32, vp, planp, vp, vp, vp, vp, vp, sz, vp]
            L.topo_reroute_layout.argtypes = [cfgp, i32, vp, planp, vp, vp, vp, vp, vp, vp, sz, vp]
            L.topo_hist_noalloc.argtypes = [cfgp, i32, vp, vp, vp, vp]
            L.topo_permute.argtypes = [cfgp, i32, i32, vp, vp, vp, vp, sz, vp]
            L.topo_dedup_layout.argtypes = [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            L.topo_gate_hist.argtypes = [cfgp, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp]
            L.topo_cooccur_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.topo_cooccur_workspace_bytes.restype = sz
            L.topo_shuffle_workspace_bytes.argtypes = [i32, i32, i32]
            L.topo_shuffle_workspace_bytes.restype = sz
            L.topo_shuffle_targets.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            L.topo_place_experts.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp]
            L.topo_combine.argtypes = [cfgp, i32, i32, vp, vp, vp, vp, vp, sz, vp]
            i64, optp = ctypes.c_int64, ctypes.POINTER(TopoRouteOpts)
            L.topo_route.argtypes = [cfgp, i32, optp, vp, i32, vp, vp, vp, vp, vp, sz, vp]
            L.topo_route_grad.argtypes = [cfgp, i32, optp, vp, i32, vp, vp, vp, vp, sz, vp]
            L.topo_permute_quantize.argtypes = [cfgp, i32, i32, vp, vp, vp, vp, vp, sz, vp]
            L.topo_quantize_rows.argtypes = [i64, i32, vp, vp, vp, vp]
            L.topo_quantize_weight.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, vp]
            L.topo_cols_capacity.argtypes = [i32, i64]
            L.topo_cols_capacity.restype = i64
            L.topo_quantize_cols.argtypes = [i32, i64, i32, vp, vp, i64, vp, vp, vp, sz, vp]
            L.topo_swiglu_quantize.argtypes = [i64, i32, vp, vp, vp, vp]
            L.topo_swiglu_grad.argtypes = [i64, i32, vp, vp, vp, vp]
            L.topo_expert_workspace_bytes.argtypes = [i32, i64, i32, i32]
            L.topo_expert_workspace_bytes.restype = sz
            L.topo_expert_gemm.argtypes = [i32, i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
            L.topo_expert_wgrad.argtypes = [i32, i64, i32, i32, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            L.topo_micro_pitch.argtypes = [i32, i32]
            L.topo_micro_pitch.restype = i64
            L.topo_quantize_rows_micro.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp]
            L.topo_permute_quantize_micro.argtypes = [cfgp, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
            L.topo_swiglu_quantize_micro.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp]
            L.topo_dequantize_micro.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp]
            L.topo_expert_gemm_micro.argtypes = [i32, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
            L.topo_few_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
            L.topo_few_workspace_bytes.restype = sz
            L.topo_expert_few.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            L.topo_read_error.argtypes = [vp]
            L.topo_strerror.argtypes = [ctypes.c_int]
            L.topo_strerror.restype = ctypes.c_char_p
            for f in ("topo_ws_reset", "topo_hist", "topo_cooccur", "topo_plan", "topo_reroute",
                      "topo_dispatch_layout", "topo_reroute_layout", "topo_read_error",
                      "topo_hist_noalloc", "topo_permute", "topo_combine", "topo_dedup_layout", "topo_gate_hist", "topo_shuffle_targets", "topo_place_experts",
                      "topo_route", "topo_route_grad", "topo_permute_quantize", "topo_quantize_rows",
                      "topo_quantize_weight", "topo_quantize_cols", "topo_swiglu_quantize", "topo_swiglu_grad",
                      "topo_expert_gemm", "topo_expert_wgrad", "topo_quantize_rows_micro",
                      "topo_permute_quantize_micro", "topo_swiglu_quantize_micro", "topo_dequantize_micro",
                      "topo_expert_gemm_micro", "topo_expert_few"):
                getattr(L, f).restype = ctypes.c_int
            _lib = L
    return _lib


def _p(x):
    if x is None:
        return None
    if type(x) is int:
        return x or None
    try:
        return x.data_ptr() or None
    except AttributeError:
        return int(x) or None


def _s(stream):
    if stream is None:
        return None
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream or None
    return int(stream) or None


def _chk(fn, rc):
    if rc != TOPO_OK:
        raise TopoError(fn, rc)
    return rc


def make_cfg(T, E, k, R, ranks_per_node, n_slot, tok_bytes=0, expert_bytes=0, c_intra=1,
             c_inter=4, max_refine_iters=0, main_rank=None, rank_offsets=None, **_ignored) -> TopoCfg:
    """topo_cfg from plain values; main_rank (int32 [E]) and rank_offsets
    (int64 [R+1]) are device pointers/tensors or None."""
    return TopoCfg(T, E, k, R, ranks_per_node, n_slot, tok_bytes, expert_bytes, c_intra, c_inter,
                   max_refine_iters, 0, _p(main_rank), _p(rank_offsets))


def make_plan(slot_expert, route_cnt, inst_load, rank_load, stats) -> TopoPlan:
    return TopoPlan(_p(slot_expert), _p(route_cnt), _p(inst_load), _p(rank_load), _p(stats))


def strerror(code: int) -> str:
    try:
        return lib().topo_strerror(code).decode()
    except RuntimeError:
        return "library not loaded"


def topo_workspace_bytes(cfg: TopoCfg | None, n_layers: int, which_call: int) -> int:
    return lib().topo_workspace_bytes(ctypes.byref(cfg) if cfg is not None else None, n_layers,
                                      which_call)


def topo_ws_reset(ws, ws_bytes: int, stream=None) -> int:
    return _chk("topo_ws_reset", lib().topo_ws_reset(_p(ws), ws_bytes, _s(stream)))


def topo_hist(cfg: TopoCfg, n_layers: int, ids, hist, ws, ws_bytes: int, stream=None) -> int:
    return _chk("topo_hist", lib().topo_hist(ctypes.byref(cfg), n_layers, _p(ids), _p(hist), _p(ws),
                                             ws_bytes, _s(stream)))


def topo_cooccur(L: int, T: int, E: int, k: int, ids, co, tr, ws, ws_bytes: int, stream=None) -> int:
    return _chk("topo_cooccur", lib().topo_cooccur(L, T, E, k, _p(ids), _p(co), _p(tr), _p(ws),
                                                   ws_bytes, _s(stream)))


def topo_plan(cfg: TopoCfg, n_layers: int, hist, plan: TopoPlan, ws, ws_bytes: int,
              stream=None) -> int:
    return _chk("topo_plan", lib().topo_plan(ctypes.byref(cfg), n_layers, _p(hist),
                                             ctypes.byref(plan), _p(ws), ws_bytes, _s(stream)))


def topo_reroute(cfg: TopoCfg, n_layers: int, ids, plan: TopoPlan, dst_inst, ws, ws_bytes: int,
                 stream=None) -> int:
    return _chk("topo_reroute", lib().topo_reroute(ctypes.byref(cfg), n_layers, _p(ids),
                                                   ctypes.byref(plan), _p(dst_inst), _p(ws),
                                                   ws_bytes, _s(stream)))


def topo_dispatch_layout(cfg: TopoCfg, n_layers: int, dst_inst, plan: TopoPlan, sorted_pairs,
                         seg_off, send_counts, layout_stats, ws, ws_bytes: int,
                         stream=None) -> int:
    return _chk("topo_dispatch_layout",
                lib().topo_dispatch_layout(ctypes.byref(cfg), n_layers, _p(dst_inst),
                                           ctypes.byref(plan), _p(sorted_pairs), _p(seg_off),
                                           _p(send_counts), _p(layout_stats), _p(ws), ws_bytes,
                                           _s(stream)))


def topo_reroute_layout(cfg: TopoCfg, n_layers: int, ids, plan: TopoPlan, dst_inst, sorted_pairs,
                        seg_off, send_counts, layout_stats, ws, ws_bytes: int, stream=None) -> int:
    return _chk("topo_reroute_layout",
                lib().topo_reroute_layout(ctypes.byref(cfg), n_layers, _p(ids), ctypes.byref(plan),
                                          _p(dst_inst), _p(sorted_pairs), _p(seg_off),
                                          _p(send_counts), _p(layout_stats), _p(ws), ws_bytes,
                                          _s(stream)))


def topo_hist_noalloc(cfg: TopoCfg, n_layers: int, ids, hist, err=None, stream=None) -> int:
    """topo_hist with the library's fixed scratch array instead of a workspace;
    err: optional device int32 that receives the device error word."""
    return _chk("topo_hist_noalloc", lib().topo_hist_noalloc(ctypes.byref(cfg), n_layers, _p(ids),
                                                             _p(hist), _p(err), _s(stream)))


def topo_place_experts(L: int, E: int, R: int, max_iters: int, co, main_rank, stats, stream=None) -> int:
    """Correlated expert placement from co-selection counts into a main-rank map."""
    return _chk("topo_place_experts",
                lib().topo_place_experts(L, E, R, max_iters, _p(co), _p(main_rank), _p(stats), _s(stream)))


def topo_shuffle_workspace_bytes(L: int, E: int, R: int) -> int:
    return int(lib().topo_shuffle_workspace_bytes(L, E, R))


def topo_cooccur_workspace_bytes(L: int, T: int, E: int, k: int) -> int:
    """Workspace bytes that let topo_cooccur use the tensor cores."""
    return int(lib().topo_cooccur_workspace_bytes(L, T, E, k))


def topo_shuffle_targets(L: int, T: int, E: int, k: int, R: int, ids, tr, main_rank, rank_offsets, target,
                         stats, ws, ws_bytes: int, stream=None) -> int:
    """Token-shuffle targets from cross-layer transition counts."""
    return _chk("topo_shuffle_targets",
                lib().topo_shuffle_targets(L, T, E, k, R, _p(ids), _p(tr), _p(main_rank), _p(rank_offsets),
                                           _p(target), _p(stats), _p(ws), ws_bytes, _s(stream)))


def topo_gate_hist(cfg: TopoCfg, n_layers: int, logits, logits_dtype: int, bias, ids, scores, hist,
                   ws, ws_bytes: int, stream=None) -> int:
    """Top-k gating of router logits (plus an optional expert bias) and Omega."""
    return _chk("topo_gate_hist",
                lib().topo_gate_hist(ctypes.byref(cfg), n_layers, _p(logits), logits_dtype, _p(bias),
                                     _p(ids), _p(scores), _p(hist), _p(ws), ws_bytes, _s(stream)))


def topo_dedup_layout(cfg: TopoCfg, n_layers: int, dst_inst, seg, row_token, row_slots, tok_dst,
                      send, stats, ws, ws_bytes: int, stream=None) -> int:
    """Deduplicated dispatch layout: one row per (token, destination rank)."""
    return _chk("topo_dedup_layout",
                lib().topo_dedup_layout(ctypes.byref(cfg), n_layers, _p(dst_inst), _p(seg),
                                        _p(row_token), _p(row_slots), _p(tok_dst), _p(send),
                                        _p(stats), _p(ws), ws_bytes, _s(stream)))


def topo_permute(cfg: TopoCfg, n_layers: int, H: int, x, sorted_pairs, y, ws, ws_bytes: int,
                 stream=None) -> int:
    """Dispatch pack: y[l][pos] = x[l][sorted_pairs[l][pos] // k] (bf16 rows)."""
    return _chk("topo_permute", lib().topo_permute(ctypes.byref(cfg), n_layers, H, _p(x),
                                                   _p(sorted_pairs), _p(y), _p(ws), ws_bytes,
                                                   _s(stream)))


def topo_combine(cfg: TopoCfg, n_layers: int, H: int, y, sorted_pairs, w, out, ws, ws_bytes: int,
                 stream=None) -> int:
    """Combine: out[l][t] = bf16(sum_j w[l][t][j] * y[l][pos(t, j)]), float, slot order."""
    return _chk("topo_combine", lib().topo_combine(ctypes.byref(cfg), n_layers, H, _p(y),
                                                   _p(sorted_pairs), _p(w), _p(out), _p(ws),
                                                   ws_bytes, _s(stream)))


def make_route(score: int, n_group: int = 1, topk_group: int = 1, group_top: int = 1, renorm: bool = True,
               scale: float = 1.0) -> TopoRouteOpts:
    """topo_route_opts from plain values."""
    return TopoRouteOpts(score, n_group, topk_group, group_top, int(bool(renorm)), scale)


def topo_route(cfg: TopoCfg, n_layers: int, opts: TopoRouteOpts, logits, logits_dtype: int, bias, ids, weights, hist,
               ws, ws_bytes: int, stream=None) -> int:
    """Routing to experts: scores, groups, top-k ids and weights (and Omega when hist is given)."""
    return _chk("topo_route", lib().topo_route(ctypes.byref(cfg), n_layers, ctypes.byref(opts), _p(logits),
                                               logits_dtype, _p(bias), _p(ids), _p(weights), _p(hist), _p(ws),
                                               ws_bytes, _s(stream)))


def topo_route_grad(cfg: TopoCfg, n_layers: int, opts: TopoRouteOpts, logits, logits_dtype: int, ids, grad_weights,
                    grad_logits, ws, ws_bytes: int, stream=None) -> int:
    """Gradient of topo_route's weights in the logits."""
    return _chk("topo_route_grad", lib().topo_route_grad(ctypes.byref(cfg), n_layers, ctypes.byref(opts), _p(logits),
                                                         logits_dtype, _p(ids), _p(grad_weights), _p(grad_logits),
                                                         _p(ws), ws_bytes, _s(stream)))


def topo_permute_quantize(cfg: TopoCfg, n_layers: int, H: int, x, sorted_pairs, q, scale, ws, ws_bytes: int,
                          stream=None) -> int:
    """Dispatch pack in 8 bits: the rows of topo_permute as e4m3 with a scale per 128 values."""
    return _chk("topo_permute_quantize",
                lib().topo_permute_quantize(ctypes.byref(cfg), n_layers, H, _p(x), _p(sorted_pairs), _p(q),
                                            _p(scale), _p(ws), ws_bytes, _s(stream)))


def topo_quantize_rows(rows: int, C: int, x, q, scale, stream=None) -> int:
    """bf16 rows as e4m3 with a scale per 128 values."""
    return _chk("topo_quantize_rows", lib().topo_quantize_rows(rows, C, _p(x), _p(q), _p(scale), _s(stream)))


def topo_quantize_weight(n_w: int, N: int, K: int, w, q, scale, qt=None, scale_t=None, stream=None) -> int:
    """bf16 weights as e4m3 with a scale per 128 x 128 block, and their transpose when qt and scale_t are given."""
    return _chk("topo_quantize_weight", lib().topo_quantize_weight(n_w, N, K, _p(w), _p(q), _p(scale), _p(qt),
                                                                   _p(scale_t), _s(stream)))


def topo_cols_capacity(n_seg: int, rows: int) -> int:
    """Columns of topo_quantize_cols' output for rows in n_seg segments."""
    return int(lib().topo_cols_capacity(n_seg, rows))


def topo_quantize_cols(n_seg: int, rows: int, C: int, x, seg_off, cap: int, q, scale, ws, ws_bytes: int,
                       stream=None) -> int:
    """bf16 rows as e4m3 down their columns in 128-row blocks of each segment, transposed."""
    return _chk("topo_quantize_cols", lib().topo_quantize_cols(n_seg, rows, C, _p(x), _p(seg_off), cap, _p(q),
                                                               _p(scale), _p(ws), ws_bytes, _s(stream)))


def topo_swiglu_quantize(rows: int, I: int, h, q, scale, stream=None) -> int:
    """silu(g) * u of rows [g | u] as e4m3 with a scale per 128 values."""
    return _chk("topo_swiglu_quantize", lib().topo_swiglu_quantize(rows, I, _p(h), _p(q), _p(scale), _s(stream)))


def topo_swiglu_grad(rows: int, I: int, h, dy, dh, stream=None) -> int:
    """Gradient of silu(g) * u in the rows [g | u]."""
    return _chk("topo_swiglu_grad", lib().topo_swiglu_grad(rows, I, _p(h), _p(dy), _p(dh), _s(stream)))


def topo_expert_workspace_bytes(n_seg: int, rows: int, N: int, K: int) -> int:
    """Workspace bytes of topo_expert_gemm and topo_expert_wgrad."""
    return int(lib().topo_expert_workspace_bytes(n_seg, rows, N, K))


def topo_expert_gemm(n_seg: int, rows: int, n_w: int, N: int, K: int, a, a_scale, seg_off, seg_w, w, w_scale, out,
                     out_dtype: int, ws, ws_bytes: int, stream=None) -> int:
    """The experts' products: each segment's e4m3 rows times its weights' transpose."""
    return _chk("topo_expert_gemm", lib().topo_expert_gemm(n_seg, rows, n_w, N, K, _p(a), _p(a_scale), _p(seg_off),
                                                           _p(seg_w), _p(w), _p(w_scale), _p(out), out_dtype,
                                                           _p(ws), ws_bytes, _s(stream)))


def topo_expert_wgrad(n_seg: int, rows: int, N: int, K: int, cap: int, dy, dy_scale, x, x_scale, seg_off, dw, ws,
                      ws_bytes: int, stream=None) -> int:
    """Each segment's weight gradient from topo_quantize_cols' operands."""
    return _chk("topo_expert_wgrad", lib().topo_expert_wgrad(n_seg, rows, N, K, cap, _p(dy), _p(dy_scale), _p(x),
                                                             _p(x_scale), _p(seg_off), _p(dw), _p(ws), ws_bytes,
                                                             _s(stream)))


def topo_micro_pitch(C: int, fmt: int) -> int:
    """Bytes of the scales of a row of C values in 4 bits."""
    return int(lib().topo_micro_pitch(C, fmt))


def topo_quantize_rows_micro(rows: int, C: int, fmt: int, x, q, scale, row_scale=None, stream=None) -> int:
    """bf16 rows (or weights) in microscaled 4 bits."""
    return _chk("topo_quantize_rows_micro", lib().topo_quantize_rows_micro(rows, C, fmt, _p(x), _p(q), _p(scale),
                                                                           _p(row_scale), _s(stream)))


def topo_permute_quantize_micro(cfg: TopoCfg, n_layers: int, H: int, fmt: int, x, sorted_pairs, q, scale, row_scale, ws,
                                ws_bytes: int, stream=None) -> int:
    """Dispatch pack in microscaled 4 bits."""
    return _chk("topo_permute_quantize_micro",
                lib().topo_permute_quantize_micro(ctypes.byref(cfg), n_layers, H, fmt, _p(x), _p(sorted_pairs), _p(q),
                                                  _p(scale), _p(row_scale), _p(ws), ws_bytes, _s(stream)))


def topo_swiglu_quantize_micro(rows: int, I: int, fmt: int, h, q, scale, row_scale=None, stream=None) -> int:
    """silu(g) * u of rows [g | u] in microscaled 4 bits."""
    return _chk("topo_swiglu_quantize_micro", lib().topo_swiglu_quantize_micro(rows, I, fmt, _p(h), _p(q), _p(scale),
                                                                               _p(row_scale), _s(stream)))


def topo_dequantize_micro(rows: int, C: int, fmt: int, q, scale, row_scale, out, stream=None) -> int:
    """The bf16 values of rows in microscaled 4 bits."""
    return _chk("topo_dequantize_micro", lib().topo_dequantize_micro(rows, C, fmt, _p(q), _p(scale), _p(row_scale),
                                                                     _p(out), _s(stream)))


def topo_expert_gemm_micro(n_seg: int, rows: int, n_w: int, N: int, K: int, fmt: int, a, a_scale, a_row, seg_off, seg_w,
                           w, w_scale, w_row, out, out_dtype: int, ws, ws_bytes: int, stream=None) -> int:
    """The experts' products of rows and weights in microscaled 4 bits."""
    return _chk("topo_expert_gemm_micro",
                lib().topo_expert_gemm_micro(n_seg, rows, n_w, N, K, fmt, _p(a), _p(a_scale), _p(a_row), _p(seg_off),
                                             _p(seg_w), _p(w), _p(w_scale), _p(w_row), _p(out), out_dtype, _p(ws),
                                             ws_bytes, _s(stream)))


def topo_few_workspace_bytes(T: int, E: int, k: int, H: int, I: int) -> int:
    """Workspace bytes of topo_expert_few."""
    return int(lib().topo_few_workspace_bytes(T, E, k, H, I))


def topo_expert_few(T: int, E: int, k: int, H: int, I: int, fmt: int, x, ids, weights, up, up_scale, up_row, down,
                    down_scale, down_row, out, ws, ws_bytes: int, stream=None) -> int:
    """The experts applied to a few tokens: out = sum_j weights_j * W_down (silu(g) * u), [g | u] = W_up x."""
    return _chk("topo_expert_few",
                lib().topo_expert_few(T, E, k, H, I, fmt, _p(x), _p(ids), _p(weights), _p(up), _p(up_scale), _p(up_row),
                                      _p(down), _p(down_scale), _p(down_row), _p(out), _p(ws), ws_bytes, _s(stream)))


def topo_read_error(ws) -> int:
    return lib().topo_read_error(_p(ws))


def topo_strerror(code: int) -> str:
    return strerror(code)
