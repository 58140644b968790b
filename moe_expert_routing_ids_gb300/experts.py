"""One mixture-of-experts layer on the planned layout, forward and backward.

The path a user of the planner runs: routing with scores and weights, the
replication plan and the dispatch layout of the chosen experts, the hidden rows
packed in 8 bits, the gate-and-up product of each expert instance, the gated
activation back in 8 bits, the down product and the weighted combine.  Every
step is a call into libtopoep; torch holds the buffers, and in the backward
pass forms the gradient of the combine (a gather and a dot product).

A layer may hold its weights in 4 bits (fmt: TOPO_FMT_MX or TOPO_FMT_NV); its rows
are then packed in 4 bits as well, and it has no backward pass.  few() is the same
layer for a few tokens, without plan, layout or packed rows: it reads the weights of
the experts in use once and keeps the activations in 16 bits.

Ranks are logical partitions of one GPU's rows, as for the planner: replicas of
an expert read the same weights, and their weight gradients are summed.
"""
from __future__ import annotations

import torch

from . import (TOPO_BLOCK, TOPO_CALL_PACK, TOPO_DTYPE_BF16, TOPO_DTYPE_F32, TOPO_FEW_MAX_TOKENS,
               TOPO_FMT_EIGHT, TOPO_FMT_MX, TOPO_FMT_NV, TopoRouteOpts, make_cfg, topo_cols_capacity, topo_combine,
               topo_expert_few, topo_expert_gemm, topo_expert_gemm_micro, topo_expert_wgrad, topo_expert_workspace_bytes,
               topo_few_workspace_bytes, topo_micro_pitch, topo_permute_quantize, topo_permute_quantize_micro,
               topo_quantize_cols, topo_quantize_rows, topo_quantize_rows_micro, topo_quantize_weight, topo_read_error,
               topo_route, topo_swiglu_grad, topo_swiglu_quantize, topo_swiglu_quantize_micro, topo_workspace_bytes,
               topo_ws_reset)
from .planner import Planner, need, ordered


def blocks(n: int) -> int:
    return (n + TOPO_BLOCK - 1) // TOPO_BLOCK


def micro_rows(shape: tuple, C: int, fmt: int, device) -> tuple:
    """Buffers of rows [*shape, C] in 4 bits: codes, scales, row scales (None for TOPO_FMT_MX)."""
    pitch = topo_micro_pitch(C, fmt)
    if pitch == 0:
        raise ValueError(f"rows in 4 bits hold a multiple of 32 values, not {C}")
    return (torch.empty((*shape, C // 2), dtype=torch.uint8, device=device),
            torch.empty((*shape, pitch), dtype=torch.uint8, device=device),
            torch.empty(shape, dtype=torch.float32, device=device) if fmt == TOPO_FMT_NV else None)


class ExpertWeights:
    """bf16 weights [E, N, K] in 8 bits with a scale per 128 x 128 block, and
    their transposes (the operand of the input gradient) when train is set; or
    (fmt) in 4 bits, row by row."""

    def __init__(self, w: torch.Tensor, train: bool = False, stream=None, fmt: int = TOPO_FMT_EIGHT):
        if not isinstance(w, torch.Tensor) or w.dim() != 3 or not w.is_cuda:
            raise ValueError("weights are a tensor [E, N, K] on a GPU")
        if fmt not in (TOPO_FMT_EIGHT, TOPO_FMT_MX, TOPO_FMT_NV):
            raise ValueError("fmt is TOPO_FMT_EIGHT, TOPO_FMT_MX or TOPO_FMT_NV")
        if train and fmt != TOPO_FMT_EIGHT:
            raise ValueError("weights in 4 bits have no backward pass")
        E, self.N, self.K = w.shape
        self.E, self.fmt, self.row = E, fmt, None
        dev, u8, f32 = w.device, torch.uint8, torch.float32
        with ordered(stream, dev, w):
            if fmt != TOPO_FMT_EIGHT:
                self.q, self.scale, self.row = micro_rows((E, self.N), self.K, fmt, dev)
                self.load(w)
                return
            self.q = torch.empty((E, self.N, self.K), dtype=u8, device=dev)
            self.scale = torch.empty((E, blocks(self.N), blocks(self.K)), dtype=f32, device=dev)
            self.qt = torch.empty((E, self.K, self.N), dtype=u8, device=dev) if train else None
            self.scale_t = torch.empty((E, blocks(self.K), blocks(self.N)), dtype=f32, device=dev) if train else None
            self.load(w)

    def load(self, w: torch.Tensor, stream=None):
        """Takes the values of w (bf16 [E, N, K]) in place of those held."""
        need("weights", w, (torch.bfloat16,), self.E * self.N, self.K, self.q.device)
        with ordered(stream, self.q.device, w):
            s = torch.cuda.current_stream(self.q.device)
            if self.fmt != TOPO_FMT_EIGHT:
                topo_quantize_rows_micro(self.E * self.N, self.K, self.fmt, w, self.q, self.scale, self.row, s)
            else:
                topo_quantize_weight(self.E, self.N, self.K, w, self.q, self.scale, self.qt, self.scale_t, s)


class ExpertLayer:
    """cfg: as for Planner (one layer per call); w_up: bf16 [E, 2 I, H], gate
    rows then up rows; w_down: bf16 [E, H, I]; route: topo_route_opts; fmt: how
    weights and packed rows are held, TOPO_FMT_EIGHT, or TOPO_FMT_MX or
    TOPO_FMT_NV (4 bits, H and I multiples of 32, without train).

    stream: every step of every call runs on it (None: torch's current stream).
    The calls take their place in the caller's current stream all the same: what
    it holds so far comes before them, what it gets next comes after.

    forward(), backward() and set_weights() work in the layer's own buffers: on one
    layer they must not overlap, on two streams or as replays of graphs that hold
    them.  few() works in buffers of its own call, and only set_weights() must not
    overlap it."""

    def __init__(self, cfg: dict, w_up: torch.Tensor, w_down: torch.Tensor, route: TopoRouteOpts, train: bool = False,
                 stream=None, fmt: int = TOPO_FMT_EIGHT):
        for name, w in (("w_up", w_up), ("w_down", w_down)):
            if not isinstance(w, torch.Tensor) or w.dim() != 3 or not w.is_cuda:
                raise ValueError(f"{name} must be a tensor of three dimensions on a GPU")
        self.E, self.H, self.I, self.device = cfg["E"], w_down.shape[1], w_down.shape[2], w_up.device
        self._need_weights(w_up, w_down)
        with ordered(stream, w_up.device, w_up, w_down):
            self._build(cfg, w_up, w_down, route, train, stream, fmt)

    def _need_weights(self, w_up, w_down):
        E, H, I = self.E, self.H, self.I
        if tuple(w_up.shape) != (E, 2 * I, H) or tuple(w_down.shape) != (E, H, I):
            raise ValueError("w_up is [E, 2 I, H] and w_down [E, H, I]")
        need("w_up", w_up, (torch.bfloat16,), E * 2 * I, H, self.device)
        need("w_down", w_down, (torch.bfloat16,), E * H, I, self.device)

    def set_weights(self, w_up: torch.Tensor, w_down: torch.Tensor):
        """New values of the weights, as after an optimiser's step; the layer keeps
        them in its format only.  A backward() belongs to the weights of its forward()."""
        self._need_weights(w_up, w_down)
        self.up.load(w_up, self.planner.stream)
        self.down.load(w_down, self.planner.stream)

    def _build(self, cfg, w_up, w_down, route, train, stream, fmt):
        self.planner = P = Planner(cfg, 1, w_up.device, stream)
        self.T, self.k, self.R = cfg["T"], cfg["k"], cfg["R"]
        self.route, self.train, self.fmt = route, train, fmt
        self.up = ExpertWeights(w_up, train, stream, fmt)
        self.down = ExpertWeights(w_down, train, stream, fmt)
        dev, rows = self.device, self.T * self.k
        self.rows, self.n_seg = rows, self.R * P.n_local
        u8, f32, bf16 = torch.uint8, torch.float32, torch.bfloat16

        def buf(*shape, dtype):
            return torch.empty(shape, dtype=dtype, device=dev)

        self.ids = buf(1, self.T, self.k, dtype=torch.int32)
        self.weights = buf(1, self.T, self.k, dtype=f32)
        if fmt == TOPO_FMT_EIGHT:
            self.xq, self.xs = buf(rows, self.H, dtype=u8), buf(rows, blocks(self.H), dtype=f32)
            self.aq, self.as_ = buf(rows, self.I, dtype=u8), buf(rows, blocks(self.I), dtype=f32)
        else:
            self.xq, self.xs, self.xr = micro_rows((rows,), self.H, fmt, dev)
            self.aq, self.as_, self.ar = micro_rows((rows,), self.I, fmt, dev)
        self.h = buf(rows, 2 * self.I, dtype=bf16)
        self.y = buf(rows, self.H, dtype=bf16)
        self.pack_bytes = topo_workspace_bytes(P.cfg, 1, TOPO_CALL_PACK)
        self.pack_ws = buf(self.pack_bytes, dtype=u8)
        self.ws_bytes = topo_expert_workspace_bytes(self.n_seg, rows, 2 * self.I, self.H)
        self.ws = buf(self.ws_bytes, dtype=u8)
        topo_ws_reset(self.pack_ws, self.pack_bytes, P._stream())
        topo_ws_reset(self.ws, self.ws_bytes, P._stream())
        self.seg_w = None
        # few(): its workspace is each call's own; 0: sizes that it does not take
        self.few_bytes = topo_few_workspace_bytes(TOPO_FEW_MAX_TOKENS, self.E, self.k, self.H, self.I)
        self.few_ids, self.few_sizes = None, {}

    def _product(self, a, a_scale, N, K, w, w_scale, out):
        topo_expert_gemm(self.n_seg, self.rows, self.E, N, K, a, a_scale, self.planner.buf.seg_off, self.seg_w, w,
                         w_scale, out, TOPO_DTYPE_BF16, self.ws, self.ws_bytes, self.planner._stream())

    def _product_micro(self, rows, w, out):
        topo_expert_gemm_micro(self.n_seg, self.rows, self.E, w.N, w.K, self.fmt, *rows, self.planner.buf.seg_off, self.seg_w,
                               w.q, w.scale, w.row, out, TOPO_DTYPE_BF16, self.ws, self.ws_bytes, self.planner._stream())

    def forward(self, x: torch.Tensor, logits: torch.Tensor, bias: torch.Tensor | None = None) -> torch.Tensor:
        """x: bf16 [T, H]; logits: float32 or bf16 [T, E]; bias: float32 [E] or
        None; returns bf16 [T, H]."""
        need("x", x, (torch.bfloat16,), self.T, self.H, self.device)
        with ordered(self.planner.stream, self.device, x, logits, bias) as outs:
            outs.append(self._forward(x, logits, bias))
        return outs[0]

    def _forward(self, x, logits, bias):
        P, s = self.planner, self.planner._stream()
        P.route(logits, self.ids, self.weights, self.route, bias)
        P.make_plan()
        P.reroute_layout(self.ids)
        self.seg_w = P.instance_experts()
        if self.fmt == TOPO_FMT_EIGHT:
            topo_permute_quantize(P.cfg, 1, self.H, x, P.buf.sorted_pairs, self.xq, self.xs, self.pack_ws,
                                  self.pack_bytes, s)
            self._product(self.xq, self.xs, 2 * self.I, self.H, self.up.q, self.up.scale, self.h)
            topo_swiglu_quantize(self.rows, self.I, self.h, self.aq, self.as_, s)
            self._product(self.aq, self.as_, self.H, self.I, self.down.q, self.down.scale, self.y)
        else:
            topo_permute_quantize_micro(P.cfg, 1, self.H, self.fmt, x, P.buf.sorted_pairs, self.xq, self.xs, self.xr,
                                        self.pack_ws, self.pack_bytes, s)
            self._product_micro((self.xq, self.xs, self.xr), self.up, self.h)
            topo_swiglu_quantize_micro(self.rows, self.I, self.fmt, self.h, self.aq, self.as_, self.ar, s)
            self._product_micro((self.aq, self.as_, self.ar), self.down, self.y)
        out = torch.empty((self.T, self.H), dtype=torch.bfloat16, device=self.device)
        topo_combine(P.cfg, 1, self.H, self.y, P.buf.sorted_pairs, self.weights, out, self.pack_ws, self.pack_bytes, s)
        return out

    def few(self, x: torch.Tensor, logits: torch.Tensor, bias: torch.Tensor | None = None) -> torch.Tensor:
        """The layer applied to n tokens, 0 to TOPO_FEW_MAX_TOKENS of them whatever
        cfg's T: x bf16 [n, H]; logits float32 or bf16 [n, E]; bias float32 [E] or
        None; returns bf16 [n, H].  The activations keep 16 bits, so the result is
        nearer to the weights' own than forward()'s.  Calls of few() may overlap one
        another and a forward(), on several streams or in graphs."""
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x must be a tensor [n, H]")
        n = x.shape[0]
        if n > TOPO_FEW_MAX_TOKENS or self.few_bytes == 0:
            raise ValueError(f"few() takes up to {TOPO_FEW_MAX_TOKENS} tokens, H and I up to 32768")
        need("x", x, (torch.bfloat16,), n, self.H, self.device)
        need("logits", logits, (torch.float32, torch.bfloat16), n, self.E, self.device)
        if bias is not None:
            need("bias", bias, (torch.float32,), 1, self.E, self.device)
        if self.planner.stream is None:                         # the caller's own: nothing to order
            return self._few(n, x, logits, bias)
        with ordered(self.planner.stream, self.device, x, logits, bias) as outs:
            outs.append(self._few(n, x, logits, bias))
        return outs[0]

    def _few(self, n, x, logits, bias):
        s, out = self.planner._stream(), torch.empty_like(x)
        if n:
            # this call's alone (a captured call's in its graph's memory): calls on several
            # streams and graphs that hold one may run at once.  The workspace, the weights behind it
            cfg, nb = self._few_sizes(n)
            ids = torch.empty((n, self.k), dtype=torch.int32, device=self.device)
            scratch = torch.empty(nb // 4 + n * self.k, dtype=torch.float32, device=self.device)
            ws = scratch.data_ptr()
            topo_route(cfg, 1, self.route, logits, TOPO_DTYPE_F32 if logits.dtype == torch.float32 else TOPO_DTYPE_BF16,
                       bias, ids, ws + nb, None, ws, nb, s)
            topo_expert_few(n, self.E, self.k, self.H, self.I, self.fmt, x, ids, ws + nb, self.up.q, self.up.scale,
                            self.up.row, self.down.q, self.down.scale, self.down.row, out, ws, nb, s)
            self.few_ids = ids                                  # the last call's
        return out

    def _few_sizes(self, n):
        """The routing's configuration and the workspace's bytes for n tokens."""
        if n not in self.few_sizes:
            self.few_sizes[n] = (make_cfg(n, self.E, self.k, 1, 1, 0),
                                 topo_few_workspace_bytes(n, self.E, self.k, self.H, self.I))
        return self.few_sizes[n]

    def _rows8(self, x):
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
        scale = torch.empty((x.shape[0], blocks(x.shape[1])), dtype=torch.float32, device=x.device)
        topo_quantize_rows(x.shape[0], x.shape[1], x, q, scale, self.planner._stream())
        return q, scale

    def _weight_grad(self, dy, x):
        """[E, N, K] from rows dy [rows, N] and x [rows, K]: instances' gradients summed by expert."""
        P, s, dev = self.planner, self.planner._stream(), dy.device
        cap = topo_cols_capacity(self.n_seg, self.rows)
        ops = []
        for v in (dy, x):
            q = torch.empty((v.shape[1], cap), dtype=torch.uint8, device=dev)
            scale = torch.empty((cap // TOPO_BLOCK, v.shape[1]), dtype=torch.float32, device=dev)
            topo_quantize_cols(self.n_seg, self.rows, v.shape[1], v, P.buf.seg_off, cap, q, scale, self.ws,
                               self.ws_bytes, s)
            ops += [q, scale]
        N, K = dy.shape[1], x.shape[1]
        dw = torch.empty((self.n_seg, N, K), dtype=torch.float32, device=dev)
        topo_expert_wgrad(self.n_seg, self.rows, N, K, cap, *ops, P.buf.seg_off, dw, self.ws, self.ws_bytes, s)
        # an expert's instances one after the other, its main one first, then its
        # replicas by rank: the same bits each time (float32 atomics would not give that)
        seg = self.seg_w.view(self.R, -1)
        inst = torch.arange(self.n_seg, device=dev).view(self.R, -1)
        m = self.E // self.R
        out = dw[inst[:, :m].reshape(-1)[torch.argsort(seg[:, :m].reshape(-1))]]
        for i, e in zip(inst[:, m:].reshape(-1).tolist(), seg[:, m:].reshape(-1).tolist()):
            if e >= 0:
                out[e] += dw[i]
        return out

    def backward(self, x: torch.Tensor, logits: torch.Tensor, dout: torch.Tensor):
        """Gradients of the last forward(x, logits) for dout ([T, H], bf16 or any
        floating type, any strides): x (bf16), logits (their type), w_up and
        w_down (float32, by expert)."""
        if not self.train:
            raise RuntimeError("ExpertLayer was built without train=True")
        need("x", x, (torch.bfloat16,), self.T, self.H, self.device)
        if not isinstance(dout, torch.Tensor) or not dout.is_floating_point():
            raise TypeError("dout must be a tensor of floating point")
        if dout.numel() != self.T * self.H or dout.shape[-1] != self.H or dout.device != x.device:
            raise ValueError(f"dout must hold {self.T} x {self.H} values on {x.device}, is {list(dout.shape)}")
        with ordered(self.planner.stream, self.device, x, logits, dout) as outs:
            outs += self._backward(x, logits, dout)
        return tuple(outs)

    def _backward(self, x, logits, dout):
        P, s = self.planner, self.planner._stream()
        pair = P.buf.sorted_pairs[0].long()
        token = pair // self.k
        # combine: out[t] = sum_j w[t, j] y[pos(t, j)]
        d = dout.reshape(self.T, self.H)[token].float()
        dw = torch.empty(self.rows, dtype=torch.float32, device=x.device)
        dw[pair] = (self.y.float() * d).sum(-1)
        dy = (d * self.weights.reshape(-1)[pair][:, None]).to(torch.bfloat16)
        dlogits = torch.empty_like(logits)
        P.route_grad(logits, self.ids, dw, dlogits, self.route)
        # down product and activation
        da = torch.empty((self.rows, self.I), dtype=torch.bfloat16, device=x.device)
        self._product(*self._rows8(dy), self.I, self.H, self.down.qt, self.down.scale_t, da)
        dh = torch.empty_like(self.h)
        topo_swiglu_grad(self.rows, self.I, self.h, da, dh, s)
        # the rows of the product as the forward pass had them, rounded to e4m3; laid out
        # for the weight gradient they are rounded a second time, down their columns
        act = (self.aq.view(torch.float8_e4m3fn).float()
               * self.as_.repeat_interleave(TOPO_BLOCK, 1)[:, :self.I]).to(torch.bfloat16)
        dw_down = self._weight_grad(dy, act)
        # up product and dispatch: a token's gradient is the sum over its pairs
        dxr = torch.empty((self.rows, self.H), dtype=torch.bfloat16, device=x.device)
        self._product(*self._rows8(dh), self.H, 2 * self.I, self.up.qt, self.up.scale_t, dxr)
        dx = torch.empty_like(x)
        topo_combine(P.cfg, 1, self.H, dxr, P.buf.sorted_pairs, torch.ones_like(self.weights), dx, self.pack_ws,
                     self.pack_bytes, s)
        dw_up = self._weight_grad(dh, x.view(self.T, self.H)[token])
        return dx, dlogits, dw_up, dw_down

    def error(self) -> int:
        """First device error word of the layer's workspaces (synchronises the device).
        few() has none to report: its ids come from the routing, all in range."""
        return self.planner.error() or topo_read_error(self.pack_ws) or topo_read_error(self.ws)
