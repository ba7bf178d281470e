"""One GPU's share of the expert-parallel MoE layer, with its buffers
allocated once (capacity-sized, so every call has static sizes and no host
synchronisation, the property the Moreh report's "Using HIP Graphs" section
asks of an EP decode step).

    route -> layout -> dispatch -> gate/up (+SwiGLU) -> down -> combine

(with int8 experts a quantisation of h between gate/up and down).  A layer made
for training also keeps 8-bit checkpoints on the way and has the backward pass:

    dgrad of down -> SwiGLU backwards -> wgrad of down -> dgrad of gate/up ->
    wgrad of gate/up -> combine of the rows' gradients -> route backwards
Every stage is one call into libmoeep; this class only owns the buffers
and orders the calls on one stream.
"""
from __future__ import annotations

import torch

from . import (CKPT_BLOCK, FP8_BLOCK, moe_checkpoint_rows, moe_combine, moe_dispatch, moe_ffn_dgrad, moe_ffn_down,
               moe_ffn_gate_up, moe_ffn_gate_up_train, moe_ffn_wgrad, moe_layout, moe_layout_masked,
               moe_layout_workspace_bytes, moe_quant_rows, moe_route, moe_route_backward, moe_route_mapped,
               moe_route_scored, moe_route_shared, moe_swiglu_backward)

_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


class MoELayer:
    """Buffers and stage order for one layer shape.

    seg_rows: tokens per simulated source segment (T = sum); E routed experts,
    K per token; H hidden, I expert intermediate; local experts
    [e_begin, e_end); act_dtype stores Xd and h ('f32' | 'bf16' | 'fp8' |
    'int8': a scale for each token in Xd and h and for each output channel of
    the weights; gate/up's bf16 h is quantised in a stage of its own);
    y_dtype / out_dtype store the expert outputs and the combined rows.
    layout: 'contiguous' (rows of the local experts back to back, cap_rows
    rows, default T*K) or 'masked' (a fixed block of cap_per_expert rows per
    local expert, default T -- no slot can be dropped).
    n_shared: always-on shared experts (every token, gate 1), run as experts
    E, E+1, ... of the same grouped FFN; the local range must end at E and the
    weights hold the shared experts after the routed ones.  self.E, self.K
    and self.e_end then count them (self.E_routed, self.K_routed do not).
    router: None routes by moe_route's rule (top-K logits, softmax over the
    picks); a dict of moe_route_scored's keywords (score, n_groups,
    topk_groups, group_top, renorm, scale) routes by that call, with the
    balance bias (E,) in self.router_bias when set.  moe_route_scored takes a
    placement map beside shared experts; the map then covers the routed ids.
    train: forward keeps 8-bit checkpoints of x (a row a token) and of the gate and
    up products, and backward() gives the gradients; 'f32' or 'bf16' storage, the
    contiguous layout.  The checkpoints, the routing and the layout of the last
    forward are what backward() works from.
    """

    def __init__(self, seg_rows, E, K, H, I, e_begin, e_end, act_dtype, y_dtype, out_dtype,
                 device="cuda", cap_rows=None, layout="contiguous", cap_per_expert=None, n_shared=0,
                 router=None, train=False):
        self.router = None if router is None else dict(router)
        if self.router is not None:
            unknown = set(self.router) - {"score", "n_groups", "topk_groups", "group_top", "renorm", "scale"}
            if unknown:
                raise ValueError(f"unknown router options {sorted(unknown)}")
        self.seg_rows = tuple(int(b) for b in seg_rows)
        self.T = sum(self.seg_rows)
        self.n_shared = int(n_shared)
        if self.n_shared and e_end != E:
            raise ValueError("shared experts need the local range to end at E")
        self.E_routed, self.K_routed = E, K
        E, K, e_end = E + self.n_shared, K + self.n_shared, e_end + self.n_shared
        self.E, self.K, self.H, self.I = E, K, H, I
        self.e_begin, self.e_end = e_begin, e_end
        self.E_loc = e_end - e_begin
        self.act_dtype, self.y_dtype, self.out_dtype = act_dtype, y_dtype, out_dtype
        if layout not in ("contiguous", "masked"):
            raise ValueError(f"unknown layout {layout!r}")
        self.masked = layout == "masked"
        self.train = bool(train)
        if self.train and (act_dtype not in ("f32", "bf16") or self.masked):
            raise ValueError("training needs f32 or bf16 storage and the contiguous layout")
        self.cap_e = (max(self.T, 1) if cap_per_expert is None else int(cap_per_expert)) if self.masked else None
        if self.masked:
            self.cap = self.E_loc * self.cap_e
        else:
            self.cap = self.T * K if cap_rows is None else int(cap_rows)
        # rows a routed local expert gets under balanced routing: the FFN tile-shape hint
        self.expected_rows = max(1, (self.T * self.K_routed) // self.E_routed)
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        # the training calls take the row count from the buffers' shapes: a row that the layout does
        # not know would count as an expert's
        T, cap = self.T, self.cap if self.train else max(self.cap, 1)
        self.topk_ids = torch.empty((T, K), **i32)
        self.topk_w = torch.empty((T, K), dtype=torch.float32, device=dev)
        self.counts = torch.empty(E, **i32)
        self.offsets = torch.empty(self.E_loc + 1, **i32)     # contiguous: offsets; masked: m (E_loc)
        self.row_of = torch.empty((T, K), **i32)
        self.src_of = torch.empty(max(cap, 1), **i32)
        self.layout_ws = torch.empty(max(moe_layout_workspace_bytes(T, K, E), 256),
                                     dtype=torch.uint8, device=dev)
        act = _TORCH[act_dtype]
        self.xd = torch.empty((cap, H), dtype=act, device=dev)
        self.h = torch.empty((cap, I), dtype=act, device=dev)
        fp8, int8 = act_dtype == "fp8", act_dtype == "int8"
        self.xd_scales = torch.empty((cap, -(-H // FP8_BLOCK)), dtype=torch.float32, device=dev) if fp8 else None
        self.h_scales = torch.empty((cap, -(-I // FP8_BLOCK)), dtype=torch.float32, device=dev) if fp8 else None
        self.h_act = None
        if int8:
            self.xd_scales = torch.empty(cap, dtype=torch.float32, device=dev)
            self.h_scales = torch.empty(cap, dtype=torch.float32, device=dev)
            self.h_act = torch.empty((cap, I), dtype=torch.bfloat16, device=dev)   # gate/up's h
        self.y = torch.empty((cap, H), dtype=_TORCH[y_dtype], device=dev)
        self.out = torch.empty((T, H), dtype=_TORCH[out_dtype], device=dev)
        # placement map (E,) int32 on the device, logical -> physical expert id; when
        # set, routing emits physical ids and [e_begin, e_end) is a physical range
        self.expert_map = None
        # balance bias (E,) fp32 on the device for the scored router (None: no bias)
        self.router_bias = None
        if self.train:
            f32 = dict(dtype=torch.float32, device=dev)
            i8 = dict(dtype=torch.int8, device=dev)
            rows = dict(dtype=act, device=dev)
            self.x_q = torch.empty((T, H), **i8)
            self.x_s = torch.empty((T, -(-H // CKPT_BLOCK)), **f32)
            self.gate_q, self.up_q = torch.empty((cap, I), **i8), torch.empty((cap, I), **i8)
            self.gate_s = torch.empty((cap, -(-I // CKPT_BLOCK)), **f32)
            self.up_s = torch.empty_like(self.gate_s)
            self.dh, self.dgate = torch.empty((cap, I), **rows), torch.empty((cap, I), **rows)
            self.dup, self.hw = torch.empty((cap, I), **rows), torch.empty((cap, I), **rows)
            self.dxd = torch.empty((cap, H), **rows)
            self.dx = torch.empty((T, H), **rows)
            self.dtopk_w = torch.empty((T, K), **f32)
            self.dlogits = torch.empty((T, self.E_routed), **f32)
            self._ones = torch.ones((T, K), **f32)

    # individual stages (each one library call) ---------------------------------
    def route(self, logits, stream=None):
        if self.router is not None:
            moe_route_scored(logits, self.K_routed, bias=self.router_bias, phys_of_logical=self.expert_map,
                             n_shared=self.n_shared, topk_ids=self.topk_ids, topk_w=self.topk_w, stream=stream,
                             **self.router)
        elif self.n_shared:
            if self.expert_map is not None:
                raise ValueError("a placement map with shared experts is not supported")
            moe_route_shared(logits, self.K_routed, self.n_shared, self.topk_ids, self.topk_w,
                             stream=stream)
        elif self.expert_map is None:
            moe_route(logits, self.K, self.topk_ids, self.topk_w, stream=stream)
        else:
            moe_route_mapped(logits, self.K, self.expert_map, self.topk_ids, self.topk_w, stream=stream)

    def layout(self, stream=None):
        if self.masked:
            moe_layout_masked(self.topk_ids, self.E, self.e_begin, self.e_end, self.cap_e, self.counts,
                              self.offsets[:self.E_loc], self.row_of, self.src_of, self.layout_ws,
                              stream=stream)
        else:
            moe_layout(self.topk_ids, self.E, self.e_begin, self.e_end, self.cap, self.counts,
                       self.offsets, self.row_of, self.src_of, self.layout_ws, stream=stream)

    @property
    def rows(self):
        """The FFN's row description: offsets (contiguous) or m (masked)."""
        return self.offsets[:self.E_loc] if self.masked else self.offsets

    def dispatch(self, x_segments, stream=None):
        x_segments = [x_segments] if isinstance(x_segments, torch.Tensor) else list(x_segments)
        moe_dispatch(x_segments, self.row_of, self.cap, self.act_dtype, self.xd, self.xd_scales,
                     stream=stream)
        if self.train:
            t = 0
            for x in x_segments:
                part = slice(t, t + x.shape[0])
                moe_checkpoint_rows(x, q=self.x_q[part], scales=self.x_s[part], stream=stream)
                t = part.stop

    def gate_up(self, w, stream=None):
        if self.train:
            moe_ffn_gate_up_train(self.xd, self.rows, w["gate"], w["up"], self.h, self.gate_q, self.gate_s, self.up_q,
                                  self.up_s, expected_rows=self.expected_rows, stream=stream)
            return
        moe_ffn_gate_up(self.xd, self.xd_scales, self.rows, w["gate"], w["up"],
                        w.get("gate_scale"), w.get("up_scale"), self.h if self.h_act is None else self.h_act,
                        self.h_scales if self.h_act is None else None, expected_rows=self.expected_rows, stream=stream, cap_per_expert=self.cap_e,
                        w_scales_pow2=bool(w.get("scales_pow2", False)))

    def quant_h(self, stream=None):
        """int8 only: gate/up's bf16 h to int8 rows and their scales."""
        moe_quant_rows(self.h_act, self.rows, cap_per_expert=self.cap_e, q=self.h, scales=self.h_scales,
                       stream=stream, E_loc=self.E_loc)

    def down(self, w, stream=None):
        moe_ffn_down(self.h, self.h_scales, self.rows, w["down"], w.get("down_scale"), self.y,
                     expected_rows=self.expected_rows, stream=stream, cap_per_expert=self.cap_e,
                     w_scales_pow2=bool(w.get("scales_pow2", False)))

    def combine(self, stream=None):
        moe_combine(self.y, self.row_of, self.topk_w, self.out, stream=stream)

    def stages(self, x_segments, logits, w):
        """(name, thunk) pairs of the six calls (int8: seven), in order."""
        quant = [("quant_h", lambda s=None: self.quant_h(s))] if self.h_act is not None else []
        return [("route", lambda s=None: self.route(logits, s)),
                ("layout", lambda s=None: self.layout(s)),
                ("dispatch", lambda s=None: self.dispatch(x_segments, s)),
                ("ffn_gate_up", lambda s=None: self.gate_up(w, s)),
                *quant,
                ("ffn_down", lambda s=None: self.down(w, s)),
                ("combine", lambda s=None: self.combine(s))]

    def forward(self, x_segments, logits, w, stream=None):
        for _, run in self.stages(x_segments, logits, w):
            run(stream)
        return self.out

    # the backward pass ----------------------------------------------------------
    def _need_dout(self, dout):
        if not isinstance(dout, torch.Tensor):
            raise TypeError("dout must be a torch.Tensor")
        # (a token's row is looked up in dout, and one that it lacks reads as zeros)
        if dout.dim() != 2 or dout.shape[0] < self.T or dout.shape[1] != self.H:
            raise ValueError(f"dout must have shape {(self.T, self.H)} (got {tuple(dout.shape)})")

    def dgrad_down(self, dout, w, stream=None):
        self._need_dout(dout)
        moe_ffn_dgrad(dout, self.offsets, w["down"], src_of=self.src_of, slots_per_token=self.K, dx=self.dh,
                      expected_rows=self.expected_rows, stream=stream)

    def swiglu_backward(self, stream=None):
        moe_swiglu_backward(self.dh, self.gate_q, self.gate_s, self.up_q, self.up_s, self.row_of, self.topk_w,
                            self.dgate, self.dup, self.hw, self.dtopk_w, stream=stream)

    def wgrad_down(self, dout, grads, accumulate=False, stream=None):
        self._need_dout(dout)
        moe_ffn_wgrad(dout, self.hw, self.offsets, src_of=self.src_of, slots_per_token=self.K, gather="dy",
                      base=grads["down"] if accumulate else None, dw=grads["down"],
                      expected_rows=self.expected_rows, stream=stream)

    def dgrad_gate_up(self, w, stream=None):
        moe_ffn_dgrad(self.dgate, self.offsets, w["gate"], dy2=self.dup, w2=w["up"], dx=self.dxd,
                      expected_rows=self.expected_rows, stream=stream)

    def wgrad_gate_up(self, grads, accumulate=False, stream=None):
        moe_ffn_wgrad(self.dgate, self.x_q, self.offsets, x_scales=self.x_s, dy2=self.dup, src_of=self.src_of,
                      slots_per_token=self.K, gather="x", base=grads["gate"] if accumulate else None,
                      base2=grads["up"] if accumulate else None, dw=grads["gate"], dw2=grads["up"],
                      expected_rows=self.expected_rows, stream=stream)

    def route_backward(self, logits, stream=None):
        kw = dict(score="picks")
        if self.router is not None:
            kw = dict(score=self.router.get("score", "sigmoid"), renorm=self.router.get("renorm", True),
                      scale=self.router.get("scale", 1.0))
        moe_route_backward(logits, self.topk_ids, self.dtopk_w, phys_of_logical=self.expert_map,
                           n_shared=self.n_shared, dlogits=self.dlogits, stream=stream, **kw)

    def backward_stages(self, dout, logits, w, grads, accumulate=False):
        """(name, thunk) pairs of the seven calls, in order."""
        if not self.train:
            raise ValueError("backward needs a layer made with train=True")
        return [("dgrad_down", lambda s=None: self.dgrad_down(dout, w, s)),
                ("swiglu_backward", lambda s=None: self.swiglu_backward(s)),
                ("wgrad_down", lambda s=None: self.wgrad_down(dout, grads, accumulate, s)),
                ("dgrad_gate_up", lambda s=None: self.dgrad_gate_up(w, s)),
                ("wgrad_gate_up", lambda s=None: self.wgrad_gate_up(grads, accumulate, s)),
                ("combine_backward", lambda s=None: moe_combine(self.dxd, self.row_of, self._ones, self.dx, stream=s)),
                ("route_backward", lambda s=None: self.route_backward(logits, s))]

    def new_grads(self, dtype=torch.float32):
        """Buffers for the weights' gradients: fp32, or bf16 for a bf16 layer."""
        kw = dict(dtype=dtype, device=self.out.device)
        return {"gate": torch.empty((self.E_loc, self.I, self.H), **kw),
                "up": torch.empty((self.E_loc, self.I, self.H), **kw),
                "down": torch.empty((self.E_loc, self.H, self.I), **kw)}

    def backward(self, dout, logits, w, grads, accumulate=False, stream=None):
        """Gradients of the last forward for dout (T, H), the loss gradient of its out in
        the storage type (rows behind the T tokens' are not read).  logits and w as
        forward took them; grads from new_grads(): the weights' gradients are written
        there (accumulate: added).  Returns dx (T, H) and dlogits (T, E), the layer's own
        buffers; dtopk_w holds the gradient of the routing weights.  dx is that of the
        experts; the router's projection, outside the layer, adds its own from dlogits."""
        for _, run in self.backward_stages(dout, logits, w, grads, accumulate):
            run(stream)
        return self.dx, self.dlogits


class MicroBatchedLayer:
    """The layer over two micro-batches on two streams (Moreh report,
    compute-communication overlapping: split the batch in two so one
    micro-batch's dispatch/combine runs under the other's expert GEMMs).

    The tokens are split at a segment boundary (or, for one segment, at its
    middle row).  Stream 0 runs micro-batch A's six calls; stream 1 runs B's
    route, layout and dispatch at once, starts B's GEMMs after A's, and B's
    combine follows them, so A's combine overlaps B's GEMMs and B's dispatch
    overlaps A's.  Per-token results equal the single-batch layer's bit for
    bit (every row is computed by the same kernels in the same order).
    Both streams have the default priority.
    """

    def __init__(self, seg_rows, *args, **kw):
        seg_rows = [int(b) for b in seg_rows]
        if len(seg_rows) > 1:
            cut = len(seg_rows) // 2
            self.parts = (seg_rows[:cut], seg_rows[cut:])
        else:
            half = seg_rows[0] // 2
            self.parts = ([half], [seg_rows[0] - half])
        if min(sum(p) for p in self.parts) < 1:
            raise ValueError("each micro-batch needs at least one token")
        self.a = MoELayer(self.parts[0], *args, **kw)
        self.b = MoELayer(self.parts[1], *args, **kw)
        self.T = self.a.T + self.b.T
        # the whole batch's tile-shape hint, so both halves use the single-batch kernels
        self.a.expected_rows = self.b.expected_rows = max(
            1, (self.T * self.a.K_routed) // self.a.E_routed)
        self.side = torch.cuda.Stream(device=self.a.out.device)   # default priority
        self._ev_a_ffn = torch.cuda.Event()
        self._ev_b_done = torch.cuda.Event()
        self._ev_start = torch.cuda.Event()

    def split_inputs(self, x_segments, logits):
        """(x segments, logits) of each micro-batch, as views of the inputs."""
        xs = list(x_segments)
        Ta = self.a.T
        if len(xs) > 1:
            cut = len(self.parts[0])
            xa, xb = xs[:cut], xs[cut:]
        else:
            xa, xb = [xs[0][:Ta]], [xs[0][Ta:]]
        return (xa, logits[:Ta]), (xb, logits[Ta:])

    def forward(self, x_segments, logits, w):
        """Enqueue both micro-batches; returns (out_a, out_b) (token order: A then B)."""
        (xa, la), (xb, lb) = self.split_inputs(x_segments, logits)
        main = torch.cuda.current_stream(self.side.device)
        self._ev_start.record(main)
        self.side.wait_event(self._ev_start)
        a, b = self.a, self.b
        a.route(la, main)
        a.layout(main)
        a.dispatch(xa, main)
        b.route(lb, self.side)
        b.layout(self.side)
        b.dispatch(xb, self.side)
        a.gate_up(w, main)
        if a.h_act is not None:
            a.quant_h(main)
        a.down(w, main)
        self._ev_a_ffn.record(main)
        a.combine(main)
        self.side.wait_event(self._ev_a_ffn)
        b.gate_up(w, self.side)
        if b.h_act is not None:
            b.quant_h(self.side)
        b.down(w, self.side)
        b.combine(self.side)
        self._ev_b_done.record(self.side)
        main.wait_event(self._ev_b_done)
        return a.out, b.out
