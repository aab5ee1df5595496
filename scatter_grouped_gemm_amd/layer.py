"""The MoE expert path as one layer over libmoe's C calls.

forward(x, logits):  route -> scatter (compact or masked; FP8: fused UE8M0
quant) -> w13 grouped GEMM -> SiLU-and-mul (FP8: fused requant) -> w2 grouped
GEMM -> weighted combine.  Every buffer has a static shape fixed at
construction from (max_tokens, k, num_local_experts, block_e), so a forward
never reads device data back to the host and can be captured in a HIP graph.

Layout choice: ``layout="auto"`` takes the policy measured on MI355X
(moe_choose_layout: masked while experts hold at most 64 rows on average and
its buffers stay within 4x the compact bound, compact beyond); ``layout="rule"``
takes the rule of "Support
DeepGEMM for standard MoE dispatch", implementation breakdown item 2 (masked
when there are non-local experts and at most 32 local ones).  The activation dtype
follows the weights ("[Feature] Support BF16 and batch-invariant inference
with DeepEP v2", implementation breakdown item 2): FP8 weights make the path
FP8, and asking for the other dtype is an error.

Training (``train=True``, BF16 weights, compact layout): forward keeps what the
gradients need in its own buffers and backward(dout) walks the same steps back --
combine, w2 (weight, then input), SiLU-and-mul, w13 (weight, then input),
scatter -- with no further host work; optimizer() gives the AdamW step over the
expert weights.  The gradient products end at 1,044,480 rows (8160 blocks of 128);
a training layer with more is refused.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .optim import AdamW


class MoELayer:
    def __init__(self, *, hidden: int, intermediate: int, num_experts: int, top_k: int,
                 max_tokens: int, num_local_experts: int | None = None, expert_start: int = 0,
                 fp8: bool = False, layout: str = "auto", block_e: int = 128,
                 max_m: int | None = None, expected_m: int = 0, fuse_silu: bool = True,
                 weight_format: str | None = None, train: bool = False,
                 grad_dtype: torch.dtype = torch.bfloat16, device="cuda"):
        self.H, self.I, self.E, self.k = hidden, intermediate, num_experts, top_k
        self.El = num_local_experts or num_experts
        self.expert_start = expert_start
        self.fp8 = fp8
        # FP8 weights: 128x128 UE8M0 blocks (default) or "mxfp8" (one exponent
        # per 32 k of a weight row); activations are FP8 with 128-channel scales
        # either way
        if weight_format not in (None, "block128", "mxfp8", "mxfp4"):
            raise ValueError(f"unknown weight format {weight_format!r}")
        if weight_format in ("mxfp8", "mxfp4") and not fp8:
            raise ValueError("MX weights need the FP8 activation path")
        self.weight_format = weight_format or ("block128" if fp8 else "bf16")
        self.mx = self.weight_format in ("mxfp8", "mxfp4")
        self.wdt = self.weight_format if self.mx else fp8
        self.block_e = block_e
        self.T_max = max_tokens
        self.device = torch.device(device)
        self.train = train
        if train:
            if fp8:
                raise ValueError("training needs BF16 weights: quantised weights have no gradient")
            if layout not in ("auto", "compact"):
                raise ValueError("training uses the compact layout")
            if grad_dtype not in (torch.bfloat16, torch.float32):
                raise ValueError(f"weight gradients are bf16 or fp32, not {grad_dtype}")
            layout, fuse_silu = "compact", False     # backward needs the gate and up halves
        self.grad_dtype = grad_dtype
        if layout == "auto":
            layout = "masked" if L.moe_choose_layout(max_tokens, top_k, self.E, self.El, block_e) else "compact"
        elif layout == "rule":
            layout = "masked" if L.moe_use_masked_layout(self.E, self.El) else "compact"
        if layout not in ("compact", "masked"):
            raise ValueError(f"unknown layout {layout!r}")
        self.layout = layout
        # w13 with SiLU-and-mul in its epilogue (bit-identical to the two calls)
        self.fuse_silu = fuse_silu
        self.max_m = max_m if max_m is not None else max_tokens
        self.expected_m = expected_m
        d, T, H, I, El, k = self.device, max_tokens, hidden, intermediate, self.El, top_k
        if layout == "compact":
            self.rows = L.moe_compact_rows_bound(T * k, El, block_e)
        else:
            self.rows = El * self.max_m
        R = self.rows
        if train:        # before any memory is taken: forward alone runs with more rows
            for n, kk in ((2 * I, H), (H, I)):
                if not L.grouped_gemm_grads_supported(R, n, kk, El):
                    raise ValueError(f"training: the gradient products do not cover {R} rows, {El} experts of {n} x {kk}")
        adt = torch.uint8 if fp8 else torch.bfloat16
        # static buffers (uninitialised: every valid row is written before it is read)
        self.topk_ids = torch.empty(T, k, dtype=torch.int32, device=d)
        self.topk_weights = torch.empty(T, k, dtype=torch.float32, device=d)
        self.src2dst = torch.empty(T, k, dtype=torch.int32, device=d)
        self.x_buf = torch.empty(R, H, dtype=adt, device=d)
        self.x_scale = torch.empty(R * (H // 128), dtype=torch.uint8, device=d) if fp8 else None
        self.gateup = None if fuse_silu else torch.empty(R, 2 * I, dtype=torch.bfloat16, device=d)
        self.act = torch.empty(R, I, dtype=adt, device=d)
        self.act_scale = torch.empty(R * (I // 128), dtype=torch.uint8, device=d) if fp8 else None
        self.y = torch.empty(R, H, dtype=torch.bfloat16, device=d)
        self.out = torch.empty(T, H, dtype=torch.bfloat16, device=d)
        if layout == "compact":
            self.m_indices = torch.empty(R, dtype=torch.int32, device=d)
            self.expert_start_loc = torch.empty(El, dtype=torch.int32, device=d)
            self.num_valid = torch.empty(El, dtype=torch.int32, device=d)
            self.masked_m = None
        else:
            self.m_indices = None
            self.masked_m = torch.empty(El, dtype=torch.int32, device=d)
        ws_bytes = L.moe_scatter_ws_bytes(T, k, El, H)
        self.ws = torch.empty((ws_bytes + 3) // 4, dtype=torch.int32, device=d)
        self.w13 = self.w2 = self.w13_scale = self.w2_scale = None
        if train:
            self.dy = torch.empty(R, H, dtype=torch.bfloat16, device=d)
            self.dx = torch.empty(T, H, dtype=torch.bfloat16, device=d)
            self.dtopk_weights = torch.empty(T, k, dtype=torch.float32, device=d)
            self.dlogits = torch.empty(T, self.E, dtype=torch.float32, device=d)
        self.dw13 = self.dw2 = None
        self._saved = None        # what the last forward left for backward
        # optional timing: name -> list of (start, end) HIP events recorded on
        # the current stream around each step of forward()
        self.marks = None

    def _mark(self, name):
        if self.marks is None:
            return _NoMark()
        return _Mark(self.marks.setdefault(name, []))

    # -- weights ---------------------------------------------------------------------

    def allocate_weights(self):
        if self.train and self.w13 is not None:      # an optimizer may hold them
            return
        d, El, H, I = self.device, self.El, self.H, self.I
        wdt = torch.uint8 if self.fp8 else torch.bfloat16
        half = 2 if self.weight_format == "mxfp4" else 1      # e2m1: two k per byte
        self.w13 = torch.empty(El, 2 * I, H // half, dtype=wdt, device=d)
        self.w2 = torch.empty(El, H, I // half, dtype=wdt, device=d)
        if self.mx:
            self.w13_scale = torch.empty(El, 2 * I // 64, H // 128, 256, dtype=torch.uint8, device=d)
            self.w2_scale = torch.empty(El, H // 64, I // 128, 256, dtype=torch.uint8, device=d)
        elif self.fp8:
            self.w13_scale = torch.empty(El, 2 * I // 128, H // 128, dtype=torch.uint8, device=d)
            self.w2_scale = torch.empty(El, H // 128, I // 128, dtype=torch.uint8, device=d)

    def set_expert(self, e: int, w13: torch.Tensor, w2: torch.Tensor):
        """Load local expert e from bf16 weights ([2I, H] and [H, I]); FP8 layers
        quantise them to 128x128 blocks with UE8M0 scales in the library."""
        if self.w13 is None:
            self.allocate_weights()
        if not self.fp8:
            self.w13[e].copy_(w13)
            self.w2[e].copy_(w2)
            return
        if self.mx:
            f = "e4m3" if self.weight_format == "mxfp8" else "e2m1"
            L.moe_quant_weight_mx(w13.contiguous()[None], f, self.w13[e:e + 1], self.w13_scale[e:e + 1])
            L.moe_quant_weight_mx(w2.contiguous()[None], f, self.w2[e:e + 1], self.w2_scale[e:e + 1])
            return
        L.moe_quant_weight_fp8_ue8m0(w13.contiguous()[None], self.w13[e:e + 1], self.w13_scale[e:e + 1])
        L.moe_quant_weight_fp8_ue8m0(w2.contiguous()[None], self.w2[e:e + 1], self.w2_scale[e:e + 1])

    def set_weights(self, w13: torch.Tensor, w2: torch.Tensor):
        for e in range(self.El):
            self.set_expert(e, w13[e], w2[e])

    def set_block_fp8_weights(self, w13q, w13s, w2q, w2s):
        """Take block-FP8 checkpoint weights (e4m3 bytes, one fp32 scale per
        128x128 block: w13 [El,2I,H] + [El,2I/128,H/128], w2 [El,H,I] +
        [El,H/128,I/128]) and requantise them in the library to UE8M0 scales
        through bf16."""
        if not self.fp8:
            raise ValueError("block-FP8 weights given to a BF16 layer: the activation dtype follows the weights")
        if self.weight_format != "block128":
            raise ValueError("block-FP8 checkpoint weights requantise to 128x128 UE8M0 blocks")
        if self.w13 is None:
            self.allocate_weights()
        L.moe_requant_weight_fp8_ue8m0(w13q.contiguous(), w13s.contiguous(), self.w13, self.w13_scale)
        L.moe_requant_weight_fp8_ue8m0(w2q.contiguous(), w2s.contiguous(), self.w2, self.w2_scale)

    def set_quantized_weights(self, w13q, w13s, w2q, w2s):
        """Take already block-quantised FP8 weights (e4m3 bytes + UE8M0 bytes)."""
        if not self.fp8:
            raise ValueError("FP8 weights given to a BF16 layer: the activation dtype follows the weights")
        self.w13, self.w13_scale, self.w2, self.w2_scale = w13q, w13s, w2q, w2s

    # -- forward ----------------------------------------------------------------------

    def route(self, logits: torch.Tensor):
        T = logits.shape[0]
        L.moe_route_topk(logits, self.k, self.topk_ids[:T], self.topk_weights[:T])

    def forward(self, x: torch.Tensor, logits: torch.Tensor | None = None, *,
                topk_ids: torch.Tensor | None = None, topk_weights: torch.Tensor | None = None):
        T = x.shape[0]
        if T > self.T_max:
            raise ValueError(f"{T} tokens exceed the layer's static capacity {self.T_max}")
        self._saved = None       # from here on the buffers are no longer the last forward's
        if topk_ids is None:
            with self._mark("route"):
                self.route(logits)
            ids, tw = self.topk_ids[:T], self.topk_weights[:T]
        else:
            ids, tw = topk_ids, topk_weights
        s2d = self.src2dst[:T]
        fp8, wdt = self.fp8, self.wdt
        I = self.I
        if self.layout == "compact":
            with self._mark("scatter"):
                L.moe_scatter_compact(x, ids, self.expert_start, self.El, self.block_e, self.rows,
                                      fp8, self.x_buf, self.x_scale, self.m_indices,
                                      self.expert_start_loc, self.num_valid, s2d, self.ws)
            if self.fuse_silu:
                with self._mark("gemm_w13_silu"):
                    L.grouped_gemm_contig_silu(wdt, self.x_buf, self.x_scale, self.w13, self.w13_scale,
                                               self.act, self.m_indices, self.act_scale)
            else:
                with self._mark("gemm_w13"):
                    L.grouped_gemm_contig(wdt, self.x_buf, self.x_scale, self.w13, self.w13_scale,
                                          self.gateup, self.m_indices)
                with self._mark("silu_and_mul"):
                    L.silu_and_mul(self.gateup, self.act, fp8, self.act_scale, m_indices=self.m_indices)
            with self._mark("gemm_w2"):
                L.grouped_gemm_contig(wdt, self.act, self.act_scale, self.w2, self.w2_scale, self.y,
                                      self.m_indices)
        else:
            El, mm = self.El, self.max_m
            with self._mark("scatter"):
                L.moe_scatter_masked(x, ids, self.expert_start, El, mm, fp8, self.x_buf,
                                     self.x_scale, self.masked_m, s2d, self.ws)
            if self.fuse_silu:
                with self._mark("gemm_w13_silu"):
                    L.grouped_gemm_masked_silu(wdt, self.x_buf.view(El, mm, self.H), self.x_scale,
                                               self.w13, self.w13_scale, self.act.view(El, mm, I),
                                               self.masked_m, self.expected_m, self.act_scale)
            else:
                with self._mark("gemm_w13"):
                    L.grouped_gemm_masked(wdt, self.x_buf.view(El, mm, self.H), self.x_scale,
                                          self.w13, self.w13_scale, self.gateup.view(El, mm, 2 * I),
                                          self.masked_m, self.expected_m)
                with self._mark("silu_and_mul"):
                    L.silu_and_mul(self.gateup, self.act, fp8, self.act_scale, masked_m=self.masked_m,
                                   max_m=mm)
            with self._mark("gemm_w2"):
                L.grouped_gemm_masked(wdt, self.act.view(El, mm, I), self.act_scale, self.w2,
                                      self.w2_scale, self.y.view(El, mm, self.H), self.masked_m,
                                      self.expected_m)
        out = self.out[:T]
        with self._mark("combine"):
            L.moe_combine(self.y, s2d, tw, out)
        if self.train:
            self._saved = (T, ids, tw, topk_ids is None)
        return out

    __call__ = forward

    # -- training ---------------------------------------------------------------------

    def allocate_grads(self):
        """The weight gradients dw13 [El, 2I, H] and dw2 [El, H, I], zero (in
        place where the layer has them).  A captured backward needs them allocated before."""
        if not self.train:
            raise ValueError("the layer was made without train=True")
        if self.dw13 is not None:        # an optimizer may hold them
            self.dw13.zero_()
            self.dw2.zero_()
            return
        self.dw13 = torch.zeros(self.El, 2 * self.I, self.H, dtype=self.grad_dtype, device=self.device)
        self.dw2 = torch.zeros(self.El, self.H, self.I, dtype=self.grad_dtype, device=self.device)

    def backward(self, dout: torch.Tensor, *, accumulate: bool = False):
        """Gradients of the last forward: writes (or, accumulate, adds to) dw13 and
        dw2 and returns (dx [T, H], dlogits [T, E]), or (dx, dtopk_weights [T, k])
        where forward was given topk_ids.  The results are the layer's own buffers.

        With a share of the experts, dx and dlogits are that share's part: both
        add up over the shares.  What forward kept is used up: one backward for
        each forward that came to its end, and ids and weights given to forward
        must still be as they were."""
        if not self.train:
            raise ValueError("the layer was made without train=True")
        if self._saved is None:
            raise ValueError("backward needs a forward of its own before it")
        T, ids, tw, routed = self._saved
        if dout.shape != (T, self.H):
            raise ValueError(f"dout: want {(T, self.H)}, got {tuple(dout.shape)}")
        if self.dw13 is None:
            # zeroed in the graph, they would be so again in every replay
            if self.device.type == "cuda" and torch.cuda.is_current_stream_capturing():
                raise ValueError("call allocate_grads() before backward is captured")
            self.allocate_grads()
        s2d, dx, dtw = self.src2dst[:T], self.dx[:T], self.dtopk_weights[:T]
        m_idx, starts, counts = self.m_indices, self.expert_start_loc, self.num_valid
        with self._mark("combine_bwd"):
            L.moe_combine_bwd(dout, self.y, s2d, tw, self.dy, dtw)
        self._saved = None
        if routed:
            with self._mark("route_bwd"):
                L.moe_route_topk_bwd(ids, tw, dtw, self.dlogits[:T])
        with self._mark("wgrad_w2"):
            L.grouped_gemm_contig_wgrad(self.dy, self.act, starts, counts, self.dw2, accumulate)
        dact = self.act          # the activation has been used: its buffer takes the gradient
        with self._mark("dgrad_w2"):
            L.grouped_gemm_contig_dgrad(self.dy, self.w2, dact, m_idx)
        with self._mark("silu_bwd"):
            L.silu_and_mul_bwd(self.gateup, dact, self.gateup, m_indices=m_idx)
        with self._mark("wgrad_w13"):
            L.grouped_gemm_contig_wgrad(self.gateup, self.x_buf, starts, counts, self.dw13, accumulate)
        with self._mark("dgrad_w13"):
            L.grouped_gemm_contig_dgrad(self.gateup, self.w13, self.y, m_idx)
        with self._mark("scatter_bwd"):
            L.moe_scatter_bwd(self.y, s2d, dx)
        return dx, (self.dlogits[:T] if routed else dtw)

    def optimizer(self, **kw) -> AdamW:
        """AdamW (optim.AdamW's arguments) over the expert weights and their gradients."""
        if not self.train:
            raise ValueError("the layer was made without train=True")
        if self.w13 is None:
            raise ValueError("set the weights first: the masters are taken from them")
        if self.dw13 is None:
            self.allocate_grads()
        return AdamW([self.w13, self.w2], [self.dw13, self.dw2], **kw)


class _NoMark:
    def __enter__(self):
        return self

    def __exit__(self, *a):
        return False


class _Mark:
    """Records a (start, end) pair of HIP events on the current stream."""

    def __init__(self, sink):
        self.sink = sink

    def __enter__(self):
        self.start = torch.cuda.Event(enable_timing=True)
        self.end = torch.cuda.Event(enable_timing=True)
        self.start.record()
        return self

    def __exit__(self, *a):
        self.end.record()
        self.sink.append((self.start, self.end))
        return False
