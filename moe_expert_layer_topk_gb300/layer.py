"""Buffers and call order of one MoE expert layer, of the block around it
(norms, gate, residual), and of a projection with per-request adapters, over
the C entry points.

`MoELayer` owns the device tensors one layer needs for a fixed token count
(outputs, activations kept for the backward pass, gradients, workspaces),
allocated once through torch, and issues the library calls in order on one
stream.  It adds no arithmetic of its own.
"""
from __future__ import annotations

import torch

from . import (moe_adapter_hidden_size, moe_adapter_linear, moe_adapter_linear_bwd,
               moe_adapter_linear_bwd_workspace_size, moe_balance_loss, moe_balance_loss_bwd, moe_balance_loss_workspace_size,
               moe_ckpt_pack, moe_ckpt_unpack, moe_combine, moe_combine_bwd,
               moe_combine_dropout, moe_combine_dropout_bwd, moe_combine_post_norm, moe_dispatch_bwd, moe_dispatch_chunked,
               moe_dispatch_e4m3_chunked, moe_dispatch_rows, moe_dropout, moe_grouped_gemm_bwd_workspace_size,
               moe_grouped_gemm_down, moe_grouped_gemm_down_bwd, moe_grouped_gemm_down_bwd_ckpt,
               moe_grouped_gemm_down_bwd_ckpt_workspace_size, moe_grouped_gemm_down_bwd_dw, moe_grouped_gemm_down_combine,
               moe_grouped_gemm_down_fp8,
               moe_grouped_gemm_swiglu, moe_grouped_gemm_swiglu_bwd_dw, moe_grouped_gemm_swiglu_bwd_dx,
               moe_grouped_gemm_swiglu_ckpt, moe_grouped_gemm_swiglu_fp8, moe_post_norm_bwd, moe_post_norm_bwd_workspace_size,
               moe_pre_norm, moe_pre_norm_bwd, moe_pre_norm_bwd_workspace_size, moe_set_gemm_sm_limit, sm_count,
               moe_grouped_gemm_swiglu_gather, moe_quantize_rows_e4m3, moe_route_topk_bwd,
               moe_route_topk_bwd_workspace_size, moe_route_topk_chunks,
               moe_route_topk_chunks_workspace_size, moe_route_topk_logits, moe_route_topk_logits_bwd)


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(256, (nbytes + 255) // 256 * 256), dtype=torch.uint8, device=device)


def _stream_of(stream, device):
    """torch's stream for what the calls take as one: None (the current one), an object, or a handle."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if hasattr(stream, "cuda_stream"):
        return stream
    return torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)


class MoELayer:
    """One layer's buffers for T tokens of hidden size H, E experts of size I, top-k.

    fused_dispatch (forward only): dispatch only ranks the slots and the
    gate/up GEMM reads its rows straight from x by token id, so x_perm is
    never written (moe_grouped_gemm_swiglu_gather).

    fp8 (forward only): dispatch writes the permuted rows as e4m3 codes with
    one scale per token (moe_dispatch_e4m3), h is quantised per row, and
    both GEMMs run on e4m3 weights prepared once by `quantize_weights` (one
    scale per output channel).

    fused_combine (forward only, bf16): the down GEMM adds each weighted row
    into its token's fp32 row and y is rounded from those
    (moe_grouped_gemm_down_combine), so y_perm is never written; the order
    of those fp32 additions is not fixed from run to run.  It saves the
    [T*k, H] y_perm buffer but measured slower than down + combine.

    balance_coef, z_coef (training): the forward also computes the router's
    load-balance loss and z-loss (`loss`, fp32 [2], unscaled) and the
    gradient of balance_coef loss[0] + z_coef loss[1] in the logits, which
    the backward adds to the router's (moe_balance_loss).  `sequences`
    packed sequences of the T tokens, told apart by the forward's
    seg_offsets, are each balanced on their own; tokens whose mask byte is 0
    take no part in the two losses.  The backward's dloss scales the two
    gradients.

    dropout (training): y = residual + D(combined rows) with the
    counter-based dropout of moe_combine_dropout; the backward computes the
    same mask again from `rng` (int64 [2] on the device: seed, offset), so
    rng has to hold the forward's words until the backward has run.
    `advance_rng` moves the offset past the layer's own counters.

    checkpoint (training): between forward and backward the layer keeps g and
    u in 8 bits (moe_grouped_gemm_swiglu_ckpt) and the routing, and nothing
    else of its activations; x_perm, h and y_perm are scratch, made again in
    the backward where it needs them.  share: another checkpointed layer of
    the same sizes on the same device, whose scratch this one uses as well
    (the layers of a model run one after another on one stream), so that
    only the kept tensors, the outputs and the gradients are a layer's own.
    checkpoint_input: x is kept in 8 bits too, and the backward's x may be
    None.  Gradients are those of the kept values: about 1% off.  With
    dropout, dy under the mask times 1/(1-p) is rounded to bf16 before it is
    permuted (the plain layer rounds the permuted rows, weighted, instead)."""

    def __init__(self, T: int, H: int, I: int, E: int, k: int, ep_size: int = 1, *,
                 training: bool = True, fused_dispatch: bool = False, fp8: bool = False,
                 fused_combine: bool = False, balance_coef: float = 0.0, z_coef: float = 0.0,
                 sequences: int = 1, dropout: float = 0.0, seed: int = 0,
                 checkpoint: bool = False, checkpoint_input: bool = False, share: "MoELayer | None" = None,
                 device: str | torch.device = "cuda"):
        if checkpoint and not training:
            raise ValueError("checkpoint belongs to a training layer")
        if (checkpoint_input or share is not None) and not checkpoint:
            raise ValueError("checkpoint_input and share belong to a checkpointed layer")
        if share is not None and (not share.checkpoint or (share.T, share.H, share.I, share.E, share.k) != (T, H, I, E, k)
                                  or share.y.device != torch.empty(0, device=device).device):
            raise ValueError("share must be a checkpointed layer of the same sizes on the same device")
        if fp8 and training:
            raise ValueError("the e4m3 path is forward only")
        if fused_combine and (training or fp8):
            raise ValueError("fused_combine is a bf16 forward-only path (the combine backward needs y_perm)")
        if fused_dispatch and training:
            raise ValueError("fused_dispatch keeps no x_perm, which the backward pass needs")
        if not training and (balance_coef or z_coef or dropout):
            raise ValueError("the balance loss, the z-loss and dropout belong to a training layer")
        self.T, self.H, self.I, self.E, self.k, self.ep_size = T, H, I, E, k, ep_size
        self.R = R = T * k
        self.training = training
        self.fused_dispatch = fused_dispatch
        self.fused_combine = fused_combine
        self.fp8 = fp8
        self.checkpoint, self.checkpoint_input = checkpoint, checkpoint_input
        self.balance_coef, self.z_coef, self.sequences, self.dropout = balance_coef, z_coef, sequences, dropout
        self.balanced = bool(balance_coef or z_coef)
        self._x = None
        self._upstream = False  # whether dlogits holds a backward's dloss
        self._side = None  # side stream of the backward's tail (created on first use)
        dev = torch.device(device)
        i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
        e = lambda *s, dt: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        self.topk_idx = e(T, k, dt=i32)
        self.topk_w = e(T, k, dt=f32)
        self.counts = e(E, dt=i32)
        self.offsets = e(E + 1, dt=i32)
        self.rank_offsets = e(ep_size + 1, dt=i32)
        own = share is None
        self.ws_route = _ws(moe_route_topk_chunks_workspace_size(T, H, E), dev) if own else share.ws_route
        # where each 16-token chunk starts in each expert's rows (from the route, for the dispatch)
        self.chunk_prefix = e(E, (T + 15) // 16, dt=i32)
        self.x_perm = None if (fused_dispatch or fp8) else e(R, H, dt=bf) if own else share.x_perm
        self.row_of_slot = e(T, k, dt=i32)
        self.token_of_row = e(R, dt=i32)
        self.h = e(R, I, dt=bf) if own else share.h
        self.gu = e(R, 2 * I, dt=bf) if training and not checkpoint else None
        self.y_perm = None if fused_combine else e(R, H, dt=bf) if own else share.y_perm
        self.y_acc = e(T, H, dt=f32) if fused_combine else None
        self.y = e(T, H, dt=bf)
        if fp8:
            u8 = torch.uint8
            self.x_q, self.x_scale = e(R, H, dt=u8), e(R, dt=f32)  # permuted rows, their tokens' scales
            self.h_q, self.h_scale = e(R, I, dt=u8), e(R, dt=f32)
        if checkpoint:
            i8 = torch.int8
            self.gu_q, self.gu_scale = e(R, 2 * I, dt=i8), e(R, 2 * I // 32, dt=bf)
            if checkpoint_input:
                self.x_kept, self.x_kept_scale = e(T, H, dt=i8), e(T, H // 32, dt=bf)
            # the tokens' values where they are made again: x from its codes, or dy under the dropout's mask
            self.tokens = e(T, H, dt=bf) if own else share.tokens
            self.row_w = e(R, dt=f32) if own else share.row_w
            self.ws_ckpt = _ws(moe_grouped_gemm_down_bwd_ckpt_workspace_size(R, I), dev) if own else share.ws_ckpt
        if training:
            self.dy_perm = e(R, H, dt=bf) if own else share.dy_perm
            self.d_w = e(T, k, dt=f32)
            self.dgu = e(R, 2 * I, dt=bf) if own else share.dgu
            self.dx_perm = e(R, H, dt=bf) if own else share.dx_perm
            self.dx_acc = e(T, H, dt=f32) if own else share.dx_acc
            self.dx = e(T, H, dt=bf)
            self.dWg = e(E, I, H, dt=f32)
            self.dWu = e(E, I, H, dt=f32)
            self.dWd = e(E, H, I, dt=f32)
            self.dWr = e(H, E, dt=f32)
            self.ws_route_bwd = _ws(moe_route_topk_bwd_workspace_size(T, H, E), dev) if own else share.ws_route_bwd
            self.ws_gemm_bwd = _ws(moe_grouped_gemm_bwd_workspace_size(E), dev) if own else share.ws_gemm_bwd
        if self.balanced:
            self.logits, self.dlogits = e(T, E, dt=f32), e(T, E, dt=f32)
            self.seq_counts, self.seq_tokens = e(sequences, E, dt=i32), e(sequences, dt=i32)
            self.prob_sum, self.loss = e(sequences, E, dt=f32), e(2, dt=f32)
            self.ws_balance = _ws(moe_balance_loss_workspace_size(T, E, sequences), dev)
        self.rng = torch.tensor([seed, 0], dtype=torch.int64, device=dev) if dropout else None

    # ---------------------------------------------------------------- forward
    def quantize_weights(self, Wg, Wu, Wd, stream=None):
        """e4m3 codes and per-output-channel scales of the expert weights."""
        E, H, I = self.E, self.H, self.I
        out = {}
        for name, W, rows, cols in (("Wg", Wg, E * I, H), ("Wu", Wu, E * I, H), ("Wd", Wd, E * H, I)):
            q = torch.empty(W.shape, dtype=torch.uint8, device=W.device)
            sc = torch.empty(rows, dtype=torch.float32, device=W.device)
            moe_quantize_rows_e4m3(W, rows, cols, q, sc, stream)
            out[name], out[name + "_scale"] = q, sc
        return out

    def route(self, x, Wr, bias=None, stream=None):
        if self.balanced:
            moe_route_topk_logits(x, Wr, bias, self.T, self.H, self.E, self.k, self.ep_size, self.topk_idx,
                                  self.topk_w, self.counts, self.offsets, self.rank_offsets, self.chunk_prefix,
                                  self.logits, self.ws_route, stream)
            return
        moe_route_topk_chunks(x, Wr, bias, self.T, self.H, self.E, self.k, self.ep_size, self.topk_idx,
                              self.topk_w, self.counts, self.offsets, self.rank_offsets, self.chunk_prefix,
                              self.ws_route, stream)

    def dispatch(self, x, stream=None):
        self._x = x  # the fused gate/up GEMM reads the rows from here
        if self.fp8:
            moe_dispatch_e4m3_chunked(x, self.topk_idx, self.offsets, self.chunk_prefix, self.T, self.H, self.E,
                                      self.k, self.x_q, self.x_scale, self.row_of_slot, self.token_of_row, stream)
            return
        if self.checkpoint_input:
            moe_ckpt_pack(x, self.T, self.H, self.x_kept, self.x_kept_scale, stream)
        moe_dispatch_chunked(x, self.topk_idx, self.offsets, self.chunk_prefix, self.T, self.H, self.E, self.k,
                             self.x_perm, self.row_of_slot, self.token_of_row, stream)

    def experts(self, Wg, Wu, Wd, stream=None, y=None):
        """Wg, Wu, Wd: bf16 expert weights, or (fp8 layers) the dict that
        `quantize_weights` returns, passed as Wg (Wu and Wd unused).
        y: the output of a fused_combine layer (default: the layer's own)."""
        if self.fp8:
            w = Wg
            T, H, I, E, R = self.T, self.H, self.I, self.E, self.R
            moe_grouped_gemm_swiglu_fp8(self.x_q, self.x_scale, None, 0, w["Wg"], w["Wg_scale"], w["Wu"],
                                        w["Wu_scale"], E, self.offsets, None, R, H, I, E, self.h, stream)
            moe_quantize_rows_e4m3(self.h, R, I, self.h_q, self.h_scale, stream)
            moe_grouped_gemm_down_fp8(self.h_q, self.h_scale, w["Wd"], w["Wd_scale"], E, self.offsets,
                                      None, R, H, I, E, self.y_perm, stream)
            return
        if self.fused_dispatch:
            moe_grouped_gemm_swiglu_gather(self._x, self.token_of_row, self.T, Wg, Wu, self.E,
                                           self.offsets, None, self.R, self.H, self.I, self.E, self.h,
                                           None, stream)
        else:
            if self.checkpoint:
                moe_grouped_gemm_swiglu_ckpt(self.x_perm, Wg, Wu, self.E, self.offsets, None, self.R, self.H, self.I, self.E,
                                             self.h, self.gu_q, self.gu_scale, stream)
            else:
                moe_grouped_gemm_swiglu(self.x_perm, Wg, Wu, self.E, self.offsets, None, self.R, self.H,
                                        self.I, self.E, self.h, self.gu, None, stream)
        if self.fused_combine:
            moe_grouped_gemm_down_combine(self.h, Wd, self.E, self.offsets, None, self.R, self.H, self.I,
                                          self.E, self.token_of_row, self.row_of_slot, self.topk_w, self.T,
                                          self.k, self.y_acc, self.y if y is None else y, stream)
            return
        moe_grouped_gemm_down(self.h, Wd, self.E, self.offsets, None, self.R, self.H, self.I,
                              self.E, self.y_perm, None, stream)

    def balance(self, mask=None, seg_offsets=None, stream=None):
        """The two router losses of the routed tokens and their gradient in the logits."""
        moe_balance_loss(self.logits, self.topk_idx, mask, self.T, self.E, self.k, self.sequences, seg_offsets,
                         self.seq_counts, self.seq_tokens, self.prob_sum, self.loss, self.balance_coef, self.z_coef,
                         self.dlogits, self.ws_balance, stream)
        self._losses_of, self._upstream = (mask, seg_offsets), False

    def advance_rng(self, stream=None):
        """Move the dropout's offset past one forward's counters, on `stream` like the other
        calls (a layer without dropout has none)."""
        if not self.dropout:
            return
        with torch.cuda.stream(_stream_of(stream, self.rng.device)):
            self.rng[1] += self.T * self.H // 8

    def combine(self, stream=None, y=None, residual=None):
        if self.dropout or residual is not None:
            moe_combine_dropout(self.y_perm, self.topk_w, self.row_of_slot, residual, self.T, self.H, self.k,
                                self.dropout, self.rng if self.dropout else self._no_rng(), self.y if y is None else y,
                                stream)
            return
        moe_combine(self.y_perm, self.topk_w, self.row_of_slot, self.T, self.H, self.k,
                    self.y if y is None else y, stream)

    def _no_rng(self):
        if self.rng is None:  # a residual without dropout: the words are read, not used
            self.rng = torch.zeros(2, dtype=torch.int64, device=self.y.device)
        return self.rng

    def forward(self, x, Wr, bias, Wg, Wu, Wd, stream=None, y=None, *, residual=None, mask=None, seg_offsets=None):
        """y: optional bf16 [T,H] output tensor (default: the layer's own).
        residual: bf16 [T,H] added to the output (its gradient is dy).
        mask, seg_offsets: uint8 [T] and int32 [sequences + 1] of the two router losses."""
        if self.fused_combine and residual is not None:
            raise ValueError("a fused_combine layer adds no residual")
        self.route(x, Wr, bias, stream)
        if self.balanced:
            self.balance(mask, seg_offsets, stream)
        self.dispatch(x, stream)
        self.experts(Wg, Wu, Wd, stream, y)
        if not self.fused_combine:
            self.combine(stream, y, residual)
        return self.y if y is None else y

    def capture_forward(self, x, Wr, bias, Wg, Wu, Wd, *, residual=None, mask=None,
                        seg_offsets=None) -> "torch.cuda.CUDAGraph":
        """Record forward() on these tensors as a CUDA graph and return it.

        `graph.replay()` then re-runs the whole forward (all its kernels,
        one launch from the host) on whatever the same tensors hold, into
        the layer's own y: for small batches, whose forward is bound by the
        host issuing one call per kernel.  One forward runs first, outside
        the capture, so that each call's first-use set-up (kernel
        attributes, the device status word) is done before it."""
        opts = dict(residual=residual, mask=mask, seg_offsets=seg_offsets)
        self.forward(x, Wr, bias, Wg, Wu, Wd, **opts)
        torch.cuda.synchronize(self.y.device)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.forward(x, Wr, bias, Wg, Wu, Wd, **opts)
        return graph

    # --------------------------------------------------------------- backward
    # SMs left free for the backward's tail (dispatch and router backward, on
    # a side stream) while the gate/up weight-gradient GEMM runs: measured at
    # T=8192 on GB300, the two together took 514 us this way against 558 us
    # one after the other (525 us on two streams with no limit).
    TAIL_SMS = 16

    def backward(self, dy, x, Wr, Wg, Wu, Wd, accumulate: bool = False, stream=None, dx=None,
                 overlap: bool = True, dloss=None):
        """dx: optional bf16 [T,H] output tensor (default: the layer's own).
        x: the forward's, or None for a checkpoint_input layer.

        dloss: fp32 [2] on the device, the upstream gradients of the two
        router losses (loss scaling, the weight of a micro-batch; default
        1), which balance_coef and z_coef are multiplied by; the forward's
        mask and seg_offsets have to hold what they held then.

        overlap: run the dispatch and router backward on a side stream beside
        the gate/up weight gradient (which then leaves TAIL_SMS SMs free);
        the results are the same either way, and the call returns with the
        work of both streams ordered before anything later on `stream`."""
        assert self.training, "layer was built without backward buffers"
        dx = self.dx if dx is None else dx
        T, H, I, E, k, R = self.T, self.H, self.I, self.E, self.k, self.R
        if dloss is not None and not self.balanced:
            raise ValueError("dloss belongs to a layer with a balance loss or a z-loss")
        if self.balanced and (dloss is not None or self._upstream):  # else dlogits is the forward's
            mask, seg_offsets = self._losses_of
            moe_balance_loss_bwd(self.logits, mask, T, E, k, self.sequences, seg_offsets, self.seq_counts, self.seq_tokens,
                                 self.balance_coef, self.z_coef, dloss, self.dlogits, stream)
            self._upstream = dloss is not None
        if x is None and not self.checkpoint_input:
            raise ValueError("the backward needs x unless the layer keeps it (checkpoint_input)")
        if self.checkpoint:
            x = self._experts_bwd_checkpointed(dy, x, Wd, accumulate, stream)
        elif self.dropout:
            moe_combine_dropout_bwd(dy, self.y_perm, self.topk_w, self.row_of_slot, T, H, k, self.dropout, self.rng,
                                    self.dy_perm, self.d_w, stream)
        else:
            moe_combine_bwd(dy, self.y_perm, self.topk_w, self.row_of_slot, T, H, k, self.dy_perm,
                            self.d_w, stream)
        if not self.checkpoint:
            moe_grouped_gemm_down_bwd(self.dy_perm, self.h, self.gu, Wd, E, self.offsets, None, R, H, I,
                                      E, self.dgu, self.dWd, accumulate, self.ws_gemm_bwd, stream)
        moe_grouped_gemm_swiglu_bwd_dx(self.dgu, Wg, Wu, E, self.offsets, None, R, H, I, E, self.dx_perm,
                                       stream)
        tail = stream
        if overlap:
            main = _stream_of(stream, self.dx_perm.device)
            if self._side is None:
                self._side = torch.cuda.Stream(self.dx_perm.device)
                self._ev_fork, self._ev_join = torch.cuda.Event(), torch.cuda.Event()
            self._ev_fork.record(main)
            self._side.wait_event(self._ev_fork)
            tail = self._side
            prev = moe_set_gemm_sm_limit(max(1, sm_count(self.dx_perm.device) - self.TAIL_SMS))
            try:
                moe_grouped_gemm_swiglu_bwd_dw(self.dgu, self.x_perm, E, self.offsets, None, R, H, I, E, self.dWg,
                                               self.dWu, accumulate, self.ws_gemm_bwd, main)
            finally:
                moe_set_gemm_sm_limit(prev)
        else:
            moe_grouped_gemm_swiglu_bwd_dw(self.dgu, self.x_perm, E, self.offsets, None, R, H, I, E, self.dWg,
                                           self.dWu, accumulate, self.ws_gemm_bwd, stream)
        moe_dispatch_bwd(self.dx_perm, self.row_of_slot, T, H, k, self.dx_acc, tail)
        if self.balanced:
            moe_route_topk_logits_bwd(self.d_w, self.topk_w, self.topk_idx, self.dlogits, x, Wr, self.dx_acc, T, H, E,
                                      k, self.dWr, dx, accumulate, self.ws_route_bwd, tail)
        else:
            moe_route_topk_bwd(self.d_w, self.topk_w, self.topk_idx, x, Wr, self.dx_acc, T, H, E, k,
                               self.dWr, dx, accumulate, self.ws_route_bwd, tail)
        if overlap:
            self._ev_join.record(self._side)
            main.wait_event(self._ev_join)
        return dx

    def _experts_bwd_checkpointed(self, dy, x, Wd, accumulate, stream):
        """The backward of combine and down projection from the kept codes (fills d_w, dgu and
        dWd), and the experts' rows of x made again; returns the x that the router's backward uses."""
        T, H, I, E, k, R = self.T, self.H, self.I, self.E, self.k, self.R
        if self.dropout:  # rounded to bf16 here, as moe_combine_dropout_bwd rounds its rows: the products take bf16
            moe_dropout(dy, None, T * H, self.dropout, self.rng, self.tokens, stream)
            dy = self.tokens
        moe_dispatch_rows(dy, None, self.row_of_slot, self.topk_w, T, H, k, self.dy_perm, self.row_w, stream)
        moe_grouped_gemm_down_bwd_ckpt(self.dy_perm, self.row_w, self.gu_q, self.gu_scale, Wd, E, self.offsets, None, R, H, I,
                                       E, self.dgu, self.h, self.d_w, self.row_of_slot, T, k, self.ws_ckpt, stream)
        moe_grouped_gemm_down_bwd_dw(self.dy_perm, self.h, E, self.offsets, None, R, H, I, E, self.dWd, accumulate,
                                     self.ws_gemm_bwd, stream)
        if x is None:
            moe_ckpt_unpack(self.x_kept, self.x_kept_scale, T, H, self.tokens, stream)
            x = self.tokens
        moe_dispatch_rows(x, None, self.row_of_slot, None, T, H, k, self.x_perm, None, stream)
        return x


class _Normed(tuple):
    """(n, rstd) as a block leaves them for the next one, and the eps that they were made with.  scratch: n is memory that
    blocks share, which holds it only until the next of them runs, forward or backward; else both stay until that block's
    own next forward."""

    def __new__(cls, n, rstd, eps, scratch):
        self = super().__new__(cls, (n, rstd))
        self.eps, self.scratch = eps, scratch
        return self


class MoEBlock:
    """An MoE layer between its norms, with the block's gate and the residual:

        out = res_scale x + out_scale sigmoid(gate) norm(MoE(norm(x) pre_gain)) post_gain

    over moe_pre_norm, MoELayer and moe_combine_post_norm.  The residual
    stream (x, out, dout, dx) is bf16, or fp32 with fp32=True.  gate: None,
    "token" (fp32 logits [T]) or "element" (bf16 logits [T,H]).  post_norm
    False leaves the second norm out (its gain stays).  Further options are
    MoELayer's (`checkpoint` and `share`, the router losses; no dropout).

    Gains are fp32 [H] or None (ones).  Blocks one after another: with
    next_norm=True a block also computes the next one's normed input on the
    way, with that one's pre_gain as next_gain, and leaves it and its rstd in
    `next_normed`, which that one's forward takes as `normed`, before any other
    block that shares their scratch runs.  One eps serves a block's two norms and the
    next one's: a block refuses a next_normed made with another eps than its
    own.  Plain and checkpointed blocks may follow one another: what a backward needs of `normed` and the block before does not
    keep (a checkpointed block's n is scratch), and any other tensors given as
    `normed`, are copied into the block's own.

    After the backward: d_pre_gain, d_post_gain (fp32 [H]), d_gate (like the
    gate), and the layer's gradients (`layer.dWg` ...).  A checkpointed
    block keeps z (bf16 [T,H]) beside what its layer keeps, and norms x
    again in the backward."""

    def __init__(self, T: int, H: int, I: int, E: int, k: int, ep_size: int = 1, *, gate: str | None = None,
                 post_norm: bool = True, eps: float = 1e-6, res_scale: float = 1.0, out_scale: float = 1.0, fp32: bool = False,
                 next_norm: bool = False, training: bool = True, share: "MoEBlock | None" = None,
                 device: str | torch.device = "cuda", **options):
        if gate not in (None, "token", "element"):
            raise ValueError("gate must be None, 'token' or 'element'")
        if options.get("dropout") or options.get("fused_combine") or options.get("checkpoint_input"):
            raise ValueError("a block takes no dropout, fused_combine or checkpoint_input")
        self.layer = MoELayer(T, H, I, E, k, ep_size, training=training, share=share.layer if share is not None else None,
                              device=device, **options)
        self.T, self.H, self.training, self.gate, self.post_norm = T, H, training, gate, post_norm
        self.eps, self.res_scale, self.out_scale = eps, res_scale, out_scale
        dev = torch.device(device)
        e = lambda *s, dt: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        f32, bf = torch.float32, torch.bfloat16
        stream_type = f32 if fp32 else bf
        self.checkpoint = self.layer.checkpoint
        self.n = share.n if share is not None else e(T, H, dt=bf)
        self.rstd = e(T, dt=f32)
        self.out = e(T, H, dt=stream_type)
        # a checkpointed block has no more use for n by then
        self.next_n = (self.n if self.checkpoint else e(T, H, dt=bf)) if next_norm else None
        self.next_rstd = e(T, dt=f32) if next_norm else None
        self._normed = None
        self.z = self.post_rstd = None
        if training:
            self.z, self.post_rstd = e(T, H, dt=bf), e(T, dt=f32) if post_norm else None
            self.dz = e(T, H, dt=bf) if share is None else share.dz
            self.dx = e(T, H, dt=stream_type)
            self.d_pre_gain, self.d_post_gain = e(H, dt=f32), e(H, dt=f32)
            self.d_gate = e(T, dt=f32) if gate == "token" else e(T, H, dt=bf) if gate == "element" else None
            self.ws_norm = _ws(max(moe_pre_norm_bwd_workspace_size(T, H), moe_post_norm_bwd_workspace_size(T, H)), dev)

    @property
    def next_normed(self):
        """The next block's normed input and its rstd (after a forward, with next_norm)."""
        return _Normed(self.next_n, self.next_rstd, self.eps, self.checkpoint)

    def _keep(self, normed, stream):
        """The normed input and the rstd, where they last until the backward: n in a plain block (a
        checkpointed one makes it again), rstd in both."""
        n, rstd = normed
        known = isinstance(normed, _Normed)
        if not (self.checkpoint or (known and not normed.scratch)):
            with torch.cuda.stream(_stream_of(stream, self.n.device)):
                n = self.n.copy_(n)
        if not known and rstd is not None:
            with torch.cuda.stream(_stream_of(stream, self.rstd.device)):
                rstd = self.rstd.copy_(rstd)
        return n, rstd

    def _check_gate(self, gate):
        if (gate is None) != (self.gate is None):
            raise ValueError("the block was built %s a gate" % ("without" if self.gate is None else "with"))
        if gate is not None and gate.dtype != (torch.float32 if self.gate == "token" else torch.bfloat16):
            raise ValueError("a token's gate is fp32, an element's bf16")

    def forward(self, x, pre_gain, post_gain, Wr, bias, Wg, Wu, Wd, gate=None, stream=None, out=None, *, normed=None,
                next_gain=None, mask=None, seg_offsets=None):
        """out (default: the block's own) of x.  normed: (n, rstd) as the block before left them
        (its next_normed, for this block's pre_gain), or tensors like them, made with this block's eps; else the block norms x itself.  next_gain:
        the next block's pre_gain, of a block with next_norm."""
        self._check_gate(gate)
        if next_gain is not None and self.next_n is None:
            raise ValueError("next_gain belongs to a block built with next_norm")
        if isinstance(normed, _Normed) and normed.eps != self.eps:
            raise ValueError("normed was made with eps %g, this block's is %g" % (normed.eps, self.eps))
        T, H, L = self.T, self.H, self.layer
        out = self.out if out is None else out
        if normed is None:
            n, rstd = self.n, self.rstd
            moe_pre_norm(x, pre_gain, self.eps, T, H, n, rstd, stream)
        else:
            n, rstd = self._keep(normed, stream) if self.training else normed
        self._normed = n, rstd
        L.route(n, Wr, bias, stream)
        if L.balanced:
            L.balance(mask, seg_offsets, stream)
        L.dispatch(n, stream)
        L.experts(Wg, Wu, Wd, stream)
        moe_combine_post_norm(L.y_perm, L.topk_w, L.row_of_slot, x, post_gain, self.post_norm, self.eps, gate, self.res_scale,
                              self.out_scale, T, H, L.k, self.z, out, self.post_rstd, next_gain, self.next_n, self.next_rstd,
                              stream)
        return out

    def backward(self, dout, x, pre_gain, post_gain, Wr, Wg, Wu, Wd, gate=None, accumulate: bool = False, stream=None, dx=None,
                 overlap: bool = True, dloss=None):
        """After the forward of the same x: the gradients of the parameters and of the gate, and dx
        (default: the block's own), which may be dout.  accumulate adds to the parameters' gradients;
        d_gate, of this batch's tokens, is overwritten."""
        assert self.training, "block was built without backward buffers"
        self._check_gate(gate)
        T, H, L = self.T, self.H, self.layer
        dx = self.dx if dx is None else dx
        n, rstd = self._normed
        moe_post_norm_bwd(dout, self.z, post_gain, self.post_norm, self.post_rstd, gate, self.out_scale, T, H, self.dz,
                          self.d_post_gain, self.d_gate, accumulate, self.ws_norm, stream)
        if self.checkpoint:  # n was scratch
            n = self.n
            moe_pre_norm(x, pre_gain, self.eps, T, H, n, None, stream)
        dn = L.backward(self.dz, n, Wr, Wg, Wu, Wd, accumulate, stream, overlap=overlap, dloss=dloss)
        moe_pre_norm_bwd(dn, x, pre_gain, rstd, dout, self.res_scale, T, H, dx, self.d_pre_gain, accumulate, self.ws_norm, stream)
        return dx


class AdapterLinear:
    """Buffers of a projection W [N,K] shared by all requests, with a low-rank
    adapter of rank r for each request, for up to T rows of up to `requests`
    requests: moe_adapter_linear and (training) moe_adapter_linear_bwd.

    The rows of a call are x's; seg_offsets (int32 [n + 1]) cuts them into n
    requests and seg_adapter (int32 [n]) names each one's adapter, -1 for
    none.  Prompts and single tokens may be mixed in one call."""

    def __init__(self, T: int, K: int, N: int, r: int, num_adapters: int, requests: int, *, training: bool = False,
                 device: str | torch.device = "cuda"):
        self.T, self.K, self.N, self.r, self.num_adapters, self.requests = T, K, N, r, num_adapters, requests
        self.training = training
        dev = torch.device(device)
        e = lambda *s, dt: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        f32, bf = torch.float32, torch.bfloat16
        self.y = e(T, N, dt=bf)
        self.hidden = _ws(moe_adapter_hidden_size(T, r), dev)
        if training:
            self.dx = e(T, K, dt=bf)
            self.dA, self.dB = e(num_adapters, r, K, dt=f32), e(num_adapters, N, r, dt=f32)
            self.ws_bwd = _ws(moe_adapter_linear_bwd_workspace_size(T, K, N, r, requests), dev)

    def forward(self, x, W, A, B, scale, seg_offsets, seg_adapter, stream=None, y=None):
        """x bf16 [rows, K], rows <= T; returns y (default: the rows of the layer's own)."""
        n = x.shape[0]
        y = self.y[:n] if y is None else y
        moe_adapter_linear(x, W, A, B, scale, seg_adapter.numel(), seg_offsets, seg_adapter, n, self.K, self.N, self.r,
                           self.num_adapters, self.hidden, y, stream)
        return y

    def backward(self, dy, x, W, A, B, scale, seg_offsets, seg_adapter, accumulate: bool = False, stream=None, dx=None):
        """After the forward of the same rows: fills dA, dB (fp32) and returns dx."""
        assert self.training, "layer was built without backward buffers"
        n = x.shape[0]
        dx = self.dx[:n] if dx is None else dx
        moe_adapter_linear_bwd(dy, x, W, A, B, scale, self.hidden, seg_adapter.numel(), seg_offsets, seg_adapter, n,
                               self.K, self.N, self.r, self.num_adapters, dx, self.dA, self.dB, accumulate, self.ws_bwd,
                               stream)
        return dx
