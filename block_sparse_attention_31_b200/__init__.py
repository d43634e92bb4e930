"""Spatial-temporal block-sparse self-attention for video diffusion transformers on B200.

The compute lives in ``libvsa.so`` (hand-written CUDA for sm_100a behind the C ABI in
``include/vsa.h``).  This package is its thin Python binding: ``_lib`` mirrors each C entry
point under the same name, and :class:`SparseAttention` owns the device buffers (from
PyTorch) of one configured call and invokes ``vsa_attention`` (``vsa_attention_host`` for
host batches).
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Sequence

import torch

from . import _lib
from ._lib import _on, _on_16_bytes
from ._lib import (VSA_BF16, VSA_CUBE, VSA_F32, VSA_SELECT_CUBE, VSA_SELECT_GIVEN, VSA_SELECT_PROFILE, VSA_SPATIAL,
                   VSA_TEMPORAL, Params, QKVO, Shape, VsaError, make_params, make_shape, qkvo, vsa_attention,
                   vsa_attention_workspace_layout, vsa_attention_workspace_size, vsa_block_order,
                   vsa_build_mask, vsa_get_device_error, vsa_layout_rows, vsa_mask_workspace_size, vsa_max_kv, vsa_num_blocks,
                   vsa_pattern_window, vsa_permute, vsa_profile_heads, vsa_profile_rows, vsa_profile_workspace_size,
                   vsa_sparse_attn_fwd, vsa_sparse_attn_fwd_natural, vsa_unpermute, SemParams, make_sem_params,
                   vsa_quantize_fp8, vsa_sparse_attn_fwd_fp8qk, QKVOGrad, qkvo_grad, vsa_sparse_attn_bwd,
                   vsa_sparse_attn_bwd_workspace_size, vsa_attention_bwd, vsa_attention_bwd_workspace_size,
                   vsa_attention_train, vsa_attention_train_workspace_size,
                   NormShape, make_norm_shape, vsa_rms_norm, vsa_rms_norm_bwd, vsa_rms_norm_bwd_workspace_size,
                   vsa_gather_rows, vsa_kmeans, vsa_kmeans_workspace_size, vsa_scatter_rows, vsa_semantic_attention,
                   vsa_semantic_mask, vsa_semantic_mask_workspace_size, vsa_semantic_workspace_size)

_SELECT = {"profile": VSA_SELECT_PROFILE, "given": VSA_SELECT_GIVEN, "cube": VSA_SELECT_CUBE}
_DTYPE = {torch.float32: VSA_F32, torch.bfloat16: VSA_BF16}


class _HostPipelined:
    """run_host for a configured call: subclasses provide __call__(q, k, v, out=, kinds=, stream=)
    and the attributes B, H, N, d, dtype and device."""

    def run_host(self, batches, outs=None, kinds: Optional[torch.Tensor] = None, timing=None):
        """Run the call on a sequence of host batches with the transfers overlapped: while call i
        computes, the inputs of call i+1 upload and the output of call i-1 downloads (three
        streams, two device buffer sets).  ``batches`` is a list of (q, k, v) CPU tensors, which
        must be pinned for the copies to overlap; ``outs`` is a list of CPU output tensors
        (pinned ones are allocated when None).  Returns ``outs`` once every output has arrived.
        The log-sum-exp, when configured, stays on the device and is not returned.  ``timing``, a
        pair of timing-enabled CUDA events, is recorded before the first upload and after the
        last download."""
        n = len(batches)
        shape = (self.B, self.H, self.N, self.d)
        if outs is None:
            outs = [torch.empty(shape, dtype=self.dtype).pin_memory() for _ in range(n)]
        if len(outs) != n:
            raise ValueError("need one output tensor per batch")
        for (q, k, v), o in zip(batches, outs):
            for t in (q, k, v, o):
                if t.device.type != "cpu" or t.dtype != self.dtype or tuple(t.shape) != shape:
                    raise ValueError(f"host tensors of shape {shape} and dtype {self.dtype} expected")
        if not hasattr(self, "_host_bufs"):
            self._host_bufs = [[torch.empty(shape, dtype=self.dtype, device=self.device) for _ in range(4)]
                               for _ in range(2)]  # q, k, v, o per buffer set
            self._streams = [torch.cuda.Stream(self.device) for _ in range(3)]  # upload, compute, download
        up, comp, down = self._streams
        ev = lambda: torch.cuda.Event()  # noqa: E731
        up_done, comp_done, down_done = [], [], []
        up.wait_stream(torch.cuda.current_stream(self.device))
        if timing is not None:
            timing[0].record(up)
        for i, ((q, k, v), o) in enumerate(zip(batches, outs)):
            dq, dk, dv, do = self._host_bufs[i % 2]
            with torch.cuda.stream(up):
                if i >= 2:
                    up.wait_event(comp_done[i - 2])  # call i-2 has read this buffer set
                dq.copy_(q, non_blocking=True)
                dk.copy_(k, non_blocking=True)
                dv.copy_(v, non_blocking=True)
                up_done.append(ev())
                up_done[i].record(up)
            with torch.cuda.stream(comp):
                comp.wait_event(up_done[i])
                if i >= 2:
                    comp.wait_event(down_done[i - 2])  # call i-2's output has left this buffer
                self(dq, dk, dv, out=do, kinds=kinds, stream=comp)
                comp_done.append(ev())
                comp_done[i].record(comp)
            with torch.cuda.stream(down):
                down.wait_event(comp_done[i])
                o.copy_(do, non_blocking=True)
                down_done.append(ev())
                down_done[i].record(down)
        if timing is not None:
            timing[1].record(down)
        down.synchronize()
        return outs


def _no_capture(what: str):
    # Autograd hands a leaf's gradient over on the stream on which the leaf's node was first used.  Under
    # capture that can be a stream outside it, which ends the process; explicit calls have no such node.
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{what} records a graph of autograd, which cannot be captured: capture the call and "
                           f"its backward method instead")


def _check_outputs(plan, out, lse):
    """Outputs that a caller gives are written as whole rows from their first address."""
    for t, dtype, n, what in ((out, plan.dtype, plan.B * plan.H * plan.N * plan.d, "out"),
                              (lse, torch.float32, plan.B * plan.H * plan.N, "lse")):
        if t is not None and (t.dtype != dtype or t.device != plan.device or t.numel() != n or not t.is_contiguous()):
            raise ValueError(f"{what} must be a contiguous {dtype} tensor of {n} elements on {plan.device}")


class _Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, q, k, v, kinds):
        ctx.set_materialize_grads(False)
        with _on(None, plan.device):
            o_lo = torch.empty_like(q, memory_format=torch.contiguous_format)
            o, lse = plan(q, k, v, kinds=kinds, o_lo=o_lo)
            ctx.plan = plan
            ctx.save_for_backward(q, k, v, o, lse, plan.kinds.clone(), o_lo)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_o):
        if d_o is None:
            return (None,) * 5
        _no_capture("attend")
        q, k, v, o, lse, kinds, o_lo = ctx.saved_tensors
        grads = ctx.plan.backward(d_o.contiguous(), q, k, v, o, lse, kinds=kinds, o_lo=o_lo)
        return (None, *(g if need else None for g, need in zip(grads, ctx.needs_input_grad[1:4])), None)


class SparseAttention(_HostPipelined):
    """One configured attention call over a B x H x (F x Hl x Wl) x d problem.

    select:  "profile" (heads pick spatial/temporal by online profiling), "given" (kinds
             passed per call) or "cube" (own cube + top-k pooled cubes for every head).
    Windows: pass ``w_s``/``w_t`` directly, or ``target`` (a kept-block fraction) to use the
             smallest windows reaching it.
    layout_in_kernel: temporal heads are gathered through the frame-major map inside the
             attention kernel instead of being permuted into copies (bf16, no cube dims).
    qk_fp8:  Q.K^T on e4m3 codes with one power-of-two scale per block; P.V stays bf16
             (bf16, d = 128, block 128).
    with_grad: the plan also holds the workspace of the gradient (``backward``, ``attend``); the
             call then always returns its log-sum-exp, and fills ``o_lo``, where it is given, with
             what rounding the output to bf16 left over (for a more exact gradient).  Not with
             qk_fp8.

    A plan's workspaces serve one call at a time: order calls on different streams, and graphs
    that captured them, before they run, or give each its own plan.  A call runs, with all that it
    reads (``kinds`` too) and allocates, on ``stream`` (a torch stream or a raw handle), by default the
    device's current one.
    """

    def __init__(self, B: int, H: int, F: int, Hl: int, Wl: int, d: int, block: int = 128, *,
                 dtype: torch.dtype = torch.bfloat16, select: str = "profile", w_s: Optional[int] = None,
                 w_t: Optional[int] = None, target: Optional[float] = None, topk: int = 0,
                 cube: Optional[Sequence[int]] = None, profile_frac: float = 0.01, scale: float = 0.0,
                 with_lse: bool = False, layout_in_kernel: bool = False, qk_fp8: bool = False,
                 with_grad: bool = False, device="cuda"):
        if dtype not in _DTYPE:
            raise ValueError(f"unsupported dtype {dtype}")
        if with_grad and qk_fp8:
            raise ValueError("the e4m3 codes of qk_fp8 have no gradient")
        self.B, self.H, self.F, self.Hl, self.Wl, self.d, self.block = B, H, F, Hl, Wl, d, block
        self.N = F * Hl * Wl
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.dtype, self.select, self.device = dtype, _SELECT[select], dev
        self.shape = make_shape(B, H, F, Hl, Wl, d, block, tuple(cube) if cube else None)
        if target is not None:
            w_s_t, self.kept_s = vsa_pattern_window(self.shape, VSA_SPATIAL, target)
            w_t_t, self.kept_t = vsa_pattern_window(self.shape, VSA_TEMPORAL, target)
            w_s = w_s_t if w_s is None else w_s
            w_t = w_t_t if w_t is None else w_t
        self.w_s, self.w_t = int(w_s or 0), int(w_t or 0)
        self.params = make_params(self.w_s, self.w_t, profile_frac, topk, scale, layout_in_kernel, qk_fp8)
        size = vsa_attention_train_workspace_size if with_grad else vsa_attention_workspace_size
        self.ws_bytes = size(self.shape, self.params, _DTYPE[dtype], self.select)
        if self.ws_bytes == 0:
            raise VsaError(_lib.VSA_ERR_INVALID_ARG, "vsa_attention_workspace_size")
        off_bits, off_idx, off_cnt, self.max_kv = vsa_attention_workspace_layout(self.shape, self.params,
                                                                                 _DTYPE[dtype], self.select)
        self.nblk = vsa_num_blocks(self.shape)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        nwords = (self.nblk + 31) // 32
        rows = B * H * self.nblk
        self.bits = self.ws[off_bits:off_bits + rows * nwords * 4].view(torch.int32).view(B, H, self.nblk, nwords)
        self.kv_idx = self.ws[off_idx:off_idx + rows * self.max_kv * 4].view(torch.int32).view(B, H, self.nblk,
                                                                                               self.max_kv)
        self.kv_cnt = self.ws[off_cnt:off_cnt + rows * 4].view(torch.int32).view(B, H, self.nblk)
        self.kinds = torch.zeros(B * H, dtype=torch.uint8, device=self.device)
        self.mse = torch.zeros(B * H * 2, dtype=torch.float32, device=self.device)
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.with_lse = with_lse or with_grad
        self.with_grad = with_grad
        if with_grad:
            self.ws_bwd_bytes = vsa_attention_bwd_workspace_size(self.shape, self.params, _DTYPE[dtype])
            if self.ws_bwd_bytes == 0:
                raise VsaError(_lib.VSA_ERR_UNSUPPORTED, "vsa_attention_bwd_workspace_size")
            self.ws_bwd = torch.empty(self.ws_bwd_bytes, dtype=torch.uint8, device=self.device)
            self.kinds_bwd = torch.full((B * H,), VSA_CUBE, dtype=torch.uint8, device=self.device)  # or given ones, cast

    def __call__(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, kinds: Optional[torch.Tensor] = None, stream=None,
                 o_lo: Optional[torch.Tensor] = None):
        if o_lo is not None and not self.with_grad:
            raise ValueError("o_lo needs with_grad=True")
        for t in (q, k, v) if o_lo is None else (q, k, v, o_lo):
            if t.dtype != self.dtype or t.device != self.device or not t.is_contiguous():
                raise ValueError("q, k, v must be contiguous tensors of the configured dtype and device")
            if tuple(t.shape) != (self.B, self.H, self.N, self.d):
                raise ValueError(f"expected shape {(self.B, self.H, self.N, self.d)}, got {tuple(t.shape)}")
        _check_outputs(self, out, lse)
        if self.select == VSA_SELECT_GIVEN and kinds is None:
            raise ValueError("select='given' needs kinds")
        with _on(stream, self.device):
            if out is None:
                out = torch.empty_like(q)
            if self.with_lse and lse is None:
                lse = torch.empty(self.B, self.H, self.N, dtype=torch.float32, device=self.device)
            if self.select == VSA_SELECT_GIVEN:
                self.kinds.copy_(kinds.reshape(-1).to(torch.uint8))
            if o_lo is not None:
                vsa_attention_train(qkvo(q, k, v, out, lse), o_lo, _DTYPE[self.dtype], self.shape, self.params, self.select,
                                    self.kinds, self.mse, self.ws, self.ws_bytes, self.err)
            else:
                vsa_attention(qkvo(q, k, v, out, lse), _DTYPE[self.dtype], self.shape, self.params, self.select, self.kinds,
                              self.mse, self.ws, self.ws_bytes, self.err)
        return (out, lse) if self.with_lse else out

    def backward(self, d_o: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                 lse: torch.Tensor, kinds: Optional[torch.Tensor] = None, d_lse: Optional[torch.Tensor] = None,
                 out: Optional[Sequence[torch.Tensor]] = None, stream=None, o_lo: Optional[torch.Tensor] = None):
        """Gradients (dq, dk, dv) of a call of this plan, from its inputs, its outputs (``o_lo`` among
        them, where the call filled it) and the gradients of those (``lse`` and ``d_lse`` with any strides).
        ``kinds`` are the call's: as given, or ``plan.kinds`` as the call left them (a copy, where another
        call comes between); they are not needed for select="cube".  Nothing else of the call is kept: the
        masks are built again.  Asynchronous on ``stream``; can be captured."""
        if not self.with_grad:
            raise ValueError("the plan was made without with_grad=True")
        shape = (self.B, self.H, self.N, self.d)
        with _on(stream, self.device):
            if out is None:
                out = tuple(torch.empty(shape, dtype=self.dtype, device=self.device) for _ in range(3))
            if len(out) != 3:
                raise ValueError("out is (dq, dk, dv)")
            for t in (d_o, q, k, v, o, *out) if o_lo is None else (d_o, q, k, v, o, *out, o_lo):
                if t.dtype != self.dtype or t.device != self.device or not t.is_contiguous() or tuple(t.shape) != shape:
                    raise ValueError(f"contiguous {self.dtype} tensors of shape {shape} on {self.device} expected")
            d_o = _on_16_bytes(d_o)  # autograd may hand over a slice
            for t in (lse, d_lse):
                if t is not None and (t.dtype != torch.float32 or t.device != self.device or tuple(t.shape) != shape[:3]):
                    raise ValueError(f"lse and d_lse are float32 tensors of shape {shape[:3]} on {self.device}")
            if self.select != VSA_SELECT_CUBE:
                if kinds is None:
                    raise ValueError("backward needs the kinds of the call")
                if kinds.numel() != self.B * self.H:
                    raise ValueError(f"{self.B * self.H} kinds expected")
                if kinds.dtype != torch.uint8 or kinds.device != self.device or not kinds.is_contiguous():
                    kinds = self.kinds_bwd.copy_(kinds.reshape(-1).to(torch.uint8))
            else:
                kinds = self.kinds_bwd  # every head is a cube head
            vsa_attention_bwd(qkvo_grad(q, k, v, o, d_o, lse, *out, d_lse=d_lse, o_lo=o_lo), _DTYPE[self.dtype], self.shape,
                              self.params, kinds, self.ws_bwd, self.ws_bwd_bytes, self.err)
        return tuple(out)

    def attend(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kinds: Optional[torch.Tensor] = None):
        """The call as a differentiable function: o whose ``backward`` fills the gradients of q, k and v
        (first derivatives; the masks count as constants).  Keeps q, k, v, o, o_lo, the log-sum-exp and
        the kinds for the gradient, and nothing where autograd does not record.  Where it does, it is
        refused under graph capture: capture the call itself and ``backward`` instead."""
        if not self.with_grad:
            raise ValueError("the plan was made without with_grad=True")
        if not (torch.is_grad_enabled() and any(t.requires_grad for t in (q, k, v))):
            return self(q, k, v, kinds=kinds)[0]
        _no_capture("attend")
        return _Attend.apply(self, q, k, v, kinds)

    def device_error(self) -> int:
        return vsa_get_device_error(self.err)

    def clear_error(self):
        self.err.zero_()

    def run_host(self, batches, outs=None, kinds: Optional[torch.Tensor] = None, timing=None):
        """The call on a sequence of host batches through the library's vsa_attention_host: the
        uploads of batch i+1 and the download of batch i-1 overlap the compute of batch i (three
        streams, two device buffer sets owned here).  ``batches`` is a list of (q, k, v) CPU
        tensors, which must be pinned for the copies to overlap; ``outs`` a list of CPU output
        tensors (pinned ones are allocated when None).  Returns ``outs`` once every output has
        arrived.  ``timing``, a pair of timing-enabled CUDA events, is recorded before the first
        upload and after the last download."""
        n = len(batches)
        shape = (self.B, self.H, self.N, self.d)
        if outs is None:
            outs = [torch.empty(shape, dtype=self.dtype).pin_memory() for _ in range(n)]
        if len(outs) != n:
            raise ValueError("need one output tensor per batch")
        for (q, k, v), o in zip(batches, outs):
            for t in (q, k, v, o):
                if t.device.type != "cpu" or t.dtype != self.dtype or tuple(t.shape) != shape or not t.is_contiguous():
                    raise ValueError(f"contiguous host tensors of shape {shape} and dtype {self.dtype} expected")
        if self.select == VSA_SELECT_GIVEN:
            if kinds is None:
                raise ValueError("select='given' needs kinds")
            self.kinds.copy_(kinds.reshape(-1).to(torch.uint8))
        if not hasattr(self, "_host_bufs"):
            self._host_bufs = [[torch.empty(shape, dtype=self.dtype, device=self.device) for _ in range(4)]
                               for _ in range(2)]  # q, k, v, o per buffer set
            self._host_lse = ([torch.empty(self.B, self.H, self.N, dtype=torch.float32, device=self.device)
                               for _ in range(2)] if self.with_lse else [None, None])
            self._streams = [torch.cuda.Stream(self.device) for _ in range(3)]  # upload, compute, download
        up, comp, down = self._streams
        cur = torch.cuda.current_stream(self.device)
        up.wait_stream(cur)
        comp.wait_stream(cur)
        if timing is not None:
            timing[0].record(up)
        sets = [qkvo(b[0], b[1], b[2], b[3], lse) for b, lse in zip(self._host_bufs, self._host_lse)]
        _lib.vsa_attention_host([(q, k, v, o) for (q, k, v), o in zip(batches, outs)], sets, _DTYPE[self.dtype],
                                self.shape, self.params, self.select, self.kinds, self.mse, self.ws, self.ws_bytes,
                                self.err, up, comp, down)
        if timing is not None:
            timing[1].record(down)
        down.synchronize()
        return outs


class SemanticAttention(_HostPipelined):
    """Block-sparse attention with the semantic-aware permutation (Sparse VideoGen2 page,
    abstract): per-head k-means of Q (``cq`` clusters) and K (``ck``), cluster-major orders,
    a ``top_p`` budget over cluster pairs, then the same attention kernel.  bf16 only, no
    cube dims."""

    def __init__(self, B: int, H: int, F: int, Hl: int, Wl: int, d: int, block: int = 128, *, cq: int = 128,
                 ck: int = 128, iters: int = 4, top_p: float = 0.6, scale: float = 0.0, with_lse: bool = False,
                 device="cuda"):
        self.B, self.H, self.F, self.Hl, self.Wl, self.d, self.block = B, H, F, Hl, Wl, d, block
        self.N = F * Hl * Wl
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device, self.dtype = dev, torch.bfloat16
        self.shape = make_shape(B, H, F, Hl, Wl, d, block)
        self.params = make_sem_params(cq, ck, iters, top_p, scale)
        self.ws_bytes = vsa_semantic_workspace_size(self.shape, self.params)
        if self.ws_bytes == 0:
            raise VsaError(_lib.VSA_ERR_INVALID_ARG, "vsa_semantic_workspace_size")
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.with_lse = with_lse

    def __call__(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, kinds=None, stream=None):
        if kinds is not None:
            raise ValueError("the semantic call chooses its blocks itself; kinds must be None")
        for t in (q, k, v):
            if t.dtype != torch.bfloat16 or t.device != self.device or not t.is_contiguous():
                raise ValueError("q, k, v must be contiguous bf16 tensors on the configured device")
            if tuple(t.shape) != (self.B, self.H, self.N, self.d):
                raise ValueError(f"expected shape {(self.B, self.H, self.N, self.d)}, got {tuple(t.shape)}")
        _check_outputs(self, out, lse)
        with _on(stream, self.device):
            if out is None:
                out = torch.empty_like(q)
            if self.with_lse and lse is None:
                lse = torch.empty(self.B, self.H, self.N, dtype=torch.float32, device=self.device)
            vsa_semantic_attention(qkvo(q, k, v, out, lse), self.shape, self.params, self.ws, self.ws_bytes, self.err)
        return (out, lse) if self.with_lse else out

    def device_error(self) -> int:
        return vsa_get_device_error(self.err)


class NormOut(NamedTuple):
    """What one RMSNorm call computed (None for what it was not asked for)."""
    y: Optional[torch.Tensor]        # [B, H, N, d] in the rows' dtype
    sum: Optional[torch.Tensor]      # x + residual, rounded to the dtype
    codes: Optional[torch.Tensor]    # [B, H, N, d] e4m3 codes (uint8) of y / 2^exps
    exps: Optional[torch.Tensor]     # [B, H, ceil(N / block)] int32
    rstd: torch.Tensor               # [B, H, N] fp32


class _Normalise(torch.autograd.Function):
    @staticmethod
    def forward(ctx, norm, x, weight, residual):
        ctx.set_materialize_grads(False)
        r = norm(x, weight, residual=residual)
        ctx.norm, ctx.has = norm, (weight is not None, residual is not None)
        ctx.save_for_backward(x if residual is None else r.sum, r.rstd, weight)
        return r.y if residual is None else (r.y, r.sum)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, d_sum=None):
        _no_capture("normalise")
        s, rstd, weight = ctx.saved_tensors
        if dy is None:
            if d_sum is None:
                return (None,) * 4
            dy = torch.zeros_like(d_sum, memory_format=torch.contiguous_format)
        dx, dw = ctx.norm.backward(dy.contiguous(), s, rstd, weight, d_sum=None if d_sum is None else d_sum.contiguous())
        need = ctx.needs_input_grad
        return (None, dx if need[1] else None, dw.to(weight.dtype) if need[2] else None, dx if need[3] else None)


class RMSNorm:
    """Root-mean-square norm of [B, H, N] rows of d elements, as in front of the attention's Q and K (H heads
    of d = 64 or 128), or of whole hidden rows (H = 1): y = s * rstd * weight, s = x + residual.

    quantize: 0 for y in the rows' dtype; 1 for e4m3 codes with one power-of-two scale per row; 64 or 128 for
              one per so many consecutive rows of a head (d = 64 or 128): with 128, the codes and exponents
              ``vsa_sparse_attn_fwd_fp8qk`` takes for spatial heads.  ``keep_y`` writes y as well.
    with_grad: the plan also holds the workspace of the weight's gradient (``backward``, ``normalise``); that
              workspace serves one call at a time.

    x and the residual are any views whose last dimension is dense, a [B, N, H, d] projection seen as
    [B, H, N, d] among them; outputs are contiguous.  A weight or gradient that does not start on 16 bytes
    (one cut out of a larger buffer) is copied first."""

    def __init__(self, B: int, H: int, N: int, d: int, *, dtype: torch.dtype = torch.bfloat16, eps: float = 1e-6,
                 quantize: int = 0, keep_y: bool = False, with_grad: bool = False, device="cuda"):
        if dtype not in _DTYPE:
            raise ValueError(f"unsupported dtype {dtype}")
        if quantize not in (0, 1, 64, 128) or (quantize > 1 and d not in (64, 128)):
            raise ValueError("quantize is 0, 1, or 64 or 128 rows of d = 64 or 128")
        if with_grad and quantize and not keep_y:
            raise ValueError("the e4m3 codes have no gradient: keep_y gives one to y")
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.B, self.H, self.N, self.d, self.dtype, self.device = B, H, N, d, dtype, dev
        self.quantize, self.keep_y, self.with_grad = quantize, keep_y or not quantize, with_grad
        self.shape = make_norm_shape(B, H, N, d, block=max(quantize, 1), eps=eps)
        need = vsa_rms_norm_bwd_workspace_size(self.shape, _DTYPE[dtype])
        if need == 0:
            raise VsaError(_lib.VSA_ERR_INVALID_ARG, "vsa_rms_norm_bwd_workspace_size")
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev) if with_grad else None

    def _shape(self, x=None, residual=None):
        strides = tuple((0, 0, 0) if t is None or t.is_contiguous() else t.stride()[:3] for t in (x, residual))
        if strides == ((0, 0, 0), (0, 0, 0)):
            return self.shape
        return make_norm_shape(self.B, self.H, self.N, self.d, *strides, block=self.shape.block, eps=self.shape.eps)

    def _rows(self, t: torch.Tensor, what: str, dense: bool = False) -> torch.Tensor:
        shape = (self.B, self.H, self.N, self.d)
        if t.dtype != self.dtype or t.device != self.device or tuple(t.shape) != shape:
            raise ValueError(f"{what} is a {self.dtype} tensor of shape {shape} on {self.device}")
        if (self.d > 1 and t.stride(3) != 1) or (dense and not t.is_contiguous()):
            raise ValueError(f"{what} must be contiguous" if dense else f"the last dimension of {what} must be dense")
        if dense:
            return _on_16_bytes(t)
        # three zero strides are how the library is told of contiguous rows
        return t.contiguous() if not any(t.stride()[:3]) else t

    def _weight(self, weight: Optional[torch.Tensor]):
        """The weight on 16 bytes (it may be cut out of a flat buffer), and its type."""
        if weight is None:
            return None, VSA_F32
        if weight.dtype not in _DTYPE or weight.device != self.device or tuple(weight.shape) != (self.d,) \
                or not weight.is_contiguous():
            raise ValueError(f"weight is a contiguous float32 or bfloat16 tensor of shape {(self.d,)} on {self.device}")
        return _on_16_bytes(weight), _DTYPE[weight.dtype]

    def __call__(self, x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                 stream=None) -> NormOut:
        shape = (self.B, self.H, self.N, self.d)
        with _on(stream, self.device):
            weight, wt = self._weight(weight)
            x = self._rows(x, "x")
            residual = None if residual is None else self._rows(residual, "the residual")
            new = lambda *sh, dtype: torch.empty(*sh, dtype=dtype, device=self.device)  # noqa: E731
            out = NormOut(new(*shape, dtype=self.dtype) if self.keep_y else None,
                          new(*shape, dtype=self.dtype) if residual is not None else None,
                          new(*shape, dtype=torch.uint8) if self.quantize else None,
                          new(*shape[:2], -(-self.N // self.quantize), dtype=torch.int32) if self.quantize else None,
                          new(*shape[:3], dtype=torch.float32))
            _lib._rms_norm(x, residual, _DTYPE[self.dtype], weight, wt, self._shape(x, residual), out.sum, out.y,
                         out.codes, out.exps, out.rstd)
        return out

    def backward(self, dy: torch.Tensor, s: torch.Tensor, rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                 d_sum: Optional[torch.Tensor] = None, stream=None, dsum: Optional[torch.Tensor] = None):
        """(dx, d_weight) of a call: s is its x, or its sum where it had a residual; dy and d_sum (or dsum, another
        name of it) the gradients of y and of sum.  dx is the residual's gradient too, and has s's order of
        dimensions where s fills its memory (else it is contiguous); d_weight is fp32 (None without a weight).
        Asynchronous on ``stream``; can be captured."""
        if not self.with_grad:
            raise ValueError("the plan was made without with_grad=True")
        if dsum is not None:
            if d_sum is not None:
                raise ValueError("d_sum and dsum are one argument")
            d_sum = dsum
        with _on(stream, self.device):
            weight, wt = self._weight(weight)
            dy = self._rows(dy, "dy", dense=True)
            d_sum = None if d_sum is None else self._rows(d_sum, "d_sum", dense=True)
            s = self._rows(s, "s")
            if rstd.dtype != torch.float32 or rstd.device != self.device or not rstd.is_contiguous() \
                    or tuple(rstd.shape) != (self.B, self.H, self.N):
                raise ValueError("rstd is the float32 tensor the call returned")
            rstd = _on_16_bytes(rstd)
            shape = (self.B, self.H, self.N, self.d)
            dx = (torch.empty_strided(shape, s.stride(), dtype=s.dtype, device=self.device) if _whole_rows(s)
                  else torch.empty(shape, dtype=s.dtype, device=self.device))
            dw = torch.empty(self.d, dtype=torch.float32, device=self.device) if weight is not None else None
            _lib._rms_norm_bwd(dy, d_sum, s, _DTYPE[self.dtype], weight, wt, rstd, self._shape(s, dx), dx, dw, self.ws,
                             self.ws.numel())
        return dx, dw

    def normalise(self, x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None):
        """The call as a differentiable function of x, weight and residual: y, or (y, sum) with a residual.  As
        SparseAttention.attend, refused under graph capture where autograd records it."""
        if not self.with_grad:
            raise ValueError("the plan was made without with_grad=True")
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, residual)):
            _no_capture("normalise")
        return _Normalise.apply(self, x, weight, residual)


def _whole_rows(t: torch.Tensor) -> bool:
    """Whether no two rows of t overlap and together they fill one piece of memory."""
    span = t.shape[3]
    for stride, size in sorted((st, n) for st, n in zip(t.stride()[:3], t.shape[:3]) if n > 1):
        if stride != span:
            return False
        span *= size
    return True


def attention(q, k, v, F: int, Hl: int, Wl: int, **kw):
    """Convenience wrapper: build a :class:`SparseAttention` for q's shape and run it once."""
    B, H, N, d = q.shape
    plan = SparseAttention(B, H, F, Hl, Wl, d, dtype=q.dtype, device=q.device, **kw)
    return plan(q, k, v)


__all__ = ["SparseAttention", "SemanticAttention", "attention", "SemParams", "make_sem_params", "vsa_gather_rows",
           "vsa_kmeans", "vsa_kmeans_workspace_size", "vsa_scatter_rows", "vsa_semantic_attention",
           "vsa_semantic_mask", "vsa_semantic_mask_workspace_size", "vsa_semantic_workspace_size", "VsaError", "Shape", "Params", "QKVO", "make_shape", "make_params", "qkvo",
           "vsa_attention", "vsa_attention_workspace_layout", "vsa_attention_workspace_size", "vsa_block_order", "vsa_build_mask",
           "vsa_get_device_error", "vsa_layout_rows", "vsa_mask_workspace_size", "vsa_max_kv", "vsa_num_blocks",
           "vsa_pattern_window", "vsa_permute", "vsa_profile_heads", "vsa_profile_rows",
           "vsa_profile_workspace_size", "vsa_sparse_attn_fwd", "vsa_sparse_attn_fwd_natural", "vsa_unpermute",
           "vsa_quantize_fp8", "vsa_sparse_attn_fwd_fp8qk", "QKVOGrad", "qkvo_grad", "vsa_sparse_attn_bwd",
           "vsa_sparse_attn_bwd_workspace_size", "vsa_attention_bwd", "vsa_attention_bwd_workspace_size",
           "vsa_attention_train", "vsa_attention_train_workspace_size",
           "RMSNorm", "NormOut", "NormShape", "make_norm_shape", "vsa_rms_norm", "vsa_rms_norm_bwd",
           "vsa_rms_norm_bwd_workspace_size", "VSA_SPATIAL", "VSA_TEMPORAL",
           "VSA_CUBE", "VSA_F32", "VSA_BF16", "VSA_SELECT_PROFILE", "VSA_SELECT_GIVEN", "VSA_SELECT_CUBE"]
