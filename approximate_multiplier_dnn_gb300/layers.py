"""Drop-in torch layers whose contractions -- the forward pass and both
gradients -- run through the LUT-simulated approximate multiplier, as the
AMDENSE and AMCONV2D layers of ApproxTrain (Sec. IV) do, plus attention built
from two approximate contractions around an exact softmax.

Each layer is a torch.autograd.Function over the C ABI: the approximate
contractions, the softmax and its gradient run in this library's kernels; bias
additions are ordinary (exact) torch additions, as they are not products.

Layouts: Dense weights are [in, out] (y = x w); Conv2D tensors are NHWC with
RSCK filters (TF's HWIO), stride/padding/dilation as in ApproxTrain's Conv2D;
depthwise filters are R x S x C x D (TF's depthwise layout, multiplier D);
attention takes Q, K, V as [batch, heads, seq, dim].

Between and after the approximate layers of a language model stand exact ones,
which are not products of the simulated multiplier: BlockNorm (the norms
around a block with its gate and the residual scale) and VocabHead (the loss
over the vocabulary); their optimizer is optim.AdamW.  Between two
contractions stand, exact as well: in attention a softmax with a learned bias by
distance (RelativeBias), key lengths, a causal mask and dropout; GroupNorm with
its activation between convolutions; Dropout after either.

Operand order of every contraction (which operand indexes the LUT's rows;
it matters only for an asymmetric user LUT): Dense forward (x, w), input
gradient (dy, w), weight gradient (x, dy); Conv2D likewise (x, w), (dy, w),
(x, dy), and the same for depthwise; attention S = (q, k), O = (p, v), dV = (p, dO), dP = (dO, v),
dQ = (dS, k), dK = (dS, q).
"""
from __future__ import annotations

import copy
import math

import torch
from torch.autograd.function import once_differentiable

from . import (ConvDesc, attention_softmax, attention_softmax_backward, block_norm, block_norm_backward, dropout,
               group_norm, group_norm_backward, relative_buckets, vocab_loss, vocab_loss_grad, amsim_conv2d_bwd_data, amsim_conv2d_bwd_filter, amsim_conv2d_fwd, amsim_conv2d_out_hw,
               amsim_conv2d_workspace_size, amsim_dwconv2d_bwd_data, amsim_dwconv2d_bwd_filter, amsim_dwconv2d_fwd,
               amsim_dwconv2d_workspace_size, amsim_gemm, amsim_gemm_strided_batched, amsim_gemm_workspace_size,
               amsim_softmax_rows, amsim_softmax_rows_backward, workspace)


def _f32(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.float32 or not t.is_cuda:
        raise TypeError("approximate layers take fp32 CUDA tensors")
    return t.contiguous()


def _gemm(tA: str, tB: str, A: torch.Tensor, B: torch.Tensor, m: int, n: int, k: int, lut, alpha=1.0):
    """C[m, n] = alpha op(A) op(B) for contiguous row-major A and B."""
    C = torch.empty((m, n), dtype=torch.float32, device=A.device)
    ws = workspace(amsim_gemm_workspace_size(tA, tB, m, n, k, 1, lut), A.device)
    amsim_gemm(tA, tB, m, n, k, alpha, A, max(1, A.shape[1]), B, max(1, B.shape[1]), 0.0, C, max(1, n), lut,
               ws=ws)
    return C


def _bgemm(tA: str, tB: str, A: torch.Tensor, B: torch.Tensor, m: int, n: int, k: int, lut, alpha=1.0):
    """C[b] = alpha op(A[b]) op(B[b]) over the leading batch dimension."""
    batch = A.shape[0]
    C = torch.empty((batch, m, n), dtype=torch.float32, device=A.device)
    ws = workspace(amsim_gemm_workspace_size(tA, tB, m, n, k, batch, lut), A.device)
    amsim_gemm_strided_batched(tA, tB, m, n, k, alpha, A, A.shape[2], A.shape[1] * A.shape[2], B, B.shape[2],
                               B.shape[1] * B.shape[2], 0.0, C, n, m * n, batch, lut, ws=ws)
    return C


# ------------------------------------------------------------------ Dense
class _DenseFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, lut):
        x, w = _f32(x), _f32(w)
        rows, fin = x.shape
        fout = w.shape[1]
        ctx.save_for_backward(x, w)
        ctx.lut = lut
        return _gemm("N", "N", x, w, rows, fout, fin, lut)

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dy = _f32(dy)
        rows, fin = x.shape
        fout = w.shape[1]
        dx = _gemm("N", "T", dy, w, rows, fin, fout, ctx.lut) if ctx.needs_input_grad[0] else None
        dw = _gemm("T", "N", x, dy, fin, fout, rows, ctx.lut) if ctx.needs_input_grad[1] else None
        return dx, dw, None


def am_dense(x: torch.Tensor, w: torch.Tensor, lut) -> torch.Tensor:
    """y = x w with approximate products (x [rows, in], w [in, out])."""
    return _DenseFn.apply(x, w, lut)


class AMDense(torch.nn.Module):
    """Fully connected layer y = x W (+ b) whose forward and backward
    contractions use the approximate multiplier (ApproxTrain's AMDENSE)."""

    def __init__(self, in_features: int, out_features: int, lut, bias: bool = True, device="cuda",
                 generator: torch.Generator | None = None):
        super().__init__()
        self.lut = lut
        bound = math.sqrt(6.0 / (in_features + out_features))          # Glorot uniform
        w = (torch.rand((in_features, out_features), generator=generator) * 2.0 - 1.0) * bound
        self.weight = torch.nn.Parameter(w.to(device))
        self.bias = torch.nn.Parameter(torch.zeros(out_features, device=device)) if bias else None

    def forward(self, x):
        y = am_dense(x, self.weight, self.lut)
        return y + self.bias if self.bias is not None else y


# ------------------------------------------------------------------ Conv2D
def _pair(v):
    return (v, v) if isinstance(v, int) else tuple(v)


class _Conv2dFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, lut, stride, padding, dilation):
        x, w = _f32(x), _f32(w)
        N, H, W, C = x.shape
        R, S, C2, K = w.shape
        if C2 != C:
            raise ValueError("filter channels differ from the input's")
        desc = ConvDesc.make(N, H, W, C, K, R, S, stride, padding, dilation)
        P, Q = amsim_conv2d_out_hw(desc)
        y = torch.empty((N, P, Q, K), dtype=torch.float32, device=x.device)
        amsim_conv2d_fwd(desc, x, w, y, lut, ws=workspace(amsim_conv2d_workspace_size(desc, 0, lut), x.device))
        ctx.save_for_backward(x, w)
        ctx.lut, ctx.desc = lut, desc
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dy = _f32(dy)
        desc, lut = ctx.desc, ctx.lut
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = torch.empty_like(x)
            amsim_conv2d_bwd_data(desc, dy, w, dx, lut,
                                  ws=workspace(amsim_conv2d_workspace_size(desc, 1, lut), x.device))
        if ctx.needs_input_grad[1]:
            dw = torch.empty_like(w)
            amsim_conv2d_bwd_filter(desc, x, dy, dw, lut,
                                    ws=workspace(amsim_conv2d_workspace_size(desc, 2, lut), x.device))
        return dx, dw, None, None, None, None


def am_conv2d(x, w, lut, stride=1, padding=0, dilation=1):
    """y = conv2d(x, w) with approximate products (x NHWC, w RSCK, y NPQK)."""
    return _Conv2dFn.apply(x, w, lut, _pair(stride), _pair(padding), _pair(dilation))


class AMConv2d(torch.nn.Module):
    """2-D convolution (cross-correlation) whose forward pass and both
    gradients use the approximate multiplier (ApproxTrain's AMCONV2D).
    NHWC input, RSCK filters."""

    def __init__(self, in_channels: int, out_channels: int, kernel_size, lut, stride=1, padding=0, dilation=1,
                 bias: bool = True, device="cuda", generator: torch.Generator | None = None):
        super().__init__()
        self.lut = lut
        R, S = _pair(kernel_size)
        self.stride, self.padding, self.dilation = _pair(stride), _pair(padding), _pair(dilation)
        std = math.sqrt(2.0 / (R * S * in_channels))                   # He normal
        w = torch.randn((R, S, in_channels, out_channels), generator=generator) * std
        self.weight = torch.nn.Parameter(w.to(device))
        self.bias = torch.nn.Parameter(torch.zeros(out_channels, device=device)) if bias else None

    def forward(self, x):
        y = _Conv2dFn.apply(x, self.weight, self.lut, self.stride, self.padding, self.dilation)
        return y + self.bias if self.bias is not None else y


# ------------------------------------------------------------------ depthwise Conv2D
class _DepthwiseConv2dFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, lut, stride, padding, dilation):
        x, w = _f32(x), _f32(w)
        N, H, W, C = x.shape
        R, S, C2, D = w.shape
        if C2 != C:
            raise ValueError("filter channels differ from the input's")
        desc = ConvDesc.make(N, H, W, C, C * D, R, S, stride, padding, dilation)
        P, Q = amsim_conv2d_out_hw(desc)
        y = torch.empty((N, P, Q, C * D), dtype=torch.float32, device=x.device)
        amsim_dwconv2d_fwd(desc, x, w, y, lut)
        ctx.save_for_backward(x, w)
        ctx.lut, ctx.desc = lut, desc
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dy = _f32(dy)
        desc, lut = ctx.desc, ctx.lut
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = torch.empty_like(x)
            amsim_dwconv2d_bwd_data(desc, dy, w, dx, lut)
        if ctx.needs_input_grad[1]:
            dw = torch.empty_like(w)
            amsim_dwconv2d_bwd_filter(desc, x, dy, dw, lut,
                                      ws=workspace(amsim_dwconv2d_workspace_size(desc, 2, lut), x.device))
        return dx, dw, None, None, None, None


def am_depthwise_conv2d(x, w, lut, stride=1, padding=0, dilation=1):
    """Depthwise y = conv2d(x, w) per channel with approximate products (x NHWC,
    w R x S x C x D for a channel multiplier D, y NPQ(C*D), output channel
    c*D + d from input channel c)."""
    return _DepthwiseConv2dFn.apply(x, w, lut, _pair(stride), _pair(padding), _pair(dilation))


class AMDepthwiseConv2d(torch.nn.Module):
    """Depthwise 2-D convolution (one filter group per input channel, channel
    multiplier D) whose forward pass and both gradients use the approximate
    multiplier; depthwise convolution is one of the layer types ApproxTrain
    simulates (Sec. III, Table I).  NHWC input, R x S x C x D filters."""

    def __init__(self, channels: int, kernel_size, lut, depth_multiplier: int = 1, stride=1, padding=0,
                 dilation=1, bias: bool = True, device="cuda", generator: torch.Generator | None = None):
        super().__init__()
        self.lut = lut
        R, S = _pair(kernel_size)
        self.stride, self.padding, self.dilation = _pair(stride), _pair(padding), _pair(dilation)
        std = math.sqrt(2.0 / (R * S))                                  # He normal over a channel's taps
        w = torch.randn((R, S, channels, depth_multiplier), generator=generator) * std
        self.weight = torch.nn.Parameter(w.to(device))
        self.bias = (torch.nn.Parameter(torch.zeros(channels * depth_multiplier, device=device)) if bias
                     else None)

    def forward(self, x):
        y = _DepthwiseConv2dFn.apply(x, self.weight, self.lut, self.stride, self.padding, self.dilation)
        return y + self.bias if self.bias is not None else y


# ------------------------------------------------------------------ attention
class _AttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lut, scale):
        q, k, v = _f32(q), _f32(k), _f32(v)
        b, h, s, d = q.shape
        t = k.shape[2]
        qf, kf, vf = q.reshape(b * h, s, d), k.reshape(b * h, t, d), v.reshape(b * h, t, d)
        S = _bgemm("N", "T", qf, kf, s, t, d, lut, alpha=scale)
        P = torch.empty_like(S)
        amsim_softmax_rows(S, P, b * h * s, t)
        O = _bgemm("N", "N", P, vf, s, d, t, lut)
        ctx.save_for_backward(qf, kf, vf, P)
        ctx.lut, ctx.scale, ctx.shape = lut, scale, (b, h, s, t, d)
        return O.reshape(b, h, s, d)

    @staticmethod
    def backward(ctx, dO):
        qf, kf, vf, P = ctx.saved_tensors
        b, h, s, t, d = ctx.shape
        lut, scale = ctx.lut, ctx.scale
        dOf = _f32(dO).reshape(b * h, s, d)
        dV = _bgemm("T", "N", P, dOf, t, d, s, lut)                   # P^T dO
        dP = _bgemm("N", "T", dOf, vf, s, t, d, lut)                  # dO V^T
        dS = torch.empty_like(dP)
        amsim_softmax_rows_backward(P, dP, dS, b * h * s, t)
        dQ = _bgemm("N", "N", dS, kf, s, d, t, lut, alpha=scale)      # scale dS K
        dK = _bgemm("T", "N", dS, qf, t, d, s, lut, alpha=scale)      # scale dS^T Q
        return dQ.reshape(b, h, s, d), dK.reshape(b, h, t, d), dV.reshape(b, h, t, d), None, None


def _seen_only(t, lengths):
    """[batch, heads, keys, dim] with zeros for the keys from a sequence's length on: a simulated product of a zero
    probability with a padded key's infinity would be NaN."""
    hidden = torch.arange(t.shape[2], device=t.device) >= lengths[:, None]
    return t.masked_fill(hidden[:, None, :, None], 0.0)


class _MaskedAttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, table, lut, scale, buckets, lengths, offset, step, causal, p, seed, call):
        q, k, v = _f32(q), _f32(k), _f32(v)
        if lengths is not None:
            k, v = _seen_only(k, lengths), _seen_only(v, lengths)
        b, h, s, d = q.shape
        t = k.shape[2]
        qf, kf, vf = q.reshape(b * h, s, d), k.reshape(b * h, t, d), v.reshape(b * h, t, d)
        ctx.lut, ctx.scale, ctx.shape = lut, scale, (b, h, s, t, d)
        if not t:                        # no row sees a key, and the contractions take none without
            ctx.save_for_backward(table)
            return torch.zeros_like(q)
        S = _bgemm("N", "T", qf, kf, s, t, d, lut, alpha=scale).view(b, h, s, t)
        args = dict(buckets=buckets, lengths=lengths, causal=causal, offset=offset, p=p, seed=seed, call=call, step=step)
        P, stats = attention_softmax(S, table=table, out=None if p else S, **args)   # dropped ones are gone: S stays
        O = _bgemm("N", "N", P.view(b * h, s, t), vf, s, d, t, lut)
        keep = [buckets, lengths, step, offset if isinstance(offset, torch.Tensor) else None]
        ctx.save_for_backward(qf, kf, vf, P, *((S, stats) if p else (None, None)), table, *keep)
        ctx.args = args
        return O.reshape(b, h, s, d)

    @staticmethod
    @once_differentiable
    def backward(ctx, dO):
        b, h, s, t, d = ctx.shape
        if not t:
            table, = ctx.saved_tensors
            none = dO.new_zeros((b, h, 0, d))
            return torch.zeros_like(dO), none, none, None if table is None else torch.zeros_like(table), *[None] * 10
        qf, kf, vf, P, S, stats, table, *_ = ctx.saved_tensors
        lut, scale = ctx.lut, ctx.scale
        dOf = _f32(dO).reshape(b * h, s, d)
        dV = _bgemm("T", "N", P.view(b * h, s, t), dOf, t, d, s, lut)
        dP = _bgemm("N", "T", dOf, vf, s, t, d, lut).view(b, h, s, t)
        source = dict(probs=P) if S is None else dict(scores=S, stats=stats)
        dS, dtable = attention_softmax_backward(dP, table=table, table_grad=ctx.needs_input_grad[3], out=dP, **source,
                                                **ctx.args)
        dS = dS.view(b * h, s, t)
        dQ = _bgemm("N", "N", dS, kf, s, d, t, lut, alpha=scale)
        dK = _bgemm("T", "N", dS, qf, t, d, s, lut, alpha=scale)
        return dQ.reshape(b, h, s, d), dK.reshape(b, h, t, d), dV.reshape(b, h, t, d), dtable, *[None] * 10


def am_attention(q, k, v, lut, scale: float | None = None, *, table=None, buckets=None, lengths=None, causal=False,
                 offset=0, dropout: float = 0.0, seed: int = 0, call: int = 0, step=None):
    """softmax(scale q k^T) v per (batch, head), contractions approximate,
    softmax exact; scale defaults to 1/sqrt(dim).

    The rest is attention_softmax's, with `dropout` for its p: a bias by distance
    (table, which gets a gradient, and buckets), lengths of the keys (cross
    attention to a padded batch of another length; what k and v hold behind a
    length has no effect and no gradient), a causal mask, the first query's
    position, dropout of the probabilities."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if (table is None) != (buckets is None):
        raise ValueError("a bias needs both its table and the buckets of its distances")
    if table is None and lengths is None and not causal and dropout == 0.0:
        return _AttentionFn.apply(q, k, v, lut, float(scale))
    if q.dim() != 4 or k.shape != (*q.shape[:2], k.shape[-2], q.shape[3]) or v.shape != k.shape:
        raise ValueError(f"k and v must be [batch, heads, keys, dim] with q's {tuple(q.shape)} but for the keys, not "
                         f"{tuple(k.shape)} and {tuple(v.shape)}")
    if lengths is not None and lengths.shape != q.shape[:1]:
        raise ValueError(f"lengths must be of shape ({q.shape[0]},), not {tuple(lengths.shape)}")
    return _MaskedAttentionFn.apply(q, k, v, table, lut, float(scale), buckets, lengths, offset, step, bool(causal),
                                    float(dropout), seed, call)


def _may_run_again() -> bool:
    """Whether torch.utils.checkpoint may be running this code, to run it again in the backward pass: it does so under
    hooks for saved tensors or (reentrant) without gradients."""
    hooks = getattr(torch._C._autograd, "_top_saved_tensors_default_hooks", None)
    return not torch.is_grad_enabled() or hooks is None or hooks(True) is not None


class _Draws(torch.nn.Module):
    """What a layer that draws keeps: a seed of its own and the number of its next call, both part of its state.

    A checkpointed block is run again in the backward pass and has to draw the same masks.  torch.utils.checkpoint
    gives torch's generator back the state that it had, so each call that may be run again takes a value from that
    generator as its mark, and a call within a backward pass takes the number of the call of the same mark.  Where that
    is not one call (the generator was seeded anew before the first one's backward pass) it is refused."""

    remembered = 1024                    # calls whose marks are known: those between a block's two runs
    replays = 2 ** 32                    # numbers that a captured call takes: its own, and one more for each step

    def __init__(self, seed, generator):
        super().__init__()
        self.seed = int(torch.randint(0, 2 ** 62, (), generator=generator)) if seed is None else int(seed)
        self.calls, self.marks = 0, {}

    def __setstate__(self, state):
        super().__setstate__({**state, "marks": {}})

    def __deepcopy__(self, memo):
        """A copy draws masks of its own, from a seed of its own: blocks are often made by copying one."""
        memo[id(self)] = new = type(self).__new__(type(self))
        new.__setstate__(copy.deepcopy({**self.__dict__, "marks": {}}, memo))
        new.seed = int(torch.randint(0, 2 ** 62, (), device="cpu"))
        return new

    def get_extra_state(self):
        return dict(seed=self.seed, calls=self.calls)

    def set_extra_state(self, state):
        self.seed, self.calls = state["seed"], state["calls"]

    def next(self, call, step) -> dict:
        """Seed and number of a call: the caller's number, or one more than the last."""
        if call is None:
            captured = torch.cuda.is_available() and torch.cuda.is_current_stream_capturing()
            if captured and step is None:
                raise RuntimeError("a captured call draws the same mask at every replay: give it a step on the device")
            if torch._C._current_graph_task_id() != -1:              # within a backward pass
                known = self.marks.get(self.mark())
                if known is None or known["call"] is None:
                    raise RuntimeError("a call within a backward pass that does not repeat one call of the forward "
                                       "pass (a checkpoint without preserve_rng_state, or torch seeded anew?) would "
                                       "draw another mask: give it the call's number")
                call, known["repeated"] = known["call"], True
            else:
                call, self.calls = self.calls, self.calls + (self.replays if captured else 1)
                if _may_run_again():
                    mark = self.mark()
                    known = self.marks.pop(mark, None)
                    self.marks[mark] = dict(call=call if known is None or known["repeated"] else None, repeated=False)
                    if len(self.marks) > self.remembered:
                        del self.marks[next(iter(self.marks))]
        return dict(seed=self.seed, call=call, step=step)

    @staticmethod
    def mark() -> int:
        return int(torch.randint(0, 2 ** 62, (), device="cpu"))


class RelativeBias(torch.nn.Module):
    """A learned bias for every head by the distance between key and query, in
    buckets (relative_buckets); several layers may share one."""

    def __init__(self, heads: int, buckets: int = 32, max_distance: int = 128, bidirectional: bool = True,
                 device="cuda", generator: torch.Generator | None = None):
        super().__init__()
        self.table = torch.nn.Parameter((torch.randn((buckets, heads), generator=generator) * 0.1).to(device))
        self.register_buffer("buckets", relative_buckets(buckets, max_distance, bidirectional).to(device),
                             persistent=False)


class AMAttention(torch.nn.Module):
    """Scaled dot-product attention over [batch, heads, seq, dim] tensors
    with approximate contractions (no projections).

    bias: a RelativeBias or None; causal: keys after a query's position are not
    seen; dropout: of the probabilities, in training.  forward(q, k, v,
    lengths=None, offset=0) takes the keys' lengths (int32 [batch]: an encoder's
    padded states) and the first query's position (an int, or int32 [batch]: a
    single token's place in its cache).  Dropout draws a new mask at each call;
    step (one int64 CUDA value, raised once a replay) does so for a captured
    one, and call repeats a given call's mask.  A block that torch.utils.checkpoint
    runs again draws what it drew; without preserve_rng_state it needs call."""

    def __init__(self, lut, scale: float | None = None, *, bias: RelativeBias | None = None, causal: bool = False,
                 dropout: float = 0.0, seed: int | None = None, generator: torch.Generator | None = None):
        super().__init__()
        if not 0.0 <= dropout < 1.0:
            raise ValueError("dropout takes a p in [0, 1)")
        self.lut, self.scale, self.bias, self.causal, self.dropout = lut, scale, bias, causal, float(dropout)
        self.draws = _Draws(seed, generator) if dropout else None

    def forward(self, q, k, v, lengths=None, offset=0, *, step=None, call=None):
        table, buckets = (None, None) if self.bias is None else (self.bias.table, self.bias.buckets)
        drawn = dict(dropout=self.dropout, **self.draws.next(call, step)) if self.draws and self.training else {}
        return am_attention(q, k, v, self.lut, self.scale, table=table, buckets=buckets, lengths=lengths,
                            causal=self.causal, offset=offset, **drawn)


# ------------------------------------------------------------------ exact: dropout
class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, step, p, seed, call):
        ctx.save_for_backward(step)      # raised before backward, the mask would be another: torch then refuses
        ctx.drawn = p, seed, call
        return dropout(x.contiguous(), p, seed=seed, call=call, step=step,
                       residual=None if residual is None else residual.contiguous())

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (step,), (p, seed, call) = ctx.saved_tensors, ctx.drawn
        dx = dropout(dy.contiguous(), p, seed=seed, call=call, step=step) if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None, None


def am_dropout(x, p: float, *, seed: int, call: int = 0, step=None, residual=None):
    """residual + dropout(x), differentiable in both; the mask is a function of
    (seed, call + step) and is drawn again in the backward pass."""
    return _DropoutFn.apply(x, residual, step, float(p), seed, call)


class Dropout(torch.nn.Module):
    """forward(x, residual=None): in training residual + x / (1 - p) where x
    stays and residual where it is dropped, with a new mask at each call; in
    evaluation residual + x.  No mask is kept.  step and call: as AMAttention's."""

    def __init__(self, p: float = 0.1, *, seed: int | None = None, generator: torch.Generator | None = None):
        super().__init__()
        if not 0.0 <= p < 1.0:
            raise ValueError("dropout takes a p in [0, 1)")
        self.p, self.draws = float(p), _Draws(seed, generator)

    def forward(self, x, residual=None, *, step=None, call=None):
        if not self.training or self.p == 0.0:
            return x if residual is None else residual + x
        return am_dropout(x, self.p, residual=residual, **self.draws.next(call, step))


# ------------------------------------------------------------------ exact: group norm
def _even_pixels(t: torch.Tensor) -> torch.Tensor:
    """A tensor whose pixels are evenly spaced with contiguous channels: t (a slice of wider pixels, say), or a copy."""
    if t.is_contiguous() or t.dim() < 2 or not t.numel():
        return t.contiguous()
    if t.shape[-1] == 1 or t.stride(-1) == 1:
        ld = at = None
        for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
            if n == 1:
                continue
            ld, at = (s, 1) if ld is None else (ld, at)
            if s != ld * at:
                return t.contiguous()
            at *= n
        if ld is None or ld >= t.shape[-1]:
            return t
    return t.contiguous()


class _GroupNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, groups, eps, activation, y_dtype):
        x = _even_pixels(x)
        y, mean, rstd = group_norm(x, groups, w, b, eps=eps, activation=activation, y_dtype=y_dtype)
        ctx.save_for_backward(x, w, b, mean, rstd)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, b, mean, rstd = ctx.saved_tensors
        dx, dw, db = group_norm_backward(_even_pixels(dy), x, w, b, mean, rstd, activation=ctx.activation)
        return dx, dw, db, None, None, None, None


class GroupNorm(torch.nn.Module):
    """Group norm with its activation over [batch, ..., channels] tensors:
    forward(x) = act(xh weight + bias), with xh the channels of a group
    normalised over all of a sample's pixels.  activation: "none", "relu" or
    "silu"; y_dtype: the output's type (x's)."""

    def __init__(self, groups: int, channels: int, *, activation: str = "none", eps: float = 1e-5, affine: bool = True,
                 y_dtype=None, device="cuda"):
        super().__init__()
        if groups < 1 or channels % groups:
            raise ValueError(f"{groups} groups do not divide {channels} channels")
        self.groups, self.activation, self.eps, self.y_dtype = groups, activation, float(eps), y_dtype
        self.weight = torch.nn.Parameter(torch.ones(channels, device=device)) if affine else None
        self.bias = torch.nn.Parameter(torch.zeros(channels, device=device)) if affine else None

    def forward(self, x):
        return _GroupNormFn.apply(x, self.weight, self.bias, self.groups, self.eps, self.activation, self.y_dtype)


# ------------------------------------------------------------------ exact: block norm
def _dense_rows(t: torch.Tensor) -> torch.Tensor:
    """A matrix whose rows are contiguous and do not overlap: t, or a copy (of a transposed or expanded one)."""
    if t.dim() != 2 or t.is_contiguous() or (t.stride(1) == 1 and t.stride(0) >= t.shape[1]):
        return t
    return t.contiguous()


class _BlockNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, w_post, w_pre, gate, alpha, eps, n_dtype):
        r, n, rstd_post, rstd_pre = block_norm(x, y, w_post, w_pre, gate=gate, alpha=alpha, eps=eps, n_dtype=n_dtype)
        ctx.save_for_backward(r, y, w_post, w_pre, gate, rstd_post, rstd_pre)
        ctx.set_materialize_grads(False)     # an output that is not used has no gradient to read
        ctx.alpha = alpha
        if r is x:                       # no block output yet: x passes through
            r = x.view_as(x)
        return r, n

    @staticmethod
    @once_differentiable
    def backward(ctx, dr, dn):
        r, y, w_post, w_pre, gate, rstd_post, rstd_pre = ctx.saved_tensors

        def rows(t):
            return None if t is None else t.contiguous()
        dx, dy, dgate, dw_post, dw_pre = block_norm_backward(rows(dr), rows(dn), r, y, w_post, w_pre, rstd_post,
                                                             rstd_pre, gate=gate, alpha=ctx.alpha)
        return dx, dy, dw_post, dw_pre, dgate, None, None, None


class BlockNorm(torch.nn.Module):
    """The norms between two blocks: forward(x, y) takes the residual stream x
    and a block's output y and returns (r, n), the new residual stream
    r = x + alpha gate rms_norm(y) w_post and the next block's input
    n = rms_norm(r) w_pre.  forward(x) alone returns (x, rms_norm(x) w_pre).
    post: norm y (else it enters as it is); gate: None, "channel" (a learnt
    gate of ones at the start), or a [groups, channels] tensor given to
    forward, one row for each rows / groups rows."""

    def __init__(self, channels: int, *, post: bool = True, gate: str | None = None, alpha: float = 1.0,
                 eps: float = 1e-6, n_dtype=None, device="cuda"):
        super().__init__()
        if gate not in (None, "channel"):
            raise ValueError('gate is None or "channel"; a gate per group of rows is given to forward')
        self.alpha, self.eps, self.n_dtype = float(alpha), float(eps), n_dtype
        self.w_pre = torch.nn.Parameter(torch.ones(channels, device=device))
        self.w_post = torch.nn.Parameter(torch.ones(channels, device=device)) if post else None
        self.gate = torch.nn.Parameter(torch.ones(1, channels, device=device)) if gate else None

    def forward(self, x, y=None, gate=None):
        shape = x.shape
        rows = _dense_rows(x.reshape(-1, shape[-1]))
        if y is None:
            r, n = _BlockNormFn.apply(rows, None, None, self.w_pre, None, self.alpha, self.eps, self.n_dtype)
        else:
            r, n = _BlockNormFn.apply(rows, _dense_rows(y.reshape(rows.shape)), self.w_post, self.w_pre,
                                      self.gate if gate is None else gate, self.alpha, self.eps, self.n_dtype)
        return r.reshape(shape), n.reshape(shape)


# ------------------------------------------------------------------ exact: vocabulary loss
class _VocabLossFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, targets, row_weight, ignore_index, reduction):
        loss, _, _, dh, dw = vocab_loss_grad(h, w, targets, row_weight=row_weight, ignore_index=ignore_index,
                                             reduction=reduction)   # the gradients for an upstream one of 1
        ctx.save_for_backward(dh, dw)
        return loss[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        def scaled(t):                   # fp32 products (a factor without dimensions would be rounded to bf16 first)
            return torch.mul(t, g.reshape(1, 1), out=torch.empty_like(t))
        dh, dw = ctx.saved_tensors
        return scaled(dh), scaled(dw), None, None, None, None


def am_vocab_loss(h, w, targets, *, row_weight=None, ignore_index=-100, reduction="mean"):
    """Cross entropy of softmax(h w^T) against the targets without keeping the
    logits, differentiable in h [tokens, dim] and w [vocab, dim] (both bf16).
    The gradients come with the loss, in the same pass, and backward scales
    them by its fp32 factor, which rounds them to bf16 once more; where none is wanted (evaluation), the loss is computed alone.
    row_weight gets no gradient, so one that requires it is refused."""
    if row_weight is not None and row_weight.requires_grad and torch.is_grad_enabled():
        raise ValueError("the vocabulary loss has no gradient for row_weight: detach it")
    h, w, targets = _dense_rows(h), _dense_rows(w), targets.contiguous()
    row_weight = None if row_weight is None else row_weight.contiguous()
    if not (torch.is_grad_enabled() and (h.requires_grad or w.requires_grad)):
        return vocab_loss(h, w, targets, row_weight=row_weight, ignore_index=ignore_index, reduction=reduction)[0][0]
    return _VocabLossFn.apply(h, w, targets, row_weight, ignore_index, reduction)


class VocabHead(torch.nn.Module):
    """The last layer of a language model with its loss: forward(h, targets)
    with h [..., dim] bf16 and targets [...] int64.  The weight is bf16;
    optim.AdamW keeps its fp32 master."""

    def __init__(self, dim: int, vocab: int, *, ignore_index: int = -100, reduction: str = "mean", device="cuda",
                 generator: torch.Generator | None = None):
        super().__init__()
        self.ignore_index, self.reduction = ignore_index, reduction
        w = torch.randn((vocab, dim), generator=generator) / math.sqrt(dim)
        self.weight = torch.nn.Parameter(w.to(device=device, dtype=torch.bfloat16))

    def forward(self, h, targets, row_weight=None):
        return am_vocab_loss(h.reshape(-1, h.shape[-1]), self.weight, targets.reshape(-1), row_weight=row_weight,
                             ignore_index=self.ignore_index, reduction=self.reduction)
