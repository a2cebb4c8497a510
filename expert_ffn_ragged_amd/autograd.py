"""torch autograd wrappers over the librd kernels: ragged_dot, trans_ragged_dot, the MoE MLP and the
routed expert layer's operators (route, dispatch_rows, combine_rows, routed_mlp).

The backward rules are the ones the SkyRL-tx page (PR #867, "Integrate
ragged_dot pallas kernel with group_offset support") states, with its
review's fix for trans_ragged_dot:

* ``out = ragged_dot(x, w)``: ``dx = ragged_dot(dout, w, trans_rhs)`` and
  ``dw = trans_ragged_dot(x, dout)``;
* ``z = trans_ragged_dot(x, y)``: ``dx = ragged_dot(y, dz, trans_rhs)`` and
  ``dy = ragged_dot(x, dz)``.

The MoE MLP (``moe_mlp``) is the expert FFN of the MaxText page (PR #5760,
"397B v7x trainer: MoE wo FSDP sharding and valid-rows-only MoE kernels"):
``fused = ragged_dot(x, wi)`` as ``[gate | up]``, ``act = silu(gate) * up``
(one kernel with the GLU as the GEMM's epilogue where the shapes allow it),
``out = ragged_dot(act, wo)``; its backward keeps the fused buffer as the GLU
residual (``act`` is recomputed from it, as the page's kernel path does) and
runs every step on the GPU kernels.  All of a layer's kernels read the same
device-resident ``group_sizes``; nothing is copied to the host, so forward
and backward can be captured in a HIP graph.

With a ``limit`` (the packed expert buffer's valid rows), rows at or past it
are neither read nor written by the GEMM and GLU kernels.  Those rows of a
forward output are left as allocated unless ``zero_tail`` is set (the
MaxText page's valid-rows commit: nothing downstream consumes them).  The
gradient of an input there is exactly zero, and that is what comes back: a
device-side kernel (``rd.zero_rows_from_limit``, limit read on the GPU)
writes those rows as +0, so no uninitialised memory reaches accumulation,
clipping or a scatter of the gradient.  Gradients come back in the dtype of
their input (bf16).

``routed_mlp`` is that MLP between the rows' way to the experts and back:
``out[t] = sum_i weights[t, i] * mlp(x[t], expert ids[t, i])``.  It keeps for
its backward pass the tokens (not their copies in the sorted buffer) and the
fused buffer in MX 8-bit elements.  With dy the output's gradient g copied to
the rows, ``d = dy @ wo^T`` is the gradient of the unweighted activation a of
a row, so the row's routing weight has the gradient <d, a> and need not see
the expert outputs, which are not kept either; w enters ``d_fused`` and the
operand ``w a`` of dwo in the GLU's backward kernel.  The activation in the
backward pass is that of the kept 8-bit values: gradients differ from the
bf16 ones by their rounding (2^-4 of an element at most).
"""

import torch
from torch.autograd.function import once_differentiable

from . import rd


def _none_grads(n):
    return (None,) * n


class RaggedDot(torch.autograd.Function):
    """out[rows of local group j] = x[rows] @ w[j] (trans_rhs: @ w[j].T)."""

    @staticmethod
    def forward(ctx, x, w, group_sizes, group_offset=None, limit=None, trans_rhs=False):
        ctx.save_for_backward(x, w, group_sizes, group_offset, limit)
        ctx.trans_rhs = trans_rhs
        return rd.ragged_dot(x, w, group_sizes, group_offset, limit, trans_rhs=trans_rhs)

    @staticmethod
    def backward(ctx, dout):
        x, w, gs, off, lim = ctx.saved_tensors
        dout = dout.contiguous()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            # d/dx of x @ w is dout @ w^T; with trans_rhs (x @ w^T) it is dout @ w
            dx = rd.zero_rows_from_limit(rd.ragged_dot(dout, w, gs, off, lim, trans_rhs=not ctx.trans_rhs), lim)
        if ctx.needs_input_grad[1]:
            gl = w.shape[0]
            if ctx.trans_rhs:   # w[j] is [n, k]: dw[j] = dout_j^T x_j
                dw = rd.trans_ragged_dot(dout, x, gs, gl, off, lim, out_dtype=w.dtype)
            else:               # w[j] is [k, n]: dw[j] = x_j^T dout_j
                dw = rd.trans_ragged_dot(x, dout, gs, gl, off, lim, out_dtype=w.dtype)
        return (dx, dw) + _none_grads(4)


class TransRaggedDot(torch.autograd.Function):
    """z[j] = x_j^T @ y_j over the rows of local group j; [num_local, k, n]."""

    @staticmethod
    def forward(ctx, x, y, group_sizes, num_local=None, group_offset=None, limit=None, out_dtype=None):
        ctx.save_for_backward(x, y, group_sizes, group_offset, limit)
        return rd.trans_ragged_dot(x, y, group_sizes, num_local, group_offset, limit,
                                   out_dtype=x.dtype if out_dtype is None else out_dtype)

    @staticmethod
    def backward(ctx, dz):
        x, y, gs, off, lim = ctx.saved_tensors
        dz = dz.to(x.dtype).contiguous()
        dx = dy = None
        if ctx.needs_input_grad[0]:
            dx = rd.zero_rows_from_limit(rd.ragged_dot(y, dz, gs, off, lim, trans_rhs=True), lim)  # y_r @ dz[j]^T
        if ctx.needs_input_grad[1]:
            dy = rd.zero_rows_from_limit(rd.ragged_dot(x, dz, gs, off, lim), lim)  # x_r @ dz[j] (the review's fix)
        return (dx, dy) + _none_grads(5)


class MoeMLP(torch.autograd.Function):
    """out = ragged_dot(silu(gate) * up, wo) with [gate | up] = ragged_dot(x, wi)."""

    @staticmethod
    def forward(ctx, x, wi, wo, group_sizes, group_offset=None, limit=None, zero_tail=False):
        m = x.shape[0]
        # one kernel (GEMM + GLU epilogue), except for decode-sized groups, whose split-contraction
        # ragged_dot path streams the weights faster than the fused tile kernel
        if m > 24 * wi.shape[0] and rd.glu_epilogue_supported(m, x.shape[1], wi.shape[2] // 2):
            act, fused = rd.ragged_dot_glu(x, wi, group_sizes, group_offset, limit, want_fused=True)
        else:
            fused = rd.ragged_dot(x, wi, group_sizes, group_offset, limit)
            act = rd.glu_fwd(fused, limit)
        out = torch.zeros((m, wo.shape[2]), dtype=x.dtype, device=x.device) if zero_tail else None
        out = rd.ragged_dot(act, wo, group_sizes, group_offset, limit, out=out)
        ctx.save_for_backward(x, wi, wo, group_sizes, group_offset, limit, fused)
        ctx.zero_tail = zero_tail
        return out

    @staticmethod
    def backward(ctx, dout):
        x, wi, wo, gs, off, lim, fused = ctx.saved_tensors
        dout = dout.contiguous()
        gl = wi.shape[0]
        act = rd.glu_fwd(fused, lim)                                         # recomputed from the residual
        d_act = rd.ragged_dot(dout, wo, gs, off, lim, trans_rhs=True)        # [m, h]
        dwo = rd.trans_ragged_dot(act, dout, gs, gl, off, lim, out_dtype=wo.dtype)
        d_fused = rd.glu_bwd(fused, d_act, lim)                              # [d_gate | d_up]
        dx = None
        if ctx.needs_input_grad[0]:
            dx = rd.zero_rows_from_limit(rd.ragged_dot(d_fused, wi, gs, off, lim, trans_rhs=True), lim)
        dwi = rd.trans_ragged_dot(x, d_fused, gs, gl, off, lim, out_dtype=wi.dtype)
        return (dx, dwi, dwo) + _none_grads(4)


def ragged_dot(x, w, group_sizes, group_offset=None, limit=None, trans_rhs=False):
    """Differentiable ragged_dot (gradients for x and w)."""
    return RaggedDot.apply(x, w, group_sizes, group_offset, limit, trans_rhs)


def trans_ragged_dot(x, y, group_sizes, num_local=None, group_offset=None, limit=None, out_dtype=None):
    """Differentiable trans_ragged_dot (gradients for x and y)."""
    return TransRaggedDot.apply(x, y, group_sizes, num_local, group_offset, limit, out_dtype)


def moe_mlp(x, wi, wo, group_sizes, group_offset=None, limit=None, zero_tail=False):
    """Differentiable MoE expert MLP over tokens sorted by expert.

    x: [m, d] bf16; wi: [num_local, d, 2h] bf16 producing [gate | up]; wo: [num_local, h, d_out] bf16;
    group_sizes: [G] int32 on the GPU; group_offset, limit: optional (1,) int32 GPU tensors.
    """
    return MoeMLP.apply(x, wi, wo, group_sizes, group_offset, limit, zero_tail)


class Route(torch.autograd.Function):
    """(weights, ids) of rd.route; the choice and the bias have no gradient."""

    @staticmethod
    def forward(ctx, logits, top_k, bias, score, groups, top_groups, renormalize, scale, limit):
        weights, ids = rd.route(logits, top_k, bias=bias, score=score, groups=groups, top_groups=top_groups,
                                renormalize=renormalize, scale=scale, limit=limit)
        ctx.save_for_backward(logits, ids)
        ctx.how = dict(score=score, renormalize=renormalize, scale=scale)
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, d_weights, _):
        logits, ids = ctx.saved_tensors
        return (rd.route_bwd(logits, ids, d_weights.contiguous(), **ctx.how),) + _none_grads(8)


class DispatchRows(torch.autograd.Function):
    """xs[slots[t, i]] = x[t]; the gradient adds the rows up again."""

    @staticmethod
    def forward(ctx, x, slots):
        ctx.save_for_backward(slots)
        return rd.dispatch_rows(x, slots)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        slots, = ctx.saved_tensors
        return rd.combine_rows(dxs.contiguous(), slots), None


class CombineRows(torch.autograd.Function):
    """out[t] = sum_i weights[t, i] * y[slots[t, i]] (weights None: a plain sum).  Rows of dy that no slot names
    are +0."""

    @staticmethod
    def forward(ctx, y, slots, weights):
        ctx.save_for_backward(y, slots, weights)
        return rd.combine_rows(y, slots, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, slots, weights = ctx.saved_tensors
        if weights is None:
            return rd.dispatch_rows(dout.contiguous(), slots, out=torch.zeros_like(y)), None, None
        dy, dw = rd.combine_rows_bwd(dout.contiguous(), y, slots, weights, dy=torch.zeros_like(y))
        return dy, None, dw


class RoutedMLP(torch.autograd.Function):
    """The expert MLP of the chosen experts of each token, weighted and added up."""

    @staticmethod
    def forward(ctx, x, weights, ids, wi, wo, experts, group_offset=None):
        sizes, rows, slots, total = rd.group_rows(ids, experts)
        xs = rd.dispatch_rows(x, slots)
        fused = rd.ragged_dot(xs, wi, sizes, group_offset, total)
        act, codes, scales = rd.glu_fwd_mx8(fused, total)
        y = rd.ragged_dot(act, wo, sizes, group_offset, total)
        ctx.save_for_backward(x, weights, wi, wo, sizes, rows, slots, total, group_offset, codes, scales)
        return rd.combine_rows(y, slots, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        x, weights, wi, wo, sizes, rows, slots, total, off, codes, scales = ctx.saved_tensors
        gl = wi.shape[0]
        dy = rd.dispatch_rows(dout.contiguous(), slots)
        d_act = rd.ragged_dot(dy, wo, sizes, off, total, trans_rhs=True)
        # slots without an expert have no row: their weights' gradient stays 0
        dot = torch.zeros(weights.numel(), dtype=torch.float32, device=x.device)
        d_fused, act, dot = rd.glu_bwd_mx8(codes, scales, d_act, total, weights=weights.view(-1), rows=rows, dot=dot)
        dx = dwi = dwo = None
        if ctx.needs_input_grad[4]:
            dwo = rd.trans_ragged_dot(act, dy, sizes, gl, off, total, out_dtype=wo.dtype)
        if ctx.needs_input_grad[3]:
            dwi = rd.trans_ragged_dot(rd.dispatch_rows(x, slots), d_fused, sizes, gl, off, total, out_dtype=wi.dtype)
        if ctx.needs_input_grad[0]:
            dx = rd.combine_rows(rd.ragged_dot(d_fused, wi, sizes, off, total, trans_rhs=True), slots)
        return dx, dot.view_as(weights), None, dwi, dwo, None, None


def route(logits, top_k, bias=None, score="softmax", groups=1, top_groups=None, renormalize=False, scale=1.0,
          limit=None):
    """Differentiable rd.route: (weights, ids), the gradient of the weights going to the logits."""
    return Route.apply(logits, top_k, bias, score, groups, top_groups, renormalize, scale, limit)


def dispatch_rows(x, slots):
    """Differentiable rd.dispatch_rows into a new buffer of tokens * top_k rows (gradient for x)."""
    return DispatchRows.apply(x, slots)


def combine_rows(y, slots, weights=None):
    """Differentiable rd.combine_rows (gradients for y and weights; weights None: a plain sum)."""
    return CombineRows.apply(y, slots, weights)


def routed_mlp(x, weights, ids, wi, wo, experts=None, group_offset=None):
    """out[t] = sum_i weights[t, i] * (silu(gate) * up) @ wo[e], [gate | up] = x[t] @ wi[e], e = ids[t, i].

    x: [tokens, d] bf16; weights, ids: [tokens, top_k] float32, int32 (route's); wi: [num_local, d, 2h] bf16,
    wo: [num_local, h, d_out] bf16, h a multiple of 32.  ids outside [0, experts) add nothing.  ``experts``
    (default num_local) counts the experts of ids where wi and wo hold a window of them that begins at
    ``group_offset`` ((1,) int32 on the GPU): experts outside the window add nothing, and their weights get a
    zero gradient.  Gradients for x, weights, wi and wo; what is kept for them is the tokens and the fused
    buffer in 8 bits.
    """
    return RoutedMLP.apply(x, weights, ids, wi, wo, wi.shape[0] if experts is None else experts, group_offset)
