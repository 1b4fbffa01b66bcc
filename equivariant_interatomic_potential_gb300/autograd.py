"""PyTorch operators over libzs, with autograd (first-order but for the grouped products).

The pull request "fused Triton zonal scatter for the GIE head" (deepmd-kit)
puts the zonal scatter behind a differentiable operator whose backward is
the edge-parallel pass and which has no double backward (sections "What"
and "Tests").  Here that operator is a ``torch.library`` custom op:

  ``zs_gie::build_csr(dst, num_nodes) -> (row_ptr, perm)``
  ``zs_gie::zonal_scatter(coup, rad, dst, row_ptr, perm, num_nodes) -> out``
  ``zs_gie::zonal_scatter_scaled(coup, rad, dst, row_ptr, perm, node_scale,
  num_nodes) -> (out, out_raw)``: the degree normalisation the pages apply
  after the operator (section "What", third bullet), fused: out[n] =
  node_scale[n] * the operator's sum, differentiable in node_scale too
  ``zs_gie::grouped_matmul(x, w, row_ptr, perm) -> y``: each row times the
  weights of its group (its species, or species and degree), the groups in a
  CSR from ``build_csr``; differentiable in x and w, its gradients again
  ``zs_gie::norm_gate_residual(h, x, gate, w_post, scale, w_pre, eps, kind) ->
  (y, u, stats)``: the norms around a block with its gate, residual scale and
  residual sum; differentiable in every tensor (``optim.AdamW`` steps them)

``zonal_scatter``'s backward is ``zs_gie::zonal_scatter_backward``, itself
an operator without a derivative, so a second backward raises.  It takes the
faster of libzs's two backward entry points for the ladder (measured on the
4096-node graph at C = 32): the CSR-order ``zs_backward_csr`` (the forward's
CSR is at hand) at lmax 2, 4 and 5, the edge-order ``zs_backward`` at lmax 1
and 3 and for every other channel count.  Every operator has a fake (meta)
implementation, so ``torch.compile`` traces through them with shapes only;
the launch grid is chosen inside libzs from the runtime sizes.  The
operators run libzs's CUDA kernels and nothing else: CPU tensors are
rejected.  Each call first reads the device's timeout flag (page-locked host
memory, no synchronisation) and raises if a bounded wait of an earlier
launch ran out.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import zs

_NS = "zs_gie"


def _cuda_only(name: str, *tensors: torch.Tensor) -> None:
    for t in tensors:
        if t.device.type != "cuda":
            raise ValueError(f"{_NS}::{name} runs on CUDA tensors only (got a {t.device.type} tensor)")
    zs.raise_on_timeout_flag(tensors[0].device)


# Ladders whose CSR-order backward is the faster one at C = 32.
CSR_BACKWARD_LADDERS = (2, 4, 5)


def uses_csr_backward(lmax: int, C: int) -> bool:
    """Whether zs_gie::zonal_scatter_backward takes zs_backward_csr for this shape."""
    return C == 32 and lmax in CSR_BACKWARD_LADDERS


@torch.library.custom_op(f"{_NS}::build_csr", mutates_args=())
def build_csr(dst: torch.Tensor, num_nodes: int) -> tuple[torch.Tensor, torch.Tensor]:
    """Stable destination CSR of int32 ``dst``: (row_ptr (N+1,), perm (E,)), int32."""
    _cuda_only("build_csr", dst)
    row_ptr, perm, _ = zs.zs_build_csr(dst.contiguous(), num_nodes)
    return row_ptr, perm


@build_csr.register_fake
def _(dst, num_nodes):
    return (dst.new_empty((num_nodes + 1,), dtype=torch.int32), dst.new_empty(dst.shape, dtype=torch.int32))


@torch.library.custom_op(f"{_NS}::zonal_scatter", mutates_args=())
def zonal_scatter(coup: torch.Tensor, rad: torch.Tensor, dst: torch.Tensor, row_ptr: torch.Tensor,
                  perm: torch.Tensor, num_nodes: int) -> torch.Tensor:
    """out (N, D, C): row 0 zero, rows 1..D-1 the zonal scatter of coup (E, D-1) x rad (E, lmax, C).

    lmax = rad.shape[1] (3 for the pages' 3/5/7 ladder), D = (lmax + 1)^2."""
    _cuda_only("zonal_scatter", coup, rad, dst, row_ptr, perm)
    return zs.zs_forward(coup.contiguous(), rad.contiguous(), row_ptr.contiguous(), perm.contiguous(), num_nodes)


@zonal_scatter.register_fake
def _(coup, rad, dst, row_ptr, perm, num_nodes):
    # ladder of degree lmax = rad.shape[1]: (lmax + 1)^2 node rows
    return coup.new_empty((num_nodes, (rad.shape[1] + 1) ** 2, rad.shape[2]))


@torch.library.custom_op(f"{_NS}::zonal_scatter_backward", mutates_args=())
def zonal_scatter_backward(grad_out: torch.Tensor, coup: torch.Tensor, rad: torch.Tensor, dst: torch.Tensor,
                           row_ptr: torch.Tensor, perm: torch.Tensor,
                           num_nodes: int) -> tuple[torch.Tensor, torch.Tensor]:
    """(d_coup (E, D-1), d_rad (E, lmax, C)) for the cotangent grad_out (N, D, C).

    row_ptr and perm are the CSR of dst (the forward's); the ladder and channel
    count pick the entry point (``uses_csr_backward``)."""
    _cuda_only("zonal_scatter_backward", grad_out, coup, rad, dst, row_ptr, perm)
    if uses_csr_backward(rad.shape[1], rad.shape[2]):
        return zs.zs_backward_csr(grad_out.contiguous(), coup.contiguous(), rad.contiguous(), row_ptr.contiguous(),
                                  perm.contiguous(), num_nodes)
    return zs.zs_backward(grad_out.contiguous(), coup.contiguous(), rad.contiguous(), dst.contiguous(), num_nodes)


@zonal_scatter_backward.register_fake
def _(grad_out, coup, rad, dst, row_ptr, perm, num_nodes):
    return coup.new_empty(coup.shape), rad.new_empty(rad.shape)


def _setup_context(ctx, inputs, output):
    coup, rad, dst, row_ptr, perm, num_nodes = inputs
    ctx.save_for_backward(coup, rad, dst, row_ptr, perm)
    ctx.num_nodes = num_nodes


def _backward(ctx, grad_out):
    coup, rad, dst, row_ptr, perm = ctx.saved_tensors
    d_coup, d_rad = zonal_scatter_backward(grad_out, coup, rad, dst, row_ptr, perm, ctx.num_nodes)
    return d_coup, d_rad, None, None, None, None


zonal_scatter.register_autograd(_backward, setup_context=_setup_context)


def zonal_scatter_from_dst(coup: torch.Tensor, rad: torch.Tensor, dst: torch.Tensor, num_nodes: int) -> torch.Tensor:
    """Build the CSR of dst, then the differentiable zonal scatter."""
    row_ptr, perm = build_csr(dst, num_nodes)
    return zonal_scatter(coup, rad, dst, row_ptr, perm, num_nodes)


@torch.library.custom_op(f"{_NS}::zonal_scatter_scaled", mutates_args=())
def zonal_scatter_scaled(coup: torch.Tensor, rad: torch.Tensor, dst: torch.Tensor, row_ptr: torch.Tensor,
                         perm: torch.Tensor, node_scale: torch.Tensor,
                         num_nodes: int) -> tuple[torch.Tensor, torch.Tensor]:
    """(out, out_raw): out[n] = node_scale[n] * out_raw[n], out_raw the zonal scatter (N, D, C)."""
    _cuda_only("zonal_scatter_scaled", coup, rad, dst, row_ptr, perm, node_scale)
    return zs.zs_forward_scaled(coup.contiguous(), rad.contiguous(), row_ptr.contiguous(), perm.contiguous(),
                                node_scale.contiguous(), num_nodes)


@zonal_scatter_scaled.register_fake
def _(coup, rad, dst, row_ptr, perm, node_scale, num_nodes):
    shape = (num_nodes, (rad.shape[1] + 1) ** 2, rad.shape[2])
    return coup.new_empty(shape), coup.new_empty(shape)


@torch.library.custom_op(f"{_NS}::zonal_scatter_scaled_backward", mutates_args=())
def zonal_scatter_scaled_backward(grad_out: torch.Tensor, coup: torch.Tensor, rad: torch.Tensor, dst: torch.Tensor,
                                  node_scale: torch.Tensor, out_raw: torch.Tensor,
                                  num_nodes: int) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(d_coup, d_rad, d_scale) for the cotangent grad_out of the scaled output."""
    _cuda_only("zonal_scatter_scaled_backward", grad_out, coup, rad, dst, node_scale, out_raw)
    return zs.zs_backward_scaled(grad_out.contiguous(), coup.contiguous(), rad.contiguous(), dst.contiguous(),
                                 node_scale.contiguous(), num_nodes, out_raw=out_raw.contiguous())


@zonal_scatter_scaled_backward.register_fake
def _(grad_out, coup, rad, dst, node_scale, out_raw, num_nodes):
    return coup.new_empty(coup.shape), rad.new_empty(rad.shape), node_scale.new_empty(node_scale.shape)


def _setup_context_scaled(ctx, inputs, output):
    coup, rad, dst, row_ptr, perm, node_scale, num_nodes = inputs
    out, out_raw = output
    ctx.mark_non_differentiable(out_raw)
    ctx.save_for_backward(coup, rad, dst, node_scale, out_raw)
    ctx.num_nodes = num_nodes


def _backward_scaled(ctx, grad_out, grad_raw):
    coup, rad, dst, node_scale, out_raw = ctx.saved_tensors
    d_coup, d_rad, d_scale = zonal_scatter_scaled_backward(grad_out, coup, rad, dst, node_scale, out_raw,
                                                           ctx.num_nodes)
    return d_coup, d_rad, None, None, None, d_scale, None


zonal_scatter_scaled.register_autograd(_backward_scaled, setup_context=_setup_context_scaled)


def degree_normalised_scatter(coup: torch.Tensor, rad: torch.Tensor, dst: torch.Tensor, node_scale: torch.Tensor,
                              num_nodes: int) -> torch.Tensor:
    """CSR of dst, then node_scale[n] * zonal scatter, differentiable in coup, rad and node_scale."""
    row_ptr, perm = build_csr(dst, num_nodes)
    return zonal_scatter_scaled(coup, rad, dst, row_ptr, perm, node_scale, num_nodes)[0]


@torch.library.custom_op(f"{_NS}::grouped_matmul", mutates_args=())
def grouped_matmul(x: torch.Tensor, w: torch.Tensor, row_ptr: torch.Tensor,
                   perm: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[i] = w[g(i)] x[i]: x (M, K), w (G, N, K), the CSR (row_ptr, perm) of the rows' groups; y (M, N)."""
    _cuda_only("grouped_matmul", x, w, row_ptr)
    return zs.zs_grouped_matmul(x.contiguous(), w.contiguous(), row_ptr.contiguous(), perm)


@grouped_matmul.register_fake
def _(x, w, row_ptr, perm=None):
    return x.new_empty((x.shape[0], w.shape[1]))


@torch.library.custom_op(f"{_NS}::grouped_matmul_backward", mutates_args=())
def grouped_matmul_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, row_ptr: torch.Tensor,
                            perm: Optional[torch.Tensor] = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(dx (M, K), dw (G, N, K)) for the cotangent dy (M, N)."""
    _cuda_only("grouped_matmul_backward", dy, x, w, row_ptr)
    return zs.zs_grouped_matmul_backward(dy.contiguous(), x.contiguous(), w.contiguous(), row_ptr.contiguous(), perm)


@grouped_matmul_backward.register_fake
def _(dy, x, w, row_ptr, perm=None):
    return x.new_empty(x.shape), w.new_empty(w.shape)


def _setup_context_grouped(ctx, inputs, output):
    ctx.save_for_backward(*inputs[:3], *(t for t in inputs[3:] if t is not None))


def _backward_grouped(ctx, dy):
    x, w, row_ptr, *perm = ctx.saved_tensors
    perm = perm[0] if perm else None
    if ctx.needs_input_grad[0] and ctx.needs_input_grad[1]:
        return (*grouped_matmul_backward(dy, x, w, row_ptr, perm), None, None)
    dx = grouped_matmul_dx(dy, w, row_ptr, perm) if ctx.needs_input_grad[0] else None   # fixed weights: the forces' path
    dw = grouped_matmul_dw(dy, x, row_ptr, perm) if ctx.needs_input_grad[1] else None
    return dx, dw, None, None


@torch.library.custom_op(f"{_NS}::grouped_matmul_dx", mutates_args=())
def grouped_matmul_dx(dy: torch.Tensor, w: torch.Tensor, row_ptr: torch.Tensor,
                      perm: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx (M, K) alone, for the cotangent dy (M, N)."""
    _cuda_only("grouped_matmul_dx", dy, w, row_ptr)
    return zs.zs_grouped_matmul_dx(dy.contiguous(), w.contiguous(), row_ptr.contiguous(), perm)


@grouped_matmul_dx.register_fake
def _(dy, w, row_ptr, perm=None):
    return dy.new_empty((dy.shape[0], w.shape[2]))


@torch.library.custom_op(f"{_NS}::grouped_matmul_dw", mutates_args=())
def grouped_matmul_dw(dy: torch.Tensor, x: torch.Tensor, row_ptr: torch.Tensor,
                      perm: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dw (G, N, K) alone, for the cotangent dy (M, N)."""
    _cuda_only("grouped_matmul_dw", dy, x, row_ptr)
    return zs.zs_grouped_matmul_dw(dy.contiguous(), x.contiguous(), row_ptr.contiguous(), perm)


@grouped_matmul_dw.register_fake
def _(dy, x, row_ptr, perm=None):
    return dy.new_empty((row_ptr.shape[0] - 1, dy.shape[1], x.shape[1]))


grouped_matmul.register_autograd(_backward_grouped, setup_context=_setup_context_grouped)


# The gradients are products of the same kind, linear in each operand, so that their own gradients are too (a potential
# trained on its forces differentiates them).

def _backward_grouped_dx(ctx, a):   # of dx = w^T dy, for the cotangent a (M, K)
    dy, w, row_ptr, *perm = ctx.saved_tensors
    perm = perm[0] if perm else None
    return (grouped_matmul(a, w, row_ptr, perm) if ctx.needs_input_grad[0] else None,
            grouped_matmul_dw(dy, a, row_ptr, perm) if ctx.needs_input_grad[1] else None, None, None)


def _backward_grouped_dw(ctx, b):   # of dw = sum dy x^T, for the cotangent b (G, N, K)
    dy, x, row_ptr, *perm = ctx.saved_tensors
    perm = perm[0] if perm else None
    return (grouped_matmul(x, b, row_ptr, perm) if ctx.needs_input_grad[0] else None,
            grouped_matmul_dx(dy, b, row_ptr, perm) if ctx.needs_input_grad[1] else None, None, None)


def _setup_context_grouped_backward(ctx, inputs, output):
    ctx.set_materialize_grads(False)
    ctx.save_for_backward(*inputs[:4], *(t for t in inputs[4:] if t is not None))


def _backward_grouped_backward(ctx, a, b):   # of both, for the cotangents a of dx and b of dw (None: zeros)
    dy, x, w, row_ptr, *perm = ctx.saved_tensors
    perm = perm[0] if perm else None
    g_dy = g_x = g_w = None
    if ctx.needs_input_grad[0]:
        parts = [grouped_matmul(r, v, row_ptr, perm) for r, v in ((a, w), (x, b)) if r is not None and v is not None]
        g_dy = sum(parts[1:], parts[0]) if parts else None
    if ctx.needs_input_grad[1] and b is not None:
        g_x = grouped_matmul_dx(dy, b, row_ptr, perm)
    if ctx.needs_input_grad[2] and a is not None:
        g_w = grouped_matmul_dw(dy, a, row_ptr, perm)
    return g_dy, g_x, g_w, None, None


grouped_matmul_dx.register_autograd(_backward_grouped_dx, setup_context=_setup_context_grouped)
grouped_matmul_dw.register_autograd(_backward_grouped_dw, setup_context=_setup_context_grouped)
grouped_matmul_backward.register_autograd(_backward_grouped_backward, setup_context=_setup_context_grouped_backward)


def species_linear(x: torch.Tensor, w: torch.Tensor, species: torch.Tensor) -> torch.Tensor:
    """CSR of the rows' species (M,) int32, then y[i] = w[species[i]] x[i], differentiable in
    x and w.  Rows whose species is outside [0, G) give zeros."""
    row_ptr, perm = build_csr(species, w.shape[0])
    return grouped_matmul(x, w, row_ptr, perm)


@torch.library.custom_op(f"{_NS}::norm_gate_residual", mutates_args=())
def norm_gate_residual(h: torch.Tensor, x: torch.Tensor, gate: Optional[torch.Tensor], w_post: torch.Tensor,
                       scale: torch.Tensor, w_pre: torch.Tensor, eps: float = 1e-6,
                       kind: str = "rms") -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, u, stats): y = x + scale * sigmoid(gate) * (norm(h) * w_post), u = norm(y) * w_pre; stats (M, 4)
    holds the rows' means and 1/roots and has no gradient."""
    _cuda_only("norm_gate_residual", h, x, w_post, scale, w_pre)
    return zs.zs_norm_gate_residual(h.contiguous(), x.contiguous(), None if gate is None else gate.contiguous(), w_post,
                                    scale, w_pre, eps=eps, kind=kind)


@norm_gate_residual.register_fake
def _(h, x, gate, w_post, scale, w_pre, eps=1e-6, kind="rms"):
    return h.new_empty(h.shape), h.new_empty(h.shape), h.new_empty((h.shape[0], 4), dtype=torch.float32)


@torch.library.custom_op(f"{_NS}::norm_gate_residual_backward", mutates_args=())
def norm_gate_residual_backward(
        dy: Optional[torch.Tensor], du: Optional[torch.Tensor], h: torch.Tensor, x: torch.Tensor, gate: Optional[torch.Tensor],
        w_post: torch.Tensor, scale: torch.Tensor, w_pre: torch.Tensor, stats: torch.Tensor, kind: str = "rms",
) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dh, dx, dgate, dw_post, dscale, dw_pre) for the cotangents dy and du (None: zeros); dgate is empty
    without a gate."""
    _cuda_only("norm_gate_residual_backward", *(t for t in (dy, du) if t is not None), h, x, w_post, scale, w_pre, stats)
    dh, dx, dgate, *sums = zs.zs_norm_gate_residual_backward(
        *(None if t is None else t.contiguous() for t in (dy, du)), h.contiguous(), x.contiguous(), None if gate is None else gate.contiguous(), w_post,
        scale, w_pre, stats, kind=kind)
    return (dh, dx, h.new_empty(0) if dgate is None else dgate, *sums)


@norm_gate_residual_backward.register_fake
def _(dy, du, h, x, gate, w_post, scale, w_pre, stats, kind="rms"):
    dgate = h.new_empty(0) if gate is None else gate.new_empty(gate.shape)
    return (h.new_empty(h.shape), x.new_empty(x.shape), dgate, *(t.new_empty(t.shape) for t in (w_post, scale, w_pre)))


def _setup_context_norm(ctx, inputs, output):
    h, x, gate, w_post, scale, w_pre, eps, kind = inputs
    ctx.set_materialize_grads(False)   # a cotangent that is not there is not read
    ctx.mark_non_differentiable(output[2])
    ctx.save_for_backward(h, x, w_post, scale, w_pre, output[2], *(() if gate is None else (gate,)))
    ctx.kind = kind


def _backward_norm(ctx, dy, du, _):
    if dy is None and du is None:
        return (None,) * 8
    h, x, w_post, scale, w_pre, stats, *gate = ctx.saved_tensors
    gate = gate[0] if gate else None
    dh, dx, dgate, dw_post, dscale, dw_pre = norm_gate_residual_backward(dy, du, h, x, gate, w_post, scale, w_pre, stats,
                                                                         ctx.kind)
    return dh, dx, None if gate is None else dgate, dw_post, dscale, dw_pre, None, None


norm_gate_residual.register_autograd(_backward_norm, setup_context=_setup_context_norm)
