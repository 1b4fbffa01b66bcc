"""GB300-native zonal scatter of the geometric initial embedding (lmax = 3).

``libzs`` (C ABI in include/zs.h, CUDA kernels for sm_103a in csrc/) holds the
three steps of the hot path and the training operators of the block after it
(products grouped by species, residual norms with a gate, the AdamW step; the
embedding, routing, exchange with experts and dropout of a sparse one);
``zs`` is its thin Python binding, ``autograd`` the differentiable
torch.library operators over it (zs_gie::build_csr, zs_gie::zonal_scatter,
zs_gie::grouped_matmul, zs_gie::norm_gate_residual, zs_gie::embedding,
zs_gie::route, zs_gie::dispatch, zs_gie::combine, zs_gie::dropout), ``optim`` the
optimiser,
and ``workloads`` draws seeded synthetic graphs.
"""
from . import autograd  # noqa: F401  (registers the zs_gie operators)
from .optim import AdamW  # noqa: F401
from .zs import (  # noqa: F401
    AdamWPlan,
    ZsError,
    declared_functions,
    library_path,
    load,
    zs_adamw_step,
    zs_backward,
    zs_backward_csr,
    zs_check_timeouts,
    zs_combine,
    zs_combine_backward,
    zs_dispatch,
    zs_dropout,
    zs_embedding,
    zs_embedding_backward,
    zs_build_csr,
    zs_build_csr_workspace_bytes,
    zs_forward,
    zs_forward_workspace_bytes,
    zs_grouped_matmul,
    zs_grouped_matmul_backward,
    zs_grouped_matmul_dw,
    zs_grouped_matmul_dx,
    zs_norm_gate_residual,
    zs_norm_gate_residual_backward,
    zs_route,
    zs_route_backward,
)
