"""Sparse Mixture-of-Experts FFN layer for MI355X (gfx950): forward,
gradient, and the training operators around them; dense linear and
feed-forward layers, and AdamW.

The layer runs in hand-written HIP kernels behind the C ABI of
include/moe.h (libmoe.so, built in-tree).  This package is the thin torch
binding: torch supplies device memory and streams only.
"""
from ._lib import (MoeDenseDesc, MoeDesc, MoeError, MoeGrads,  # noqa: F401
                   MoeLinearDesc, MoeRouting, MoeTensor, MoeWeights, lib)
from .dense import (DenseGrads, DenseLayer, DenseWeights,  # noqa: F401
                    LinearGrads, LinearWeights, make_dense_desc,
                    make_linear_desc, moe_dense_backward, moe_dense_forward,
                    moe_dense_grad_workspace_size, moe_dense_workspace_size,
                    moe_linear, moe_linear_grad,
                    moe_linear_grad_workspace_size, moe_linear_workspace_size)
from .layer import (Grads, MoeLayer, RouterWeights, Routing,  # noqa: F401
                    Weights, make_desc, moe_backward,
                    moe_bias_update, moe_capacity, moe_clip_grads,
                    moe_clip_workspace_size, moe_combine, moe_combine_rows,
                    moe_combine_rows_grad, moe_dispatch_rows,
                    moe_dispatch_rows_grad,
                    moe_ffn_down, moe_ffn_up, moe_forward, moe_forward_noalloc,
                    moe_gemm_tail_split,
                    moe_gemm_variant, moe_grad_norm, moe_grad_workspace_size,
                    moe_grouped_ffn, moe_permute, moe_route_dispatch,
                    moe_router_grad, moe_router_grad_workspace_size,
                    moe_router_topk,
                    moe_workspace_size)
from .optim import AdamW  # noqa: F401

__version__ = "0.1.0"
