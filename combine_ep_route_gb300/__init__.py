"""Routed MoE expert-parallel dispatch / combine for one GB300 GPU.

All W expert-parallel ranks live as blocks of one GPU's memory; the kernels
(sm_103a) sit behind the C-ABI in ``include/ep.h`` and this package binds it
for PyTorch tensors. See ``ep.EpContext``; ``product`` and ``router`` hold the operators of
the layer around it (experts' and linear products with their gradients, top-k routing).
"""
from .ep import (EpConfig, EpContext, DispatchOut, AgrsBuffers, agrs, alloc_agrs_buffers,  # noqa: F401
                 capacities, workspace_bytes)
from .product import (act_grad, check_products, experts_product, experts_product_dgrad,  # noqa: F401
                      experts_product_wgrad, linear, linear_dgrad, linear_wgrad, product_status,
                      set_product_wait_limit)
from .router import route_topk, route_topk_backward  # noqa: F401
from .balance import balance_loss, balance_loss_backward  # noqa: F401
from .product_w4 import (dequantize_weight4, experts_product_w4, linear_w4, pack_weight4,  # noqa: F401
                         quantize_weight4)
from .gradnorm import clip_grad_norm  # noqa: F401
from ._lib import EpError  # noqa: F401
