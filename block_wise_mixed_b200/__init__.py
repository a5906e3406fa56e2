"""block_wise_mixed_b200 -- block-wise mixed-precision weight-only quantized
linear layer (64x128 blocks, per-block bits in {0,1,2,3,4,5,6,8} plus 16-bit passthrough blocks, RTN-g128,
fp16 scale/zero, bi-directional channel reordering) on NVIDIA B200.

The computation lives in the C-ABI library ``libmpq.so`` (include/mpq.h); this
package only marshals arguments to it.  The ``i8_*`` calls are the 8-bit integer
operators for layers that stay at 8 bits throughout: row quantizer, linear, gated
feed-forward block and their gradients.  ``synth`` draws seeded workloads.
"""
from ._lib import (ACT_GELU_TANH, ACT_SILU, I8_WS_ZERO, I8Matrix, i8_dequantize, i8_empty, i8_gated,  # noqa: F401
                   i8_gated_backward, i8_gated_backward_workspace_size, i8_gated_workspace_size, i8_linear,
                   i8_linear_backward, i8_linear_backward_workspace_size, i8_linear_workspace_size, i8_matrix,
                   i8_plan, i8_quantize)
from ._lib import (GROUP_MAX, Y_BF16, Y_F32, MpqError, PackedLayer, allocate_bits, check, fold_orders,  # noqa: F401
                   linear,
                   linear_group, linear_group_workspace_size, linear_host, linear_host_workspace_size,
                   linear_timed, linear_typed_workspace_size, linear_workspace_size, pack, plan,
                   with_orders)
