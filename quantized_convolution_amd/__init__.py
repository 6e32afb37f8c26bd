"""quantized_convolution_amd: group-wise fully quantized 8-bit Winograd
convolution F(4,3) / F(6,3) with diagonal transform scales, on MI355X.

The compute path is the HIP library libwino_q8_conv.so (C ABI declared in
include/wino_q8_conv.h); `binding` marshals torch tensors into it. `ops` does
so for the operators around the convolution in a UNet (include/wino_q8_ops.h):
group norm with an activation, and the matrix product with bias, activation
and residual, forward and backward; `token_ops` for those on 8-bit codes
(include/wino_q8_tokens.h): packing, the root-mean-square norm, and the product
of codes with its backward. Importing this package does not load the library;
the first call does, and raises if it has not been built.
"""
from .binding import (Plan, Wq8Error, load, wq8_conv_forward, wq8_direct_conv, wq8_direct_forward,
                      wq8_direct_quantize_x, wq8_direct_weights_prepare, wq8_plan_bt_codes, wq8_plan_matrices,
                      wq8_stage1, wq8_stage2, wq8_stage2_i32, wq8_stage3, wq8_stage23,
                      wq8_weights_prepare)
from .ops import (LinearPlan, NormPlan, wq8_linear_backward, wq8_linear_forward, wq8_norm_backward,
                  wq8_norm_forward)
from .token_ops import (Q8LinearPlan, QuantPlan, RmsPlan, wq8_q8linear_backward, wq8_q8linear_forward, wq8_quant_pack,
                        wq8_quant_unpack, wq8_rms_backward, wq8_rms_forward)

__all__ = ["Plan", "Wq8Error", "load", "wq8_conv_forward", "wq8_direct_conv", "wq8_direct_forward",
           "wq8_direct_quantize_x", "wq8_direct_weights_prepare", "wq8_plan_bt_codes", "wq8_plan_matrices", "wq8_stage1",
           "wq8_stage2", "wq8_stage2_i32", "wq8_stage3", "wq8_stage23", "wq8_weights_prepare", "NormPlan", "LinearPlan",
           "wq8_norm_forward", "wq8_norm_backward", "wq8_linear_forward", "wq8_linear_backward", "QuantPlan", "RmsPlan",
           "Q8LinearPlan", "wq8_quant_pack", "wq8_quant_unpack", "wq8_rms_forward", "wq8_rms_backward",
           "wq8_q8linear_forward", "wq8_q8linear_backward"]
