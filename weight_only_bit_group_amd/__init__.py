"""weight_only_bit_group_amd -- group-wise INT4 (W4A16), AWQ calibration, FP4 decode, MXFP4 and FP8 products and routing to
experts on MI355X.

The compute lives in libaq.so (hand-written HIP kernels for gfx950 behind the C
ABI of include/aq.h).  ``binding`` exposes the entry points to torch under the
same names; ``layer`` builds on it the quantized linear modules, the experts of a
mixture and the norm-group AWQ apply step; ``synth`` holds the seeded synthetic inputs.  Importing this package
does not load the library; the first binding call does, and fails loudly if it
has not been built.
"""

__all__ = ["aq_quantize_pack", "aq_w4a16_gemv", "aq_w4a16_gemm", "aq_w4a16_gemm_workspace", "aq_act_absmean",
           "aq_act_absmean_workspace", "aq_awq_search", "aq_awq_search_workspace", "aq_fp4_gemm",
           "aq_fp4_gemm_workspace", "aq_fp4_quantize", "aq_fp4_quantize_workspace", "aq_quantize_pack8",
           "aq_w8a16_gemv", "aq_w8a16_gemm", "aq_w8a16_gemm_workspace", "aq_mxfp4_quantize", "aq_mxfp4_dequantize",
           "aq_mxfp4_gemm", "aq_mxfp4_gemm_a4", "aq_mxfp4_grouped_gemm", "aq_mxfp4_grouped_gemm_a4",
           "aq_fp8_quantize", "aq_fp8_dequantize", "aq_fp8_gemm", "aq_fp8_linear",
           "aq_fp8_linear_workspace", "aq_fp8_grouped_gemm", "aq_fp8_swiglu_quantize",
           "aq_fp8_experts", "aq_fp8_experts_workspace", "aq_moe_route", "aq_moe_route_backward",
           "aq_moe_group", "aq_moe_group_workspace", "aq_moe_combine", "aq_moe_combine_backward"]


def __getattr__(name):
    if name in __all__:
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)
