"""libzq: ZeRO++ / LoCo block-quantized gradient and weight communication
kernels, llm.c-style stochastic-rounding accumulation, embedding lookup and
gradient, and gradient-norm clipping for MI355X (gfx950).

The compute lives in ``libzq.so`` (hand-written HIP kernels behind the C ABI
in ``include/zq.h`` and ``include/zq_train.h``); this package is its thin
ctypes binding.
"""
from .zq import (  # noqa: F401
    ZQ_BF16, ZQ_FP32, ZQ_GRAD_ADD, ZQ_GRAD_ADD_SR, ZQ_GRAD_WRITE, DrSegmentTable, EfqSegmentTable,
    GradSegmentTable, SrSegmentTable, ZQError, embed_grad_workspace, grad_sumsq_workspace,
    int4_code_bytes, lib, num_blocks, zeropp_slots, zq_dequant_int8, zq_dequant_reduce,
    zq_dequant_reduce_batched, zq_embed_grad, zq_embed_lookup, zq_embed_lookup_int8,
    zq_grad_clip_batched, zq_grad_sumsq_batched, zq_quant_int8, zq_quantize_ef_int4,
    zq_quantize_ef_int4_batched, zq_quantize_ef_int4_permuted, zq_sr_accumulate,
    zq_sr_accumulate_batched,
)
