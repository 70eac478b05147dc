// zq_train_launch.h -- internal launchers behind include/zq_train.h (host
// side).  Each one assumes that the ABI layer has validated its arguments and
// only enqueues kernels on the given stream.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/zq_train.h"
#include "zq_launch.h"

namespace zq {

// Element type of a lookup's table beside ElemType: qwZ int8 codes.
constexpr int kQ8 = 3;

enum GradMode : int { kGradWrite = 0, kGradAdd = 1, kGradAddSr = 2 };

struct LookupArgs {
    const void* table;    // values, or int8 codes
    const float* scales;  // block scales of the codes
    uint32_t log2b;
    uint32_t id64;        // ids are int64 (else int32)
    const void* ids;
    uint64_t n_tok, rows, dim;
    float scale;
    void* out;
};

hipError_t launch_embed_lookup(const LookupArgs& a, int table_type, int out_type,
                               hipStream_t stream);

struct EmbedGradArgs {
    const void* dout;
    const void* ids;
    uint32_t id64;
    uint64_t n_tok, rows, dim;
    float scale;
    void* grad;
    uint64_t seed, cbase;
    void* workspace;
};

size_t embed_grad_workspace(uint64_t n_tok, uint64_t rows, uint64_t dim);

hipError_t launch_embed_grad(const EmbedGradArgs& a, int d_type, int grad_type, int mode,
                             hipStream_t stream);

// One tensor of a norm or clip; n == 0 is skipped.
using GradSegment = zq_grad_segment;

size_t grad_sumsq_workspace(uint32_t n_seg);

hipError_t launch_grad_sumsq(const GradSegment* segs, uint32_t n_seg, int g_type, bool accumulate,
                             double* sumsq, double* partials, hipStream_t stream);

hipError_t launch_grad_clip(const GradSegment* segs, uint32_t n_seg, int g_type,
                            const double* sumsq, float max_norm, float eps, float* norm,
                            hipStream_t stream);

}  // namespace zq
