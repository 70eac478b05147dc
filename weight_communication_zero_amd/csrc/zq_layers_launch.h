// zq_layers_launch.h -- internal launchers behind include/zq_layers.h (host
// side).  Each one assumes that the ABI layer has validated its arguments and
// only enqueues kernels on the given stream.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/zq_layers.h"
#include "zq_train_launch.h"

namespace zq {

struct SwigluArgs {
    const void *gate, *up;
    uint64_t n;
    void* h;
    int8_t* gate_codes;
    float* gate_scales;
    int8_t* up_codes;
    float* up_scales;
};

hipError_t launch_swiglu(const SwigluArgs& a, int type, uint32_t block, hipStream_t stream);

struct SwigluGradArgs {
    const int8_t* gate_codes;
    const float* gate_scales;
    const int8_t* up_codes;
    const float* up_scales;
    uint32_t log2b;
    const void* dh;
    uint64_t n;
    void *dgate, *dup, *h;
};

hipError_t launch_swiglu_grad(const SwigluGradArgs& a, int type, hipStream_t stream);

struct LinearGradArgs {
    const void* dy;
    const int8_t* codes;
    const float* scales;
    uint32_t log2b;
    uint32_t n_tok, out_dim, in_dim;
    void* grad;
    void* workspace;
};

size_t linear_grad_workspace(uint32_t n_tok, uint32_t out_dim, uint32_t in_dim);

hipError_t launch_linear_grad(const LinearGradArgs& a, int type, int grad_type, int mode,
                              hipStream_t stream);

// The projection: 16-bit values, or codes and scales (w_type kQ8).
struct CeArgs {
    const void* x;
    uint32_t n_tok, dim, rows;
    const void* w;
    const float* w_scales;
    uint32_t log2b;
    const void* ids;
    uint32_t id64;
    float scale;
    float* loss;         // loss call
    float* lse_out;
    const float* lse;    // gradient call
    const float* dloss;
    void* dx;
    void* dw;
    uint64_t piece;
    void* workspace;
};

size_t ce_loss_workspace(uint32_t n_tok, uint32_t rows, uint32_t dim, uint64_t piece);
size_t ce_grad_workspace(uint32_t n_tok, uint32_t rows, uint32_t dim, uint64_t piece);

hipError_t launch_ce_loss(const CeArgs& a, int type, int w_type, hipStream_t stream);
hipError_t launch_ce_grad(const CeArgs& a, int type, int w_type, int dw_type, int mode,
                          hipStream_t stream);

// Clears `bytes` bytes (a kernel: memset nodes of a captured graph are not used).
hipError_t launch_clear(void* p, uint64_t bytes, hipStream_t stream);

}  // namespace zq
