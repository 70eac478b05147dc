// zq_stage.h -- operands of the matrix products laid out in a call's workspace:
// rows of 16-bit values of the product's type with zeros up to a padded width, from
// rows of any width or from qwZ codes, all rows or those of a list.  HBM's: 180 M codes
// into bf16 take 91 us (5.9 TB/s), 67 M 16-bit values 42 us (6.4).
#pragma once

#include "zq_layers_launch.h"
#include "zq_rows.h"

namespace zq {

struct StageArgs {
    const void* src;        // values or codes, rows of `dim` elements
    const float* scales;
    uint32_t log2b;
    uint64_t dim, row0;     // the first row taken
    uint32_t rows, ld;      // rows and width of the result, a multiple of 8
    uint16_t* out;
    const uint32_t* list;   // row r is src's row list[r], for r < *count
    const uint32_t* count;
    uint16_t* clear;        // where set, rows list[r] of `dim` elements, r from *count on,
                            // are cleared in it
    uint32_t twice;         // 1: every row stands twice, one behind the other
};

// A lane per group of 8 elements of the result; the calling workgroup is wg of wgs.
template <int T, int IN, bool WHOLE>
__device__ __forceinline__ void stage_rows(const StageArgs& a, uint32_t wg, uint32_t wgs) {
    const uint32_t rows = a.count ? min(a.rows, *a.count) : a.rows;
    const uint32_t per_row = a.ld / 8;
    const uint64_t groups = (uint64_t)((a.clear ? a.rows : rows) << a.twice) * per_row;
    for (uint64_t g = wg * 256ull + threadIdx.x; g < groups; g += wgs * 256ull) {
        const uint32_t r2 = (uint32_t)(g / per_row), r = r2 >> a.twice;
        const uint32_t c = (uint32_t)(g - (uint64_t)r2 * per_row) * 8;
        Raw<T, 8> v = {{0, 0, 0, 0}};
        if (r >= rows) {
            if (c < a.dim && (r << a.twice) == r2)
                store_group<T, 8, WHOLE, false>(v, a.clear, a.list[r] * a.dim + c,
                                                (uint32_t)(a.dim - c));
            continue;
        }
        if (c < a.dim) {
            const uint64_t e = ((a.list ? a.list[r] : r) + a.row0) * a.dim + c;
            const uint32_t left = (uint32_t)(a.dim - c);
            Raw<IN, 8> x = load_group<IN, 8, WHOLE, false>(a.src, e, left);
            if constexpr (!WHOLE)
                whole<IN, 8>(x, left);
            if constexpr (IN == kQ8) {
                // A group touches two blocks at most (a block has 32 elements or more).
                const uint64_t last = e + (left < 8 ? left : 8) - 1;
                const float s0 = a.scales[e >> a.log2b];
                const float s1 = WHOLE ? s0 : a.scales[last >> a.log2b];
                float y[8];
                widen<IN, 8>(x, y);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = j < (int)left ? y[j] * ((e + j) >> a.log2b == e >> a.log2b ? s0 : s1)
                                         : 0.0f;
                v = narrow<T, 8>(y);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v.w[i] = x.w[i];
            }
        }
        store_group<T, 8, true, false>(v, a.out, g * 8, 8);
    }
}

template <int T, int IN, bool WHOLE>
__global__ __launch_bounds__(256) void stage_kernel(StageArgs a) {
    stage_rows<T, IN, WHOLE>(a, blockIdx.x, gridDim.x);
}

inline uint32_t stage_wgs(const StageArgs& a) {
    const uint64_t wgs = (((uint64_t)a.rows << a.twice) * (a.ld / 8) + 255) / 256;
    return (uint32_t)(wgs < 65536 ? wgs : 65536);
}

// in: T, or kQ8.
template <int T>
hipError_t launch_stage(const StageArgs& a, int in, hipStream_t stream) {
    if (a.rows == 0)
        return hipSuccess;
    const bool whole = a.dim % 8 == 0;
    const void* fn = in == kQ8 ? whole ? (const void*)&stage_kernel<T, kQ8, true>
                                       : (const void*)&stage_kernel<T, kQ8, false>
                     : whole   ? (const void*)&stage_kernel<T, T, true>
                               : (const void*)&stage_kernel<T, T, false>;
    StageArgs k = a;
    void* args[] = {&k};
    return hipLaunchKernel(fn, dim3(stage_wgs(a)), dim3(256), args, 0, stream);
}

// Two operands in one launch: the first by the first `wgs` workgroups.
template <int T, int IN1, bool WHOLE1, int IN2, bool WHOLE2>
__global__ __launch_bounds__(256) void stage_both_kernel(StageArgs a, StageArgs b, uint32_t wgs) {
    if (blockIdx.x < wgs)
        stage_rows<T, IN1, WHOLE1>(a, blockIdx.x, wgs);
    else
        stage_rows<T, IN2, WHOLE2>(b, blockIdx.x - wgs, gridDim.x - wgs);
}

// a of type IN1 (T or kQ8), b of type IN2.
template <int T, int IN1, int IN2>
hipError_t launch_stage_both(const StageArgs& a, const StageArgs& b, hipStream_t stream) {
    const bool wa = a.dim % 8 == 0, wb = b.dim % 8 == 0;
    const void* fn =
        wa   ? wb ? (const void*)&stage_both_kernel<T, IN1, true, IN2, true>
                  : (const void*)&stage_both_kernel<T, IN1, true, IN2, false>
        : wb ? (const void*)&stage_both_kernel<T, IN1, false, IN2, true>
             : (const void*)&stage_both_kernel<T, IN1, false, IN2, false>;
    StageArgs ka = a, kb = b;
    uint32_t wgs = stage_wgs(a);
    void* args[] = {&ka, &kb, &wgs};
    return hipLaunchKernel(fn, dim3(wgs + stage_wgs(b)), dim3(256), args, 0, stream);
}

}  // namespace zq
