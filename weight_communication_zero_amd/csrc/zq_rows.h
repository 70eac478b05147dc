// zq_rows.h -- device access to rows of a [rows, dim] array by groups of eight
// consecutive elements, shared by the embedding kernels.
//
// Where dim is a multiple of 8 every group starts on a 16-byte boundary and is
// whole (WHOLE).  Otherwise a row may start at any element: a whole group is
// then read and written through vector types of the element's alignment (the
// hardware takes unaligned global accesses), and the row's last group, which
// has fewer elements, one by one.
#pragma once

#include "zq_device.h"
#include "zq_train_launch.h"

namespace zq {

typedef uint32_t u4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u2a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef float f4a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ uint32_t word(const u4& w, int i) {
    return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
}

// Raw bits of eight elements: 32 bytes for fp32, 16 for the 16-bit types.
template <int T>
struct Raw8 {
    u4 w[T == kF32 ? 2 : 1];
};

// Elements e .. e + 7 of p, of which the first `left` exist.
template <int T, bool WHOLE>
__device__ __forceinline__ Raw8<T> load8(const void* __restrict__ p, uint64_t e, uint32_t left) {
    Raw8<T> r;
    if constexpr (WHOLE) {
        if constexpr (T == kF32) {
            r.w[0] = ((const u4*)((const float*)p + e))[0];
            r.w[1] = ((const u4*)((const float*)p + e))[1];
        } else {
            r.w[0] = *(const u4*)((const uint16_t*)p + e);
        }
    } else if (left >= 8) {
        if constexpr (T == kF32) {
            const float* q = (const float*)p + e;
            r.w[0] = __builtin_bit_cast(u4, (f4)*(const f4a4*)q);
            r.w[1] = __builtin_bit_cast(u4, (f4)*(const f4a4*)(q + 4));
        } else {
            r.w[0] = (u4)*(const u4a2*)((const uint16_t*)p + e);
        }
    } else {
        uint32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (uint32_t j = 0; j < 7; ++j)
            if (j < left) {
                if constexpr (T == kF32)
                    v[j] = fbits(((const float*)p)[e + j]);
                else
                    v[j >> 1] |= (uint32_t)((const uint16_t*)p)[e + j] << (16 * (j & 1));
            }
        r.w[0] = u4{v[0], v[1], v[2], v[3]};
        if constexpr (T == kF32)
            r.w[1] = u4{v[4], v[5], v[6], v[7]};
    }
    return r;
}

template <int T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float x[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (T == kF32) {
            x[i] = bitsf(word(r.w[0], i));
            x[4 + i] = bitsf(word(r.w[T == kF32 ? 1 : 0], i));
        } else {
            x[2 * i] = half_lo<T>(word(r.w[0], i));
            x[2 * i + 1] = half_hi<T>(word(r.w[0], i));
        }
    }
}

// A binary32 product about to be rounded to fp16, kept apart from the rounding:
// the compiler otherwise joins the two into one v_fma_mixlo_f16 with a +0
// addend, which turns a product of -0 into +0.
__device__ __forceinline__ float apart(float x) {
    asm("" : "+v"(x));
    return x;
}

// Two fp32 products in type T's bits, rounded to nearest even.
template <int T>
__device__ __forceinline__ uint32_t pack_products(float lo, float hi) {
    if constexpr (T == kF16)
        return pack_f16_rne(apart(lo), apart(hi));
    else
        return pack_bf16_rne(lo, hi);
}

// Eight fp32 values in type T's bits, rounded to nearest even.
template <int T>
__device__ __forceinline__ Raw8<T> narrow8(const float x[8]) {
    Raw8<T> r;
    if constexpr (T == kF32) {
        r.w[0] = u4{fbits(x[0]), fbits(x[1]), fbits(x[2]), fbits(x[3])};
        r.w[T == kF32 ? 1 : 0] = u4{fbits(x[4]), fbits(x[5]), fbits(x[6]), fbits(x[7])};
    } else {
        r.w[0] = u4{pack_products<T>(x[0], x[1]), pack_products<T>(x[2], x[3]),
                    pack_products<T>(x[4], x[5]), pack_products<T>(x[6], x[7])};
    }
    return r;
}

template <int T, bool WHOLE>
__device__ __forceinline__ void store8(const Raw8<T>& r, void* __restrict__ p, uint64_t e,
                                       uint32_t left) {
    if constexpr (WHOLE) {
        if constexpr (T == kF32) {
            st_stream(r.w[0], (u4*)((float*)p + e));
            st_stream(r.w[T == kF32 ? 1 : 0], (u4*)((float*)p + e + 4));
        } else {
            st_stream(r.w[0], (u4*)((uint16_t*)p + e));
        }
    } else if (left >= 8) {
        if constexpr (T == kF32) {
            float* q = (float*)p + e;
            *(f4a4*)q = __builtin_bit_cast(f4, r.w[0]);
            *(f4a4*)(q + 4) = __builtin_bit_cast(f4, r.w[T == kF32 ? 1 : 0]);
        } else {
            *(u4a2*)((uint16_t*)p + e) = r.w[0];
        }
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 7; ++j)
            if (j < left) {
                if constexpr (T == kF32)
                    ((uint32_t*)p)[e + j] = word(r.w[j >> 2], j & 3);
                else
                    ((uint16_t*)p)[e + j] = (uint16_t)(word(r.w[0], j >> 1) >> (16 * (j & 1)));
            }
    }
}

// Token id of position t as an unsigned number: negative ids become large, so
// one comparison with the number of rows tells whether it names a row.
__device__ __forceinline__ uint64_t token_id(const void* __restrict__ ids, uint32_t id64,
                                             uint64_t t) {
    return id64 ? ((const uint64_t*)ids)[t] : (uint64_t)(int64_t)((const int32_t*)ids)[t];
}

}  // namespace zq
