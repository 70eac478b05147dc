// zq_rows.h -- device access to rows of a [rows, dim] array by groups of G = 4
// or 8 consecutive elements, shared by the embedding kernels.
//
// Where dim is a multiple of G every group starts on a boundary of its own size
// (16 bytes at most) and is whole (WHOLE).  Otherwise a row may start at any
// element: a whole group is then read and written through vector types of the
// element's alignment (the hardware takes unaligned global accesses), and the
// row's last group, which has fewer elements, one by one.
//
// NT marks the access nontemporal.  It pays where a wave's instruction covers
// whole cache lines, and costs where it covers half of each (8 fp32 values a
// lane take two instructions, each with every other 16 bytes): the line then
// travels twice.
#pragma once

#include "zq_device.h"
#include "zq_train_launch.h"

namespace zq {

// Bytes of an element: 4, 2, or 1 for qwZ codes.
template <int T>
constexpr int elem_bytes() {
    return T == kF32 ? 4 : T == kQ8 ? 1 : 2;
}

// The bits of G elements.
template <int T, int G>
struct Raw {
    static constexpr int kWords = G * elem_bytes<T>() / 4;
    uint32_t w[kWords];
};

// N 32-bit words at p, which is aligned to A bytes (NT: to the vector's size).
template <int N, int A, bool NT>
__device__ __forceinline__ void load_words(const void* __restrict__ p, uint32_t* w) {
    constexpr int V = N < 4 ? N : 4;
    typedef uint32_t vec __attribute__((ext_vector_type(V)));
    typedef uint32_t vec_a __attribute__((ext_vector_type(V), aligned(A)));
#pragma unroll
    for (int i = 0; i < N / V; ++i) {
        vec v;
        if constexpr (NT)
            v = __builtin_nontemporal_load((const vec*)p + i);
        else
            v = *((const vec_a*)p + i);
#pragma unroll
        for (int j = 0; j < V; ++j)
            w[i * V + j] = v[j];
    }
}

template <int N, int A, bool NT>
__device__ __forceinline__ void store_words(const uint32_t* w, void* __restrict__ p) {
    constexpr int V = N < 4 ? N : 4;
    typedef uint32_t vec_a __attribute__((ext_vector_type(V), aligned(A)));
#pragma unroll
    for (int i = 0; i < N / V; ++i) {
        if constexpr (NT && V == 4)
            st_stream(u4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]}, (u4*)p + i);
        else if constexpr (NT && V == 2)
            st_stream(u2{w[0], w[1]}, (u2*)p);
        else if constexpr (NT)
            st_stream(w[0], (uint32_t*)p);
        else {
            vec_a v;
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] = w[i * V + j];
            *((vec_a*)p + i) = v;
        }
    }
}

// Elements e .. e + G - 1 of p, of which the first `left` exist.
template <int T, int G, bool WHOLE, bool NT>
__device__ __forceinline__ Raw<T, G> load_group(const void* __restrict__ p, uint64_t e,
                                                uint32_t left) {
    constexpr int B = elem_bytes<T>(), N = Raw<T, G>::kWords;
    const char* q = (const char*)p + e * B;
    Raw<T, G> r;
    if constexpr (WHOLE) {
        load_words<N, (N < 4 ? 4 * N : 16), NT>(q, r.w);
    } else if (left >= G) {
        load_words<N, B, false>(q, r.w);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            r.w[i] = 0;
#pragma unroll
        for (uint32_t j = 0; j < G - 1; ++j)
            if (j < left) {
                if constexpr (B == 4)
                    r.w[j] = ((const uint32_t*)q)[j];
                else if constexpr (B == 2)
                    r.w[j / 2] |= (uint32_t)((const uint16_t*)q)[j] << (16 * (j & 1));
                else
                    r.w[j / 4] |= (uint32_t)((const uint8_t*)q)[j] << (8 * (j & 3));
            }
    }
    return r;
}

template <int T, int G, bool WHOLE, bool NT>
__device__ __forceinline__ void store_group(const Raw<T, G>& r, void* __restrict__ p, uint64_t e,
                                            uint32_t left) {
    constexpr int B = elem_bytes<T>(), N = Raw<T, G>::kWords;
    char* q = (char*)p + e * B;
    if constexpr (WHOLE) {
        store_words<N, (N < 4 ? 4 * N : 16), NT>(r.w, q);
    } else if (left >= G) {
        store_words<N, B, false>(r.w, q);
    } else {
#pragma unroll
        for (uint32_t j = 0; j < G - 1; ++j)
            if (j < left) {
                if constexpr (B == 4)
                    ((uint32_t*)q)[j] = r.w[j];
                else
                    ((uint16_t*)q)[j] = (uint16_t)(r.w[j / 2] >> (16 * (j & 1)));
            }
    }
}

// The elements' values (of codes: the integers).
template <int T, int G>
__device__ __forceinline__ void widen(const Raw<T, G>& r, float* x) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
        if constexpr (T == kF32)
            x[j] = bitsf(r.w[j]);
        else if constexpr (T == kQ8)
            x[j] = (float)((int32_t)(r.w[j / 4] << (24 - 8 * (j & 3))) >> 24);
        else
            x[j] = j & 1 ? half_hi<T>(r.w[j / 2]) : half_lo<T>(r.w[j / 2]);
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

// G fp32 values in type T's bits, rounded to nearest even.
template <int T, int G>
__device__ __forceinline__ Raw<T, G> narrow(const float* x) {
    Raw<T, G> r;
#pragma unroll
    for (int i = 0; i < Raw<T, G>::kWords; ++i) {
        if constexpr (T == kF32)
            r.w[i] = fbits(x[i]);
        else
            r.w[i] = pack_products<T>(x[2 * i], x[2 * i + 1]);
    }
    return r;
}

// Token ids of positions at(0) .. at(K - 1) as unsigned numbers: negative ids
// become large, so one comparison with the number of rows tells whether an id
// names a row.  The loads stand together behind the one branch on the type.
template <int K, typename F>
__device__ __forceinline__ void load_ids(const void* __restrict__ ids, uint32_t id64, F at,
                                         uint64_t* id) {
    if (id64) {
#pragma unroll
        for (int u = 0; u < K; ++u)
            id[u] = ((const uint64_t*)ids)[at(u)];
    } else {
        int32_t v[K];
#pragma unroll
        for (int u = 0; u < K; ++u)
            v[u] = ((const int32_t*)ids)[at(u)];
#pragma unroll
        for (int u = 0; u < K; ++u)
            id[u] = (uint64_t)(int64_t)v[u];
    }
}

}  // namespace zq
