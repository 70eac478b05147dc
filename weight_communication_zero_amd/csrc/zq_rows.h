// zq_rows.h -- device access to rows of a [rows, dim] array by groups of G = 4
// or 8 consecutive elements, shared by the embedding kernels.
//
// Where dim is a multiple of G every group starts on a boundary of its own size
// (16 bytes at most) and is whole (WHOLE).  Otherwise a row may start at any
// element: a whole group is then read and written through vector types of the
// element's alignment (the hardware takes unaligned global accesses), and the
// row's last group, which has fewer elements, in pieces of 4, 2 and 1.
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

// a or b by value.  (c ? a : b of two array elements is an lvalue, a choice of
// addresses, which can push a register array out into LDS.)
__device__ __forceinline__ uint32_t pick(bool c, uint32_t a, uint32_t b) { return c ? a : b; }

// The bits of G elements.  After a load of fewer than G, the words hold the piece
// of 4 (where there is one), then that of 2, then that of 1, each from a word of
// its own on, until whole() joins them.  (Codes are joined at once.)
template <int T, int G>
struct Raw {
    static constexpr int kWords = G * elem_bytes<T>() / 4;
    static constexpr int kTwo = G == 8 ? kWords / 2 : 0;                  // first word of the 2
    static constexpr int kOne = kTwo + (elem_bytes<T>() == 4 ? 2 : 1);  // word of the 1
    uint32_t w[kWords];
};

// Vectors of N 32-bit words, and the same at any address of A bytes' alignment.
// make() builds one in a single expression: a vector filled word by word is
// split up again by the compiler, which then drops a store's nontemporal mark.
template <int N, int A>
struct Vec;
#define ZQ_VEC(N, A, ...)                                                          \
    template <>                                                                    \
    struct Vec<N, A> {                                                             \
        typedef uint32_t type __attribute__((ext_vector_type(N)));                 \
        typedef uint32_t at __attribute__((ext_vector_type(N), aligned(A)));       \
        static __device__ __forceinline__ type load_nt(const void* p) {            \
            return __builtin_nontemporal_load((const at*)p);                       \
        }                                                                          \
        static __device__ __forceinline__ type make(const uint32_t* w) {           \
            return type{__VA_ARGS__};                                              \
        }                                                                          \
        static __device__ __forceinline__ void store_nt(type v, void* p) {         \
            __builtin_nontemporal_store((at)v, (at*)p);                            \
        }                                                                          \
    };
ZQ_VEC(4, 16, w[0], w[1], w[2], w[3])
ZQ_VEC(4, 4, w[0], w[1], w[2], w[3])
ZQ_VEC(4, 2, w[0], w[1], w[2], w[3])
ZQ_VEC(2, 8, w[0], w[1])
ZQ_VEC(2, 4, w[0], w[1])
ZQ_VEC(2, 2, w[0], w[1])
ZQ_VEC(2, 1, w[0], w[1])
ZQ_VEC(1, 4, w[0])
ZQ_VEC(1, 2, w[0])
ZQ_VEC(1, 1, w[0])
#undef ZQ_VEC

// N 32-bit words at p, which is aligned to A bytes.
template <int N, int A, bool NT>
__device__ __forceinline__ void load_words(const void* __restrict__ p, uint32_t* w) {
    constexpr int V = N < 4 ? N : 4;
    typedef Vec<V, A> X;
#pragma unroll
    for (int i = 0; i < N / V; ++i) {
        const typename X::at* q = (const typename X::at*)p + i;
        typename X::type v;
        if constexpr (NT)
            v = X::load_nt(q);
        else
            v = *q;
#pragma unroll
        for (int j = 0; j < V; ++j)
            w[i * V + j] = v[j];
    }
}

template <int N, int A, bool NT>
__device__ __forceinline__ void store_words(const uint32_t* w, void* __restrict__ p) {
    constexpr int V = N < 4 ? N : 4;
    typedef Vec<V, A> X;
#pragma unroll
    for (int i = 0; i < N / V; ++i) {
        typename X::at* q = (typename X::at*)p + i;
        const typename X::type v = X::make(w + i * V);
        if constexpr (NT)
            X::store_nt(v, q);
        else
            *q = v;
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
        if constexpr (G == 8)
            if (left & 4)
                load_words<B, B, false>(q, r.w);
        const char* q2 = q + (left & 4) * B;
        const char* q1 = q + (left & 6) * B;
        constexpr int two = Raw<T, G>::kTwo, one = Raw<T, G>::kOne;
        if constexpr (B == 4) {
            if (left & 2)
                load_words<2, 4, false>(q2, r.w + two);
            if (left & 1)
                r.w[one] = *(const uint32_t*)q1;
        } else if constexpr (B == 2) {
            if (left & 2)
                load_words<1, 2, false>(q2, r.w + two);
            if (left & 1)
                r.w[one] = *(const uint16_t*)q1;
        } else {
            r.w[two] = 0;
            if (left & 2)
                r.w[two] = (uint32_t)(uint8_t)q2[0] | (uint32_t)(uint8_t)q2[1] << 8;
            if (left & 1)
                r.w[two] |= (uint32_t)(uint8_t)*q1 << (8 * (left & 2));
        }
    }
    return r;
}

// Joins the pieces of a load of `left` < G elements; the others become 0.
template <int T, int G>
__device__ __forceinline__ void whole(Raw<T, G>& r, uint32_t left) {
    if (left >= G)
        return;
    constexpr int B = elem_bytes<T>(), N = Raw<T, G>::kWords, H = Raw<T, G>::kTwo;
    const bool four = G == 8 && (left & 4), two = left & 2, one = left & 1;
    uint32_t c[3] = {0, 0, 0};  // the last one to three elements
    if constexpr (B == 1) {
        c[0] = r.w[H];
    } else {
        const uint32_t last = pick(one, r.w[Raw<T, G>::kOne], 0);
        c[0] = pick(two, r.w[H], last);
        if constexpr (B == 4)
            c[1] = pick(two, r.w[H + 1], 0);
        c[B == 4 ? 2 : 1] = pick(two, last, 0);
    }
#pragma unroll
    for (int i = N - 1; i >= 0; --i) {
        const uint32_t low = i < 3 ? c[i < 3 ? i : 0] : 0;
        const uint32_t high = i >= H && i - H < 3 ? c[i >= H && i - H < 3 ? i - H : 0] : 0;
        r.w[i] = i >= H ? pick(H && !four, low, high) : pick(four, r.w[i], low);
    }
}

template <int T, int G, bool WHOLE, bool NT>
__device__ __forceinline__ void store_group(const Raw<T, G>& r, void* __restrict__ p, uint64_t e,
                                            uint32_t left) {
    constexpr int B = elem_bytes<T>(), N = Raw<T, G>::kWords;
    static_assert(B == 2 || (B == 4 && G == 4), "the outputs there are");
    char* q = (char*)p + e * B;
    if constexpr (WHOLE) {
        store_words<N, (N < 4 ? 4 * N : 16), NT>(r.w, q);
    } else if (left >= G) {
        store_words<N, B, NT && B == 4>(r.w, q);
    } else if constexpr (B == 4) {
        if (left & 2)
            store_words<2, 4, false>(r.w, q);
        if (left & 1)
            *(uint32_t*)(q + (left & 2) * 4) = pick(left & 2, r.w[2], r.w[0]);
    } else {
        const bool four = G == 8 && (left & 4);
        if (four)
            store_words<2, 2, false>(r.w, q);
        // The words of the last one to three elements.
        const uint32_t c0 = pick(four, r.w[N - 2], r.w[0]), c1 = pick(four, r.w[N - 1], r.w[1]);
        if (left & 2)
            *(Vec<1, 2>::at*)(q + (left & 4) * 2) = Vec<1, 2>::type{c0};
        if (left & 1)
            *(uint16_t*)(q + (left & 6) * 2) = (uint16_t)pick(left & 2, c1, c0);
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
