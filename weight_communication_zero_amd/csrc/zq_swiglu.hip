// zq_swiglu.hip -- SwiGLU with its inputs kept as int8 blocks, and its gradient
// from them.
//   forward   h = g sg(g) u;  codes and scales of g and of u
//   backward  dg = dh u sg (1 + g (1 - sg)),  du = dh g sg,  [h = g sg u]
//
// Both are single passes over the data.  Forward moves 3 E + 2 (1 + 4/B) bytes an
// element (E = 4 or 2 bytes of the type), backward 2 (1 + 4/B) + 3 E or 4 E.  A
// lane owns 8 consecutive elements of a 512-element part of its wave's tile, as in
// the plain int8 quantizer: a block is a group of adjacent lanes, or several parts
// of the whole wave.  No LDS.
//
// Bound by HBM: 46 M elements in bf16, block 128, take 70 us forward (372 MB at 5.3
// TB/s) and 58 us backward (6.4); 180 M elements backward with h 315 us (1.81 GB at
// 5.7).  A copy of the same card runs at 4.9.
#include "zq_device.h"
#include "zq_layers_launch.h"
#include "zq_rows.h"

namespace zq {
namespace {

// exp(x) for x <= 0, off by 1.5 ulp or so: the product with log2(e) is kept in two
// parts, so that its rounding does not grow with |x| (4 instructions more than
// exp2(x log2(e)), which at x = -80 is off by 40 ulp).  Below -100 (and for NaN) that of
// -100, which is 0 to within 2^-140: nothing is multiplied by an infinity.
__device__ __forceinline__ float exp_neg(float x) {
    constexpr float kHi = 0x1.715476p0f, kLo = 0x1.4ae0cp-26f, kLn2 = 0x1.62e430p-1f;
    x = __builtin_fmaxf(x, -100.0f);
    const float t = x * kHi;
    const float r = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, r * kLn2, e);
}

// sigmoid(g) and 1 - sigmoid(g), neither by subtraction, so that both keep their
// relative precision and nothing overflows.  (Of a NaN they are 0 and 1: every use
// multiplies by g itself.)
__device__ __forceinline__ void sigmoid(float g, float* s, float* not_s) {
    const float a = exp_neg(-__builtin_fabsf(g));
    const float r = __builtin_amdgcn_rcpf(1.0f + a);
    const float q = a * r;
    *s = g >= 0.0f ? r : q;
    *not_s = g >= 0.0f ? q : r;
}

template <int B>
struct SwGeom {
    static constexpr int SUB = kWave * 8;
    static constexpr int LPB = B <= SUB ? B / 8 : kWave;  // lanes of a block
    static constexpr int SPB = B <= SUB ? 1 : B / SUB;    // parts of a block
    static constexpr int U = SPB;
    static constexpr int TILE = SUB * U;
};

// The largest magnitude of 16-bit values, two a word, as binary32 bits: magnitudes
// order like their bits (NaN above all), also after widening.
template <int T>
__device__ __forceinline__ uint32_t top_of(u4 w) {
    typedef uint16_t us2 __attribute__((ext_vector_type(2)));
    us2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(us2, w[i] & 0x7FFF7FFFu));
    const uint32_t top = max((uint32_t)m.x, (uint32_t)m.y);
    return fbits(half_lo<T>(top));
}

// 8 elements from element e on; of the last ones, those at n and after are 0.  Gives
// their largest magnitude's bits where TOP says so.
template <int T, bool MASK, bool TOP = false>
__device__ __forceinline__ uint32_t load8(const void* __restrict__ p, uint64_t e, uint64_t n,
                                          float* x) {
    uint32_t top = 0;
    if constexpr (!MASK) {
        if constexpr (T == kF32) {
            const f4 a = ld_stream((const f4*)((const float*)p + e));
            const f4 b = ld_stream((const f4*)((const float*)p + e + 4));
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
            const u4 w = ld_stream((const u4*)((const uint16_t*)p + e));
            x[0] = half_lo<T>(w.x); x[1] = half_hi<T>(w.x);
            x[2] = half_lo<T>(w.y); x[3] = half_hi<T>(w.y);
            x[4] = half_lo<T>(w.z); x[5] = half_hi<T>(w.z);
            x[6] = half_lo<T>(w.w); x[7] = half_hi<T>(w.w);
            if constexpr (TOP)
                return top_of<T>(w);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = 0.0f;
            if (e + j < n) {
                if constexpr (T == kF32)
                    x[j] = ((const float*)p)[e + j];
                else
                    x[j] = half_lo<T>(((const uint16_t*)p)[e + j]);
            }
        }
    }
    if constexpr (TOP) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, absbits(x[j]));
    }
    return top;
}

template <int T, bool MASK>
__device__ __forceinline__ void store8(const float* x, void* __restrict__ p, uint64_t e,
                                       uint64_t n) {
    if constexpr (T == kF32) {
        if constexpr (!MASK) {
            st_stream(f4{x[0], x[1], x[2], x[3]}, (f4*)((float*)p + e));
            st_stream(f4{x[4], x[5], x[6], x[7]}, (f4*)((float*)p + e + 4));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e + j < n)
                    ((float*)p)[e + j] = x[j];
        }
    } else {
        const u4 v = {pack_products<T>(x[0], x[1]), pack_products<T>(x[2], x[3]),
                      pack_products<T>(x[4], x[5]), pack_products<T>(x[6], x[7])};
        if constexpr (!MASK) {
            st_stream(v, (u4*)((uint16_t*)p + e));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e + j < n)
                    ((uint16_t*)p)[e + j] = (uint16_t)(v[j / 2] >> (16 * (j & 1)));
        }
    }
}

// The kept form of a tile, of which this lane's largest magnitude is `top`: scales, then
// codes.  Adding 1.5 2^23 to a quotient rounds it to the nearest integer, ties to even,
// and leaves its two's complement in the low bits: the codes' bytes are picked from
// there.
template <int B, bool MASK>
__device__ __forceinline__ void keep(const float (&x)[SwGeom<B>::U][8], uint32_t top,
                                     uint64_t base, int lane, uint64_t n,
                                     int8_t* __restrict__ codes, float* __restrict__ scales) {
    using G = SwGeom<B>;
    constexpr float kInt = 0x1.8p23f;
    const BlockScale s = block_scale<127>(group_max<G::LPB>(top));
    const uint64_t first = base + (uint64_t)lane * 8;
    if (lane % G::LPB == 0 && (!MASK || first < n))
        scales[first / B] = s.s;

    bool redo = false;
    float f[G::U][8];
#pragma unroll
    for (int u = 0; u < G::U; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = x[u][j] * s.inv;
            f[u][j] = y + kInt;
            redo |= __builtin_fabsf(y - (f[u][j] - kInt)) > tie_band<127>();
        }
    if (redo | s.exact) {
#pragma unroll
        for (int u = 0; u < G::U; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[u][j] = code_fix<127>(x[u][j], s, f[u][j] - kInt) + kInt;
    }
#pragma unroll
    for (int u = 0; u < G::U; ++u) {
        const uint64_t e = base + (uint64_t)u * G::SUB + (uint64_t)lane * 8;
        u2 v;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v[h] = __builtin_amdgcn_perm(fbits(f[u][4 * h + 1]), fbits(f[u][4 * h]), 0x0C0C0400u) |
                   __builtin_amdgcn_perm(fbits(f[u][4 * h + 3]), fbits(f[u][4 * h + 2]),
                                         0x04000C0Cu);
        if constexpr (!MASK) {
            st_stream(v, (u2*)(codes + e));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e + j < n)
                    codes[e + j] = (int8_t)(v[j / 4] >> (8 * (j & 3)));
        }
    }
}

template <int T, int B, bool MASK>
__device__ __forceinline__ void forward_tile(const SwigluArgs& a, uint64_t tile) {
    using G = SwGeom<B>;
    const int lane = lane_id();
    const uint64_t base = tile * G::TILE;
    float g[G::U][8], v[G::U][8];
    uint32_t g_top = 0, v_top = 0;
#pragma unroll
    for (int u = 0; u < G::U; ++u) {
        const uint64_t e = base + (uint64_t)u * G::SUB + (uint64_t)lane * 8;
        g_top = max(g_top, load8<T, MASK, true>(a.gate, e, a.n, g[u]));
        v_top = max(v_top, load8<T, MASK, true>(a.up, e, a.n, v[u]));
    }
#pragma unroll
    for (int u = 0; u < G::U; ++u) {
        float h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float s, r;
            sigmoid(g[u][j], &s, &r);
            h[j] = g[u][j] * s * v[u][j];
        }
        store8<T, MASK>(h, a.h, base + (uint64_t)u * G::SUB + (uint64_t)lane * 8, a.n);
    }
    keep<B, MASK>(g, g_top, base, lane, a.n, a.gate_codes, a.gate_scales);
    keep<B, MASK>(v, v_top, base, lane, a.n, a.up_codes, a.up_scales);
}

template <int T, int B>
__global__ __launch_bounds__(kBlockThreads) void forward_kernel(SwigluArgs a) {
    using G = SwGeom<B>;
    const uint64_t full = a.n / G::TILE;
    uint64_t t = stream_wave_id<kGeomStream.threads>();
    for (; t < full; t += wave_count())
        forward_tile<T, B, false>(a, t);
    if (t == full && a.n % G::TILE)
        forward_tile<T, B, true>(a, t);
}

constexpr int kGradU = 1;
constexpr int kGradTile = kWave * 8 * kGradU;

// 8 kept values (one block: blocks have 32 elements or more).
template <bool MASK>
__device__ __forceinline__ u2 load_codes(const int8_t* __restrict__ p, uint64_t e, uint64_t n) {
    if constexpr (!MASK)
        return ld_stream((const u2*)(p + e));
    u2 v = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (e + j < n)
            v[j / 4] |= (uint32_t)(uint8_t)p[e + j] << (8 * (j & 3));
    return v;
}

__device__ __forceinline__ float code_at(u2 v, int j) {
    return (float)((int32_t)(v[j / 4] << (24 - 8 * (j & 3))) >> 24);
}

template <int T, bool H, bool MASK>
__device__ __forceinline__ void backward_tile(const SwigluGradArgs& a, uint64_t tile) {
    const uint64_t base = tile * kGradTile + (uint64_t)lane_id() * 8;
    u2 gc[kGradU], uc[kGradU];
    float gs[kGradU], us[kGradU], d[kGradU][8];
#pragma unroll
    for (int u = 0; u < kGradU; ++u) {
        const uint64_t e = base + (uint64_t)u * kWave * 8;
        gc[u] = load_codes<MASK>(a.gate_codes, e, a.n);
        uc[u] = load_codes<MASK>(a.up_codes, e, a.n);
        gs[u] = us[u] = 0.0f;
        if (!MASK || e < a.n) {
            gs[u] = a.gate_scales[e >> a.log2b];
            us[u] = a.up_scales[e >> a.log2b];
        }
        load8<T, MASK>(a.dh, e, a.n, d[u]);
    }
#pragma unroll
    for (int u = 0; u < kGradU; ++u) {
        const uint64_t e = base + (uint64_t)u * kWave * 8;
        float dg[8], du[8], h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float g = code_at(gc[u], j) * gs[u], v = code_at(uc[u], j) * us[u];
            float s, r;
            sigmoid(g, &s, &r);
            const float silu = g * s;
            // The sigmoid's part, 1.1 at most, first: dh u alone may leave binary32.
            dg[j] = d[u][j] * (s * (1.0f + g * r)) * v;
            du[j] = d[u][j] * silu;
            h[j] = silu * v;
        }
        store8<T, MASK>(dg, a.dgate, e, a.n);
        store8<T, MASK>(du, a.dup, e, a.n);
        if constexpr (H)
            store8<T, MASK>(h, a.h, e, a.n);
    }
}

template <int T, bool H>
__global__ __launch_bounds__(kBlockThreads) void backward_kernel(SwigluGradArgs a) {
    const uint64_t full = a.n / kGradTile;
    uint64_t t = stream_wave_id<kGeomStream.threads>();
    for (; t < full; t += wave_count())
        backward_tile<T, H, false>(a, t);
    if (t == full && a.n % kGradTile)
        backward_tile<T, H, true>(a, t);
}

template <int T>
const void* forward_fn(uint32_t block, uint32_t* tile) {
    switch (block) {
#define ZQ_SW(B)                                          \
    case B:                                               \
        *tile = SwGeom<B>::TILE;                          \
        return (const void*)&forward_kernel<T, B>;
        ZQ_SW(32) ZQ_SW(64) ZQ_SW(128) ZQ_SW(256) ZQ_SW(512) ZQ_SW(1024) ZQ_SW(2048) ZQ_SW(4096)
#undef ZQ_SW
        default: return nullptr;
    }
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, int type, uint32_t block, hipStream_t stream) {
    uint32_t tile = 1;
    const void* fn = type == kF32    ? forward_fn<kF32>(block, &tile)
                     : type == kBF16 ? forward_fn<kBF16>(block, &tile)
                     : type == kF16  ? forward_fn<kF16>(block, &tile)
                                     : nullptr;
    if (!fn)
        return hipErrorInvalidValue;
    SwigluArgs k = a;
    void* args[] = {&k};
    return hipLaunchKernel(fn, grid_for_tiles((a.n + tile - 1) / tile, kGeomStream),
                           dim3(kGeomStream.threads), args, 0, stream);
}

hipError_t launch_swiglu_grad(const SwigluGradArgs& a, int type, hipStream_t stream) {
    const bool h = a.h != nullptr;
    const void* fn = type == kF32    ? h ? (const void*)&backward_kernel<kF32, true>
                                         : (const void*)&backward_kernel<kF32, false>
                     : type == kBF16 ? h ? (const void*)&backward_kernel<kBF16, true>
                                         : (const void*)&backward_kernel<kBF16, false>
                     : type == kF16  ? h ? (const void*)&backward_kernel<kF16, true>
                                         : (const void*)&backward_kernel<kF16, false>
                                     : nullptr;
    if (!fn)
        return hipErrorInvalidValue;
    SwigluGradArgs k = a;
    void* args[] = {&k};
    return hipLaunchKernel(fn, grid_for_tiles((a.n + kGradTile - 1) / kGradTile, kGeomStream),
                           dim3(kGeomStream.threads), args, 0, stream);
}

}  // namespace zq
