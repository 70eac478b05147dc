// zq_embed.hip -- embedding lookup with scaling, from a table of fp32, bf16 or
// fp16 rows or from the table's qwZ int8 codes and block scales.
//   out[t, j] = rne(fl(scale * w)),  w = table[id, j]  or  fl(k * s)
//
// Pure data movement: it reads each named row (4 / 2 / 1 + 4/B bytes an
// element) and writes 4 / 2 bytes an element.  The output is walked as one
// flat run of 8-element groups, a lane per group, so any dim fills the waves;
// a wave finds its first group's token by one scalar division and a lane its
// own from there.
#include "zq_rows.h"

namespace zq {
namespace {

constexpr int kLookU = 4;  // groups a lane has in flight

template <int IN, int OUT, bool WHOLE>
__global__ __launch_bounds__(kBlockThreads) void lookup_kernel(LookupArgs a) {
    const uint32_t per_row = (uint32_t)((a.dim + 7) / 8);
    const uint64_t groups = a.n_tok * per_row;
    const uint32_t lane = (uint32_t)lane_id();
    for (uint64_t w = wave_id(); w * (kWave * kLookU) < groups; w += wave_count()) {
        const uint64_t g0 = w * (kWave * kLookU);
        const uint64_t t0 = g0 / per_row;
        const uint32_t r0 = (uint32_t)(g0 - t0 * per_row) + lane;
        uint64_t tok[kLookU], row[kLookU];
        uint32_t col[kLookU];
        bool in[kLookU], there[kLookU];
#pragma unroll
        for (int u = 0; u < kLookU; ++u) {
            const uint32_t r = r0 + u * kWave;
            const uint32_t q = r / per_row;
            tok[u] = t0 + q;
            col[u] = (r - q * per_row) * 8;
            in[u] = g0 + (uint64_t)u * kWave + lane < groups;
            row[u] = in[u] ? token_id(a.ids, a.id64, tok[u]) : UINT64_MAX;
            there[u] = row[u] < a.rows;
        }
        float x[kLookU][8];
#pragma unroll
        for (int u = 0; u < kLookU; ++u) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[u][j] = 0.0f;
            if (!there[u])
                continue;
            const uint64_t e = row[u] * a.dim + col[u];
            const uint32_t left = (uint32_t)a.dim - col[u];
            if constexpr (IN == kQ8) {
                const int8_t* c = (const int8_t*)a.table + e;
                uint32_t v[2] = {0, 0};
                if (WHOLE) {
                    const u2 k = *(const u2*)c;
                    v[0] = k.x;
                    v[1] = k.y;
                } else if (left >= 8) {
                    const u2 k = (u2) * (const u2a1*)c;
                    v[0] = k.x;
                    v[1] = k.y;
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < 7; ++j)
                        if (j < left)
                            v[j >> 2] |= (uint32_t)(uint8_t)c[j] << (8 * (j & 3));
                }
                // Eight elements touch two blocks at most (a block has 32 or more).
                const uint64_t last = e + (left < 8 ? left : 8) - 1;
                const float s0 = a.scales[e >> a.log2b];
                const float s1 = WHOLE ? s0 : a.scales[last >> a.log2b];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float s = (WHOLE || (e + j) >> a.log2b == e >> a.log2b) ? s0 : s1;
                    x[u][j] = (float)((int32_t)(v[j >> 2] << (24 - 8 * (j & 3))) >> 24) * s;
                }
            } else {
                widen8<IN>(load8<IN, WHOLE>(a.table, e, left), x[u]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[u][j] *= a.scale;
        }
#pragma unroll
        for (int u = 0; u < kLookU; ++u)
            if (in[u])
                store8<OUT, WHOLE>(narrow8<OUT>(x[u]), a.out, tok[u] * a.dim + col[u],
                                   (uint32_t)a.dim - col[u]);
    }
}

template <int IN, int OUT>
hipError_t lookup_t(const LookupArgs& a, hipStream_t st) {
    const uint64_t per_wave = kWave * kLookU;
    const uint64_t tiles = (a.n_tok * ((a.dim + 7) / 8) + per_wave - 1) / per_wave;
    const void* fn = a.dim % 8 == 0 ? (const void*)&lookup_kernel<IN, OUT, true>
                                    : (const void*)&lookup_kernel<IN, OUT, false>;
    void* args[] = {(void*)&a};
    return hipLaunchKernel(fn, grid_for_tiles(tiles, kGeomReduce), dim3(kGeomReduce.threads), args,
                           0, st);
}

template <int IN>
hipError_t lookup_in(const LookupArgs& a, int out_type, hipStream_t st) {
    switch (out_type) {
        case kF32: return lookup_t<IN, kF32>(a, st);
        case kBF16: return lookup_t<IN, kBF16>(a, st);
        case kF16: return lookup_t<IN, kF16>(a, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_embed_lookup(const LookupArgs& a, int table_type, int out_type,
                               hipStream_t stream) {
    switch (table_type) {
        case kF32: return lookup_in<kF32>(a, out_type, stream);
        case kBF16: return lookup_in<kBF16>(a, out_type, stream);
        case kF16: return lookup_in<kF16>(a, out_type, stream);
        case kQ8: return lookup_in<kQ8>(a, out_type, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace zq
