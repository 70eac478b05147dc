// zq_embed.hip -- embedding lookup with scaling, from a table of fp32, bf16 or
// fp16 rows or from the table's qwZ int8 codes and block scales.
//   out[t, j] = rne(fl(scale * w)),  w = table[id, j]  or  fl(k * s)
//
// Pure data movement: it reads each named row (4 / 2 / 1 + 4/B bytes an
// element) and writes 4 / 2 bytes an element.  The output is walked as one
// flat run of groups of G elements, a lane per group, so any dim fills the
// waves; a wave finds its first group's token by one scalar division and a
// lane its own from there.  G is 4 where an element has four bytes on either
// side, so that every access covers whole lines, else 8.
//
// 16384 tokens x 4096 from int8 codes into bf16 take 26 us in most bursts of
// calls, 157 MB at 6.0 TB/s, and up to 32 in others on the same inputs (41 us
// with plain in place of nontemporal stores: the output then displaces the rows
// that are read again); 8192 x 768 from fp32 6.7 us; one token 2.3 us.
#include "zq_rows.h"

namespace zq {
namespace {

constexpr int kLookU = 4;  // groups a lane has in flight

template <int IN, int OUT>
constexpr int group_elems() {
    return IN == kF32 || OUT == kF32 ? 4 : 8;
}

template <int IN, int OUT, bool WHOLE>
__global__ __launch_bounds__(kBlockThreads) void lookup_kernel(LookupArgs a) {
    constexpr int G = group_elems<IN, OUT>();
    const uint32_t per_row = (uint32_t)((a.dim + G - 1) / G);
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
            col[u] = (r - q * per_row) * G;
            in[u] = g0 + (uint64_t)u * kWave + lane < groups;
        }
        // Loads without branches around them stay in flight together: past the
        // end the last token is read, and row 0 for an id of no row.
        load_ids<kLookU>(a.ids, a.id64, [&](int u) { return min(tok[u], a.n_tok - 1); }, row);
#pragma unroll
        for (int u = 0; u < kLookU; ++u) {
            there[u] = row[u] < a.rows;
            row[u] = there[u] ? row[u] : 0;
        }
        Raw<IN, G> v[kLookU];
        float s0[kLookU], s1[kLookU];
#pragma unroll
        for (int u = 0; u < kLookU; ++u) {
            const uint64_t e = row[u] * a.dim + col[u];
            const uint32_t left = (uint32_t)a.dim - col[u];
            v[u] = load_group<IN, G, WHOLE, false>(a.table, e, left);
            if constexpr (IN == kQ8) {
                // A group touches two blocks at most (a block has 32 elements or more).
                s0[u] = a.scales[e >> a.log2b];
                s1[u] = WHOLE ? s0[u] : a.scales[(e + (left < G ? left : G) - 1) >> a.log2b];
            }
        }
#pragma unroll
        for (int u = 0; u < kLookU; ++u) {
            float x[G];
            if constexpr (!WHOLE)
                whole<IN, G>(v[u], (uint32_t)a.dim - col[u]);
            widen<IN, G>(v[u], x);
            if constexpr (IN == kQ8) {
                const uint64_t e = row[u] * a.dim + col[u];
#pragma unroll
                for (int j = 0; j < G; ++j)
                    x[j] *= WHOLE || (e + j) >> a.log2b == e >> a.log2b ? s0[u] : s1[u];
            }
#pragma unroll
            for (int j = 0; j < G; ++j)
                x[j] = there[u] ? a.scale * x[j] : 0.0f;
            if (in[u])
                store_group<OUT, G, WHOLE, true>(narrow<OUT, G>(x), a.out, tok[u] * a.dim + col[u],
                                                 (uint32_t)a.dim - col[u]);
        }
    }
}

template <int IN, int OUT>
hipError_t lookup_t(const LookupArgs& a, hipStream_t st) {
    constexpr int G = group_elems<IN, OUT>();
    const uint64_t per_wave = kWave * kLookU;
    const uint64_t tiles = (a.n_tok * ((a.dim + G - 1) / G) + per_wave - 1) / per_wave;
    const void* fn = a.dim % G == 0 ? (const void*)&lookup_kernel<IN, OUT, true>
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
