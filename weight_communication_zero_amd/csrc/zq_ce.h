// zq_ce.h -- what the cross entropy's loss and gradient share: the tokens that
// count, gathered; the plan of a call's workspace; pieces of the projection.
#pragma once

#include <cmath>

#include "zq_mm_plan.h"
#include "zq_stage.h"

namespace zq {

// Scalars in the workspace.
struct CeScalars {
    uint32_t count;    // tokens that count
    uint32_t twice;    // two times that
    float up, down;    // the power of two that scales q, and its inverse
};

// The tokens that count, in order: the r-th of them is token list[r].  Behind them
// stand the tokens that are left out, the last one first.
struct CeTokens {
    CeScalars* scalars;
    uint32_t* list;
    uint32_t* target;
    float *lse, *dloss;  // gradient only
};

struct CePrepArgs {
    const void* ids;
    uint32_t id64, n_tok, rows, scaled;
    const float *lse, *dloss;
    float *loss, *lse_out;  // loss only: cleared where a token is left out
    CeTokens t;
};

// Gathers the tokens that count.  One workgroup: positions need no second pass, and
// 2^14 tokens take two rounds of 8192 ids, J = 8 a thread in flight together (J = 1 for
// 1024 tokens or fewer, whose 7 loads a thread past the end would be for nothing).
template <bool GRAD, int J>
__global__ __launch_bounds__(1024) void ce_prep_kernel(CePrepArgs a) {
    __shared__ uint32_t sums[16], maxima[16];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t count = 0, top = 0;
    for (uint32_t base = 0; base < a.n_tok; base += 1024 * J) {
        const uint32_t first = base + wave * (64 * J) + lane;
        const uint32_t last = a.n_tok - 1;
        uint64_t id[J];
        load_ids<J>(a.ids, a.id64, [&](int j) { return min(first + j * 64, last); }, id);
        float lse[J], g[J];
        if constexpr (GRAD) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                lse[j] = a.lse[min(first + j * 64, last)];
                g[j] = a.dloss[min(first + j * 64, last)];
            }
        }
        uint64_t there[J];
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            there[j] = __builtin_amdgcn_ballot_w64(first + j * 64 < a.n_tok && id[j] < a.rows);
            mine += (uint32_t)__builtin_popcountll(there[j]);
        }
        if (lane == 0)
            sums[wave] = mine;
        __syncthreads();
        uint32_t at = count;
#pragma unroll
        for (uint32_t w = 0; w < 16; ++w) {
            at += w < wave ? sums[w] : 0;
            count += sums[w];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t t = first + j * 64;
            const uint32_t r = at + (uint32_t)__builtin_popcountll(
                                        there[j] & (((uint64_t)1 << lane) - 1));
            at += (uint32_t)__builtin_popcountll(there[j]);
            if (there[j] >> lane & 1) {
                a.t.list[r] = t;
                a.t.target[r] = (uint32_t)id[j];
                if constexpr (GRAD) {
                    a.t.lse[r] = lse[j];
                    a.t.dloss[r] = g[j];
                    top = max(top, absbits(g[j]) < 0x7F800000u ? absbits(g[j]) : 0);
                }
            } else if (t < a.n_tok) {
                // t - r tokens before this one are left out.
                a.t.list[last - (t - r)] = t;
                if constexpr (!GRAD) {
                    a.loss[t] = 0.0f;
                    a.lse_out[t] = 0.0f;
                }
            }
        }
    }
    if constexpr (GRAD) {
        top = group_max<64>(top);
        if (lane == 0)
            maxima[wave] = top;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        a.t.scalars->count = count;
        a.t.scalars->twice = 2 * count;
        if constexpr (GRAD) {
            for (int w = 0; w < 16; ++w)
                top = max(top, maxima[w]);
            // 2^(14 - exponent): exponents of a power of two and of its inverse stay
            // normal.
            int shift = 0;
            if (a.scaled && top)
                shift = min(max(141 - (int)(top >> 23), -120), 120);
            a.t.scalars->up = bitsf((uint32_t)(127 + shift) << 23);
            a.t.scalars->down = bitsf((uint32_t)(127 - shift) << 23);
        }
    }
}

// Byte offsets in the workspace.
struct CeLayout {
    uint64_t kp;              // width of staged rows: dim up to a multiple of 64
    uint32_t piece, n_pieces;
    uint32_t parts;           // of q: 1 or 2 (gradient)
    MmPlan logits;
    uint64_t scalars, list, target, lse, dloss, x, w;
    uint64_t part, run, z_target;   // loss
    uint64_t q, acc, x_sums, w_sums;  // gradient
    uint64_t ldacc;
    uint64_t total;

    uint32_t rows_of(uint32_t i, uint32_t rows) const {
        return i + 1 < n_pieces ? piece : rows - i * piece;
    }
};

struct CeTake {
    uint64_t at = 0;
    uint64_t operator()(uint64_t bytes) {
        const uint64_t here = at;
        at += round_up(bytes, 256);
        return here;
    }
};

// Pieces of `rows` of at most `most` rows each (multiples of 256), of one size but
// for the last.
inline void ce_pieces(CeLayout& l, uint32_t rows, uint64_t most) {
    most = std::max<uint64_t>(std::min<uint64_t>(most, (uint64_t)1 << 22) / 256 * 256, 256);
    l.n_pieces = (uint32_t)div_up(rows, most);
    l.piece = (uint32_t)round_up(div_up(rows, l.n_pieces), 256);
    l.n_pieces = (uint32_t)div_up(rows, l.piece);
}

inline void ce_take_tokens(CeLayout& l, CeTake& take, uint32_t n_tok, bool grad) {
    l.scalars = take(sizeof(CeScalars));
    l.list = take((uint64_t)n_tok * 4);
    l.target = take((uint64_t)n_tok * 4);
    l.lse = take(grad ? (uint64_t)n_tok * 4 : 0);
    l.dloss = take(grad ? (uint64_t)n_tok * 4 : 0);
    l.x = take(n_tok * l.kp * 2 * l.parts);
    l.w = take(l.piece * l.kp * 2);
}

inline CeTokens ce_tokens(const CeLayout& l, char* ws) {
    return {(CeScalars*)(ws + l.scalars), (uint32_t*)(ws + l.list), (uint32_t*)(ws + l.target),
            (float*)(ws + l.lse), (float*)(ws + l.dloss)};
}

template <bool GRAD>
hipError_t ce_prep(const CeArgs& a, const CeTokens& t, bool scaled, hipStream_t stream) {
    CePrepArgs p = {a.ids, a.id64, a.n_tok, a.rows, scaled, a.lse, a.dloss, a.loss, a.lse_out, t};
    void* args[] = {&p};
    const void* fn = a.n_tok <= 1024 ? (const void*)&ce_prep_kernel<GRAD, 1>
                                     : (const void*)&ce_prep_kernel<GRAD, 8>;
    return hipLaunchKernel(fn, dim3(1), dim3(1024), args, 0, stream);
}

// The hidden states of the tokens that count, and zeros for dx where one is left out.
inline StageArgs ce_stage_x(const CeArgs& a, const CeLayout& l, const CeTokens& t, char* ws) {
    StageArgs s = {};
    s.src = a.x;
    s.dim = a.dim;
    s.rows = a.n_tok;
    s.ld = (uint32_t)l.kp;
    s.out = (uint16_t*)(ws + l.x);
    s.list = t.list;
    s.count = &t.scalars->count;
    s.clear = (uint16_t*)a.dx;
    s.twice = l.parts - 1;
    return s;
}

// Whether the projection is an operand where it lies: else (codes, widths that are no
// multiple of 64) its pieces are staged.
inline bool w_in_place(const CeArgs& a, int w_type) {
    return w_type != kQ8 && a.dim % kMmK == 0;
}

// Rows v0 .. v0 + n - 1 of the projection as an operand.
inline MmOperand ce_piece(const CeArgs& a, int w_type, const CeLayout& l, uint32_t v0, char* ws) {
    if (w_in_place(a, w_type))
        return {(const uint16_t*)a.w + (uint64_t)v0 * a.dim, a.dim};
    return {(const uint16_t*)(ws + l.w), l.kp};
}

inline StageArgs ce_stage_w(const CeArgs& a, const CeLayout& l, uint32_t v0, uint32_t n, char* ws) {
    StageArgs s = {};
    s.src = a.w;
    s.scales = a.w_scales;
    s.log2b = a.log2b;
    s.dim = a.dim;
    s.row0 = v0;
    s.rows = n;
    s.ld = (uint32_t)l.kp;
    s.out = (uint16_t*)(ws + l.w);
    return s;
}

// Stages what piece i needs: its rows where the projection is not in place, and with the
// first piece the hidden states where `x` says so.
template <int T>
hipError_t ce_stage(const CeArgs& a, int w_type, const CeLayout& l, uint32_t i, bool x,
                    const CeTokens& t, char* ws, hipStream_t stream) {
    const uint32_t v0 = i * l.piece;
    const StageArgs sw = ce_stage_w(a, l, v0, l.rows_of(i, a.rows), ws);
    const StageArgs sx = ce_stage_x(a, l, t, ws);
    const bool w = !w_in_place(a, w_type);
    if (w && x && i == 0)
        return w_type == kQ8 ? launch_stage_both<T, kQ8, T>(sw, sx, stream)
                             : launch_stage_both<T, T, T>(sw, sx, stream);
    if (w)
        return launch_stage<T>(sw, w_type == kQ8 ? kQ8 : T, stream);
    return x && i == 0 ? launch_stage<T>(sx, T, stream) : hipSuccess;
}

// A logit is unit * (pre * sum): pre is the scale's sign and power of two, so that the
// inner product is exact (but for what leaves binary32's range), and unit, in [1, 2), is
// never a factor that makes NaN of an infinity.  A scale of 0 and one that is not finite
// stand in pre as they are.
struct CeScale {
    float pre, unit;
};

inline CeScale ce_scale(float scale) {
    if (scale == 0.0f || !std::isfinite(scale))
        return {scale, 1.0f};
    int e;
    const float unit = 2.0f * std::frexp(std::fabs(scale), &e);
    return {std::copysign(std::ldexp(1.0f, e - 1), scale), unit};
}

// Exponentials are taken in base 2: a factor or an exponent times log2(e), rounded once.
__device__ __forceinline__ float base2(float x) { return x * 0x1.715476p0f; }

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

}  // namespace zq
