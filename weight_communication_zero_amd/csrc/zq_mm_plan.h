// zq_mm_plan.h -- host side of the matrix products: which tile a product takes,
// into how many parts its k's are split, and the launches.
#pragma once

#include <algorithm>

#include "zq_mm.h"

namespace zq {

// The tiles there are: 256 x 256 by 8 waves (160 KiB of LDS, one workgroup a CU),
// 128 x 128 by 4 waves (80 KiB, two a CU), and for few rows or columns 32 x 64 by 4
// waves (56 KiB).
enum MmTileKind : int { kTile256 = 0, kTile128 = 1, kTileSmall = 2 };

struct MmPlan {
    int kind;
    uint32_t splits;
};

constexpr uint32_t kMaxSplits = 32;

constexpr uint32_t tile_rows(int kind) {
    return kind == kTile256 ? 256 : kind == kTile128 ? 128 : 32;
}
constexpr uint32_t tile_cols(int kind) {
    return kind == kTile256 ? 256 : kind == kTile128 ? 128 : 64;
}

inline uint64_t div_up(uint64_t a, uint64_t b) { return (a + b - 1) / b; }
inline uint64_t round_up(uint64_t a, uint64_t b) { return div_up(a, b) * b; }

// Floats of partial sums that a plan needs.
inline uint64_t part_floats(const MmPlan& p, uint64_t M, uint64_t N) {
    return p.splits > 1 ? p.splits * M * round_up(N, 4) : 0;
}

// The tile and the splits of the least time by a simple model: the workgroups that a CU
// works through, each of its steps of 64 k's and of what lies around them, and for a
// split the partial sums' way to memory and back.  Operands' bytes have no term in it: it
// is fitted to products that the matrix units bound, and where one of few rows waits for
// memory it may choose too many splits or too large a tile.  Measured; the chosen
// and the next best of some products, in us (tile edge / splits):
//   2048 x 2048 x 8192     128/2   73    256/4   75
//   256 x 4096 x 16384     128/8   49    256/8   60
//   321 x 515 x 1001       32/1    7.3   128/4   12
//   65 x 513 x 1000        32/1    6.6   128/4   11
//   256 x 32000 x 2048     128/1   37    256/1   50
//   512 x 32000 x 2048     256/1   59    128/1   67
inline MmPlan mm_plan(uint64_t M, uint64_t N, uint64_t K, bool may_split) {
    struct Cost {
        double step, around;  // of a workgroup, its CU shared out
        double alone;         // a step of a workgroup that has a CU to itself
    };
    constexpr Cost kCost[3] = {{1.5, 4.0, 1.25}, {0.475, 2.0, 0.62}, {0.185, 2.0, 0.19}};
    const uint64_t steps = std::max<uint64_t>(div_up(K, kMmK), 1);
    MmPlan best = {kTile256, 1};
    double least = 1e30;
    for (int kind : {kTile256, kTile128, kTileSmall}) {
        const Cost& c = kCost[kind];
        const uint64_t tiles = div_up(M, tile_rows(kind)) * div_up(N, tile_cols(kind));
        for (uint64_t s = 1; s <= (may_split ? kMaxSplits : 1) && (s == 1 || steps / s >= 4); ++s) {
            const double per_cu = (double)div_up(tiles * s, 256), n = (double)div_up(steps, s);
            double us = std::max(per_cu * (n * c.step + c.around), n * c.alone + 4.0);
            if (s > 1)
                us += 3.0 + (double)(2 * s * M * N) * 4 / 5e6;
            if (us < least) {
                least = us;
                best = {kind, (uint32_t)s};
            }
        }
    }
    return best;
}

template <int T, bool TA, bool TB>
using MmShape256 = MmShape<T, 256, 256, 2, 4, 2, TA, TB>;
template <int T, bool TA, bool TB>
using MmShape128 = MmShape<T, 128, 128, 2, 2, 2, TA, TB>;
template <int T, bool TA, bool TB>
using MmShapeSmall = MmShape<T, 32, 64, 1, 4, 4, TA, TB>;

constexpr uint32_t tile_threads(int kind) { return kind == kTile256 ? 512 : 256; }

// The product with its plan's grid.
inline MmArgs mm_planned(MmArgs a, const MmPlan& p) {
    a.wgs = (uint32_t)div_up(div_up(a.M, tile_rows(p.kind)) * div_up(a.N, tile_cols(p.kind)), 8) * 8;
    a.splits = p.splits;
    return a;
}

template <int T, bool TA, bool TB, class Epi>
hipError_t launch_mm(const MmArgs& a, const typename Epi::Args& e, const MmPlan& p,
                     hipStream_t stream) {
    const void* fn = p.kind == kTile256   ? (const void*)&mm_kernel<MmShape256<T, TA, TB>, Epi>
                     : p.kind == kTile128 ? (const void*)&mm_kernel<MmShape128<T, TA, TB>, Epi>
                                          : (const void*)&mm_kernel<MmShapeSmall<T, TA, TB>, Epi>;
    MmArgs k = mm_planned(a, p);
    typename Epi::Args ke = e;
    void* args[] = {&k, &ke};
    return hipLaunchKernel(fn, dim3(k.wgs * k.splits), dim3(tile_threads(p.kind)), args, 0, stream);
}

// A product into MmOut, its partial sums (where split) in `part`.
struct MmInto {
    MmArgs a;
    MmOut o;
    MmPlan plan;
    float* part;
    bool pairs = false;  // MmSum's

    MmSum::Args sum() const {
        return {o, plan.splits > 1 ? part : nullptr, a.M, round_up(a.N, 4), pairs};
    }
};

inline hipError_t launch_mm_join(const MmInto& p, hipStream_t stream) {
    if (p.plan.splits == 1)
        return hipSuccess;
    MmSum::Args e = p.sum();
    uint32_t splits = p.plan.splits, M = p.a.M, N = p.a.N;
    const uint32_t* dyn = p.a.dyn_m;
    void* args[] = {&e, &splits, &M, &N, &dyn};
    const uint64_t wgs = std::min<uint64_t>(div_up((uint64_t)M * div_up(N, 4), 256), 8192);
    return hipLaunchKernel((const void*)&mm_join_kernel, dim3((uint32_t)wgs), dim3(256), args, 0,
                           stream);
}

template <int T, bool TA, bool TB>
hipError_t launch_mm_sum(const MmInto& p, hipStream_t stream) {
    const hipError_t st = launch_mm<T, TA, TB, MmSum>(p.a, p.sum(), p.plan, stream);
    return st == hipSuccess ? launch_mm_join(p, stream) : st;
}

// Two products that do not need each other, p of a plain and a transposed operand, q of
// two transposed ones: in one launch where they take tiles of one kind.
template <int T>
hipError_t launch_mm_two_sums(const MmInto& p, const MmInto& q, hipStream_t stream) {
    hipError_t st;
    if (p.plan.kind != q.plan.kind) {
        st = launch_mm_sum<T, false, true>(p, stream);
        return st == hipSuccess ? launch_mm_sum<T, true, true>(q, stream) : st;
    }
    const void* fn =
        p.plan.kind == kTile256
            ? (const void*)&mm_pair_kernel<MmShape256<T, false, true>, MmShape256<T, true, true>, MmSum>
        : p.plan.kind == kTile128
            ? (const void*)&mm_pair_kernel<MmShape128<T, false, true>, MmShape128<T, true, true>, MmSum>
            : (const void*)&mm_pair_kernel<MmShapeSmall<T, false, true>, MmShapeSmall<T, true, true>, MmSum>;
    MmArgs a1 = mm_planned(p.a, p.plan), a2 = mm_planned(q.a, q.plan);
    MmSum::Args e1 = p.sum(), e2 = q.sum();
    void* args[] = {&a1, &e1, &a2, &e2};
    st = hipLaunchKernel(fn, dim3(a1.wgs * a1.splits + a2.wgs * a2.splits),
                         dim3(tile_threads(p.plan.kind)), args, 0, stream);
    if (st == hipSuccess)
        st = launch_mm_join(p, stream);
    return st == hipSuccess ? launch_mm_join(q, stream) : st;
}

}  // namespace zq
