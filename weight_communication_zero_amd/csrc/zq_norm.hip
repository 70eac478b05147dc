// zq_norm.hip -- the global norm of many gradient tensors, and clipping by it.
//   sumsq = [sumsq +] sum over all tensors of x * x            (binary64)
//   norm = sqrt(sumsq);  c = fl32(min(1, max_norm / (norm + eps)))
//   out = fl(c * x), rounded to nearest even in a 16-bit type
//
// The sum is binary64 from the first product on: a binary32 value's square is
// exact there and cannot overflow, and the order of the additions (tiles dealt
// round robin to a fixed number of waves, a tree in the wave and the
// workgroup, the workgroups' partials in a fixed order) depends on the
// segments' sizes alone, so equal inputs give equal bits.  No atomics.
//
// Both are bound by memory.  The sum reads 4 / 2 B/elem: 0.85 G elements in 494 us
// (fp32) or 246 (bf16), 6.9 TB/s.  The clip reads and writes them: 1071 us in
// fp32, 6.35 TB/s, 1074 in place.  28 MB of fp16 in 111 ragged tensors take 8 + 2
// us (sum and join) and 12 us (clip, a copy's rate).  A ragged last tile goes
// element by element; with every tensor filled up to whole tiles the three take
// 0.8 us and 0.7 us less.
// A clip in place with c = 1 touches no tensor, but the grid is the same: 0.85 G
// fp32 elements are 1.6 million workgroups, which come and go in 352 us.
#include <algorithm>

#include "zq_rows.h"

namespace zq {
namespace {

// Segments of a launch: the table travels in the kernel arguments (4 KB).
constexpr int kSumSegs = 192;
constexpr int kClipSegs = 144;
// Vectors of 16 bytes that a lane has in flight.  The clip's waves take one tile
// each in 1-wave workgroups, XCD by XCD (stream_wave_id), which the dispatcher
// keeps coming: 0.85 G fp32 elements, norm and clip together, took 1837 us with
// 2048 looping workgroups, 1640 / 1562 / 1613 us so with 4 / 2 / 1 vectors.
constexpr int kNormU = 4;
constexpr int kClipU = 2;
constexpr uint32_t kClipMaxWgs = 1u << 24;
// Workgroups of the sum, each looping over tiles: 0.85 G bf16 elements took
// 249.4 / 262.5 / 248.9 us with 1024 / 2048 / 4096 of them (6.8 TB/s; a fill
// writes 6.9), and with plain loads in place of nontemporal ones 274.
constexpr uint32_t kNormMaxWgs = 4096;
// Most tiles that one workgroup sums by itself, in one launch: 16 / 64 / 128 tiles
// take 2.7 / 4.2 / 6.4 us in a graph so, and 4.1 / 4.3 / 4.4 us as sum and join.
constexpr uint32_t kNormOneWg = 64;

// A tile is 64 lanes x U 16-byte vectors.
template <int T, int U>
struct NormGeom {
    static constexpr int VEC = T == kF32 ? 4 : 8;
    static constexpr int SUB = kWave * VEC;
    static constexpr int TILE = SUB * U;
};

// The segment of a tile, as SegmentFinder gives it, for tables of up to 192
// segments: lane l holds the cumulative tile counts l, l + 64 and l + 128, and
// a tile's segment is the number of counts that it has passed.
template <int N>
struct TileFinder {
    static constexpr int E = (N + kWave - 1) / kWave;
    uint32_t e[E];
    __device__ __forceinline__ explicit TileFinder(const uint32_t (&ends)[N]) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const uint32_t k = (uint32_t)lane_id() + i * kWave;
            e[i] = k < N ? ends[k] : UINT32_MAX;
        }
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t t) const {
        uint32_t s = 0;
#pragma unroll
        for (int i = 0; i < E; ++i)
            s += (uint32_t)__builtin_popcountll(__builtin_amdgcn_ballot_w64(t >= e[i]));
        return s;
    }
};

template <int T>
__device__ __forceinline__ float load1(const void* p, uint64_t i) {
    if constexpr (T == kF32)
        return ((const float*)p)[i];
    else
        return half_lo<T>(((const uint16_t*)p)[i]);
}

struct NormBatch {
    static constexpr int kSegs = kSumSegs, kU = kNormU;
    const void* g[kSegs];
    uint64_t n[kSegs];
    uint32_t tile_end[kSegs];  // cumulative tiles; unused entries hold UINT32_MAX
    uint32_t total;
};

// The value of the lane that a DPP control, or the swap of the two 32-lane
// halves, pairs with this one.
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the wave's lanes, the same tree on every call; every lane has it.
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp<0xB1>(v);   // quad_perm: lane ^ 1
    v += dpp<0x4E>(v);   // quad_perm: lane ^ 2
    v += dpp<0x141>(v);  // half mirror: the other quad of eight lanes
    v += dpp<0x140>(v);  // mirror: the other eight of sixteen
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// Sum over the workgroup; thread 0 has it.
__device__ __forceinline__ double group_sum(double v) {
    __shared__ double part[16];
    v = wave_sum(v);
    if (lane_id() == 0)
        part[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (uint32_t w = 1; w < blockDim.x >> 6; ++w)
            v += part[w];
    return v;
}

// out: one partial per workgroup, or (last) the result itself.
template <int T>
__global__ __launch_bounds__(1024) void sumsq_kernel(NormBatch b, double* out, uint32_t last,
                                                     uint32_t accumulate) {
    using G = NormGeom<T, kNormU>;
    const TileFinder<kSumSegs> find(b.tile_end);
    const int lane = lane_id();
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    for (size_t ts = wave_id(); ts < b.total; ts += wave_count()) {
        const uint32_t t = (uint32_t)ts, s = find(t);
        const uint64_t base = (uint64_t)(t - (s ? b.tile_end[s - 1] : 0u)) * G::TILE;
        const void* g = b.g[s];
        const uint64_t n = b.n[s];
        if (base + G::TILE <= n) {
            Raw<T, G::VEC> w[kNormU];
#pragma unroll
            for (int u = 0; u < kNormU; ++u) {
                const uint64_t i0 = base + (uint64_t)u * G::SUB + (uint64_t)lane * G::VEC;
                w[u] = load_group<T, G::VEC, true, true>(g, i0, G::VEC);
            }
#pragma unroll
            for (int u = 0; u < kNormU; ++u) {
                float x[G::VEC];
                widen<T, G::VEC>(w[u], x);
#pragma unroll
                for (int j = 0; j < G::VEC; ++j)
                    acc[j & 3] = __builtin_fma((double)x[j], (double)x[j], acc[j & 3]);
            }
        } else {
            for (uint64_t i = base + lane; i < n; i += kWave) {
                const double x = (double)load1<T>(g, i);
                acc[0] = __builtin_fma(x, x, acc[0]);
            }
        }
    }
    const double v = group_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
    if (threadIdx.x == 0) {
        if (last)
            *out = accumulate ? *out + v : v;
        else
            out[blockIdx.x] = v;
    }
}

// Joins the workgroups' partials: one workgroup, a fixed order.
__global__ __launch_bounds__(1024) void sumsq_join_kernel(const double* __restrict__ part,
                                                          uint64_t n, double* sumsq,
                                                          uint32_t accumulate) {
    double a = 0.0;
    for (uint64_t i = threadIdx.x; i < n; i += 4 * blockDim.x) {
        double v[4];  // four in flight; past the end the last one again, not added
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u)
            v[u] = part[min(i + u * blockDim.x, n - 1)];
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u)
            a += i + u * blockDim.x < n ? v[u] : 0.0;
    }
    a = group_sum(a);
    if (threadIdx.x == 0)
        *sumsq = accumulate ? *sumsq + a : a;
}

struct ClipBatch {
    static constexpr int kSegs = kClipSegs, kU = kClipU;
    const void* g[kSegs];
    void* out[kSegs];
    uint64_t n[kSegs];
    uint32_t tile_end[kSegs];
    uint32_t total;
    float max_norm, eps;
    const double* sumsq;
    float* norm;
};

template <int T>
__global__ __launch_bounds__(kWave) void clip_kernel(ClipBatch b) {
    using G = NormGeom<T, kClipU>;
    const double norm = __builtin_sqrt(*b.sumsq);
    if (b.norm && blockIdx.x == 0 && threadIdx.x == 0)
        *b.norm = (float)norm;
    const double q = (double)b.max_norm / (norm + (double)b.eps);
    const float c = q >= 1.0 ? 1.0f : (float)q;  // a NaN stays one
    const TileFinder<kClipSegs> find(b.tile_end);
    const int lane = lane_id();
    for (size_t ts = stream_wave_id<kWave>(); ts < b.total; ts += wave_count()) {
        const uint32_t t = (uint32_t)ts, s = find(t);
        const uint64_t base = (uint64_t)(t - (s ? b.tile_end[s - 1] : 0u)) * G::TILE;
        const void* g = b.g[s];
        void* out = b.out[s];
        const uint64_t n = b.n[s];
        if (c == 1.0f && out == g)
            continue;
        if (base + G::TILE <= n) {
            Raw<T, G::VEC> w[kClipU];
#pragma unroll
            for (int u = 0; u < kClipU; ++u) {
                const uint64_t i0 = base + (uint64_t)u * G::SUB + (uint64_t)lane * G::VEC;
                w[u] = load_group<T, G::VEC, true, true>(g, i0, G::VEC);
            }
#pragma unroll
            for (int u = 0; u < kClipU; ++u) {
                const uint64_t i0 = base + (uint64_t)u * G::SUB + (uint64_t)lane * G::VEC;
                float x[G::VEC];
                widen<T, G::VEC>(w[u], x);
#pragma unroll
                for (int j = 0; j < G::VEC; ++j)
                    x[j] = c * x[j];
                store_group<T, G::VEC, true, true>(narrow<T, G::VEC>(x), out, i0, G::VEC);
            }
        } else {
            for (uint64_t i = base + lane; i < n; i += kWave) {
                const float x = c * load1<T>(g, i);
                if constexpr (T == kF32)
                    ((float*)out)[i] = x;
                else
                    ((uint16_t*)out)[i] = (uint16_t)pack_products<T>(x, 0.0f);
            }
        }
    }
}

void set_out(NormBatch&, uint32_t, void*) {}
void set_out(ClipBatch& b, uint32_t k, void* out) { b.out[k] = out; }

// Fills a launch's table with the non-empty segments from segs[i] on and
// returns the first segment that the next launch takes.  The ABI layer holds a
// call to 2^40 elements, so the tiles of a launch (of 512 elements at least,
// and a ragged one a segment) stay below 2^32.
template <int T, typename B>
uint32_t fill(B& b, const GradSegment* segs, uint32_t i, uint32_t n_seg) {
    constexpr uint64_t kTile = NormGeom<T, B::kU>::TILE;
    uint64_t tiles = 0;
    uint32_t k = 0;
    for (; i < n_seg && k < (uint32_t)B::kSegs; ++i) {
        if (segs[i].n == 0)
            continue;
        b.g[k] = segs[i].g;
        b.n[k] = segs[i].n;
        set_out(b, k, segs[i].out);
        tiles += (segs[i].n + kTile - 1) / kTile;
        b.tile_end[k++] = (uint32_t)tiles;
    }
    for (; k < (uint32_t)B::kSegs; ++k)
        b.tile_end[k] = UINT32_MAX;
    b.total = (uint32_t)tiles;
    return i;
}

inline uint32_t norm_wgs(uint64_t tiles) {
    return (uint32_t)std::min<uint64_t>((tiles + 3) / 4, kNormMaxWgs);
}

template <int T>
hipError_t sumsq_t(const GradSegment* segs, uint32_t n_seg, uint32_t accumulate, double* sumsq,
                   double* partials, hipStream_t st) {
    uint64_t np = 0;
    for (uint32_t i = 0; i < n_seg;) {
        NormBatch b = {};
        const uint32_t first = i;
        i = fill<T>(b, segs, i, n_seg);
        // Few tiles: one workgroup sums them and writes the result, one launch
        // in place of two.
        uint32_t last = first == 0 && i == n_seg && b.total <= kNormOneWg;
        if (b.total == 0 && !last)
            continue;
        const uint32_t wgs = last ? 1 : norm_wgs(b.total);
        double* out = last ? sumsq : partials + np;
        void* args[] = {(void*)&b, (void*)&out, (void*)&last, (void*)&accumulate};
        const hipError_t e = hipLaunchKernel((const void*)&sumsq_kernel<T>, dim3(wgs),
                                             dim3(last ? 1024 : kBlockThreads), args, 0, st);
        if (e != hipSuccess || last)
            return e;
        np += wgs;
    }
    void* args[] = {(void*)&partials, (void*)&np, (void*)&sumsq, (void*)&accumulate};
    return hipLaunchKernel((const void*)&sumsq_join_kernel, dim3(1),
                           dim3(np > 256 ? 1024 : 256), args, 0, st);
}

template <int T>
hipError_t clip_t(const GradSegment* segs, uint32_t n_seg, const double* sumsq, float max_norm,
                  float eps, float* norm, hipStream_t st) {
    uint32_t i = 0;
    do {  // at least one launch: it writes the norm
        ClipBatch b = {};
        b.max_norm = max_norm;
        b.eps = eps;
        b.sumsq = sumsq;
        b.norm = i == 0 ? norm : nullptr;
        i = fill<T>(b, segs, i, n_seg);
        void* args[] = {(void*)&b};
        const hipError_t e =
            hipLaunchKernel((const void*)&clip_kernel<T>,
                            dim3(std::min(std::max(b.total, 1u), kClipMaxWgs)), dim3(kWave), args, 0,
                            st);
        if (e != hipSuccess)
            return e;
    } while (i < n_seg);
    return hipSuccess;
}

}  // namespace

// One partial for each workgroup of each launch.
size_t grad_sumsq_workspace(uint32_t n_seg) {
    const size_t launches = std::max<size_t>(1, (n_seg + (size_t)kSumSegs - 1) / kSumSegs);
    return sizeof(double) * kNormMaxWgs * launches;
}

hipError_t launch_grad_sumsq(const GradSegment* segs, uint32_t n_seg, int g_type, bool accumulate,
                             double* sumsq, double* partials, hipStream_t stream) {
    switch (g_type) {
        case kF32: return sumsq_t<kF32>(segs, n_seg, accumulate, sumsq, partials, stream);
        case kBF16: return sumsq_t<kBF16>(segs, n_seg, accumulate, sumsq, partials, stream);
        case kF16: return sumsq_t<kF16>(segs, n_seg, accumulate, sumsq, partials, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_grad_clip(const GradSegment* segs, uint32_t n_seg, int g_type,
                            const double* sumsq, float max_norm, float eps, float* norm,
                            hipStream_t stream) {
    switch (g_type) {
        case kF32: return clip_t<kF32>(segs, n_seg, sumsq, max_norm, eps, norm, stream);
        case kBF16: return clip_t<kBF16>(segs, n_seg, sumsq, max_norm, eps, norm, stream);
        case kF16: return clip_t<kF16>(segs, n_seg, sumsq, max_norm, eps, norm, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace zq
