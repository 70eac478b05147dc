// zq_embed_grad.hip -- the embedding table's gradient, summed by sorted tokens.
//   S[v, j] = sum over the tokens t with id v, ascending, of dout[t, j]
//   G = fl(scale * S);  grad = rne(G) | rne(fl(grad + G)) | SR(fl(grad + G))
//
// 1. Sort.  The tokens' positions are sorted by row with a stable counting
//    sort, least significant digit first, so a row's tokens keep ascending
//    order; ids that name no row take the key `rows` and come last.  Up to
//    kSmallTokens tokens one workgroup sorts in LDS in one launch; more are
//    split over at most kSortBlocks workgroups, two launches a digit (count,
//    scatter; every workgroup adds up the counts before it by itself).
// 2. Sum.  The sorted positions are cut into chunks of kChunk.  A wave takes a
//    chunk and 512 columns and sums the runs (equal rows) that begin in its
//    chunk, up to the end of the next chunk, in registers, and writes a run
//    that ends there to the table.  A longer run leaves fp32 partials: the
//    wave it began in one, and each later chunk that it reaches one.  In the
//    write mode the same launch clears the rows that no token names.
// 3. Join.  The partials of each long run are added in order and written.
// Every row is written by one wave per column group, and the grouping depends
// on the ids alone, so equal inputs give equal bits; integer atomics only
// count.
#include <algorithm>

#include "zq_rows.h"

namespace zq {
namespace {

constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr uint32_t kDigitBits = 9;
constexpr uint32_t kBins = 1u << kDigitBits;
constexpr uint32_t kSmallThreads = 1024;
constexpr uint32_t kSmallTokens = 8192;
constexpr uint32_t kSortThreads = 512;
constexpr uint32_t kSortItems = 4;
constexpr uint32_t kSortRound = kSortThreads * kSortItems;
constexpr uint32_t kSortBlocks = 256;
constexpr uint32_t kChunk = 32;
constexpr uint32_t kCols = kWave * 8;
constexpr uint32_t kJoinThreads = 512;
constexpr uint64_t kClearBytes = 64 << 10;

// How the caller's workspace is laid out; every part on a 256-byte boundary.
struct Layout {
    uint64_t key[2], pos[2];  // ping-pong buffers of the sort, u32 [n_tok]
    uint64_t count;           // u32 [kSortBlocks][kBins]
    uint64_t named;           // one byte per row: some token names it
    uint64_t runs;            // u32 [1 + chunks]: number of long runs, first chunks
    uint64_t part;            // fp32 [chunks + 1][pitch]: partials of the long runs
    uint64_t pitch, chunks, bytes;
};

Layout layout(uint64_t n_tok, uint64_t rows, uint64_t dim) {
    Layout l = {};
    uint64_t at = 0;
    const auto take = [&at](uint64_t bytes) {
        const uint64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    l.chunks = (n_tok + kChunk - 1) / kChunk;
    l.pitch = (dim + 7) / 8 * 8;
    const bool small = n_tok <= kSmallTokens;
    for (int i = 0; i < 2; ++i) {
        l.key[i] = small && i ? l.key[0] : take(4 * n_tok);
        l.pos[i] = small && i ? l.pos[0] : take(4 * n_tok);
    }
    l.count = small ? at : take(4ull * kSortBlocks * kBins);
    l.named = take(rows);
    l.runs = take(4 * (1 + l.chunks));
    l.part = take(n_tok > 2 * kChunk ? 4 * l.pitch * (l.chunks + 1) : 0);
    l.bytes = at;
    return l;
}

struct SortArgs {
    const void* ids;
    uint32_t id64;
    uint32_t n, rows;
    uint32_t per_block;  // tokens of a workgroup, a multiple of kSortRound
    uint32_t shift, bits;
    const uint32_t* key_in;  // nullptr: the first digit, keys come from ids
    const uint32_t* pos_in;
    uint32_t* key_out;
    uint32_t* pos_out;
    uint32_t* count;
    uint8_t* named;  // nullptr: not wanted
    uint32_t* runs;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i) {
    if (a.key_in)
        return a.key_in[i];
    const uint64_t id = token_id(a.ids, a.id64, i);
    return id < a.rows ? (uint32_t)id : a.rows;
}

// Lanes of the wave whose digit equals this lane's.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint32_t bits) {
    uint64_t m = ~0ull;
    for (uint32_t b = 0; b < bits; ++b) {
        const bool one = (d >> b) & 1;
        const uint64_t v = __builtin_amdgcn_ballot_w64(one);
        m &= one ? v : ~v;
    }
    return m;
}

// Rank of this lane's item among the wave's items of the same digit so far,
// counted in the wave's own row of LDS counters.  The wave's LDS accesses are
// performed in order; the fences keep the compiler from reordering them.
__device__ __forceinline__ uint32_t wave_rank(uint16_t* mine, uint32_t d, uint32_t bits) {
    const uint64_t m = same_digit(d, bits);
    const uint32_t below = (uint32_t)__builtin_popcountll(m & ((1ull << lane_id()) - 1));
    const uint32_t base = mine[d];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (below == 0)
        mine[d] = (uint16_t)(base + (uint32_t)__builtin_popcountll(m));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return base + below;
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    const int lane = lane_id();
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint32_t o = __shfl_up(v, d);
        if (lane >= d)
            v += o;
    }
    return v;
}

// Exclusive sum over the first kBins threads' values (a multiple of 64 of
// them); called by the whole workgroup.
__device__ __forceinline__ uint32_t bins_scan(uint32_t v, uint32_t* tmp) {
    const uint32_t t = threadIdx.x;
    const uint32_t inc = wave_scan(t < kBins ? v : 0);
    if (t < kBins && lane_id() == kWave - 1)
        tmp[t >> 6] = inc;
    __syncthreads();
    uint32_t before = 0;
    for (uint32_t w = 0; w < kBins / kWave; ++w)
        if (w < (t >> 6))
            before += tmp[w];
    __syncthreads();
    return before + inc - v;
}

// One workgroup sorts up to kSmallTokens tokens: kItems a thread, in LDS.
template <int kItems>
__global__ __launch_bounds__(kSmallThreads) void sort_small_kernel(SortArgs a, uint32_t passes) {
    constexpr uint32_t kWaves = kSmallThreads / kWave;
    __shared__ uint16_t cnt[kWaves][kBins];
    __shared__ uint32_t tmp[kBins / kWave];
    __shared__ uint32_t key_s[kItems * kSmallThreads];
    __shared__ uint16_t pos_s[kItems * kSmallThreads];
    const uint32_t t = threadIdx.x, wave = t / kWave, lane = t % kWave;
    const uint32_t first = wave * kWave * kItems + lane;
    uint32_t key[kItems], pos[kItems], rank[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        pos[i] = first + i * kWave;
        key[i] = pos[i] < a.n ? sort_key(a, pos[i]) : kNone;  // past the end: sorts last
    }
    if (a.named)
        for (uint32_t r = t; r < a.rows; r += kSmallThreads)
            a.named[r] = 0;
    if (t == 0)
        a.runs[0] = 0;
    const uint32_t mask = (1u << a.bits) - 1;
    for (uint32_t p = 0; p < passes; ++p) {
        const uint32_t shift = p * a.bits;
        for (uint32_t i = t; i < kWaves * kBins; i += kSmallThreads)
            (&cnt[0][0])[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            rank[i] = wave_rank(cnt[wave], (key[i] >> shift) & mask, a.bits);
        __syncthreads();
        uint32_t sum = 0;
        if (t < kBins)
            for (uint32_t w = 0; w < kWaves; ++w)
                sum += cnt[w][t];
        uint32_t at = bins_scan(sum, tmp);
        if (t < kBins)
            for (uint32_t w = 0; w < kWaves; ++w) {
                const uint32_t c = cnt[w][t];
                cnt[w][t] = (uint16_t)at;
                at += c;
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const uint32_t to = cnt[wave][(key[i] >> shift) & mask] + rank[i];
            key_s[to] = key[i];
            pos_s[to] = (uint16_t)pos[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            key[i] = key_s[first + i * kWave];
            pos[i] = pos_s[first + i * kWave];
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t o = first + i * kWave;
        if (o < a.n) {
            a.key_out[o] = key[i];
            a.pos_out[o] = pos[i];
            if (a.named && key[i] < a.rows)
                a.named[key[i]] = 1;  // after the clearing: barriers lie between
        }
    }
}

// Counts one digit of a workgroup's tokens.  The first digit's launch also
// clears the row flags and the number of long runs.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
    __shared__ uint32_t cnt[kBins];
    const uint32_t t = threadIdx.x;
    for (uint32_t i = t; i < kBins; i += kSortThreads)
        cnt[i] = 0;
    if (!a.key_in) {
        if (a.named)
            for (uint64_t r = (uint64_t)blockIdx.x * kSortThreads + t; r < a.rows;
                 r += (uint64_t)gridDim.x * kSortThreads)
                a.named[r] = 0;
        if (blockIdx.x == 0 && t == 0)
            a.runs[0] = 0;
    }
    __syncthreads();
    const uint64_t lo = (uint64_t)blockIdx.x * a.per_block;
    const uint64_t hi = min(lo + a.per_block, (uint64_t)a.n);
    const uint32_t mask = (1u << a.bits) - 1;
    for (uint64_t i = lo + t; i < hi; i += kSortThreads)
        atomicAdd(&cnt[(sort_key(a, (uint32_t)i) >> a.shift) & mask], 1u);
    __syncthreads();
    for (uint32_t i = t; i < kBins; i += kSortThreads)
        a.count[blockIdx.x * kBins + i] = cnt[i];
}

__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(SortArgs a) {
    static_assert(kSortThreads == kBins, "a thread per digit value");
    constexpr uint32_t kWaves = kSortThreads / kWave;
    __shared__ uint16_t cnt[kWaves][kBins];
    __shared__ uint32_t base[kBins];
    __shared__ uint32_t tmp[kBins / kWave];
    const uint32_t t = threadIdx.x, wave = t / kWave, lane = t % kWave;
    // Where this workgroup's first token of digit value t goes: all tokens of
    // smaller digits, then those of this digit in earlier workgroups.
    uint32_t total = 0, earlier = 0;
    for (uint32_t b = 0; b < gridDim.x; ++b) {
        const uint32_t c = a.count[b * kBins + t];
        total += c;
        earlier += b < blockIdx.x ? c : 0;
    }
    base[t] = bins_scan(total, tmp) + earlier;
    const uint64_t lo = (uint64_t)blockIdx.x * a.per_block;
    const uint64_t hi = min(lo + a.per_block, (uint64_t)a.n);
    const uint32_t mask = (1u << a.bits) - 1;
    for (uint64_t r = lo; r < hi; r += kSortRound) {
        for (uint32_t i = t; i < kWaves * kBins; i += kSortThreads)
            (&cnt[0][0])[i] = 0;
        __syncthreads();
        uint32_t key[kSortItems], pos[kSortItems], rank[kSortItems];
#pragma unroll
        for (uint32_t i = 0; i < kSortItems; ++i) {
            const uint64_t at = r + wave * kWave * kSortItems + i * kWave + lane;
            key[i] = at < hi ? sort_key(a, (uint32_t)at) : kNone;
            pos[i] = at < hi ? (a.pos_in ? a.pos_in[at] : (uint32_t)at) : 0;
            // Past the end: ranked last, and not written.
            rank[i] = wave_rank(cnt[wave], (key[i] >> a.shift) & mask, a.bits);
        }
        __syncthreads();
        uint32_t sum = 0;
        for (uint32_t w = 0; w < kWaves; ++w) {
            const uint32_t c = cnt[w][t];
            cnt[w][t] = (uint16_t)sum;
            sum += c;
        }
        __syncthreads();
#pragma unroll
        for (uint32_t i = 0; i < kSortItems; ++i) {
            const uint64_t at = r + wave * kWave * kSortItems + i * kWave + lane;
            if (at >= hi)
                continue;
            const uint32_t d = (key[i] >> a.shift) & mask;
            const uint32_t to = base[d] + cnt[wave][d] + rank[i];
            a.key_out[to] = key[i];
            a.pos_out[to] = pos[i];
            if (a.named && key[i] < a.rows)
                a.named[key[i]] = 1;
        }
        __syncthreads();
        base[t] += sum;  // the pads counted in it belong to the last round only
    }
}

struct SumArgs {
    const uint32_t* key;
    const uint32_t* pos;
    const uint8_t* named;
    uint32_t* runs;
    float* part;
    uint64_t pitch;
    uint32_t n, chunks, rows;
    uint32_t col_tiles;
    uint64_t dim;
    const void* dout;
    void* grad;
    float scale;
    uint64_t seed, cbase;
    uint32_t sum_wgs;    // the workgroups after these clear rows
    uint32_t clear_rows; // rows a workgroup clears at a time
};

// The eight 16-bit random numbers of indices q .. q + 7 (the layout of
// zq_sr_accumulate: eight from each Philox call).  q mod 8 is the same on
// every lane of a wave.
__device__ __forceinline__ void random8(uint64_t q, uint64_t seed, uint32_t r[8]) {
    const uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    const uint64_t c = q >> 3;
    const uint32_t phase = __builtin_amdgcn_readfirstlane((uint32_t)(q & 7));
    const Philox4 a = philox4x32_10((uint32_t)c, (uint32_t)(c >> 32), 0u, 0u, k0, k1);
    uint32_t w[8] = {a.w[0], a.w[1], a.w[2], a.w[3], 0, 0, 0, 0};
    if (phase) {
        const uint64_t c1 = c + 1;
        const Philox4 b = philox4x32_10((uint32_t)c1, (uint32_t)(c1 >> 32), 0u, 0u, k0, k1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[4 + i] = b.w[i];
        if (phase & 4) {
#pragma unroll
            for (int i = 0; i < 6; ++i)
                w[i] = w[i + 2];
        }
        if (phase & 2) {
#pragma unroll
            for (int i = 0; i < 5; ++i)
                w[i] = w[i + 1];
        }
        if (phase & 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (w[i] >> 16) | (w[i + 1] << 16);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        r[j] = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu;
}

// Writes a row's eight sums at element e = row * dim + col, of which `left`
// exist; `old` are the buffer's values there (add modes).
template <int OUT, int MODE, bool WHOLE>
__device__ __forceinline__ void finish(const SumArgs& a, const float s[8], const Raw8<OUT>& old,
                                       uint64_t e, uint32_t left) {
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        g[j] = a.scale * s[j];
    if constexpr (MODE != kGradWrite) {
        float o[8];
        widen8<OUT>(old, o);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            g[j] = o[j] + g[j];
    }
    if constexpr (MODE == kGradAddSr) {
        uint32_t r[8];
        random8(a.cbase + e, a.seed, r);
        Raw8<OUT> w;
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[j] = sr_bf16(g[2 * j], r[2 * j]) | (sr_bf16(g[2 * j + 1], r[2 * j + 1]) << 16);
        w.w[0] = u4{h[0], h[1], h[2], h[3]};
        store8<OUT, WHOLE>(w, a.grad, e, left);
    } else {
        store8<OUT, WHOLE>(narrow8<OUT>(g), a.grad, e, left);
    }
}

constexpr int kSumU = 4;  // tokens a wave has in flight

// Sums positions [p, e) of the wave's window, one run after the other, each
// run's sum going to `done(last position, sums)`.  ends has a bit at each
// run's last position.
template <int IN, int OUT, int MODE, bool WHOLE>
struct Walker {
    const SumArgs& a;
    uint32_t key, pos;  // lane l: the window's l-th sorted token
    uint32_t col, left;
    bool on;            // the lane has columns

    __device__ __forceinline__ uint32_t key_at(uint32_t p) const {
        return __builtin_amdgcn_readlane(key, p);
    }

    __device__ __forceinline__ void run(uint32_t p, uint32_t e, uint64_t ends, float* long_part,
                                        uint32_t long_end) const {
        float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        while (p < e) {
            Raw8<IN> x[kSumU];
            Raw8<OUT> old[kSumU];
#pragma unroll
            for (int u = 0; u < kSumU; ++u) {
                if (p + u >= e)
                    continue;
                const uint64_t t = __builtin_amdgcn_readlane(pos, p + u);
                if (on)
                    x[u] = load8<IN, WHOLE>(a.dout, t * a.dim + col, left);
                if constexpr (MODE != kGradWrite)
                    if (on && ((ends >> (p + u)) & 1) && p + u != long_end)
                        old[u] = load8<OUT, WHOLE>(a.grad, (uint64_t)key_at(p + u) * a.dim + col,
                                                   left);
            }
#pragma unroll
            for (int u = 0; u < kSumU; ++u) {
                if (p + u >= e)
                    continue;
                float v[8];
                widen8<IN>(x[u], v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[j] += v[j];
                if ((ends >> (p + u)) & 1) {
                    if (on) {
                        if (p + u == long_end) {
                            *(f4*)(long_part + col) = f4{s[0], s[1], s[2], s[3]};
                            *(f4*)(long_part + col + 4) = f4{s[4], s[5], s[6], s[7]};
                        } else {
                            finish<OUT, MODE, WHOLE>(
                                a, s, old[u], (uint64_t)key_at(p + u) * a.dim + col, left);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        s[j] = 0.0f;
                }
            }
            p += kSumU;
        }
    }
};

template <int IN, int OUT, int MODE, bool WHOLE>
__device__ __forceinline__ void sum_chunk(const SumArgs& a, uint32_t k, uint32_t tile) {
    static_assert(2 * kChunk == kWave, "a chunk and its successor fill the lanes");
    const uint32_t lane = (uint32_t)lane_id();
    const uint32_t i0 = k * kChunk;
    const uint32_t i = i0 + lane;
    Walker<IN, OUT, MODE, WHOLE> w = {a, kNone, 0, tile * kCols + lane * 8, 0, false};
    w.on = w.col < a.dim;
    w.left = w.on ? (uint32_t)a.dim - w.col : 0;
    if (i < a.n) {
        w.key = a.key[i];
        w.pos = a.pos[i];
    }
    const uint32_t first = w.key_at(0);
    if (first >= a.rows)
        return;  // ids that name no row, to the end
    const bool cont = k > 0 && a.key[i0 - 1] == first;
    // Bit p: a run starts at position p (the first kNone is one too).
    uint32_t prev = __shfl_up(w.key, 1);
    const uint64_t starts =
        __builtin_amdgcn_ballot_w64(lane == 0 ? !cont : w.key != prev);
    const uint64_t ends = starts >> 1;
    const uint32_t own = (uint32_t)(starts & ((1ull << kChunk) - 1));
    uint32_t p = own ? (uint32_t)__builtin_ctz(own) : kChunk;
    if (cont && k > 1 && a.key[i0 - kChunk - 1] == first) {
        // The run began before the previous chunk: this chunk's part of it.
        const uint32_t here = min(p, a.n - i0);
        w.run(0, here, 1ull << (here - 1), a.part + (uint64_t)k * a.pitch, here - 1);
    }
    if (!own)
        return;
    // The runs that start here; the last one may reach into the next chunk.
    const uint64_t later = starts >> kChunk;
    uint32_t e = later ? kChunk + (uint32_t)__builtin_ctzll(later) : kWave;
    uint32_t long_end = kNone;
    if (e == kWave && i0 + kWave < a.n && a.key[i0 + kWave] == w.key_at(kWave - 1) &&
        w.key_at(kWave - 1) < a.rows) {
        long_end = kWave - 1;
        if (tile == 0 && lane == 0)
            a.runs[1 + atomicAdd(&a.runs[0], 1u)] = k;
    }
    // Ids that name no row, and positions past the end, are not summed.
    const uint64_t bad = __builtin_amdgcn_ballot_w64(w.key >= a.rows);
    if (bad)
        e = min(e, (uint32_t)__builtin_ctzll(bad));
    w.run(p, e, ends | (1ull << (kWave - 1)), a.part + (uint64_t)(k + 1) * a.pitch, long_end);
}

template <int OUT, bool WHOLE>
__device__ __forceinline__ void clear_rows(const SumArgs& a, uint32_t job) {
    const uint64_t r0 = (uint64_t)job * a.clear_rows;
    const uint32_t nr = (uint32_t)min((uint64_t)a.clear_rows, a.rows - r0);
    const Raw8<OUT> zero = {};
    const uint32_t per_row = (uint32_t)((a.dim + 7) / 8);
    for (uint32_t r = 0; r < nr; ++r) {
        if (a.named[r0 + r])
            continue;
        for (uint32_t g = threadIdx.x; g < per_row; g += kBlockThreads)
            store8<OUT, WHOLE>(zero, a.grad, (r0 + r) * a.dim + (uint64_t)g * 8,
                               (uint32_t)a.dim - g * 8);
    }
}

template <int IN, int OUT, int MODE, bool WHOLE>
__global__ __launch_bounds__(kBlockThreads) void sum_kernel(SumArgs a) {
    if (MODE != kGradWrite || blockIdx.x < a.sum_wgs) {
        const uint64_t jobs = (uint64_t)a.chunks * a.col_tiles;
        const uint64_t waves = (uint64_t)a.sum_wgs * (kBlockThreads / kWave);
        for (uint64_t j = wave_id(); j < jobs; j += waves) {
            const uint32_t k = (uint32_t)(j / a.col_tiles);
            sum_chunk<IN, OUT, MODE, WHOLE>(a, k, (uint32_t)(j - (uint64_t)k * a.col_tiles));
        }
    } else {
        const uint32_t jobs = (uint32_t)(((uint64_t)a.rows + a.clear_rows - 1) / a.clear_rows);
        for (uint32_t j = blockIdx.x - a.sum_wgs; j < jobs; j += gridDim.x - a.sum_wgs)
            clear_rows<OUT, WHOLE>(a, j);
    }
}

// Adds the partials of each long run in order.  The run that began in chunk k
// has them in slots k + 1 (chunks k and k + 1), k + 2, ..., as far as chunks
// begin with its row.  Each wave of the workgroup adds a stretch of the slots,
// then the stretches are added in order.
template <int OUT, int MODE, bool WHOLE>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(SumArgs a) {
    constexpr uint32_t kWaves = kJoinThreads / kWave;
    __shared__ float part[kWaves][kCols];
    const uint32_t wave = threadIdx.x / kWave, lane = (uint32_t)lane_id();
    const uint64_t jobs = (uint64_t)a.runs[0] * a.col_tiles;
    for (uint64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
        const uint32_t k = a.runs[1 + j / a.col_tiles];
        const uint32_t tile = (uint32_t)(j % a.col_tiles);
        const uint32_t row = a.key[(k + 2) * kChunk];
        // The chunks from k + 2 on that begin with the row: the first one
        // does, and the keys are sorted, so 64 probes narrow the end down.
        uint32_t lo = k + 2, hi = a.chunks;  // lo begins with the row; hi does not, or is the end
        while (hi - lo > 1) {
            const uint32_t step = (hi - lo + kWave - 1) / kWave;
            const uint64_t at = (uint64_t)lo + (uint64_t)lane * step;
            const bool yes = at < hi && a.key[at * kChunk] == row;
            const uint32_t c = (uint32_t)__builtin_popcountll(__builtin_amdgcn_ballot_w64(yes));
            hi = (uint32_t)min((uint64_t)hi, (uint64_t)lo + (uint64_t)c * step);
            lo += (c - 1) * step;
        }
        const uint32_t slots = hi - (k + 1);
        const uint32_t s0 = k + 1 + (uint32_t)((uint64_t)slots * wave / kWaves);
        const uint32_t s1 = k + 1 + (uint32_t)((uint64_t)slots * (wave + 1) / kWaves);
        const uint32_t col = tile * kCols + lane * 8;
        const bool on = col < a.dim;
        float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (on) {
#pragma unroll 4
            for (uint32_t i = s0; i < s1; ++i) {
                const f4* q = (const f4*)(a.part + (uint64_t)i * a.pitch + col);
                const f4 x = q[0], y = q[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[e] += x[e];
                    s[4 + e] += y[e];
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            part[wave][e * kWave + lane] = s[e];
        __syncthreads();
        if (wave == 0 && on) {
            for (uint32_t w = 1; w < kWaves; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[e] += part[w][e * kWave + lane];
            const uint64_t at = (uint64_t)row * a.dim + col;
            const uint32_t left = (uint32_t)a.dim - col;
            Raw8<OUT> old = {};
            if constexpr (MODE != kGradWrite)
                old = load8<OUT, WHOLE>(a.grad, at, left);
            finish<OUT, MODE, WHOLE>(a, s, old, at, left);
        }
        __syncthreads();
    }
}

// ZQ_GRAD_WRITE without tokens.
__global__ __launch_bounds__(kBlockThreads) void clear_kernel(char* p, uint64_t bytes) {
    const uint64_t n16 = bytes / 16, step = (uint64_t)gridDim.x * kBlockThreads;
    for (uint64_t i = (uint64_t)blockIdx.x * kBlockThreads + threadIdx.x; i < n16; i += step)
        st_stream(u4{0, 0, 0, 0}, (u4*)p + i);
    const uint64_t at = n16 * 16 + 2 * threadIdx.x;
    if (blockIdx.x == 0 && at < bytes)
        *(uint16_t*)(p + at) = 0;
}

hipError_t launch(const void* fn, uint64_t wgs, uint32_t threads, void** args, hipStream_t st) {
    return hipLaunchKernel(fn, dim3((uint32_t)wgs), dim3(threads), args, 0, st);
}

hipError_t sort_small(SortArgs& s, uint32_t passes, hipStream_t st) {
    const void* fn = s.n <= 1024   ? (const void*)&sort_small_kernel<1>
                     : s.n <= 2048 ? (const void*)&sort_small_kernel<2>
                     : s.n <= 4096 ? (const void*)&sort_small_kernel<4>
                                   : (const void*)&sort_small_kernel<8>;
    void* args[] = {(void*)&s, (void*)&passes};
    return launch(fn, 1, kSmallThreads, args, st);
}

// Sorts the tokens; *key, *pos get the buffers that hold them in order.
hipError_t sort(const EmbedGradArgs& a, const Layout& l, bool want_named, const uint32_t** key,
                const uint32_t** pos, hipStream_t st) {
    char* ws = (char*)a.workspace;
    SortArgs s = {};
    s.ids = a.ids;
    s.id64 = a.id64;
    s.n = (uint32_t)a.n_tok;
    s.rows = (uint32_t)a.rows;
    s.count = (uint32_t*)(ws + l.count);
    s.named = want_named ? (uint8_t*)(ws + l.named) : nullptr;
    s.runs = (uint32_t*)(ws + l.runs);
    // Keys run from 0 to rows: as many digits as their bits need, of equal width.
    uint32_t bits = 1;
    while ((s.rows >> bits) != 0)
        ++bits;
    const uint32_t passes = (bits + kDigitBits - 1) / kDigitBits;
    s.bits = (bits + passes - 1) / passes;
    if (a.n_tok <= kSmallTokens) {
        s.key_out = (uint32_t*)(ws + l.key[0]);
        s.pos_out = (uint32_t*)(ws + l.pos[0]);
        *key = s.key_out;
        *pos = s.pos_out;
        return sort_small(s, passes, st);
    }
    const uint32_t rounds = (s.n + kSortRound - 1) / kSortRound;
    s.per_block = (rounds + kSortBlocks - 1) / kSortBlocks * kSortRound;
    const uint32_t wgs = (s.n + s.per_block - 1) / s.per_block;
    uint8_t* named = s.named;
    for (uint32_t p = 0; p < passes; ++p) {
        s.shift = p * s.bits;
        s.key_out = (uint32_t*)(ws + l.key[p & 1]);
        s.pos_out = (uint32_t*)(ws + l.pos[p & 1]);
        void* args[] = {(void*)&s};
        hipError_t e = launch((const void*)&sort_count_kernel, wgs, kSortThreads, args, st);
        if (e != hipSuccess)
            return e;
        s.named = p + 1 == passes ? named : nullptr;
        e = launch((const void*)&sort_scatter_kernel, wgs, kSortThreads, args, st);
        if (e != hipSuccess)
            return e;
        s.key_in = s.key_out;
        s.pos_in = s.pos_out;
    }
    *key = s.key_out;
    *pos = s.pos_out;
    return hipSuccess;
}

template <int IN, int OUT, int MODE, bool WHOLE>
hipError_t grad_t(const EmbedGradArgs& a, hipStream_t st) {
    const Layout l = layout(a.n_tok, a.rows, a.dim);
    char* ws = (char*)a.workspace;
    SumArgs s = {};
    hipError_t e = sort(a, l, MODE == kGradWrite, &s.key, &s.pos, st);
    if (e != hipSuccess)
        return e;
    s.named = (const uint8_t*)(ws + l.named);
    s.runs = (uint32_t*)(ws + l.runs);
    s.part = (float*)(ws + l.part);
    s.pitch = l.pitch;
    s.n = (uint32_t)a.n_tok;
    s.chunks = (uint32_t)l.chunks;
    s.rows = (uint32_t)a.rows;
    s.dim = a.dim;
    s.col_tiles = (uint32_t)((a.dim + kCols - 1) / kCols);
    s.dout = a.dout;
    s.grad = a.grad;
    s.scale = a.scale;
    s.seed = a.seed;
    s.cbase = a.cbase;
    constexpr uint64_t kMaxWgs = 1 << 20;
    const uint64_t jobs = (uint64_t)s.chunks * s.col_tiles;
    s.sum_wgs = (uint32_t)std::min(kMaxWgs, (jobs + 3) / 4);
    uint64_t clear = 0;
    if (MODE == kGradWrite) {
        const uint64_t row_bytes = a.dim * (OUT == kF32 ? 4 : 2);
        s.clear_rows = (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(64, kClearBytes / row_bytes));
        clear = std::min(kMaxWgs, (a.rows + s.clear_rows - 1) / s.clear_rows);
    }
    void* args[] = {(void*)&s};
    e = launch((const void*)&sum_kernel<IN, OUT, MODE, WHOLE>, s.sum_wgs + clear, kBlockThreads, args,
               st);
    if (e != hipSuccess || a.n_tok <= 2 * kChunk)
        return e;  // no run is longer than a chunk and its successor
    return launch((const void*)&join_kernel<OUT, MODE, WHOLE>, std::min<uint64_t>(512, jobs),
                  kJoinThreads, args, st);
}

template <int IN, int OUT, int MODE>
hipError_t grad_m(const EmbedGradArgs& a, hipStream_t st) {
    return a.dim % 8 == 0 ? grad_t<IN, OUT, MODE, true>(a, st) : grad_t<IN, OUT, MODE, false>(a, st);
}

template <int IN, int OUT>
hipError_t grad_io(const EmbedGradArgs& a, int mode, hipStream_t st) {
    if (mode == kGradWrite)
        return grad_m<IN, OUT, kGradWrite>(a, st);
    if (mode == kGradAdd)
        return grad_m<IN, OUT, kGradAdd>(a, st);
    if constexpr (OUT == kBF16)
        if (mode == kGradAddSr)
            return grad_m<IN, OUT, kGradAddSr>(a, st);
    return hipErrorInvalidValue;
}

template <int IN>
hipError_t grad_in(const EmbedGradArgs& a, int grad_type, int mode, hipStream_t st) {
    switch (grad_type) {
        case kF32: return grad_io<IN, kF32>(a, mode, st);
        case kBF16: return grad_io<IN, kBF16>(a, mode, st);
        case kF16: return grad_io<IN, kF16>(a, mode, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

size_t embed_grad_workspace(uint64_t n_tok, uint64_t rows, uint64_t dim) {
    return layout(n_tok, rows, dim).bytes;
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, int d_type, int grad_type, int mode,
                             hipStream_t stream) {
    if (a.n_tok == 0) {
        char* p = (char*)a.grad;
        uint64_t bytes = a.rows * a.dim * (grad_type == kF32 ? 4 : 2);
        void* args[] = {(void*)&p, (void*)&bytes};
        return launch((const void*)&clear_kernel, std::min<uint64_t>(8192, bytes / 4096 + 1),
                      kBlockThreads, args, stream);
    }
    switch (d_type) {
        case kF32: return grad_in<kF32>(a, grad_type, mode, stream);
        case kBF16: return grad_in<kBF16>(a, grad_type, mode, stream);
        case kF16: return grad_in<kF16>(a, grad_type, mode, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace zq
