// zq_embed_grad.hip -- the embedding table's gradient, summed by sorted tokens.
//   S[v, j] = sum over the tokens t with id v, ascending, of dout[t, j]
//   G = fl(scale * S);  grad = rne(G) | rne(fl(grad + G)) | SR(fl(grad + G))
//
// 1. Sort.  The tokens' positions are ordered by row, ascending within a row;
//    ids that name no row take the key `rows` and come last.  One launch up to
//    kRangeTokens tokens, two a digit beyond (below, at the kernels).
// 2. Sum.  The sorted positions are cut into chunks.  A wave takes a chunk and
//    512 columns and sums the runs (equal rows) that begin in its chunk, up to
//    the end of the next chunk, in registers, and writes a run that ends there
//    to the table.  A longer run leaves fp32 partials: the wave it began in
//    one, and each later chunk that it reaches one.
// 3. Join.  The partials of each long run are added in order and written.
// In the write mode the sort notes which rows the tokens name, and workgroups of
// the sum's launch clear the others while the sums wait for their loads.
// Every row is written by one wave per column group, and the grouping depends
// on the ids and sizes alone, so equal inputs give equal bits; integer atomics
// only count.
//
// Bound by memory where there is much of it: 32768 bf16 tokens x 4096 added into
// fp32 move 557 MB in the sum's 120 us (4.7 TB/s, a copy's rate); counters show no
// byte twice but the partials'.  Around it the sort takes 15 us and the join 9;
// with 8192 tokens x 768 the three launches take 6 + 12 + 5 us.  The sum there is
// 2048 waves, half of which have only 32 lanes with columns.
// A row that most tokens name is slow: one workgroup sorts its tokens and one per
// 512 columns joins its partials (32768 bf16 tokens x 768 added into fp32 take
// 113 us when all name one row, 47 with text's ids).
#include <algorithm>

#include "zq_rows.h"

namespace zq {
namespace {

constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr uint32_t kCols = kWave * 8;

// Sort by ranges: its workgroups, one for every kRangeBins rows at least, each
// read all the tokens.  A whole gradient call (bf16 added into 16 fp32 columns,
// ids drawn evenly) took, by ranges / by digits: 32768 tokens 31.8 / 37.7 us with 2^17 rows, 40.9 / 37.7 with 2^18; 8192
// tokens 29.1 / 36.9 with 2^19, 45.4 / 37.4 with 2^20; 2048 tokens 25.0 / 31.2
// with 2^20; and 65536 bf16 tokens written into fp32 [32000, 1024] 87.5 / 79.0.
constexpr uint64_t kRangeTokens = 1 << 15;
constexpr uint64_t kRangeRows = 1 << 20;
constexpr uint64_t kRangeWork = 1ull << 32;  // tokens times rows
constexpr uint32_t kRangeBins = 512;  // most rows a workgroup takes
constexpr uint32_t kRangeWgs = 64;    // where the rows ask for no more; 32 to 256 are alike
constexpr uint32_t kRangeThreads = 1024;

// Sort by digits.
constexpr uint32_t kDigitBits = 9;
constexpr uint32_t kBins = 1u << kDigitBits;
constexpr uint32_t kSortThreads = 512;
constexpr uint32_t kSortItems = 4;
constexpr uint32_t kSortRound = kSortThreads * kSortItems;
constexpr uint32_t kSortBlocks = 256;

constexpr uint32_t kJoinThreads = 512;  // 256 and 1024 took 0 to 2 us more a call
// A workgroup clears rows of about this size together, with nontemporal stores:
// 16384 tokens into fp32 [32000, 2048] took 70.2 / 71.7 / 73.1 us with 8 / 16 /
// 32 KB, and 80.4 with plain stores.
constexpr uint64_t kClearBytes = 8 << 10;
constexpr uint64_t kMaxWgs = 1 << 20;

// Threads of a sum workgroup, whose waves work apart.  Adding, 128 beat 256 by up
// to 1.5 % and 512 by 3 to 6 %; writing, where most workgroups clear rows, 256
// beat 64 / 128 / 512 by 5 / 3 / 5 %.
template <int MODE>
constexpr uint32_t sum_threads() {
    return MODE == kGradWrite ? 256 : 128;
}

// Tokens of a chunk: 32, or as many less (16, 8) as it takes for kWantWaves waves.
// Short chunks give more waves, each with a shorter chain of loads and stores;
// long ones leave fewer partials of long runs.  With 4096 / 8192 / 16384 waves
// wanted, 16384 tokens written into fp32 [32000, 2048] took 67.5 / 70.4 / 70.4
// us, 32768 added into [32000, 4096] 144.4 / 144.4 / 148.8, 200000 added into
// [32000, 1024] 176 / 176 / 196 (bf16 tokens in all three).
constexpr uint64_t kWantWaves = 4096;
uint32_t chunk_tokens(uint64_t n_tok, uint64_t col_tiles) {
    for (uint32_t c = 32; c > 8; c /= 2)
        if ((n_tok + c - 1) / c * col_tiles >= kWantWaves)
            return c;
    return 8;
}

bool sorts_by_range(uint64_t n_tok, uint64_t rows) {
    return n_tok <= kRangeTokens && rows <= kRangeRows && n_tok * rows <= kRangeWork;
}

// How the caller's workspace is laid out; every part on a 256-byte boundary.
struct Layout {
    uint64_t key[2], pos[2];  // u32 [n_tok] each; the second pair for the sort by digits
    uint64_t count;           // u32 [kSortBlocks][kBins], for the sort by digits
    uint64_t named;           // one byte per row: some token names it
    uint64_t runs;            // u32 [1 + chunks]: number of long runs, their first chunks
    uint64_t part;            // fp32 [chunks + 1][pitch]: partials of the long runs
    uint64_t pitch, col_tiles, chunk, chunks, bytes;
};

uint64_t part_floats(uint64_t n_tok, uint64_t chunk, uint64_t pitch) {
    return n_tok > 2 * chunk ? ((n_tok + chunk - 1) / chunk + 1) * pitch : 0;
}

Layout layout(uint64_t n_tok, uint64_t rows, uint64_t dim) {
    Layout l = {};
    uint64_t at = 0;
    const auto take = [&at](uint64_t bytes) {
        const uint64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    l.col_tiles = (dim + kCols - 1) / kCols;
    l.chunk = chunk_tokens(n_tok, l.col_tiles);
    l.chunks = (n_tok + l.chunk - 1) / l.chunk;
    l.pitch = (dim + 7) / 8 * 8;
    l.key[0] = take(4 * n_tok);
    l.pos[0] = take(4 * n_tok);
    l.named = take(rows);
    l.runs = take(4 * (2 + n_tok / 8));
    const bool digits = !sorts_by_range(n_tok, rows);
    l.key[1] = digits ? take(4 * n_tok) : 0;
    l.pos[1] = digits ? take(4 * n_tok) : 0;
    l.count = digits ? take(4ull * kSortBlocks * kBins) : 0;
    // A workspace made for some number of tokens serves every smaller number:
    // the most tokens that still take a shorter chunk may need more partials.
    uint64_t part = part_floats(n_tok, l.chunk, l.pitch);
    for (uint64_t c = 8; c < l.chunk; c *= 2)
        part = std::max(part, part_floats((kWantWaves - 1) / l.col_tiles * 2 * c, c, l.pitch));
    l.part = take(4 * part);
    l.bytes = at;
    return l;
}

struct SortArgs {
    const void* ids;
    uint32_t id64;
    uint32_t n, rows;
    uint32_t per_wg;     // rows (range sort) or tokens (digits: a multiple of kSortRound)
    uint32_t shift, bits;
    const uint32_t* key_in;  // nullptr: the first digit, keys come from ids
    const uint32_t* pos_in;
    uint32_t* key_out;
    uint32_t* pos_out;
    uint32_t* count;
    uint8_t* named;          // nullptr: not wanted
    uint32_t* runs;
};

// Keys of positions at(0) .. at(K - 1): the row, or `rows` for an id of none.
template <int K, typename F>
__device__ __forceinline__ void sort_keys(const SortArgs& a, F at, uint32_t* key) {
    if (a.key_in) {
#pragma unroll
        for (int u = 0; u < K; ++u)
            key[u] = a.key_in[at(u)];
        return;
    }
    uint64_t id[K];
    load_ids<K>(a.ids, a.id64, at, id);
#pragma unroll
    for (int u = 0; u < K; ++u)
        key[u] = id[u] < a.rows ? (uint32_t)id[u] : a.rows;
}

// Lanes of the wave, of those in `among`, whose digit equals this lane's.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint32_t bits, uint64_t among) {
    for (uint32_t b = 0; b < bits; ++b) {
        const bool one = (d >> b) & 1;
        const uint64_t v = __builtin_amdgcn_ballot_w64(one);
        among &= one ? v : ~v;
    }
    return among;
}

// Where this lane's item goes among the items of the same digit: the wave's
// own LDS counter, plus the lanes before it in `same`; the counter moves on.
// The wave's LDS accesses are performed in order; the fences keep the compiler
// from reordering them.
template <typename C>
__device__ __forceinline__ uint32_t next_place(C* counter, uint64_t same, bool on) {
    const uint32_t below = (uint32_t)__builtin_popcountll(same & ((1ull << lane_id()) - 1));
    const uint32_t base = on ? *counter : 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (on && below == 0)
        *counter = (C)(base + (uint32_t)__builtin_popcountll(same));
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

// Exclusive sum over the values of the workgroup's first kBins threads;
// called by the whole workgroup.
__device__ __forceinline__ uint32_t bins_scan(uint32_t v, uint32_t* tmp) {
    const uint32_t t = threadIdx.x;
    const uint32_t inc = wave_scan(t < kBins ? v : 0);
    if (t < kBins && lane_id() == kWave - 1)
        tmp[t >> 6] = inc;
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (uint32_t w = 0; w < kBins / kWave; ++w)
        before += w < (t >> 6) ? tmp[w] : 0;
    __syncthreads();
    return before + inc - v;
}

// Sort by ranges: workgroup w orders the tokens of rows [w, w + 1) * per_wg.
// Every workgroup reads every id (from L2), so that nothing has to be exchanged
// between workgroups and one launch does it all.  Each of its waves holds a
// stretch of 64 K ids in registers and walks it twice.  The first walk counts
// the range's rows, and the tokens of smaller keys, which go before the
// workgroup's.  The second gathers the range's few tokens in an LDS ring, in
// order, and places them 64 at a time.
template <int K>
__global__ __launch_bounds__(kRangeThreads) void sort_range_kernel(SortArgs a) {
    constexpr uint32_t kWaves = kRangeThreads / kWave;
    constexpr int B = K < 8 ? K : 8;              // steps between looks at the ring
    constexpr uint32_t kRing = 2 * kWave * B;     // holds 63 + 64 B entries
    static_assert(kRangeBins == kBins, "bins_scan");
    __shared__ uint32_t cnt[kWaves][kRangeBins];
    __shared__ uint32_t ring_s[kWaves][kRing];
    __shared__ uint32_t tmp[kRangeBins / kWave];
    __shared__ uint32_t smaller[kWaves];
    const uint32_t t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t / kWave);
    const uint32_t lane = t % kWave;
    const uint32_t v0 = blockIdx.x * a.per_wg;
    const uint32_t bins = min(a.per_wg, a.rows + 1 - v0);
    const uint32_t lo = wave * (K * kWave);
    uint32_t k[K];  // key - v0: below bins in the range; larger for smaller keys
    constexpr int L = K < 16 ? K : 16;  // loads together
#pragma unroll
    for (int u = 0; u < K; u += L) {
        const uint32_t i = lo + u * kWave + lane;
        sort_keys<L>(a, [&](int j) { return min(i + j * kWave, a.n - 1); }, k + u);
#pragma unroll
        for (int j = 0; j < L; ++j)
            k[u + j] = i + j * kWave < a.n ? k[u + j] : kNone;
    }
    for (uint32_t i = t; i < kWaves * kRangeBins; i += kRangeThreads)
        (&cnt[0][0])[i] = 0;
    if (blockIdx.x == 0 && t == 0)
        a.runs[0] = 0;
    __syncthreads();
    uint32_t less = 0;
#pragma unroll
    for (int u = 0; u < K; ++u) {
        less += k[u] < v0;
        k[u] -= v0;
        if (k[u] < bins)
            atomicAdd(&cnt[wave][k[u]], 1u);
    }
    less = wave_scan(less);
    if (lane == kWave - 1)
        smaller[wave] = less;
    __syncthreads();
    uint32_t sum = 0;
    if (t < kRangeBins) {
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w)
            sum += cnt[w][t];
    }
    if (a.named && t < bins && v0 + t < a.rows)
        a.named[v0 + t] = sum != 0;
    uint32_t at = bins_scan(sum, tmp);
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w)
        at += smaller[w];
    if (t < kRangeBins) {
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w) {
            const uint32_t c = cnt[w][t];
            cnt[w][t] = at;
            at += c;
        }
    }
    __syncthreads();
    uint32_t bits = 0;
    while ((bins - 1) >> bits)
        ++bits;
    // The wave's own ring: its LDS accesses are performed in order.
    uint32_t* ring = ring_s[wave];
    uint32_t put = 0, got = 0;
    const auto place = [&](uint32_t n) {  // the ring's next n <= 64 entries
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const bool in = lane < n;
        const uint32_t e = in ? ring[(got + lane) % kRing] : 0;
        const uint32_t bin = e % kRangeBins;
        const uint64_t same = same_digit(bin, bits, __builtin_amdgcn_ballot_w64(in));
        const uint32_t to = next_place(&cnt[wave][bin], same, in);
        if (in) {
            a.key_out[to] = bin + v0;
            a.pos_out[to] = lo + e / kRangeBins;
        }
        got += n;
    };
#pragma unroll
    for (int u = 0; u < K; u += B) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const bool in = k[u + b] < bins;
            const uint64_t any = __builtin_amdgcn_ballot_w64(in);
            if (any) {
                const uint32_t before = (uint32_t)__builtin_popcountll(any & ((1ull << lane) - 1));
                if (in)
                    ring[(put + before) % kRing] = k[u + b] + ((u + b) * kWave + lane) * kRangeBins;
                put += (uint32_t)__builtin_popcountll(any);
            }
        }
        while (put - got >= kWave)
            place(kWave);
    }
    if (put != got)
        place(put - got);
}

// Sort by digits: a stable counting sort, least significant digit first, over
// at most kSortBlocks workgroups.  Counts one digit of a workgroup's tokens; the
// first digit's launch also clears the row flags, which the last one sets.  The
// number of tokens alone sets the grid, so few tokens clear the flags of many
// rows slowly: 64 tokens written into fp32 [2^20, 16] take 30 us (by ranges),
// into [2^20 + 1, 16] 102, into [2^22, 16] 338.
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
    const uint64_t lo = (uint64_t)blockIdx.x * a.per_wg;
    const uint64_t hi = min(lo + a.per_wg, (uint64_t)a.n);
    const uint32_t mask = (1u << a.bits) - 1;
    for (uint64_t i = lo + t; i < hi; i += kSortRound) {
        uint32_t key[kSortItems];
        sort_keys<kSortItems>(a, [&](int j) { return min(i + j * kSortThreads, hi - 1); }, key);
#pragma unroll
        for (uint32_t j = 0; j < kSortItems; ++j)
            if (i + j * kSortThreads < hi)
                atomicAdd(&cnt[(key[j] >> a.shift) & mask], 1u);
    }
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
#pragma unroll 8
    for (uint32_t b = 0; b < gridDim.x; ++b) {
        const uint32_t c = a.count[b * kBins + t];
        total += c;
        earlier += b < blockIdx.x ? c : 0;
    }
    base[t] = bins_scan(total, tmp) + earlier;
    const uint64_t lo = (uint64_t)blockIdx.x * a.per_wg;
    const uint64_t hi = min(lo + a.per_wg, (uint64_t)a.n);
    const uint32_t mask = (1u << a.bits) - 1;
    for (uint64_t r = lo; r < hi; r += kSortRound) {
        for (uint32_t i = t; i < kWaves * kBins; i += kSortThreads)
            (&cnt[0][0])[i] = 0;
        __syncthreads();
        uint32_t key[kSortItems], pos[kSortItems], rank[kSortItems];
        const uint64_t r0 = r + wave * kWave * kSortItems + lane;
        sort_keys<kSortItems>(a, [&](int j) { return min(r0 + j * kWave, hi - 1); }, key);
#pragma unroll
        for (uint32_t i = 0; i < kSortItems; ++i) {
            const uint64_t at = r0 + i * kWave;
            key[i] = at < hi ? key[i] : kNone;
            pos[i] = a.pos_in ? a.pos_in[min(at, hi - 1)] : (uint32_t)at;
        }
#pragma unroll
        for (uint32_t i = 0; i < kSortItems; ++i) {
            // Past the end: all bits set, ranked last, and not written.
            const uint32_t d = (key[i] >> a.shift) & mask;
            rank[i] = next_place(&cnt[wave][d], same_digit(d, a.bits, ~0ull), true);
        }
        __syncthreads();
        uint32_t sum = 0;
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w) {
            const uint32_t c = cnt[w][t];
            cnt[w][t] = (uint16_t)sum;
            sum += c;
        }
        __syncthreads();
#pragma unroll
        for (uint32_t i = 0; i < kSortItems; ++i) {
            if (r0 + i * kWave >= hi)
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
    uint32_t n, rows;
    uint32_t chunk, chunks;  // tokens of a chunk (8, 16 or 32), number of chunks
    uint32_t col_tiles;
    uint64_t dim;
    const void* dout;
    void* grad;
    float scale;
    uint64_t seed, cbase;
    uint32_t sum_wgs;     // the workgroups after these clear rows
    uint32_t clear_rows;  // rows of such a workgroup, at most 64
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

// The eight columns of a lane in its wave's group of kCols: eight consecutive
// ones, or with an fp32 gradient two fours, kCols / 2 apart, so that each
// access covers whole lines.
template <int OUT>
struct Cols {
    static constexpr bool kSplit = OUT == kF32;
    static constexpr int H = kSplit ? 2 : 1, G = 8 / H;
    uint32_t col[H], left[H];  // first column, columns from there to the row's end
    bool on[H];                // there is one (else the lane reads column 0, and writes nothing)

    __device__ __forceinline__ Cols(uint32_t tile, uint32_t dim) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            col[h] = tile * kCols + h * (kCols / 2) + (uint32_t)lane_id() * G;
            on[h] = col[h] < dim;
            if (!on[h])
                col[h] = 0;
            left[h] = dim - col[h];
        }
    }
};

// A lane's columns of one row of an array of type T.
template <int T, int OUT>
struct RowBits {
    Raw<T, Cols<OUT>::G> h[Cols<OUT>::H];
};

template <int T, int OUT, bool WHOLE, bool NT>
__device__ __forceinline__ RowBits<T, OUT> load_row(const void* __restrict__ p, uint64_t row,
                                                    uint64_t dim, const Cols<OUT>& c) {
    RowBits<T, OUT> r;
#pragma unroll
    for (int h = 0; h < Cols<OUT>::H; ++h)
        r.h[h] = load_group<T, Cols<OUT>::G, WHOLE, NT>(p, row * dim + c.col[h], c.left[h]);
    return r;
}

template <int T, int OUT, bool WHOLE>
__device__ __forceinline__ void widen_row(RowBits<T, OUT> r, const Cols<OUT>& c, float x[8]) {
#pragma unroll
    for (int h = 0; h < Cols<OUT>::H; ++h) {
        if constexpr (!WHOLE)
            whole<T, Cols<OUT>::G>(r.h[h], c.left[h]);
        widen<T, Cols<OUT>::G>(r.h[h], x + h * Cols<OUT>::G);
    }
}

// A long run's partial sums.
template <int OUT>
__device__ __forceinline__ void store_part(const float s[8], float* p, const Cols<OUT>& c) {
#pragma unroll
    for (int h = 0; h < Cols<OUT>::H; ++h)
        if (c.on[h])
#pragma unroll
            for (int i = 0; i < Cols<OUT>::G; i += 4) {
                const float* q = s + h * Cols<OUT>::G + i;
                *(f4*)(p + c.col[h] + i) = f4{q[0], q[1], q[2], q[3]};
            }
}

// dout is read nontemporally where an access covers whole lines (see zq_rows.h).
// The gradient's rows are read and written plainly: 32768 tokens x 4096 added
// into fp32 took 171.8 us with nontemporal reads of them, 168.5 with plain ones;
// written (16384 x 2048) 81.4 us with nontemporal stores, 79.4 with plain ones.
template <int IN, int OUT>
constexpr bool dout_nt() {
    return IN != kF32 || OUT == kF32;
}

// Writes a row's eight sums; `old` are the buffer's values there (add modes).
template <int OUT, int MODE, bool WHOLE>
__device__ __forceinline__ void finish(const SumArgs& a, const float s[8],
                                       const RowBits<OUT, OUT>& old, uint64_t row,
                                       const Cols<OUT>& c) {
    constexpr int H = Cols<OUT>::H, G = Cols<OUT>::G;
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        g[j] = a.scale * s[j];
    if constexpr (MODE != kGradWrite) {
        float o[8];
        widen_row<OUT, OUT, WHOLE>(old, c, o);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            g[j] = o[j] + g[j];
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const uint64_t e = row * a.dim + c.col[h];
        Raw<OUT, G> r;
        if constexpr (MODE == kGradAddSr) {
            uint32_t r16[8];
            random8(a.cbase + e, a.seed, r16);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r.w[j] = sr_bf16(g[2 * j], r16[2 * j]) | (sr_bf16(g[2 * j + 1], r16[2 * j + 1]) << 16);
        } else {
            r = narrow<OUT, G>(g + h * G);
        }
        if (c.on[h])
            store_group<OUT, G, WHOLE, false>(r, a.grad, e, c.left[h]);
    }
}

// A wave's window of the sorted tokens: lane l holds the l-th from its chunk's
// first on, two chunks of them.
template <int IN, int OUT, int MODE, bool WHOLE>
struct Window {
    static constexpr int U = 8;  // tokens in flight
    const SumArgs& a;
    uint32_t key, pos;
    Cols<OUT> cols;

    __device__ __forceinline__ uint32_t key_at(uint32_t p) const {
        return __builtin_amdgcn_readlane(key, p);
    }

    // Sums positions [p, e), p < e, one run after the other; `ends` has a bit at
    // each run's last position.  A run that ends at long_end goes to long_part,
    // the others to the table.
    __device__ __forceinline__ void sum(uint32_t p, uint32_t e, uint64_t ends, float* long_part,
                                        uint32_t long_end) const {
        float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (; p < e; p += U) {
            RowBits<IN, OUT> x[U];
            RowBits<OUT, OUT> old[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t q = min(p + u, e - 1);  // past the end: read, not used
                const uint64_t t = __builtin_amdgcn_readlane(pos, q);
                x[u] = load_row<IN, OUT, WHOLE, dout_nt<IN, OUT>()>(a.dout, t, a.dim, cols);
                if constexpr (MODE != kGradWrite)
                    if (((ends >> q) & 1) && q != long_end)
                        old[u] = load_row<OUT, OUT, WHOLE, false>(a.grad, key_at(q), a.dim, cols);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p + u >= e)
                    break;
                float v[8];
                widen_row<IN, OUT, WHOLE>(x[u], cols, v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[j] += v[j];
                if (!((ends >> (p + u)) & 1))
                    continue;
                if (p + u == long_end)
                    store_part<OUT>(s, long_part, cols);
                else
                    finish<OUT, MODE, WHOLE>(a, s, old[u], key_at(p + u), cols);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[j] = 0.0f;
            }
        }
    }
};

template <int IN, int OUT, int MODE, bool WHOLE>
__device__ __forceinline__ void sum_chunk(const SumArgs& a, uint32_t k, uint32_t tile) {
    const uint32_t lane = (uint32_t)lane_id();
    const uint32_t c = a.chunk, span = 2 * c;  // span <= 64
    const uint32_t i0 = k * c;
    Window<IN, OUT, MODE, WHOLE> w = {a, kNone, 0, Cols<OUT>(tile, (uint32_t)a.dim)};
    if (lane < span && i0 + lane < a.n) {
        w.key = a.key[i0 + lane];
        w.pos = a.pos[i0 + lane];
    }
    // The neighbours that decide how runs cross the window's borders, read at
    // once with it: the tokens before this chunk and before the previous one,
    // and the first one after the window.
    const uint32_t before = k > 0 ? a.key[i0 - 1] : kNone;
    const uint32_t before2 = k > 1 ? a.key[i0 - c - 1] : kNone;
    const uint32_t after = i0 + span < a.n ? a.key[i0 + span] : kNone;
    const uint32_t first = w.key_at(0);
    if (first >= a.rows)
        return;  // ids that name no row, to the end
    const bool cont = before == first;
    // Bit p: a run starts at position p.  Lanes without a token hold kNone, the
    // first of them is a start too.
    const uint32_t prev = __shfl_up(w.key, 1);
    const uint64_t starts = __builtin_amdgcn_ballot_w64(lane == 0 ? !cont : w.key != prev);
    const uint64_t ends = starts >> 1;
    const uint32_t own = (uint32_t)(starts & ((1ull << c) - 1));
    const uint32_t p = own ? (uint32_t)__builtin_ctz(own) : c;
    if (cont && before2 == first) {
        // The run began before the previous chunk: this chunk's part of it.
        const uint32_t here = min(p, a.n - i0);
        w.sum(0, here, 1ull << (here - 1), a.part + (uint64_t)k * a.pitch, here - 1);
    }
    if (!own)
        return;
    // The runs that start here; the last one may reach into the next chunk.
    const uint64_t later = starts >> c;
    uint32_t e = later ? min(c + (uint32_t)__builtin_ctzll(later), span) : span;
    uint32_t long_end = kNone;
    const uint32_t last = w.key_at(span - 1);
    if (e == span && last < a.rows && after == last) {
        long_end = span - 1;
        if (tile == 0 && lane == 0)
            a.runs[1 + atomicAdd(&a.runs[0], 1u)] = k;
    }
    // Ids that name no row, and positions past the end, are not summed.
    const uint64_t bad = __builtin_amdgcn_ballot_w64(w.key >= a.rows);
    if (bad)
        e = min(e, (uint32_t)__builtin_ctzll(bad));
    if (p < e)
        w.sum(p, e, ends | (1ull << (span - 1)), a.part + (uint64_t)(k + 1) * a.pitch, long_end);
}

// Clears the rows of job j that no token names: a thread per group of G columns,
// over all the job's rows as one run of groups.
template <int OUT, bool WHOLE>
__device__ __forceinline__ void clear_rows(const SumArgs& a, uint32_t j) {
    constexpr int G = Cols<OUT>::G;
    constexpr uint32_t kThreads = sum_threads<kGradWrite>();
    const uint32_t r0 = j * a.clear_rows, rows = min(a.clear_rows, a.rows - r0);
    const uint32_t lane = (uint32_t)lane_id();
    const uint64_t named = __builtin_amdgcn_ballot_w64(lane < rows && a.named[r0 + lane]);
    const uint32_t per_row = (uint32_t)((a.dim + G - 1) / G);
    uint32_t row = threadIdx.x / per_row, group = threadIdx.x % per_row;
    const uint32_t row_step = kThreads / per_row, group_step = kThreads % per_row;
    const Raw<OUT, G> zero = {};
    while (row < rows) {
        if (!((named >> row) & 1))
            store_group<OUT, G, WHOLE, true>(zero, a.grad,
                                             (uint64_t)(r0 + row) * a.dim + (uint64_t)group * G,
                                             (uint32_t)a.dim - group * G);
        row += row_step;
        group += group_step;
        if (group >= per_row) {
            group -= per_row;
            ++row;
        }
    }
}

template <int IN, int OUT, int MODE, bool WHOLE>
__global__ __launch_bounds__(sum_threads<MODE>()) void sum_kernel(SumArgs a) {
    if (MODE == kGradWrite && blockIdx.x >= a.sum_wgs) {
        const uint32_t jobs = (a.rows - 1) / a.clear_rows + 1;
        for (uint32_t j = blockIdx.x - a.sum_wgs; j < jobs; j += gridDim.x - a.sum_wgs)
            clear_rows<OUT, WHOLE>(a, j);
        return;
    }
    const uint64_t jobs = (uint64_t)a.chunks * a.col_tiles;
    const uint64_t waves = (uint64_t)a.sum_wgs * (sum_threads<MODE>() / kWave);
    for (uint64_t j = wave_id(); j < jobs; j += waves) {
        const uint32_t k = (uint32_t)(j / a.col_tiles);
        sum_chunk<IN, OUT, MODE, WHOLE>(a, k, (uint32_t)(j - (uint64_t)k * a.col_tiles));
    }
}

// Adds the partials of each long run in order.  The run that began in chunk k
// has them in slots k + 1 (chunks k and k + 1), k + 2, ..., as far as chunks
// begin with its row.  Each wave of the workgroup adds a stretch of the slots,
// then the stretches are added in order.
template <int OUT, int MODE, bool WHOLE>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(SumArgs a) {
    constexpr uint32_t kWaves = kJoinThreads / kWave;
    constexpr int G = Cols<OUT>::G;
    __shared__ float part[kWaves][kCols];
    const uint32_t wave = threadIdx.x / kWave, lane = (uint32_t)lane_id();
    const uint32_t list = min(blockIdx.x / a.col_tiles, a.chunks - 1);
    const uint32_t k0 = a.runs[1 + list];  // read beside the number of runs: a guess at most
    const uint64_t jobs = (uint64_t)a.runs[0] * a.col_tiles;
    for (uint64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
        const uint32_t k = j == blockIdx.x ? k0 : a.runs[1 + j / a.col_tiles];
        const uint32_t tile = (uint32_t)(j % a.col_tiles);
        // The chunks from k + 2 on that begin with the run's row: chunk k + 2 does,
        // and the keys are sorted, so 64 probes at a time find the end; mostly
        // within the next 64 chunks.
        const uint32_t probe = a.key[min(k + 2 + lane, a.chunks - 1) * a.chunk];
        const uint32_t row = __builtin_amdgcn_readfirstlane(probe);
        const Cols<OUT> c(tile, (uint32_t)a.dim);
        RowBits<OUT, OUT> old = {};
        if constexpr (MODE != kGradWrite)
            if (wave == 0)
                old = load_row<OUT, OUT, WHOLE, false>(a.grad, row, a.dim, c);
        const uint32_t near = (uint32_t)__builtin_popcountll(
            __builtin_amdgcn_ballot_w64(k + 2 + lane < a.chunks && probe == row));
        uint32_t hi = k + 2 + near;
        if (near == kWave) {
            uint32_t lo = hi - 1;  // begins with the row; hi does not, or is the end
            hi = a.chunks;
            while (hi - lo > 1) {
                const uint32_t step = (hi - lo + kWave - 1) / kWave;
                const uint64_t at = (uint64_t)lo + (uint64_t)lane * step;
                const bool yes = at < hi && a.key[at * a.chunk] == row;
                const uint32_t n = (uint32_t)__builtin_popcountll(__builtin_amdgcn_ballot_w64(yes));
                hi = (uint32_t)min((uint64_t)hi, (uint64_t)lo + (uint64_t)n * step);
                lo += (n - 1) * step;
            }
        }
        const uint32_t slots = hi - (k + 1);
        const uint32_t s0 = k + 1 + (uint32_t)((uint64_t)slots * wave / kWaves);
        const uint32_t s1 = k + 1 + (uint32_t)((uint64_t)slots * (wave + 1) / kWaves);
        float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (uint32_t i = s0; i < s1; i += 4) {
            f4 x[4][2];  // four slots in flight; past the end the last one again, not added
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) {
                const float* q = a.part + (uint64_t)min(i + u, s1 - 1) * a.pitch;
                x[u][0] = *(const f4*)(q + c.col[0]);
                x[u][1] = *(const f4*)(q + c.col[4 / G] + 4 % G);
            }
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[e] += i + u < s1 ? x[u][e / 4][e % 4] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            part[wave][e * kWave + lane] = s[e];
        __syncthreads();
        if (wave == 0) {
            for (uint32_t w = 1; w < kWaves; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[e] += part[w][e * kWave + lane];
            finish<OUT, MODE, WHOLE>(a, s, old, row, c);
        }
        __syncthreads();
    }
}

// ZQ_GRAD_WRITE without tokens.  One store a thread: 262 MB took 39.7 us so (as
// long as torch's fill), 45 to 50 us with loops over 16 to 1024 KB a workgroup.
__global__ __launch_bounds__(kBlockThreads) void clear_kernel(char* p, uint64_t bytes) {
    const uint64_t units = bytes / 16;
    for (uint64_t i = (uint64_t)blockIdx.x * kBlockThreads + threadIdx.x; i < units;
         i += (uint64_t)gridDim.x * kBlockThreads)
        ((u4*)p)[i] = u4{0, 0, 0, 0};
    if (blockIdx.x == 0 && 2 * threadIdx.x < bytes % 16)
        *(uint16_t*)(p + units * 16 + 2 * threadIdx.x) = 0;
}

hipError_t launch(const void* fn, uint64_t wgs, uint32_t threads, void** args, hipStream_t st) {
    return hipLaunchKernel(fn, dim3((uint32_t)wgs), dim3(threads), args, 0, st);
}

// The range sort that holds n tokens.
const void* sort_range_of(uint32_t n) {
    static_assert(kRangeTokens <= 32 * kRangeThreads, "the largest K");
    return n <= 1024    ? (const void*)&sort_range_kernel<1>
           : n <= 2048  ? (const void*)&sort_range_kernel<2>
           : n <= 4096  ? (const void*)&sort_range_kernel<4>
           : n <= 8192  ? (const void*)&sort_range_kernel<8>
           : n <= 16384 ? (const void*)&sort_range_kernel<16>
                        : (const void*)&sort_range_kernel<32>;
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
    s.named = want_named ? (uint8_t*)(ws + l.named) : nullptr;
    s.runs = (uint32_t*)(ws + l.runs);
    s.key_out = (uint32_t*)(ws + l.key[0]);
    s.pos_out = (uint32_t*)(ws + l.pos[0]);
    void* args[] = {(void*)&s};
    if (sorts_by_range(a.n_tok, a.rows)) {
        // Keys run from 0 to rows.  A workgroup for every 32 tokens, at most
        // kRangeWgs of them unless that gives one over kRangeBins keys.
        const uint32_t keys = s.rows + 1;
        const uint32_t want = std::max(std::min((s.n + 31) / 32, kRangeWgs),
                                       (keys + kRangeBins - 1) / kRangeBins);
        s.per_wg = (keys + want - 1) / want;
        *key = s.key_out;
        *pos = s.pos_out;
        return launch(sort_range_of(s.n), (keys + s.per_wg - 1) / s.per_wg, kRangeThreads, args, st);
    }
    // As many digits as the keys' bits need, of equal width.
    uint32_t bits = 1;
    while ((s.rows >> bits) != 0)
        ++bits;
    const uint32_t passes = (bits + kDigitBits - 1) / kDigitBits;
    s.bits = (bits + passes - 1) / passes;
    s.count = (uint32_t*)(ws + l.count);
    const uint32_t rounds = (s.n + kSortRound - 1) / kSortRound;
    s.per_wg = (rounds + kSortBlocks - 1) / kSortBlocks * kSortRound;
    const uint32_t wgs = (s.n + s.per_wg - 1) / s.per_wg;
    uint8_t* named = s.named;
    for (uint32_t p = 0; p < passes; ++p) {
        s.shift = p * s.bits;
        s.key_out = (uint32_t*)(ws + l.key[p & 1]);
        s.pos_out = (uint32_t*)(ws + l.pos[p & 1]);
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
    s.chunk = (uint32_t)l.chunk;
    s.chunks = (uint32_t)l.chunks;
    s.rows = (uint32_t)a.rows;
    s.dim = a.dim;
    s.col_tiles = (uint32_t)l.col_tiles;
    s.dout = a.dout;
    s.grad = a.grad;
    s.scale = a.scale;
    s.seed = a.seed;
    s.cbase = a.cbase;
    const uint64_t jobs = l.chunks * l.col_tiles;
    constexpr uint32_t kThreads = sum_threads<MODE>(), kWaves = kThreads / kWave;
    s.sum_wgs = (uint32_t)std::min(kMaxWgs, (jobs + kWaves - 1) / kWaves);
    uint64_t wgs = s.sum_wgs;
    if (MODE == kGradWrite) {
        const uint64_t row_bytes = a.dim * (OUT == kF32 ? 4 : 2);
        s.clear_rows = (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(kWave, kClearBytes / row_bytes));
        wgs += std::min(kMaxWgs, (a.rows - 1) / s.clear_rows + 1);
    }
    void* args[] = {(void*)&s};
    e = launch((const void*)&sum_kernel<IN, OUT, MODE, WHOLE>, wgs, kThreads, args, st);
    if (e != hipSuccess || a.n_tok <= 2 * l.chunk)
        return e;  // no run is longer than a chunk and its successor
    return launch((const void*)&join_kernel<OUT, MODE, WHOLE>, std::min<uint64_t>(512, jobs),
                  kJoinThreads, args, st);
}

template <int IN, int OUT, int MODE>
hipError_t grad_m(const EmbedGradArgs& a, hipStream_t st) {
    return a.dim % Cols<OUT>::G == 0 ? grad_t<IN, OUT, MODE, true>(a, st)
                                     : grad_t<IN, OUT, MODE, false>(a, st);
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
        return launch((const void*)&clear_kernel, std::min(kMaxWgs, bytes / 4096 + 1), kBlockThreads,
                      args, stream);
    }
    switch (d_type) {
        case kF32: return grad_in<kF32>(a, grad_type, mode, stream);
        case kBF16: return grad_in<kBF16>(a, grad_type, mode, stream);
        case kF16: return grad_in<kF16>(a, grad_type, mode, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace zq
