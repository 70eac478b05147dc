// zq_mm.h -- the matrix product of libzq's layer kernels, on gfx950's MFMA
// units:  C[m, n] = sum_k A(m, k) B(n, k)  of bf16 or fp16 operands, summed in
// binary32, with what becomes of C left to an epilogue.
#pragma once

#include "zq_device.h"

namespace zq {

typedef short h4 __attribute__((ext_vector_type(4)));
typedef short h8 __attribute__((ext_vector_type(8)));
typedef int i4v __attribute__((ext_vector_type(4)));

constexpr uint32_t kMmK = 64;  // k's per step

// An operand: element (r, k) at p[r * ld + k], or with TRANSPOSED at
// p[k * ld + r].  ld is a multiple of 8, p 16-byte aligned.
// A plain operand's K is a multiple of 64; where the other operand is transposed, a
// plain one holds zeros from the last k on up to that multiple.
struct MmOperand {
    const uint16_t* p;
    uint64_t ld;
};

struct MmArgs {
    MmOperand a, b;
    uint32_t M, N, K;
    uint32_t a_cols, b_cols;   // of a transposed operand: stored columns (a multiple of 8)
    const uint32_t* a_rows;    // where set, row m of a plain a is stored row a_rows[m]
                               // (all of them within 4 GiB)
    const uint32_t* dyn_m;     // where set, M (K) is the smaller of M (K) and this
    const uint32_t* dyn_k;
    uint32_t wgs, splits;      // workgroups of a split (a multiple of 8, one for each
                               // tile or more); parts that the k's are split into
};

typedef __attribute__((address_space(3))) unsigned char lds_byte;

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(const lds_byte*)p;
}

// 16 bytes a lane from global memory to LDS: lane l's to lds + 16 l.
__device__ __forceinline__ void dma16(i4v srd, uint32_t voff, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
        :
        : "v"(voff), "s"(srd), "s"(lds)
        : "memory", "m0");
}

__device__ __forceinline__ i4v buffer_of(const void* p) {
    const uint64_t a = (uint64_t)(uintptr_t)p;
    i4v r = {(int)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
             (int)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)), -1, 0x00020000};
    // Should a vector instruction have written the words, a load that reads them has to
    // stay 5 cycles behind; the compiler does not see the loads in dma16.
    asm volatile("s_nop 4" : "+s"(r));
    return r;
}

// The buffer `bytes` further on (scalar instructions, which need no distance).
__device__ __forceinline__ i4v advanced(i4v r, uint64_t bytes) {
    const uint64_t a = ((uint64_t)(uint32_t)r.y << 32 | (uint32_t)r.x) + bytes;
    r.x = (int)(uint32_t)a;
    r.y = (int)(uint32_t)(a >> 32);
    return r;
}

// Waits until at most N of the wave's loads are under way.
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// All waves' arrival; no access to memory moves across it.
__device__ __forceinline__ void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int T>
__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) {
    if constexpr (T == kBF16) {
        typedef __bf16 b8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a),
                                                       __builtin_bit_cast(b8, b), c, 0, 0, 0);
    } else {
        typedef _Float16 g8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(g8, a),
                                                      __builtin_bit_cast(g8, b), c, 0, 0, 0);
    }
}

// The turn of a transposed tile's row of ROWS / 16 pairs: the 16 k's of one read are
// 8 q + 0 .. 3 for q = 0 .. 3.
template <int ROWS>
__device__ __forceinline__ uint32_t mm_turn(uint32_t k) {
    return ((k & 3) + 4 * ((k >> 3) & 1)) & (ROWS >= 128 ? 7 : ROWS / 16 - 1);
}

// The LDS side of one operand of ROWS rows.  Stored by 16-byte chunks so that
// the reads below meet no bank twice (transposed tiles of fewer than 128 rows apart):
//   plain       row r, chunk c of 8 at (r, c ^ (r & 7))
//   transposed  k, pair of chunks q at (k, q ^ mm_turn(k))
template <int ROWS, bool TR, int WAVES>
struct MmTile {
    static constexpr uint32_t kBytes = ROWS * kMmK * 2;
    static constexpr int kLoads = (int)(kBytes / (WAVES * 1024));
    static_assert(kLoads * WAVES * 1024 == kBytes, "whole loads");

    uint32_t voff[kLoads];

    // rows: rows (plain) or columns (transposed) there are from the tile's first on;
    // list: where set, the stored rows of a plain operand.
    __device__ __forceinline__ void init(uint32_t wave, uint32_t lane, uint64_t ld, uint32_t rows,
                                         const uint32_t* list) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t u = (j * WAVES + wave) * 64 + lane;
            if constexpr (TR) {
                const uint32_t k = u / (ROWS / 8), c = u % (ROWS / 8);
                const uint32_t col = ((c / 2) ^ mm_turn<ROWS>(k)) * 16 + (c & 1) * 8;
                voff[j] = k * (uint32_t)ld * 2 + min(col, rows - 8) * 2;
            } else {
                const uint32_t c = (u & 7) ^ ((u >> 3) & 7);
                uint32_t r = min(u >> 3, rows - 1);
                if (list)
                    r = list[r];
                voff[j] = r * (uint32_t)ld * 2 + c * 16;
            }
        }
    }

    // Load j of the wave's kLoads of the step whose first k `srd` points to; left: k's
    // there are from it on (past the last one, a transposed operand's last is taken).
    __device__ __forceinline__ void load(i4v srd, int j, uint64_t ld, uint32_t left, uint32_t lds,
                                         uint32_t wave) const {
        uint32_t v = voff[j];
        if constexpr (TR)
            if (left < kMmK) {
                const uint32_t k = ((j * WAVES + wave) * 64 + (threadIdx.x & 63)) / (ROWS / 8);
                v -= (k - min(k, left - 1)) * (uint32_t)ld * 2;
            }
        dma16(srd, v, lds + (j * WAVES + wave) * 1024);
    }

    __device__ __forceinline__ void load_all(i4v srd, uint64_t ld, uint32_t left, uint32_t lds,
                                             uint32_t wave) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            load(srd, j, ld, left, lds, wave);
    }

    // Clears the k's from `left` on of a loaded transposed step.
    static __device__ __forceinline__ void clear_tail(unsigned char* lds, uint32_t left,
                                                      uint32_t tid) {
        for (uint32_t i = left * (ROWS / 8) + tid; i < kMmK * (ROWS / 8); i += WAVES * 64)
            *(u4*)(lds + i * 16) = u4{0, 0, 0, 0};
    }
};

// A wave's fragments of COUNT groups of 16 rows.
template <int ROWS, bool TR, int COUNT>
struct MmFrags {
    uint32_t at[TR ? 1 : 2];

    __device__ __forceinline__ void init(uint32_t row0, uint32_t lane) {
        if constexpr (TR) {
            const uint32_t kq = (lane >> 4) * 8 + ((lane & 15) >> 2);
            at[0] = kq * (ROWS * 2) + (((row0 / 16) ^ mm_turn<ROWS>(kq)) * 32) + (lane & 3) * 8;
        } else {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
                at[kk] = (row0 + (lane & 15)) * 128 + (((kk * 4 + (lane >> 4)) ^ (lane & 7)) << 4);
        }
    }

    // A transposed group i lies at the first one's address with the bits of 32 i
    // flipped: row0 / 16 is a multiple of COUNT, at most 8 and a power of two, and a
    // stage starts on a multiple of 256 bytes.
    __device__ __forceinline__ h8 read(uint32_t lds, int i, int kk) const {
        static_assert(COUNT == 8 || COUNT == 4 || COUNT == 2 || COUNT == 1, "a power of two");
        if constexpr (TR) {
            typedef __attribute__((address_space(3))) h4 lds_h4;
            lds_h4* p = (lds_h4*)(uintptr_t)((lds + at[0]) ^ (i * 32));
            const h4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p + kk * 8 * ROWS);
            const h4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p + kk * 8 * ROWS + ROWS);
            return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            typedef __attribute__((address_space(3))) h8 lds_h8;
            return ((const lds_h8*)(uintptr_t)(lds + at[kk]))[i * 128];
        }
    }
};

// Tile t of tm x tn in an order that keeps neighbours together: 4 tiles down,
// then the next column (the 32 tiles that an XCD works on then share 4 row and 8
// column panels in its L2; 8 x 4 measured 1 to 2 % slower, 16 x 2 3 %).
__device__ __forceinline__ void mm_tile_of(uint32_t t, uint32_t tm, uint32_t tn, uint32_t* m,
                                           uint32_t* n) {
    constexpr uint32_t G = 4;
    const uint32_t g = t / (G * tn), r = t - g * G * tn;
    const uint32_t h = min(G, tm - g * G);
    *n = r / h;
    *m = g * G + r - *n * h;
}

// A workgroup's tile of BM x BN, shared out to WM x WN waves; DEPTH steps of loads
// under way.
template <int T_, int BM_, int BN_, int WM_, int WN_, int DEPTH_, bool TA_, bool TB_>
struct MmShape {
    static constexpr int T = T_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, DEPTH = DEPTH_;
    static constexpr bool TA = TA_, TB = TB_;
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
    static constexpr uint32_t kLds = (DEPTH * BM + (DEPTH + 1) * BN) * kMmK * 2;
    // What mm_rows takes of it: of each wave kGroup rows of fragments at a time.
    static constexpr int kGroup = MI < 4 ? MI : 4;
    static constexpr uint32_t kRowsLds = kGroup * 16 * NI * 64 * kWaves;
    static_assert(kRowsLds <= kLds, "fits");
};

template <int V>
struct MmInt {
    static constexpr int value = V;
};

// The kernel.  LDS holds DEPTH stages of a's steps and DEPTH + 1 of b's.  A step is
// two phases of 32 k's; in each, a wave multiplies one set of fragments while it
// reads the other set from LDS and issues loads, all between its matrix
// instructions, a few for every row of fragments:
//   phase 0 of step s   multiplies its first half, reads its second, loads step
//                       s + DEPTH of b (into the stage that step s - 1 has left)
//   (the one barrier of a step: step s + 1 has arrived for all waves, and all have
//   read what they need of step s)
//   phase 1             multiplies the second half, reads the first half of step
//                       s + 1, loads step s + DEPTH of a (into step s's stage)
// so that the matrix units wait neither for LDS nor for the loads' issue.  16384 x
// 32000 x 4096 in bf16: 3.55 ms with all reads of a half step before its products, 3.45
// with the reads half a step ahead, 3.20 with the loads spread among the products, 3.09
// to 3.13 (1370 to 1390 TFLOP/s) with the last steps, which load nothing, in a loop of
// their own.  The matrix units are then busy 75 % of the cycles, at 1.74 GHz of 2.4; the
// library's product takes 2.85 to 2.95 ms.
template <class S, class Epi>
__device__ __forceinline__ void mm_run(const MmArgs& a, const typename Epi::Args& e, uint32_t wg,
                                       unsigned char* lds) {
    using TileA = MmTile<S::BM, S::TA, S::kWaves>;
    using TileB = MmTile<S::BN, S::TB, S::kWaves>;
    constexpr uint32_t kA = TileA::kBytes, kB = TileB::kBytes;
    constexpr int kLoadsA = TileA::kLoads, kLoadsB = TileB::kLoads;
    constexpr uint32_t D = S::DEPTH;
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    uint32_t M = a.M, K = a.K;
    if (a.dyn_m)
        M = min(M, *a.dyn_m);
    if (a.dyn_k)
        K = min(K, *a.dyn_k);
    const uint32_t split = wg / a.wgs;
    wg -= split * a.wgs;
    // Workgroup b runs on XCD b % 8: each XCD takes an eighth of the tiles in a row.
    const uint32_t tm = (M + S::BM - 1) / S::BM, tn = (a.N + S::BN - 1) / S::BN;
    const uint32_t total = tm * tn, per = (total + 7) / 8;
    const uint32_t t = (wg & 7) * per + (wg >> 3);
    if ((wg >> 3) >= per || t >= total)
        return;
    uint32_t im, in;
    mm_tile_of(t, tm, tn, &im, &in);
    const uint32_t m0 = im * S::BM, n0 = in * S::BN;

    // This split's k's.
    const uint32_t steps_all = (K + kMmK - 1) / kMmK;
    const uint32_t per_split = (steps_all + a.splits - 1) / a.splits;
    const uint32_t s0 = min(split * per_split, steps_all);
    const uint32_t steps = min(per_split, steps_all - s0);
    const uint32_t count = K - s0 * kMmK;  // k's from the split's first on

    TileA la;
    TileB lb;
    const bool listed = !S::TA && a.a_rows;
    la.init(wave, lane, a.a.ld, S::TA ? a.a_cols - m0 : M - m0, listed ? a.a_rows + m0 : nullptr);
    lb.init(wave, lane, a.b.ld, S::TB ? a.b_cols - n0 : a.N - n0, nullptr);
    const uint64_t step_a = S::TA ? kMmK * a.a.ld : kMmK, step_b = S::TB ? kMmK * a.b.ld : kMmK;
    i4v pa = buffer_of(a.a.p + (S::TA ? (uint64_t)m0 : listed ? 0 : m0 * a.a.ld) + s0 * step_a);
    i4v pb = buffer_of(a.b.p + (S::TB ? (uint64_t)n0 : n0 * a.b.ld) + s0 * step_b);
    const typename Epi::Row row = Epi::row(e, M, m0, tid);

    const uint32_t wm = wave / S::WN, wn = wave % S::WN;
    MmFrags<S::BM, S::TA, S::MI> fa;
    MmFrags<S::BN, S::TB, S::NI> fb;
    fa.init(wm * (S::BM / S::WM), lane);
    fb.init(wn * (S::BN / S::WN), lane);

    f4 acc[S::MI][S::NI];
#pragma unroll
    for (int i = 0; i < S::MI; ++i)
#pragma unroll
        for (int j = 0; j < S::NI; ++j)
            acc[i][j] = f4{0, 0, 0, 0};

    const uint32_t base_a = lds_offset(lds), base_b = base_a + D * kA;
    h8 x[2][S::MI], y[2][S::NI];
    constexpr int kReads = (S::MI + S::NI + S::MI - 1) / S::MI;  // a row of fragments
    auto phase = [&](auto set, uint32_t sa, uint32_t sb, auto half, auto&& issue) {
        constexpr int cur = decltype(set)::value, kk = decltype(half)::value;
#pragma unroll
        for (int i = 0; i < S::MI; ++i) {
#pragma unroll
            for (int r = i * kReads; r < (i + 1) * kReads && r < S::MI + S::NI; ++r) {
                if (r < S::NI)
                    y[1 - cur][r < S::NI ? r : 0] = fb.read(sb, r, kk);
                else
                    x[1 - cur][r < S::NI ? 0 : r - S::NI] = fa.read(sa, r - S::NI, kk);
            }
            issue(i);
#pragma unroll
            for (int j = 0; j < S::NI; ++j)
                acc[i][j] = mfma<S::T>(y[cur][j], x[cur][i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Clears what a loaded step s of transposed operands has past the last k.
    auto clear = [&](uint32_t s, uint32_t oa, uint32_t ob) {
        const uint32_t here = count - s * kMmK;
        if ((S::TA || S::TB) && s < steps && here < kMmK) {
            if constexpr (S::TA)
                TileA::clear_tail(lds + oa, here, tid);
            if constexpr (S::TB)
                TileB::clear_tail(lds + D * kA + ob, here, tid);
            __syncthreads();
        }
    };
    if (steps) {
#pragma unroll
        for (uint32_t s = 0; s < D; ++s)
            if (s < steps) {
                la.load_all(pa, a.a.ld, count - s * kMmK, base_a + s * kA, wave);
                lb.load_all(pb, a.b.ld, count - s * kMmK, base_b + s * kB, wave);
                pa = advanced(pa, step_a * 2);
                pb = advanced(pb, step_b * 2);
            }
        if (steps >= D)
            wait_vm<(D - 1) * (kLoadsA + kLoadsB)>();
        else
            wait_vm<0>();
        meet();
        clear(0, 0, 0);
#pragma unroll
        for (int i = 0; i < S::MI; ++i)
            x[0][i] = fa.read(base_a, i, 0);
#pragma unroll
        for (int j = 0; j < S::NI; ++j)
            y[0][j] = fb.read(base_b, j, 0);
    }
    uint32_t oa = 0, ob = 0, ob_new = D * kB;  // stages of step s, and of step s + D of b
    auto step = [&](uint32_t s, auto more) {
        constexpr bool kMore = decltype(more)::value;  // step s + D is there to load
        const uint32_t left = count - (s + D) * kMmK;
        const uint32_t oa1 = oa == (D - 1) * kA ? 0 : oa + kA, ob1 = ob == D * kB ? 0 : ob + kB;
        __builtin_amdgcn_sched_barrier(0);
        phase(MmInt<0>(), base_a + oa, base_b + ob, MmInt<1>(), [&](int i) {
            if constexpr (kMore)
#pragma unroll
                for (int j = 0; j < kLoadsB; ++j)
                    if (j * S::MI / kLoadsB == i)
                        lb.load(pb, j, a.b.ld, left, base_b + ob_new, wave);
        });
        // Past step s + 1's loads, those of steps s + 2 to s + D - 1 and the ones just
        // issued may be under way.
        wait_lds();
        if constexpr (kMore)
            wait_vm<(D - 2) * (kLoadsA + kLoadsB) + kLoadsB>();
        else
            wait_vm<0>();
        meet();
        if constexpr (!kMore)
            clear(s + 1, oa1, ob1);
        __builtin_amdgcn_sched_barrier(0);
        phase(MmInt<1>(), base_a + oa1, base_b + ob1, MmInt<0>(), [&](int i) {
            if constexpr (kMore)
#pragma unroll
                for (int j = 0; j < kLoadsA; ++j)
                    if (j * S::MI / (2 * kLoadsA) == i)
                        la.load(pa, j, a.a.ld, left, base_a + oa, wave);
        });
        pa = advanced(pa, step_a * 2);
        pb = advanced(pb, step_b * 2);
        oa = oa1;
        ob_new = ob;
        ob = ob1;
    };
    uint32_t s = 0;
    for (; s + D < steps; ++s)
        step(s, MmInt<1>());
    for (; s < steps; ++s)
        step(s, MmInt<0>());
    wait_lds();
    meet();
    // acc[i][j][r] is C at m = m0 + wm BM / WM + 16 i + (lane & 15),
    // n = n0 + wn BN / WN + 16 j + 4 (lane >> 4) + r.
    Epi::template finish<S>(e, row, acc, M, a.N, m0, n0, split, wm, wn, lane, lds);
}

// Two waves a SIMD are asked for (LDS lets no more in): with 512 registers to give, the
// compiler would keep the sums in accumulation registers and move fragments to and fro.
template <class S, class Epi>
__global__ __launch_bounds__(S::kThreads, 2) void mm_kernel(MmArgs a, typename Epi::Args e) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S::kLds];
    mm_run<S, Epi>(a, e, blockIdx.x, lds);
}

// Two products in one launch, so that the second's tiles fill the CUs that the first's
// last ones leave idle.
template <class S1, class S2, class Epi>
__global__ __launch_bounds__(S1::kThreads, 2) void mm_pair_kernel(MmArgs a1, typename Epi::Args e1,
                                                                  MmArgs a2,
                                                                  typename Epi::Args e2) {
    static_assert(S1::kThreads == S2::kThreads && S1::kLds == S2::kLds, "tiles of one kind");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S1::kLds];
    const uint32_t first = a1.wgs * a1.splits;
    if (blockIdx.x < first)
        mm_run<S1, Epi>(a1, e1, blockIdx.x, lds);
    else
        mm_run<S2, Epi>(a2, e2, blockIdx.x - first, lds);
}

// Hands each f4 of a wave's sums to put(m in the tile, n in the tile, f4, what
// fetch(m, n) gave), through LDS: 16 lanes then hold 64 neighbours of one row, so that
// whole lines are stored, and the code stands 4 times instead of 32 (it runs once and
// comes from memory).  Four at a time, so that their fetches are under way together.
// Four rows of fragments in a part of LDS of the wave's own, chunk c of 16 bytes of a row
// at c ^ (row & 15) (or a smaller mask), which meets no bank twice.
// With `pairs`, rows 2 r and 2 r + 1 of the tile are added and handed over as row r.
template <class S, class G, class F>
__device__ __forceinline__ void mm_rows(f4 (&acc)[S::MI][S::NI], uint32_t wm, uint32_t wn,
                                        uint32_t lane, unsigned char* lds, bool pairs, G&& fetch,
                                        F&& put) {
    constexpr int kGroup = S::kGroup;
    constexpr uint32_t kChunks = S::NI * 4;           // of 16 bytes in a row
    constexpr uint32_t kMask = kChunks < 16 ? kChunks - 1 : 15;
    constexpr uint32_t kAll = kGroup * 16 * kChunks;  // of a wave
    constexpr int kBatch = kAll / 64 < 4 ? kAll / 64 : 4;
    static_assert(kAll % (64 * kBatch) == 0, "whole batches");
    unsigned char* mine = lds + (wm * S::WN + wn) * kAll * 16;
    const uint32_t r = lane & 15, q = lane >> 4;
    const uint32_t mw = wm * (S::BM / S::WM), nw = wn * (S::BN / S::WN);
#pragma unroll
    for (int g = 0; g < S::MI / kGroup; ++g) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
#pragma unroll
            for (int j = 0; j < S::NI; ++j)
                *(f4*)(mine + ((i * 16 + r) * kChunks + ((j * 4 + q) ^ (r & kMask))) * 16) =
                    acc[g * kGroup + i][j];
        wait_lds();
#pragma unroll 1
        for (uint32_t c0 = lane; c0 < kAll; c0 += 64 * kBatch) {
            f4 v[kBatch], old[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const uint32_t row = (c0 + k * 64) / kChunks, chunk = (c0 + k * 64) % kChunks;
                v[k] = *(const f4*)(mine + (row * kChunks + (chunk ^ (row & kMask))) * 16);
                if (pairs)  // (an odd row adds its own other half, and is not handed over)
                    v[k] += *(const f4*)(mine + ((row ^ 1) * kChunks + (chunk ^ ((row ^ 1) & kMask))) * 16);
                old[k] = fetch((mw + g * kGroup * 16 + row) >> pairs, nw + chunk * 4);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const uint32_t row = (c0 + k * 64) / kChunks, chunk = (c0 + k * 64) % kChunks;
                if (!pairs || row % 2 == 0)
                    put((mw + g * kGroup * 16 + row) >> pairs, nw + chunk * 4, v[k], old[k]);
            }
        }
        wait_lds();
    }
}

// An epilogue has Args; Row, what a thread loads for row m0 + tid before the sums
// (where it needs something); and finish.
struct MmNoRow {};

// What becomes of a sum: C[m, n .. n + 3], of which the first `count` exist.
struct MmOut {
    const float* acc_in;    // sums of earlier pieces to add, or NULL
    float* acc_out;         // where to keep the sum for later pieces, or NULL
    uint64_t ldacc;         // a multiple of 4
    void* out;              // else: times scale (and *factor) into out's row list[m],
    uint64_t ldo;           // added to what is there where `add` is set
    const uint32_t* list;
    const float* factor;
    float scale;
    int type, add;

    __device__ __forceinline__ uint64_t at(uint32_t m, uint32_t n) const {
        return (list ? list[m] : m) * ldo + n;
    }

    // What put needs of memory: the earlier pieces' sums, or what out holds.  (Both never
    // occur together: dx has pieces, dw is added to.)
    __device__ __forceinline__ f4 fetch(uint32_t m, uint32_t n, uint32_t count) const {
        if (acc_in)
            return *(const f4*)(acc_in + m * ldacc + n);
        f4 v = {0, 0, 0, 0};
        if (!add)
            return v;
        const uint64_t e = at(m, n);
        if (type == kF32) {
            typedef f4 any __attribute__((aligned(4)));
            const float* p = (const float*)out + e;
            if (count >= 4)
                return *(const any*)p;
#pragma unroll
            for (uint32_t r = 0; r < 3; ++r)
                if (r < count)
                    v[r] = p[r];
        } else {
            typedef u2 any __attribute__((aligned(2)));
            const uint16_t* p = (const uint16_t*)out + e;
            u2 o = {0, 0};
            if (count >= 4) {
                o = *(const any*)p;
            } else {
                o.x = p[0];
                if (count > 1)
                    o.x |= (uint32_t)p[1] << 16;
                if (count > 2)
                    o.y = p[2];
            }
            v = type == kBF16 ? f4{bf16lo(o.x), bf16hi(o.x), bf16lo(o.y), bf16hi(o.y)}
                              : f4{f16lo(o.x), f16hi(o.x), f16lo(o.y), f16hi(o.y)};
        }
        return v;
    }

    __device__ __forceinline__ void put(uint32_t m, uint32_t n, uint32_t count, f4 v,
                                        f4 old) const {
        if (acc_in)
            v += old;
        if (acc_out) {
            *(f4*)(acc_out + m * ldacc + n) = v;
            return;
        }
        v *= factor ? scale * *factor : scale;
        if (add)
            v += old;
        const uint64_t e = at(m, n);
        if (type == kF32) {
            typedef f4 any __attribute__((aligned(4)));
            float* p = (float*)out + e;
            if (count >= 4) {
                *(any*)p = v;
                return;
            }
#pragma unroll
            for (uint32_t r = 0; r < 3; ++r)
                if (r < count)
                    p[r] = v[r];
        } else {
            typedef u2 any __attribute__((aligned(2)));
            uint16_t* p = (uint16_t*)out + e;
            const u2 o = type == kBF16
                             ? u2{pack_bf16_rne(v[0], v[1]), pack_bf16_rne(v[2], v[3])}
                             : u2{pack_f16_rne(apart(v[0]), apart(v[1])),
                                  pack_f16_rne(apart(v[2]), apart(v[3]))};
            if (count >= 4) {
                *(any*)p = o;
                return;
            }
            p[0] = (uint16_t)o.x;
            if (count > 1)
                p[1] = (uint16_t)(o.x >> 16);
            if (count > 2)
                p[2] = (uint16_t)o.y;
        }
    }
};

// The epilogue of sums: put, or with part set (K is split) the split's
// partial sums at part[(split * rows + m) * ld + n], for mm_join_kernel.
struct MmSum {
    struct Args {
        MmOut o;
        float* part;
        uint64_t rows, ld;
        bool pairs;  // rows 2 m and 2 m + 1 of the product are row m's two parts
    };
    using Row = MmNoRow;
    static __device__ __forceinline__ Row row(const Args&, uint32_t, uint32_t, uint32_t) {
        return {};
    }
    template <class S>
    static __device__ __forceinline__ void finish(const Args& e, const Row&,
                                                  f4 (&acc)[S::MI][S::NI], uint32_t M, uint32_t N,
                                                  uint32_t m0, uint32_t n0, uint32_t split,
                                                  uint32_t wm, uint32_t wn, uint32_t lane,
                                                  unsigned char* lds) {
        const bool part = e.part != nullptr;
        m0 >>= e.pairs;
        M >>= e.pairs;
        mm_rows<S>(
            acc, wm, wn, lane, lds, e.pairs,
            [&](uint32_t r, uint32_t c) {
                const uint32_t m = m0 + r, n = n0 + c;
                return !part && m < M && n < N ? e.o.fetch(m, n, N - n) : f4{0, 0, 0, 0};
            },
            [&](uint32_t r, uint32_t c, f4 v, f4 old) {
                const uint32_t m = m0 + r, n = n0 + c;
                if (m >= M || n >= N)
                    return;
                if (part)
                    *(f4*)(e.part + (split * e.rows + m) * e.ld + n) = v;
                else
                    e.o.put(m, n, N - n, v, old);
            });
    }
};

// Adds the splits' partial sums in their order and puts the result.
__global__ __launch_bounds__(256) static void mm_join_kernel(MmSum::Args e, uint32_t splits,
                                                             uint32_t M, uint32_t N,
                                                             const uint32_t* dyn_m) {
    if (dyn_m)
        M = min(M, *dyn_m);
    M >>= e.pairs;
    const uint32_t groups = (N + 3) / 4;
    const uint64_t total = (uint64_t)M * groups;
    for (uint64_t g = blockIdx.x * 256ull + threadIdx.x; g < total; g += gridDim.x * 256ull) {
        const uint32_t m = (uint32_t)(g / groups), n = (uint32_t)(g - (uint64_t)m * groups) * 4;
        const f4 old = e.o.fetch(m, n, N - n);
        f4 v = *(const f4*)(e.part + m * e.ld + n);
        for (uint32_t s = 1; s < splits; ++s)
            v += *(const f4*)(e.part + (s * e.rows + m) * e.ld + n);
        e.o.put(m, n, N - n, v, old);
    }
}

}  // namespace zq
