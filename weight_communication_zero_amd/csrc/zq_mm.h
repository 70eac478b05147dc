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
    const uint32_t* dyn_m;     // where set, M (K) is the smaller of M (K) and this
    const uint32_t* dyn_k;
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
    return r;
}

// Waits until at most N of the wave's loads are under way.
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

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

__device__ __forceinline__ h4 lds_read_tr(uint32_t at) {
    typedef __attribute__((address_space(3))) h4 lds_h4;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_h4*)(uintptr_t)at);
}

// The LDS side of one operand of ROWS rows.  Stored by 16-byte chunks so that
// the reads below meet no bank twice:
//   plain       row r, chunk c of 8 at (r, c ^ (r & 7))
//   transposed  k, pair of chunks q at (k, q ^ ((k & 3) + 4 (k >> 3 & 1)))
template <int ROWS, bool TR, int WAVES>
struct MmTile {
    static constexpr uint32_t kBytes = ROWS * kMmK * 2;
    static constexpr int kLoads = (int)(kBytes / (WAVES * 1024));
    static_assert(kLoads * WAVES * 1024 == kBytes, "whole loads");

    uint32_t voff[kLoads];
    uint32_t klane[TR ? kLoads : 1], coff[TR ? kLoads : 1];

    // rows: rows (plain) or columns (transposed) there are from the tile's first on.
    __device__ __forceinline__ void init(uint32_t wave, uint32_t lane, uint64_t ld, uint32_t rows) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t u = (j * WAVES + wave) * 64 + lane;
            if constexpr (TR) {
                const uint32_t k = u / (ROWS / 8), c = u % (ROWS / 8);
                const uint32_t sw = (k & 3) + 4 * ((k >> 3) & 1);
                uint32_t col = ((c / 2) ^ sw) * 16 + (c & 1) * 8;
                col = min(col, rows - 8);
                klane[j] = k;
                coff[j] = col * 2;
                voff[j] = k * (uint32_t)ld * 2 + col * 2;
            } else {
                const uint32_t r = u >> 3, c = (u & 7) ^ (r & 7);
                voff[j] = min(r, rows - 1) * (uint32_t)ld * 2 + c * 16;
            }
        }
    }

    // Loads the step at `p` (the operand's first element of the step's first
    // k); left: k's there are, where fewer than a step's.
    __device__ __forceinline__ void load(const uint16_t* p, uint64_t ld, uint32_t left,
                                         uint32_t lds, uint32_t wave) const {
        const i4v srd = buffer_of(p);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            uint32_t v = voff[j];
            if constexpr (TR)
                if (left < kMmK)
                    v = min(klane[j], left - 1) * (uint32_t)ld * 2 + coff[j];
            dma16(srd, v, lds + (j * WAVES + wave) * 1024);
        }
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
    uint32_t at[TR ? COUNT : 2];

    __device__ __forceinline__ void init(uint32_t row0, uint32_t lane) {
        if constexpr (TR) {
            const uint32_t kq = (lane >> 4) * 8 + ((lane & 15) >> 2);
            const uint32_t sw = (kq & 3) + 4 * ((kq >> 3) & 1);
#pragma unroll
            for (int i = 0; i < COUNT; ++i)
                at[i] = kq * (ROWS * 2) + (((row0 / 16 + i) ^ sw) * 32) + (lane & 3) * 8;
        } else {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
                at[kk] = (row0 + (lane & 15)) * 128 + (((kk * 4 + (lane >> 4)) ^ (lane & 7)) << 4);
        }
    }

    __device__ __forceinline__ h8 read(uint32_t lds, int i, int kk) const {
        if constexpr (TR) {
            const uint32_t p = lds + at[i] + kk * 32 * ROWS * 2;
            const h4 x = lds_read_tr(p), y = lds_read_tr(p + 4 * ROWS * 2);
            return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            typedef __attribute__((address_space(3))) h8 lds_h8;
            return *(const lds_h8*)(uintptr_t)(lds + at[kk] + i * 2048);
        }
    }
};

// Tile t of tm x tn in an order that keeps neighbours together: 8 tiles down,
// then the next column.
__device__ __forceinline__ void mm_tile_of(uint32_t t, uint32_t tm, uint32_t tn, uint32_t* m,
                                           uint32_t* n) {
    constexpr uint32_t G = 8;
    const uint32_t g = t / (G * tn), r = t - g * G * tn;
    const uint32_t h = min(G, tm - g * G);
    *n = r / h;
    *m = g * G + r - *n * h;
}

// A workgroup's tile of BM x BN, shared out to WM x WN waves; STAGES steps of the
// operands in LDS.
template <int T_, int BM_, int BN_, int WM_, int WN_, int STAGES_, bool TA_, bool TB_>
struct MmShape {
    static constexpr int T = T_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
    static constexpr bool TA = TA_, TB = TB_;
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
    static constexpr uint32_t kStage = (BM + BN) * kMmK * 2;
};

template <class S, class Epi>
__global__ __launch_bounds__(S::kThreads) void mm_kernel(MmArgs a, typename Epi::Args e) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S::STAGES * S::kStage];
    using TileA = MmTile<S::BM, S::TA, S::kWaves>;
    using TileB = MmTile<S::BN, S::TB, S::kWaves>;
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    uint32_t M = a.M, K = a.K;
    if (a.dyn_m)
        M = min(M, *a.dyn_m);
    if (a.dyn_k)
        K = min(K, *a.dyn_k);
    const uint32_t tm = (M + S::BM - 1) / S::BM, tn = (a.N + S::BN - 1) / S::BN;
    const uint32_t total = tm * tn, per = (total + 7) / 8;
    const uint32_t t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || t >= total)
        return;
    uint32_t im, in;
    mm_tile_of(t, tm, tn, &im, &in);
    const uint32_t m0 = im * S::BM, n0 = in * S::BN;

    // This split's k's.
    const uint32_t steps_all = (K + kMmK - 1) / kMmK;
    const uint32_t per_split = (steps_all + gridDim.y - 1) / gridDim.y;
    const uint32_t s0 = min(blockIdx.y * per_split, steps_all);
    const uint32_t steps = min(per_split, steps_all - s0);

    TileA la;
    TileB lb;
    la.init(wave, lane, a.a.ld, S::TA ? a.a_cols - m0 : M - m0);
    lb.init(wave, lane, a.b.ld, S::TB ? a.b_cols - n0 : a.N - n0);
    const uint64_t step_a = S::TA ? kMmK * a.a.ld : kMmK, step_b = S::TB ? kMmK * a.b.ld : kMmK;
    const uint16_t* pa = a.a.p + (S::TA ? (uint64_t)m0 : m0 * a.a.ld) + s0 * step_a;
    const uint16_t* pb = a.b.p + (S::TB ? (uint64_t)n0 : n0 * a.b.ld) + s0 * step_b;

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

    const uint32_t base = lds_offset(lds);
    uint32_t left = K - s0 * kMmK;  // k's from the next step to load on
    auto load = [&](uint32_t buf) {
        la.load(pa, a.a.ld, left, base + buf * S::kStage, wave);
        lb.load(pb, a.b.ld, left, base + buf * S::kStage + TileA::kBytes, wave);
        pa += step_a;
        pb += step_b;
        left -= kMmK;
    };
    constexpr uint32_t kAhead = S::STAGES - 1;
#pragma unroll
    for (uint32_t s = 0; s < kAhead; ++s)
        if (s < steps)
            load(s);
    uint32_t buf = 0;
    for (uint32_t s = 0; s < steps; ++s) {
        // Step s has arrived for this wave, then for all; the reads of step s - 1
        // are over, so its buffer can be loaded.
        if (s + kAhead <= steps)
            wait_vm<(S::STAGES - 2) * (TileA::kLoads + TileB::kLoads)>();
        else
            wait_vm<0>();
        wait_lds();
        __builtin_amdgcn_s_barrier();
        if (s + kAhead < steps)
            load(buf == 0 ? kAhead : buf - 1);
        const uint32_t here = K - (s0 + s) * kMmK;
        if ((S::TA || S::TB) && here < kMmK) {
            if constexpr (S::TA)
                TileA::clear_tail(lds + buf * S::kStage, here, tid);
            if constexpr (S::TB)
                TileB::clear_tail(lds + buf * S::kStage + TileA::kBytes, here, tid);
            __syncthreads();
        }
        const uint32_t sa = base + buf * S::kStage, sb = sa + TileA::kBytes;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            h8 x[S::MI], y[S::NI];
#pragma unroll
            for (int j = 0; j < S::NI; ++j)
                y[j] = fb.read(sb, j, kk);
#pragma unroll
            for (int i = 0; i < S::MI; ++i)
                x[i] = fa.read(sa, i, kk);
#pragma unroll
            for (int i = 0; i < S::MI; ++i)
#pragma unroll
                for (int j = 0; j < S::NI; ++j)
                    acc[i][j] = mfma<S::T>(y[j], x[i], acc[i][j]);
        }
        buf = buf + 1 == S::STAGES ? 0 : buf + 1;
    }
    wait_lds();
    __builtin_amdgcn_s_barrier();
    // acc[i][j][r] is C at m = mw + 16 i + (lane & 15), n = nw + 16 j + 4 (lane >> 4) + r.
    Epi::template finish<S>(e, acc, M, a.N, m0, n0, wm, wn, lane, lds);
}


// What becomes of a sum: C[m, n .. n + 3], of which the first `count` exist.
struct MmOut {
    const float* acc_in;    // sums of earlier pieces to add, or NULL
    float* acc_out;         // where to keep the sum for later pieces, or NULL
    uint64_t ldacc;         // a multiple of 4
    void* out;              // else: times scale (and *factor) into out's row list[m]
    uint64_t ldo;
    const uint32_t* list;
    const float* factor;
    float scale;
    int type, add;

    __device__ __forceinline__ void put(uint32_t m, uint32_t n, uint32_t count, f4 v) const {
        if (acc_in)
            v += *(const f4*)(acc_in + m * ldacc + n);
        if (acc_out) {
            *(f4*)(acc_out + m * ldacc + n) = v;
            return;
        }
        const float f = factor ? scale * *factor : scale;
        v *= f;
        const uint64_t e = (list ? list[m] : m) * ldo + n;
        if (type == kF32) {
            typedef f4 at __attribute__((aligned(4)));
            float* p = (float*)out + e;
            if (count >= 4) {
                if (add)
                    v += *(const at*)p;
                *(at*)p = v;
            } else {
                for (uint32_t r = 0; r < 3; ++r)
                    if (r < count)
                        p[r] = add ? p[r] + v[r] : v[r];
            }
        } else {
            typedef u2 at __attribute__((aligned(2)));
            uint16_t* p = (uint16_t*)out + e;
            if (count >= 4) {
                if (add) {
                    const u2 o = *(const at*)p;
                    if (type == kBF16)
                        v += f4{bf16lo(o.x), bf16hi(o.x), bf16lo(o.y), bf16hi(o.y)};
                    else
                        v += f4{f16lo(o.x), f16hi(o.x), f16lo(o.y), f16hi(o.y)};
                }
                *(at*)p = type == kBF16 ? u2{pack_bf16_rne(v[0], v[1]), pack_bf16_rne(v[2], v[3])}
                                        : u2{pack_f16_rne(apart(v[0]), apart(v[1])),
                                             pack_f16_rne(apart(v[2]), apart(v[3]))};
            } else {
                for (uint32_t r = 0; r < 3; ++r)
                    if (r < count) {
                        float x = v[r];
                        if (add)
                            x += type == kBF16 ? bf16lo(p[r]) : f16lo(p[r]);
                        p[r] = (uint16_t)(type == kBF16 ? pack_bf16_rne(x, x)
                                                        : pack_f16_rne(apart(x), apart(x)));
                    }
            }
        }
    }
};

// The epilogue of sums: put, or with part set (K split over gridDim.y) the split's
// partial sums at part[(split * rows + m) * ld + n], for mm_join_kernel.
struct MmSum {
    struct Args {
        MmOut o;
        float* part;
        uint64_t rows, ld;
    };
    template <class S>
    static __device__ __forceinline__ void finish(const Args& e, f4 (&acc)[S::MI][S::NI],
                                                  uint32_t M, uint32_t N, uint32_t m0, uint32_t n0,
                                                  uint32_t wm, uint32_t wn, uint32_t lane,
                                                  unsigned char*) {
        const uint32_t mw = m0 + wm * (S::BM / S::WM) + (lane & 15);
        const uint32_t nw = n0 + wn * (S::BN / S::WN) + (lane >> 4) * 4;
#pragma unroll
        for (int i = 0; i < S::MI; ++i) {
            const uint32_t m = mw + i * 16;
            if (m >= M)
                continue;
#pragma unroll
            for (int j = 0; j < S::NI; ++j) {
                const uint32_t n = nw + j * 16;
                if (n >= N)
                    continue;
                if (e.part)
                    *(f4*)(e.part + (blockIdx.y * e.rows + m) * e.ld + n) = acc[i][j];
                else
                    e.o.put(m, n, N - n, acc[i][j]);
            }
        }
    }
};

// Adds the splits' partial sums in their order and puts the result.
__global__ __launch_bounds__(256) static void mm_join_kernel(MmSum::Args e, uint32_t splits,
                                                             uint32_t M, uint32_t N,
                                                             const uint32_t* dyn_m) {
    if (dyn_m)
        M = min(M, *dyn_m);
    const uint32_t groups = (N + 3) / 4;
    const uint64_t total = (uint64_t)M * groups;
    for (uint64_t g = blockIdx.x * 256ull + threadIdx.x; g < total; g += gridDim.x * 256ull) {
        const uint32_t m = (uint32_t)(g / groups), n = (uint32_t)(g - (uint64_t)m * groups) * 4;
        f4 v = *(const f4*)(e.part + m * e.ld + n);
        for (uint32_t s = 1; s < splits; ++s)
            v += *(const f4*)(e.part + (s * e.rows + m) * e.ld + n);
        e.o.put(m, n, N - n, v);
    }
}

}  // namespace zq
