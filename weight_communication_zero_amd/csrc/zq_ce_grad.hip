// zq_ce_grad.hip -- the gradient of the vocabulary projection's cross entropy.
//
// For each piece of the vocabulary three products on one tile engine:
//   q  = dloss (exp(scale x w^T - lse) - [target])   rounded to 16 bits, in the
//        workspace: tokens x piece
//   dx += q w        (kept in binary32 between pieces)
//   dw  = q^T x      (this piece's rows, whole)
// The second and third take their operands as they lie, by transposed reads from
// LDS, so nothing is stored transposed; neither needs the other, so they share a launch.
//
// Bound by the matrix units: 16384 tokens, 4096 x 32000, take 9.54 to 9.88 ms in two
// pieces, by the card (1300 to 1350 TFLOP/s over all), 8192 tokens, 2048 x 32000, with
// 10 % left out 2.26 to 2.36 ms.  Few tokens are bound by memory and by steps that wait
// for each other: 64 tokens, 2048 x 32000, take 177 us, one read of w and one write of dw
// 54 us at a copy's rate.
#include "zq_ce.h"

namespace zq {
namespace {

// Up to this many tokens q is kept in two 16-bit parts (rows 2 t and 2 t + 1, which dx's
// product adds up in pairs and dw's sums over, x's rows standing twice), so that its
// rounding is off by 2^-16 (bf16) or 2^-22 (fp16) of it.  With few tokens one rounding
// weighs more, as nothing averages out, and the products wait for memory and launches:
// 64 tokens, 2048 x 32000 in bf16, take 175 us in two parts and 169 in one, 128 tokens
// 205 and 178, 256 tokens 261 and 211.
constexpr uint32_t kTwoParts = 128;

// What a first part leaves of q: nothing where it is infinite or NaN.
__device__ __forceinline__ float rest(float q, float first) {
    const float r = q - first;
    return __builtin_fabsf(r) < __builtin_inff() ? r : 0.0f;
}

struct Residual {
    struct Args {
        float scale;
        uint16_t* q;
        uint64_t ldq;
        uint32_t parts;
        CeTokens t;
        uint32_t v0;
    };

    // A token's target in the piece, its lse, and its scaled loss gradient.
    struct Row {
        uint32_t target;
        float lse, g;
    };
    static __device__ __forceinline__ Row row(const Args& e, uint32_t M, uint32_t m0,
                                              uint32_t tid) {
        const uint32_t m = min(m0 + tid, M - 1);
        return {e.t.target[m] - e.v0, e.t.lse[m], e.t.dloss[m] * e.t.scalars->up};
    }

    template <class S>
    static __device__ __forceinline__ void finish(const Args& e, const Row& mine,
                                                  f4 (&acc)[S::MI][S::NI], uint32_t M, uint32_t N,
                                                  uint32_t m0, uint32_t n0, uint32_t,
                                                  uint32_t wm, uint32_t wn, uint32_t lane,
                                                  unsigned char* lds) {
        // The rows' values behind the part of LDS that the sums go through.
        static_assert(S::kThreads >= S::BM && S::kRowsLds + S::BM * sizeof(Row) <= S::kLds, "fits");
        Row* rows = (Row*)(lds + S::kRowsLds);
        if (threadIdx.x < S::BM)
            rows[threadIdx.x] = mine;
        __syncthreads();
        const uint32_t end = (N + kMmK - 1) / kMmK * kMmK;  // zeros from N up to here
        mm_rows<S>(
            acc, wm, wn, lane, lds, false, [](uint32_t, uint32_t) { return f4{0, 0, 0, 0}; },
            [&](uint32_t r, uint32_t c, f4 z, f4) {
                const uint32_t m = m0 + r, n = n0 + c;
                if (m >= M || n >= end)
                    return;
                const Row t = rows[r];
                float q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // The logit is rounded as the loss rounds it: of a sure token it is
                    // lse, and p is 1, however large it is.  (In one fma of base 2 the
                    // roundings of lse log2 e and of the factor stay in the exponent.)
                    const float p = exp2_of(base2(e.scale * z[k] - t.lse));
                    q[k] = t.g * (n + k == t.target ? p - 1.0f : p);
                    q[k] = n + k < N ? q[k] : 0.0f;
                }
                const u2 first = {pack_half_rne<S::T>(q[0], q[1]), pack_half_rne<S::T>(q[2], q[3])};
                uint16_t* out = e.q + (uint64_t)m * e.parts * e.ldq + n;
                *(u2*)out = first;
                if (e.parts == 2)
                    *(u2*)(out + e.ldq) =
                        u2{pack_half_rne<S::T>(rest(q[0], half_lo<S::T>(first.x)),
                                               rest(q[1], half_hi<S::T>(first.x))),
                           pack_half_rne<S::T>(rest(q[2], half_lo<S::T>(first.y)),
                                               rest(q[3], half_hi<S::T>(first.y)))};
            });
    }
};

CeLayout layout(uint32_t n_tok, uint32_t rows, uint32_t dim, uint64_t piece) {
    CeLayout l = {};
    l.kp = round_up(dim, kMmK);
    l.parts = n_tok <= kTwoParts ? 2 : 1;
    const uint64_t n_pad = round_up(n_tok, 256);
    // The library's choice: 512 MiB of q and of staged rows.
    uint64_t most = piece ? round_up(std::min<uint64_t>(piece, rows), 256)
                          : ((uint64_t)1 << 28) / std::max(n_pad, l.kp);
    most = std::min(most, ((uint64_t)1 << 36) / std::max(n_pad, l.kp));
    ce_pieces(l, rows, most);
    l.logits = mm_plan(n_tok, l.piece, l.kp, false);
    CeTake take;
    ce_take_tokens(l, take, n_tok, true);
    l.q = take((uint64_t)n_tok * l.piece * 2 * l.parts);
    l.ldacc = round_up(dim, 4);
    l.acc = take(l.n_pieces > 1 ? n_tok * l.ldacc * 4 : 0);
    uint64_t x_floats = 0, w_floats = 0;
    for (uint32_t n : {l.piece, l.rows_of(l.n_pieces - 1, rows)}) {
        const uint32_t k = n_tok * l.parts;
        x_floats = std::max(x_floats, part_floats(mm_plan(k, dim, n, true), k, dim));
        w_floats = std::max(w_floats, part_floats(mm_plan(n, dim, k, true), n, dim));
    }
    l.x_sums = take(x_floats * 4);
    l.w_sums = take(w_floats * 4);
    l.total = take.at;
    return l;
}

template <int T>
hipError_t launch(const CeArgs& a, int w_type, int dw_type, int mode, hipStream_t stream) {
    const CeLayout l = layout(a.n_tok, a.rows, a.dim, a.piece);
    char* ws = (char*)a.workspace;
    const CeTokens tok = ce_tokens(l, ws);
    hipError_t st = ce_prep<true>(a, tok, T == kF16, stream);
    const MmOperand x = {(const uint16_t*)(ws + l.x), l.kp};
    const MmOperand q = {(const uint16_t*)(ws + l.q), l.piece};
    float* acc = (float*)(ws + l.acc);
    const uint32_t* count = &tok.scalars->count;
    for (uint32_t i = 0; i < l.n_pieces && st == hipSuccess; ++i) {
        const uint32_t v0 = i * l.piece, n = l.rows_of(i, a.rows);
        st = ce_stage<T>(a, w_type, l, i, true, tok, ws, stream);
        if (st != hipSuccess)
            break;
        const MmOperand w = ce_piece(a, w_type, l, v0, ws);
        MmArgs m = {};
        m.a = {x.p, x.ld * l.parts};  // each row's first copy
        m.b = w;
        m.M = a.n_tok;
        m.N = n;
        m.K = (uint32_t)l.kp;
        m.dyn_m = count;
        Residual::Args e = {a.scale, (uint16_t*)(ws + l.q), l.piece, l.parts, tok, v0};
        st = launch_mm<T, false, false, Residual>(m, e, l.logits, stream);
        if (st != hipSuccess)
            break;
        MmOut o = {};
        o.ldacc = l.ldacc;
        o.ldo = a.dim;
        o.factor = &tok.scalars->down;
        o.scale = a.scale;
        const uint32_t q_rows = a.n_tok * l.parts;
        const uint32_t* q_count = l.parts == 2 ? &tok.scalars->twice : count;
        MmInto to_x = {m, o, mm_plan(q_rows, a.dim, n, true), (float*)(ws + l.x_sums), l.parts == 2};
        to_x.a.a = q;
        to_x.a.M = q_rows;
        to_x.a.dyn_m = q_count;
        to_x.a.N = a.dim;
        to_x.a.K = n;
        to_x.a.b_cols = (uint32_t)l.kp;
        to_x.o.acc_in = i ? acc : nullptr;
        to_x.o.acc_out = i + 1 < l.n_pieces ? acc : nullptr;
        to_x.o.out = a.dx;
        to_x.o.list = tok.list;
        to_x.o.type = T;
        MmInto to_w = {{}, o, mm_plan(n, a.dim, q_rows, true), (float*)(ws + l.w_sums)};
        to_w.a.a = q;
        to_w.a.b = x;
        to_w.a.M = n;
        to_w.a.N = a.dim;
        to_w.a.K = q_rows;
        to_w.a.a_cols = l.piece;
        to_w.a.b_cols = (uint32_t)l.kp;
        to_w.a.dyn_k = q_count;
        if (a.dw)
            to_w.o.out = (char*)a.dw + (uint64_t)v0 * a.dim * (dw_type == kF32 ? 4 : 2);
        to_w.o.type = dw_type;
        to_w.o.add = mode == kGradAdd;
        if (a.dx && a.dw)
            st = launch_mm_two_sums<T>(to_x, to_w, stream);
        else if (a.dx)
            st = launch_mm_sum<T, false, true>(to_x, stream);
        else
            st = launch_mm_sum<T, true, true>(to_w, stream);
    }
    return st;
}

__global__ __launch_bounds__(256) void clear_kernel(uint32_t* p, uint64_t words, uint32_t rest) {
    const uint64_t first = blockIdx.x * 256ull + threadIdx.x;
    for (uint64_t i = first; i < words; i += gridDim.x * 256ull)
        p[i] = 0;
    if (first < rest)
        ((uint8_t*)(p + words))[first] = 0;
}

}  // namespace

hipError_t launch_clear(void* p, uint64_t bytes, hipStream_t stream) {
    uint32_t* q = (uint32_t*)p;
    uint64_t words = bytes / 4;
    uint32_t rest = bytes % 4;
    void* args[] = {&q, &words, &rest};
    const uint64_t wgs = std::min<uint64_t>(words / 256 + 1, 16384);
    return hipLaunchKernel((const void*)&clear_kernel, dim3((uint32_t)wgs), dim3(256), args, 0,
                           stream);
}

size_t ce_grad_workspace(uint32_t n_tok, uint32_t rows, uint32_t dim, uint64_t piece) {
    return layout(n_tok, rows, dim, piece).total;
}

hipError_t launch_ce_grad(const CeArgs& a, int type, int w_type, int dw_type, int mode,
                          hipStream_t stream) {
    return type == kBF16 ? launch<kBF16>(a, w_type, dw_type, mode, stream)
                         : launch<kF16>(a, w_type, dw_type, mode, stream);
}

}  // namespace zq
