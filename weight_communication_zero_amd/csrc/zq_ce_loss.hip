// zq_ce_loss.hip -- softmax cross entropy of the vocabulary projection.
//
// The logits of a tile of tokens x vocabulary stay in the matrix product's
// registers: the epilogue takes each token's largest sum m over the tile's columns but the
// target's, the sum s of 2^(f (a - m)) over them, f = unit log2 e, and the target's sum
// t where it lies there.  A second kernel joins the tiles' pairs,
// (m, s) + (m', s') = (M, s 2^(f (m - M)) + s' 2^(f (m' - M))),
// and forms  loss = log1p(s 2^(f (m - t))),  or where t < m
//            loss = unit (m - t) + log(s + 2^(f (t - m))),
// in which nothing cancels: the loss of a nearly sure token keeps its digits (taken as
// lse - z it is off by half a unit of the logit's last place, 100 % of a loss of 1e-6).
//
// Bound by the matrix units with many tokens (16384 x 4096 x 32000 from int8 in 3.04 to
// 3.16 ms, by the card: 1360 to 1410 TFLOP/s, 0.07 ms of it the dequantization; the
// differences before the factor are 0.02 of it), by the read of w with few (one token,
// 4096 x 32000 in bf16: 56 us, of which 41 read the 262 MB, at 6.3 TB/s, and 6 join).  Few
// tokens from codes wait for the widened copy of w, which is written and read again: one
// token 119 us, where the codes alone are 27 us at a copy's rate.
#include "zq_ce.h"

namespace zq {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));

// What the exponentials are taken relative to: the maximum, where it is finite (an
// infinite one would give inf - inf).
__device__ __forceinline__ float reference(float m) {
    return __builtin_fabsf(m) < __builtin_inff() ? m : 0.0f;
}

// 2^(factor (a - ref)) of two sums.  The difference is taken before the factor: factor a
// and factor ref, each rounded, would leave half a unit of the largest logit's last place
// in the exponent, which is 1e-6 at logits of 14 and whole powers of two beyond 10^9.
__device__ __forceinline__ float relative(float factor, float a, float ref) {
    return exp2_of(factor * (a - ref));
}

// A pair's sum relative to another reference.  With an infinite maximum the sum is
// 0, infinity or NaN, and stays so.
__device__ __forceinline__ float rebased(float factor, f2 p, float ref) {
    return __builtin_fabsf(p.x) < __builtin_inff() ? p.y * relative(factor, p.x, ref) : p.y;
}

struct Stats {
    struct Args {
        CeScale scale;
        f2* part;          // [tile of the piece][ld]
        uint64_t ld;
        uint32_t v0;       // the piece's first row
        float* z_target;
        const uint32_t* target;  // of the tokens that count, or NULL: all tokens, by
        const void* ids;         // their ids
        uint32_t id64;
    };

    // A token's target in the piece (a large number where it lies outside).
    struct Row {
        uint32_t target;
    };
    static __device__ __forceinline__ Row row(const Args& e, uint32_t M, uint32_t m0,
                                              uint32_t tid) {
        const uint32_t m = min(m0 + tid, M - 1);
        if (e.target)
            return {e.target[m] - e.v0};
        uint64_t id[1];
        load_ids<1>(e.ids, e.id64, [&](int) { return m; }, id);
        return {id[0] <= 0x7FFFFFFFu ? (uint32_t)id[0] - e.v0 : 0xFFFFFFFFu};
    }

    template <class S>
    static __device__ __forceinline__ void finish(const Args& e, const Row& mine,
                                                  f4 (&acc)[S::MI][S::NI], uint32_t M, uint32_t N,
                                                  uint32_t m0, uint32_t n0, uint32_t,
                                                  uint32_t wm, uint32_t wn, uint32_t lane,
                                                  unsigned char* lds) {
        f2* pair = (f2*)lds;                              // [WN][BM]
        uint32_t* targets = (uint32_t*)(pair + S::WN * S::BM);  // [BM]
        static_assert(S::kThreads >= S::BM && S::BM * (8 * S::WN + 4) <= S::kLds, "fits");
        if (threadIdx.x < S::BM)
            targets[threadIdx.x] = mine.target;
        __syncthreads();
        const uint32_t nw = n0 + wn * (S::BN / S::WN) + (lane >> 4) * 4;
        const bool whole = n0 + S::BN <= N;
        const float factor = base2(e.scale.unit);
#pragma unroll
        for (int i = 0; i < S::MI; ++i) {
            const uint32_t r = wm * (S::BM / S::WM) + i * 16 + (lane & 15), m = m0 + r;
#pragma unroll
            for (int j = 0; j < S::NI; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[i][j][k] *= e.scale.pre;
                    if (!whole)
                        acc[i][j][k] =
                            nw + j * 16 + k < N ? acc[i][j][k] : -__builtin_inff();
                }
            // The target's sum stands apart.  Few waves hold a target of their 16 rows.
            const uint32_t target = m < M && targets[r] < N ? targets[r] : 0xFFFFFFFFu;
            const uint32_t off = target - nw;
            const bool here = off < S::NI * 16 && (off & 15) < 4;
            if (__builtin_amdgcn_ballot_w64(here)) {
                float z = 0.0f;
#pragma unroll
                for (int j = 0; j < S::NI; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bool it = off == j * 16 + k;
                        z = it ? acc[i][j][k] : z;
                        acc[i][j][k] = it ? -__builtin_inff() : acc[i][j][k];
                    }
                if (here)
                    e.z_target[m] = z;
            }
            float top = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < S::NI; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    top = __builtin_fmaxf(top, acc[i][j][k]);
            top = __builtin_fmaxf(top, __shfl_xor(top, 16));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            const float ref = reference(top);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < S::NI; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sum += relative(factor, acc[i][j][k], ref);
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (lane < 16)
                pair[wn * S::BM + r] = f2{top, sum};
        }
        __syncthreads();
        for (uint32_t r = threadIdx.x; r < S::BM; r += S::kThreads) {
            float top = pair[r].x;
#pragma unroll
            for (int w = 1; w < S::WN; ++w)
                top = __builtin_fmaxf(top, pair[w * S::BM + r].x);
            const float ref = reference(top);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < S::WN; ++w)
                sum += rebased(factor, pair[w * S::BM + r], ref);
            if (m0 + r < M)
                e.part[(uint64_t)(n0 / S::BN) * e.ld + m0 + r] = f2{top, sum};
        }
    }
};

struct JoinArgs {
    const f2* part;
    uint64_t ld;
    uint32_t tiles, first, last, n_tok, rows;
    f2* run;
    const float* z_target;
    const uint32_t *list, *count;  // of the tokens that count, or NULL: all tokens, by
    const void* ids;               // their ids
    uint32_t id64;
    float *loss, *lse;
    float unit;
};

// Joins a piece's tiles with what earlier pieces gave.  ROWS tokens a workgroup,
// K = 256 / ROWS threads each: thread k takes tiles k, k + K, ..., and the threads'
// pairs are joined by halves.
template <uint32_t ROWS>
__global__ __launch_bounds__(256) void join_kernel(JoinArgs a) {
    constexpr uint32_t K = 256 / ROWS;
    __shared__ f2 part[K][ROWS];
    const uint32_t row = threadIdx.x % ROWS, k = threadIdx.x / ROWS;
    const uint32_t m = blockIdx.x * ROWS + row;
    const uint32_t count = a.count ? *a.count : a.n_tok;
    f2 mine = {-__builtin_inff(), 0.0f};
    const float factor = base2(a.unit);
    auto add = [&mine, factor](f2 p) {
        const float top = __builtin_fmaxf(mine.x, p.x), ref = reference(top);
        mine = f2{top, rebased(factor, mine, ref) + rebased(factor, p, ref)};
    };
    if (m < count) {
        uint32_t t = k;
        for (; t + 3 * K < a.tiles; t += 4 * K) {  // four loads under way
            f2 p[4];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                p[j] = a.part[(t + j * K) * a.ld + m];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                add(p[j]);
        }
        for (; t < a.tiles; t += K)
            add(a.part[t * a.ld + m]);
    }
#pragma unroll
    for (uint32_t h = K / 2; h > 0; h /= 2) {
        part[k][row] = mine;
        __syncthreads();
        if (k < h)
            add(part[k + h][row]);
        __syncthreads();
    }
    if (k != 0 || m >= count)
        return;
    if (!a.first)
        add(a.run[m]);
    if (!a.last) {
        a.run[m] = mine;
        return;
    }
    uint32_t t = m;
    if (a.list) {
        t = a.list[m];
    } else {
        uint64_t id[1];
        load_ids<1>(a.ids, a.id64, [&](int) { return m; }, id);
        if (id[0] >= a.rows) {
            a.lse[t] = 0.0f;
            a.loss[t] = 0.0f;
            return;
        }
    }
    const float z = a.z_target[m];
    float loss, lse;
    if (__builtin_fabsf(z) < __builtin_inff() && mine.x < __builtin_inff()) {
        if (z >= mine.x) {
            loss = log1pf(mine.y * relative(factor, mine.x, z));
            lse = __builtin_fmaf(a.unit, z, loss);
        } else {
            const float l = logf(mine.y + relative(factor, z, mine.x));
            loss = __builtin_fmaf(a.unit, mine.x - z, l);
            lse = __builtin_fmaf(a.unit, mine.x, l);
        }
    } else {  // infinite or NaN: what the formula gives
        const float ref = reference(__builtin_fmaxf(mine.x, z));
        const float sum = rebased(factor, mine, ref) + relative(factor, z, ref);
        lse = __builtin_fmaf(a.unit, ref, logf(sum));
        loss = lse - a.unit * z;
    }
    a.lse[t] = lse;
    a.loss[t] = loss;
}

// Up to this many tokens the loss is formed for all of them, also those that are left
// out: no tile's worth of work is saved by gathering, and its launch is (a token, 4096
// x 32000: 67 us in place of 77).
constexpr uint32_t kAllTokens = 512;

// Whether the hidden states are read where they lie (else staged): rows whose width is a
// whole number of steps, within the 4 GiB that a list's rows may span.
bool x_in_place(uint32_t n_tok, uint32_t dim) {
    return dim % kMmK == 0 && (n_tok <= kAllTokens || (uint64_t)n_tok * dim * 2 < (uint64_t)1 << 32);
}

CeLayout layout(uint32_t n_tok, uint32_t rows, uint32_t dim, uint64_t piece) {
    CeLayout l = {};
    l.kp = round_up(dim, kMmK);
    l.parts = 1;
    const uint64_t n_pad = round_up(n_tok, 256);
    // The library's choice: at most 256 MiB of staged rows, and of pairs 128 (256-tiles),
    // 256 or 512 MiB (small tiles).
    uint64_t most = piece ? round_up(std::min<uint64_t>(piece, rows), 256)
                          : std::min(((uint64_t)1 << 27) / l.kp, ((uint64_t)1 << 32) / n_pad);
    most = std::min(most, ((uint64_t)1 << 36) / n_pad);
    ce_pieces(l, rows, most);
    l.logits = mm_plan(n_tok, l.piece, l.kp, false);
    CeTake take;
    ce_take_tokens(l, take, n_tok, false);
    l.part = take(div_up(l.piece, tile_cols(l.logits.kind)) * n_pad * 8);
    l.run = take(n_pad * 8);
    l.z_target = take(n_pad * 4);
    l.total = take.at;
    return l;
}

template <int T>
hipError_t launch(const CeArgs& a, int w_type, hipStream_t stream) {
    const CeLayout l = layout(a.n_tok, a.rows, a.dim, a.piece);
    char* ws = (char*)a.workspace;
    const CeTokens tok = ce_tokens(l, ws);
    const bool all = a.n_tok <= kAllTokens && x_in_place(a.n_tok, a.dim);
    hipError_t st = all ? hipSuccess : ce_prep<false>(a, tok, false, stream);
    const uint32_t* count = all ? nullptr : &tok.scalars->count;
    for (uint32_t i = 0; i < l.n_pieces && st == hipSuccess; ++i) {
        const uint32_t v0 = i * l.piece, n = l.rows_of(i, a.rows);
        MmArgs m = {};
        st = ce_stage<T>(a, w_type, l, i, !x_in_place(a.n_tok, a.dim), tok, ws, stream);
        if (st != hipSuccess)
            break;
        m.b = ce_piece(a, w_type, l, v0, ws);
        m.a = {(const uint16_t*)(ws + l.x), l.kp};
        if (x_in_place(a.n_tok, a.dim)) {
            m.a.p = (const uint16_t*)a.x;
            m.a_rows = all ? nullptr : tok.list;
        }
        m.M = a.n_tok;
        m.N = n;
        m.K = (uint32_t)l.kp;
        m.dyn_m = count;
        Stats::Args e = {ce_scale(a.scale),
                         (f2*)(ws + l.part),
                         round_up(a.n_tok, 256),
                         v0,
                         (float*)(ws + l.z_target),
                         all ? nullptr : tok.target,
                         a.ids,
                         a.id64};
        st = launch_mm<T, false, false, Stats>(m, e, l.logits, stream);
        if (st != hipSuccess)
            break;
        JoinArgs j = {e.part, e.ld, (uint32_t)div_up(n, tile_cols(l.logits.kind)), i == 0,
                      i + 1 == l.n_pieces, a.n_tok, a.rows, (f2*)(ws + l.run), e.z_target,
                      all ? nullptr : tok.list, count, a.ids, a.id64, a.loss, a.lse_out,
                      e.scale.unit};
        void* args[] = {&j};
        // Few tokens: more threads each, so that no thread walks a long line of tiles.
        const uint32_t rows = a.n_tok <= 512 ? 2 : 16;
        st = hipLaunchKernel(rows == 2 ? (const void*)&join_kernel<2> : (const void*)&join_kernel<16>,
                             dim3((a.n_tok + rows - 1) / rows), dim3(256), args, 0, stream);
    }
    return st;
}

}  // namespace

size_t ce_loss_workspace(uint32_t n_tok, uint32_t rows, uint32_t dim, uint64_t piece) {
    return layout(n_tok, rows, dim, piece).total;
}

hipError_t launch_ce_loss(const CeArgs& a, int type, int w_type, hipStream_t stream) {
    return type == kBF16 ? launch<kBF16>(a, w_type, stream) : launch<kF16>(a, w_type, stream);
}

}  // namespace zq
