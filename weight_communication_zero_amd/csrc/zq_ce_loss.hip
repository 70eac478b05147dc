// zq_ce_loss.hip -- softmax cross entropy of the vocabulary projection.
//
// The logits of a tile of tokens x vocabulary stay in the matrix product's
// registers: the epilogue takes each token's maximum m over the tile's columns, the
// sum s of exp(z - m), and the target's logit where it lies there.  A second kernel
// joins the tiles' pairs,  (m, s) + (m', s') = (M, s e^(m-M) + s' e^(m'-M)).
#include "zq_ce.h"

namespace zq {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));

// What the exponentials are taken relative to: the maximum, where it is finite (an
// infinite one would give inf - inf).
__device__ __forceinline__ float reference(float m) {
    return __builtin_fabsf(m) < __builtin_inff() ? m : 0.0f;
}

// A pair's sum relative to another reference.  With an infinite maximum the sum is
// 0, infinity or NaN, and stays so.
__device__ __forceinline__ float rebased(f2 p, float ref) {
    return __builtin_fabsf(p.x) < __builtin_inff() ? p.y * exp_of(p.x - ref) : p.y;
}

struct Stats {
    struct Args {
        float scale;
        f2* part;          // [tile of the piece][ld]
        uint64_t ld;
        const uint32_t* target;
        uint32_t v0;       // the piece's first row
        float* z_target;
    };

    using Row = MmNoRow;
    static __device__ __forceinline__ Row row(const Args&, uint32_t, uint32_t, uint32_t) {
        return {};
    }

    template <class S>
    static __device__ __forceinline__ void finish(const Args& e, const Row&,
                                                  f4 (&acc)[S::MI][S::NI], uint32_t M, uint32_t N,
                                                  uint32_t m0, uint32_t n0, uint32_t wm,
                                                  uint32_t wn, uint32_t lane, unsigned char* lds) {
        f2* pair = (f2*)lds;  // [WN][BM]
        const uint32_t nw = n0 + wn * (S::BN / S::WN) + (lane >> 4) * 4;
#pragma unroll
        for (int i = 0; i < S::MI; ++i) {
            const uint32_t r = wm * (S::BM / S::WM) + i * 16 + (lane & 15), m = m0 + r;
            uint32_t target = m < M ? e.target[m] - e.v0 : N;
            target = target < N ? target : 0xFFFFFFFFu;
            float top = -__builtin_inff(), z_target = 0.0f;
#pragma unroll
            for (int j = 0; j < S::NI; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t n = nw + j * 16 + k;
                    const float z = e.scale * acc[i][j][k];
                    acc[i][j][k] = n < N ? z : -__builtin_inff();
                    if (n < N)
                        top = __builtin_fmaxf(top, z);
                    z_target = n == target ? z : z_target;
                }
            const uint32_t off = target - nw;
            if (off < S::NI * 16 && (off & 15) < 4)
                e.z_target[m] = z_target;
            top = __builtin_fmaxf(top, __shfl_xor(top, 16));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            const float ref = reference(top);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < S::NI; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sum += exp_of(acc[i][j][k] - ref);
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
                sum += rebased(pair[w * S::BM + r], ref);
            if (m0 + r < M)
                e.part[(uint64_t)(n0 / S::BN) * e.ld + m0 + r] = f2{top, sum};
        }
    }
};

struct JoinArgs {
    const f2* part;
    uint64_t ld;
    uint32_t tiles, first, last;
    f2* run;
    const float* z_target;
    CeTokens t;
    float *loss, *lse;
};

// Joins a piece's tiles with what earlier pieces gave.  16 tokens a workgroup, 16
// threads each: thread k takes tiles k, k + 16, ...
__global__ __launch_bounds__(256) void join_kernel(JoinArgs a) {
    __shared__ f2 part[16][17];
    const uint32_t row = threadIdx.x & 15, k = threadIdx.x >> 4;
    const uint32_t m = blockIdx.x * 16 + row, count = a.t.scalars->count;
    f2 mine = {-__builtin_inff(), 0.0f};
    auto add = [&mine](f2 p) {
        const float top = __builtin_fmaxf(mine.x, p.x), ref = reference(top);
        mine = f2{top, rebased(mine, ref) + rebased(p, ref)};
    };
    if (m < count)
        for (uint32_t t = k; t < a.tiles; t += 16)
            add(a.part[t * a.ld + m]);
    part[k][row] = mine;
    __syncthreads();
    if (k != 0 || m >= count)
        return;
    for (int j = 1; j < 16; ++j)
        add(part[j][row]);
    if (!a.first)
        add(a.run[m]);
    if (!a.last) {
        a.run[m] = mine;
        return;
    }
    const float ref = reference(mine.x), log_sum = logf(mine.y);
    const uint32_t t = a.t.list[m];
    a.lse[t] = ref + log_sum;
    a.loss[t] = (ref - a.z_target[m]) + log_sum;
}

CeLayout layout(uint32_t n_tok, uint32_t rows, uint32_t dim, uint64_t piece) {
    CeLayout l = {};
    l.kp = round_up(dim, kMmK);
    const uint64_t n_pad = round_up(n_tok, 256);
    // The library's choice: 256 MiB each of staged rows and of pairs.
    uint64_t most = piece ? round_up(std::min<uint64_t>(piece, rows), 256)
                          : std::min(((uint64_t)1 << 27) / l.kp, ((uint64_t)1 << 32) / n_pad);
    most = std::min(most, ((uint64_t)1 << 36) / n_pad);
    ce_pieces(l, rows, most);
    l.logits = mm_plan(n_tok, l.piece, l.kp, false);
    CeTake take;
    ce_take_tokens(l, take, n_tok, false);
    l.part = take(div_up(l.piece, tile_edge(l.logits.kind)) * n_pad * 8);
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
    hipError_t st = ce_prep(a, tok, false, stream);
    if (st == hipSuccess)
        st = ce_stage_x<T>(a, l, tok, ws, stream);
    for (uint32_t i = 0; i < l.n_pieces && st == hipSuccess; ++i) {
        const uint32_t v0 = i * l.piece, n = l.rows_of(i, a.rows);
        MmArgs m = {};
        st = ce_piece<T>(a, w_type, l, v0, n, ws, &m.b, stream);
        if (st != hipSuccess)
            break;
        m.a = {(const uint16_t*)(ws + l.x), l.kp};
        m.M = a.n_tok;
        m.N = n;
        m.K = (uint32_t)l.kp;
        m.dyn_m = &tok.scalars->count;
        Stats::Args e = {a.scale, (f2*)(ws + l.part), round_up(a.n_tok, 256), tok.target, v0,
                         (float*)(ws + l.z_target)};
        st = launch_mm<T, false, false, Stats>(m, e, l.logits, stream);
        if (st != hipSuccess)
            break;
        JoinArgs j = {e.part, e.ld, (uint32_t)div_up(n, tile_edge(l.logits.kind)), i == 0,
                      i + 1 == l.n_pieces, (f2*)(ws + l.run), e.z_target, tok, a.loss, a.lse_out};
        void* args[] = {&j};
        st = hipLaunchKernel((const void*)&join_kernel, dim3((a.n_tok + 15) / 16), dim3(256), args,
                             0, stream);
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
