// zq_linear_grad.hip -- a linear layer's weight gradient from its input kept as
// int8 blocks:  grad[o, i] (+)= sum_t dy[t, o] x[t, i].
//
// Both operands lie with the summed index t outermost, so the product takes both as
// transposed operands: no transposed copy is made.  The kept input is dequantized
// once into the workspace (3 bytes an element) and read from there: of the 1.25 to 1.32 ms
// of 16384 tokens, 11008 -> 4096, that takes 0.09 (540 MB at 5.9 TB/s) and the product the
// rest (1.23 ms in a trace: 1200 TFLOP/s; its 688 tiles are 2.7 rounds of the 256 CUs, so
// 10 % of the CUs' time is idle in the third).
#include "zq_mm_plan.h"
#include "zq_stage.h"

namespace zq {
namespace {

struct Layout {
    uint64_t ldx, ldy;
    bool stage_dy;
    MmPlan plan;
    uint64_t x, dy, part, total;  // byte offsets
};

Layout layout(uint32_t n_tok, uint32_t out_dim, uint32_t in_dim) {
    Layout l;
    l.ldx = round_up(in_dim, 8);
    l.ldy = round_up(out_dim, 8);
    l.stage_dy = out_dim % 8 != 0;
    l.plan = mm_plan(out_dim, in_dim, n_tok, true);
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    l.x = take(n_tok * l.ldx * 2);
    l.dy = take(l.stage_dy ? n_tok * l.ldy * 2 : 0);
    l.part = take(part_floats(l.plan, out_dim, in_dim) * 4);
    l.total = at;
    return l;
}

template <int T>
hipError_t launch(const LinearGradArgs& a, int grad_type, int mode, hipStream_t stream) {
    const Layout l = layout(a.n_tok, a.out_dim, a.in_dim);
    char* ws = (char*)a.workspace;
    StageArgs s = {};
    s.src = a.codes;
    s.scales = a.scales;
    s.log2b = a.log2b;
    s.dim = a.in_dim;
    s.rows = a.n_tok;
    s.ld = (uint32_t)l.ldx;
    s.out = (uint16_t*)(ws + l.x);
    MmArgs m = {};
    m.a = {(const uint16_t*)a.dy, a.out_dim};
    hipError_t st;
    if (l.stage_dy) {
        StageArgs d = {};
        d.src = a.dy;
        d.dim = a.out_dim;
        d.rows = a.n_tok;
        d.ld = (uint32_t)l.ldy;
        d.out = (uint16_t*)(ws + l.dy);
        m.a = {d.out, l.ldy};
        st = launch_stage_both<T, kQ8, T>(s, d, stream);
    } else {
        st = launch_stage<T>(s, kQ8, stream);
    }
    if (st != hipSuccess)
        return st;
    m.b = {(const uint16_t*)(ws + l.x), l.ldx};
    m.M = a.out_dim;
    m.N = a.in_dim;
    m.K = a.n_tok;
    m.a_cols = (uint32_t)l.ldy;
    m.b_cols = (uint32_t)l.ldx;
    MmOut o = {};
    o.out = a.grad;
    o.ldo = a.in_dim;
    o.scale = 1.0f;
    o.type = grad_type;
    o.add = mode == kGradAdd;
    return launch_mm_sum<T, true, true>({m, o, l.plan, (float*)(ws + l.part)}, stream);
}

}  // namespace

size_t linear_grad_workspace(uint32_t n_tok, uint32_t out_dim, uint32_t in_dim) {
    return layout(n_tok, out_dim, in_dim).total;
}

hipError_t launch_linear_grad(const LinearGradArgs& a, int type, int grad_type, int mode,
                              hipStream_t stream) {
    return type == kBF16 ? launch<kBF16>(a, grad_type, mode, stream)
                         : launch<kF16>(a, grad_type, mode, stream);
}

}  // namespace zq
