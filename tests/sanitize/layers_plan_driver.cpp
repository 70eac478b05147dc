// layers_plan_driver.cpp -- the host side of the layer kernels' launches (tiles and splits,
// pieces, the workspace's parts, grids) under AddressSanitizer and
// UndefinedBehaviorSanitizer, without a GPU.  hipLaunchKernel is a stub here: it looks at
// each launch's arguments and checks that everything the kernel addresses lies in the
// buffer, or in the part of the workspace, that it is meant for, that offsets which the
// kernels hold in 32 bits fit, and that the grid covers the work and stays in range.
// Buffers are fake addresses that are never dereferenced.  Test infrastructure only
// (built and run by tests/test_layers_plan.py); PART says which of the three calls.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#if PART == 0
#include "../../weight_communication_zero_amd/csrc/zq_linear_grad.hip"
#elif PART == 1
#include "../../weight_communication_zero_amd/csrc/zq_ce_loss.hip"
#else
#include "../../weight_communication_zero_amd/csrc/zq_ce_grad.hip"
#endif

namespace {

int failures = 0;
uint64_t launches = 0, calls = 0;
char now[256];

#define CHECK(c)                                                                                \
    do {                                                                                        \
        if (!(c) && ++failures < 20)                                                            \
            std::fprintf(stderr, "check failed at line %d: %s (%s)\n", __LINE__, #c, now);      \
    } while (0)

struct Region {
    const char* name;
    uint64_t lo, hi;
};
std::vector<Region> regions;

void region(const char* name, uint64_t lo, uint64_t bytes) { regions.push_back({name, lo, lo + bytes}); }

// [p, p + bytes) lies in the region of one of these names ("a|b").
void inside(const void* p, uint64_t bytes, const char* names, int line) {
    const uint64_t lo = (uint64_t)(uintptr_t)p;
    for (const char* name = names; name; name = std::strchr(name, '|') ? std::strchr(name, '|') + 1 : nullptr) {
        const size_t length = std::strcspn(name, "|");
        for (const Region& r : regions)
            if (std::strlen(r.name) == length && !std::strncmp(r.name, name, length) && r.lo <= lo &&
                lo + bytes <= r.hi && lo + bytes >= lo)
                return;
    }
    if (++failures < 20)
        std::fprintf(stderr, "line %d: %llu bytes do not lie in %s (%s)\n", line,
                     (unsigned long long)bytes, names, now);
}
#define INSIDE(p, bytes, names) inside(p, bytes, names, __LINE__)

constexpr uint64_t k32 = (uint64_t)1 << 32;
using namespace zq;
constexpr int T = kBF16;
uint64_t n_tok, wide;  // of the call: tokens, stored width of the hidden states

void grid_ok(dim3 grid, dim3 block) {
    CHECK(grid.y == 1 && grid.z == 1 && grid.x >= 1);
    CHECK((uint64_t)grid.x * block.x < k32);
}

void operand(const MmOperand& o, bool tr, uint64_t rows, uint64_t cols, uint64_t K, bool listed,
             const char* names) {
    CHECK((uintptr_t)o.p % 16 == 0 && o.ld % 8 == 0 && o.ld < k32);
    if (tr) {
        CHECK(cols % 8 == 0 && cols >= rows && cols <= o.ld);
        CHECK(63 * o.ld * 2 + 512 < k32);
        INSIDE(o.p, ((K - 1) * o.ld + cols) * 2, names);
    } else {
        CHECK(round_up(K, kMmK) <= o.ld);
        CHECK((listed ? rows : 256) * o.ld * 2 <= k32);
        INSIDE(o.p, ((rows - 1) * o.ld + round_up(K, kMmK)) * 2, names);
    }
}

// The product's grid and operands.
uint64_t product(const MmArgs& a, int kind, bool ta, bool tb, const char* in_a, const char* in_b) {
    CHECK(a.M && a.N && a.K);
    const uint64_t tiles = div_up(a.M, tile_rows(kind)) * div_up(a.N, tile_cols(kind));
    CHECK(a.wgs % 8 == 0 && a.wgs >= tiles && a.wgs < tiles + 8);
    CHECK(a.splits >= 1 && a.splits <= kMaxSplits);
    CHECK(ta || tb || a.K % kMmK == 0);
    CHECK(!(a.a_rows && ta));
    operand(a.a, ta, a.M, a.a_cols, a.K, a.a_rows != nullptr, in_a);
    operand(a.b, tb, a.N, a.b_cols, a.K, false, in_b);
    if (a.a_rows)
        INSIDE(a.a_rows, a.M * 4ull, "list");
    for (const uint32_t* d : {a.dyn_m, a.dyn_k})
        if (d)
            INSIDE(d, 4, "scalars");
    return (uint64_t)a.wgs * a.splits;
}

void sums(const MmSum::Args& e, const MmArgs& a, const char* parts, const char* out) {
    const uint64_t M = a.M >> e.pairs, elem = e.o.type == kF32 ? 4 : 2;
    CHECK((e.part != nullptr) == (a.splits > 1));
    if (e.part) {
        CHECK(e.ld % 4 == 0 && e.ld >= a.N && e.rows >= M && (uintptr_t)e.part % 16 == 0);
        INSIDE(e.part, ((a.splits - 1) * e.rows + M) * e.ld * 4, parts);
    }
    for (const float* p : {e.o.acc_in, (const float*)e.o.acc_out})
        if (p) {
            CHECK(e.o.ldacc % 4 == 0 && e.o.ldacc >= a.N);
            INSIDE(p, M * e.o.ldacc * 4, "acc");
        }
    if (!e.o.acc_out)
        INSIDE(e.o.out, ((M - 1) * e.o.ldo + a.N) * elem, out);
    if (e.o.list)
        INSIDE(e.o.list, M * 4, "list");
    if (e.o.factor)
        INSIDE(e.o.factor, 4, "scalars");
}

void staged(const StageArgs& a, uint64_t wgs, int in) {
    CHECK(a.ld % 8 == 0 && a.ld >= a.dim && a.rows && wgs >= 1);
    const uint64_t rows = (uint64_t)a.rows << a.twice;
    INSIDE(a.out, rows * a.ld * 2, a.list || (PART == 0 && in == kQ8) ? "x" : PART == 0 ? "dy_staged" : "w");
    const uint64_t n = a.list ? n_tok * a.dim : (a.row0 + a.rows) * a.dim;
    INSIDE(a.src, n * (in == kQ8 ? 1 : 2), a.list ? "in_x" : PART == 0 && in != kQ8 ? "in_dy" : "in_w");
    if (in == kQ8)
        INSIDE(a.scales, (((n - 1) >> a.log2b) + 1) * 4, "in_scales");
    if (a.list) {
        INSIDE(a.list, a.rows * 4ull, "list");
        INSIDE(a.count, 4, "scalars");
    }
    if (a.clear)
        INSIDE(a.clear, n * 2, "out_dx");
}

template <int IN, bool W>
bool staged_alone(const void* fn, dim3 grid, void** args) {
    if (fn != (const void*)&stage_kernel<T, IN, W>)
        return false;
    const StageArgs& a = *(const StageArgs*)args[0];
    CHECK(!W || a.dim % 8 == 0);
    staged(a, grid.x, IN);
    return true;
}
template <int IN1, bool W1, int IN2, bool W2>
bool staged_both(const void* fn, dim3 grid, void** args) {
    if (fn != (const void*)&stage_both_kernel<T, IN1, W1, IN2, W2>)
        return false;
    const StageArgs &a = *(const StageArgs*)args[0], &b = *(const StageArgs*)args[1];
    const uint64_t wgs = *(const uint32_t*)args[2];
    CHECK((!W1 || a.dim % 8 == 0) && (!W2 || b.dim % 8 == 0) && wgs < grid.x);
    staged(a, wgs, IN1);
    staged(b, grid.x - wgs, IN2);
    return true;
}
template <int IN1, int IN2>
bool any_both(const void* fn, dim3 grid, void** args) {
    return staged_both<IN1, true, IN2, true>(fn, grid, args) ||
           staged_both<IN1, true, IN2, false>(fn, grid, args) ||
           staged_both<IN1, false, IN2, true>(fn, grid, args) ||
           staged_both<IN1, false, IN2, false>(fn, grid, args);
}
bool any_stage(const void* fn, dim3 grid, void** args) {
    return staged_alone<kQ8, true>(fn, grid, args) || staged_alone<kQ8, false>(fn, grid, args) ||
           staged_alone<T, true>(fn, grid, args) || staged_alone<T, false>(fn, grid, args) ||
           any_both<kQ8, T>(fn, grid, args)
#if PART > 0
           || any_both<T, T>(fn, grid, args)
#endif
        ;
}

template <bool TA, bool TB, class Epi>
int kind_of(const void* fn) {
    return fn == (const void*)&mm_kernel<MmShape256<T, TA, TB>, Epi>     ? kTile256
           : fn == (const void*)&mm_kernel<MmShape128<T, TA, TB>, Epi>   ? kTile128
           : fn == (const void*)&mm_kernel<MmShapeSmall<T, TA, TB>, Epi> ? kTileSmall
                                                                         : -1;
}

void joined(void** args, const char* parts, const char* out) {
    const MmSum::Args& e = *(const MmSum::Args*)args[0];
    MmArgs a = {};
    a.splits = *(const uint32_t*)args[1];
    a.M = *(const uint32_t*)args[2];
    a.N = *(const uint32_t*)args[3];
    CHECK(a.splits > 1);
    sums(e, a, parts, out);
}

#if PART == 0
void launch_ok(const void* fn, dim3 grid, dim3 block, void** args) {
    if (any_stage(fn, grid, args))
        return;
    if (fn == (const void*)&mm_join_kernel)
        return joined(args, "part", "out_grad");
    const int kind = kind_of<true, true, MmSum>(fn);
    CHECK(kind >= 0);
    if (kind < 0)
        return;
    const MmArgs& a = *(const MmArgs*)args[0];
    CHECK(product(a, kind, true, true, "in_dy|dy_staged", "x") == grid.x && block.x == tile_threads(kind));
    sums(*(const MmSum::Args*)args[1], a, "part", "out_grad");
}
#else
template <bool GRAD>
bool prepared(const void* fn, void** args) {
    if (fn != (const void*)&ce_prep_kernel<GRAD, 1> && fn != (const void*)&ce_prep_kernel<GRAD, 8>)
        return false;
    const CePrepArgs& p = *(const CePrepArgs*)args[0];
    CHECK(p.n_tok == n_tok);
    INSIDE(p.t.scalars, sizeof(CeScalars), "scalars");
    INSIDE(p.t.list, n_tok * 4, "list");
    INSIDE(p.t.target, n_tok * 4, "target");
    if (GRAD) {
        INSIDE(p.t.lse, n_tok * 4, "lse");
        INSIDE(p.t.dloss, n_tok * 4, "dloss");
    }
    return true;
}
#endif

#if PART == 1
void launch_ok(const void* fn, dim3 grid, dim3 block, void** args) {
    if (any_stage(fn, grid, args) || prepared<false>(fn, args))
        return;
    if (fn == (const void*)&join_kernel<2> || fn == (const void*)&join_kernel<16>) {
        const JoinArgs& j = *(const JoinArgs*)args[0];
        const uint64_t rows = fn == (const void*)&join_kernel<2> ? 2 : 16;
        CHECK(grid.x * rows >= n_tok && block.x == 256 && j.tiles >= 1);
        INSIDE(j.part, ((j.tiles - 1) * j.ld + n_tok) * 8, "part");
        INSIDE(j.run, n_tok * 8, "run");
        INSIDE(j.z_target, n_tok * 4, "z_target");
        if (j.list)
            INSIDE(j.list, n_tok * 4, "list");
        return;
    }
    const int kind = kind_of<false, false, Stats>(fn);
    CHECK(kind >= 0);
    if (kind < 0)
        return;
    const MmArgs& a = *(const MmArgs*)args[0];
    const Stats::Args& e = *(const Stats::Args*)args[1];
    CHECK(product(a, kind, false, false, "in_x|x", "in_w|w") == grid.x && block.x == tile_threads(kind));
    CHECK(a.splits == 1 && e.ld >= a.M);
    INSIDE(e.part, ((a.N - 1) / tile_cols(kind) * e.ld + a.M) * 8, "part");
    INSIDE(e.z_target, a.M * 4ull, "z_target");
}
#elif PART == 2
template <int KIND, class S1, class S2>
bool paired(const void* fn, dim3 grid, dim3 block, void** args) {
    if (fn != (const void*)&mm_pair_kernel<S1, S2, MmSum>)
        return false;
    const MmArgs &a = *(const MmArgs*)args[0], &b = *(const MmArgs*)args[2];
    const uint64_t wgs = product(a, KIND, false, true, "q", "in_w|w") +
                         product(b, KIND, true, true, "q", "x");
    CHECK(wgs == grid.x && block.x == tile_threads(KIND));
    sums(*(const MmSum::Args*)args[1], a, "x_sums", "out_dx");
    sums(*(const MmSum::Args*)args[3], b, "w_sums", "out_dw");
    return true;
}
void launch_ok(const void* fn, dim3 grid, dim3 block, void** args) {
    if (any_stage(fn, grid, args) || prepared<true>(fn, args))
        return;
    if (fn == (const void*)&mm_join_kernel)
        return joined(args, "x_sums|w_sums", "out_dx|out_dw");
    if (paired<kTile256, MmShape256<T, false, true>, MmShape256<T, true, true>>(fn, grid, block, args) ||
        paired<kTile128, MmShape128<T, false, true>, MmShape128<T, true, true>>(fn, grid, block, args) ||
        paired<kTileSmall, MmShapeSmall<T, false, true>, MmShapeSmall<T, true, true>>(fn, grid, block, args))
        return;
    const MmArgs& a = *(const MmArgs*)args[0];
    int kind = kind_of<false, false, Residual>(fn);
    if (kind >= 0) {
        const Residual::Args& e = *(const Residual::Args*)args[1];
        CHECK(product(a, kind, false, false, "x", "in_w|w") == grid.x && block.x == tile_threads(kind));
        CHECK(a.splits == 1 && e.ldq % 64 == 0 && e.ldq >= round_up(a.N, 64));
        INSIDE(e.q, ((a.M * (uint64_t)e.parts - 1) * e.ldq + round_up(a.N, 64)) * 2, "q");
        return;
    }
    kind = kind_of<false, true, MmSum>(fn);
    if (kind >= 0) {
        CHECK(product(a, kind, false, true, "q", "in_w|w") == grid.x && block.x == tile_threads(kind));
        return sums(*(const MmSum::Args*)args[1], a, "x_sums", "out_dx");
    }
    kind = kind_of<true, true, MmSum>(fn);
    CHECK(kind >= 0);
    if (kind >= 0) {
        CHECK(product(a, kind, true, true, "q", "x") == grid.x && block.x == tile_threads(kind));
        sums(*(const MmSum::Args*)args[1], a, "w_sums", "out_dw");
    }
}
#endif

std::mt19937_64 rng(1);
uint64_t upto(uint64_t n) { return rng() % (n + 1); }
// From 1 to `most`, over its logarithm, now and then a power of two, its neighbours or the
// end.
uint64_t size(uint64_t most) {
    int bits = 0;
    while ((uint64_t)2 << bits <= most)
        ++bits;
    uint64_t v = ((uint64_t)1 << upto(bits));
    switch (upto(5)) {
        case 0: break;
        case 1: v -= 1; break;
        case 2: v += 1; break;
        case 3: v = most - (upto(1) ? 0 : upto(most < 300 ? most - 1 : 299)); break;
        default: v += upto(v);
    }
    return v < 1 ? 1 : v > most ? most : v;
}

constexpr uint64_t kAt = (uint64_t)1 << 50;
void* at(int i) { return (void*)(uintptr_t)(kAt * i); }

struct Part {
    const char* name;
    uint64_t lo;
};
// The workspace's parts in the order in which they were taken.
void parts(std::vector<Part> p, uint64_t total) {
    for (size_t i = 0; i < p.size(); ++i) {
        const uint64_t hi = i + 1 < p.size() ? p[i + 1].lo : total;
        CHECK(p[i].lo <= hi && p[i].lo % 256 == 0);
        region(p[i].name, kAt * 1 + p[i].lo, hi - p[i].lo);
    }
}

// False where the call would be one of more launches than the test has time for (their
// pieces are all alike but for the last).
bool one(uint64_t n, uint64_t b, uint64_t c, uint64_t piece, bool q8, int which, uint32_t log2b,
         uint32_t most_pieces) {
#if PART > 0
    if (layout((uint32_t)n, (uint32_t)b, (uint32_t)c, piece).n_pieces > most_pieces)
        return false;
#else
    (void)most_pieces;
#endif
    std::snprintf(now, sizeof now, "tokens %llu, %llu x %llu, piece %llu, q8 %d, which %d",
                  (unsigned long long)n, (unsigned long long)b, (unsigned long long)c,
                  (unsigned long long)piece, (int)q8, which);
    regions.clear();
    n_tok = n;
    ++calls;
#if PART == 0
    const uint64_t o = b, i = c;
    (void)piece, (void)q8;
    const Layout l = layout((uint32_t)n, (uint32_t)o, (uint32_t)i);
    CHECK(l.total == linear_grad_workspace((uint32_t)n, (uint32_t)o, (uint32_t)i));
    parts({{"x", l.x}, {"dy_staged", l.dy}, {"part", l.part}}, l.total);
    region("in_dy", kAt * 2, n * o * 2);
    region("in_w", kAt * 3, n * i);
    region("in_scales", kAt * 4, (((n * i - 1) >> log2b) + 1) * 4);
    const int type = which % 2 ? kF32 : kBF16;
    region("out_grad", kAt * 5, o * i * (type == kF32 ? 4 : 2));
    const LinearGradArgs a = {at(2), (const int8_t*)at(3), (const float*)at(4), log2b, (uint32_t)n,
                              (uint32_t)o, (uint32_t)i, at(5), at(1)};
    CHECK(launch_linear_grad(a, T, type, which / 2, nullptr) == hipSuccess);
#else
    const uint64_t rows = b, dim = c;
    CeArgs a = {};
    a.x = at(2);
    a.n_tok = (uint32_t)n;
    a.dim = (uint32_t)dim;
    a.rows = (uint32_t)rows;
    a.w = at(3);
    a.w_scales = (const float*)at(4);
    a.log2b = log2b;
    a.ids = at(6);
    a.scale = 1.0f;
    a.piece = piece;
    a.workspace = at(1);
    region("in_x", kAt * 2, n * dim * 2);
    region("in_w", kAt * 3, rows * dim * (q8 ? 1 : 2));
    region("in_scales", kAt * 4, (((rows * dim - 1) >> log2b) + 1) * 4);
    const CeLayout l = layout((uint32_t)n, (uint32_t)rows, (uint32_t)dim, piece);
    CHECK(l.piece % 256 == 0 && (uint64_t)l.piece * l.n_pieces >= rows);
    CHECK((uint64_t)l.piece * (l.n_pieces - 1) < rows && l.kp % 64 == 0 && l.kp >= dim);
#if PART == 1
    (void)which;
    CHECK(l.total == ce_loss_workspace((uint32_t)n, (uint32_t)rows, (uint32_t)dim, piece));
    parts({{"scalars", l.scalars}, {"list", l.list}, {"target", l.target}, {"lse", l.lse}, {"dloss", l.dloss},
           {"x", l.x}, {"w", l.w}, {"part", l.part}, {"run", l.run}, {"z_target", l.z_target}}, l.total);
    a.loss = (float*)at(7);
    a.lse_out = (float*)at(8);
    CHECK(launch_ce_loss(a, T, q8 ? kQ8 : T, nullptr) == hipSuccess);
#else
    CHECK(l.total == ce_grad_workspace((uint32_t)n, (uint32_t)rows, (uint32_t)dim, piece));
    parts({{"scalars", l.scalars}, {"list", l.list}, {"target", l.target}, {"lse", l.lse}, {"dloss", l.dloss},
           {"x", l.x}, {"w", l.w}, {"q", l.q}, {"acc", l.acc}, {"x_sums", l.x_sums}, {"w_sums", l.w_sums}},
          l.total);
    const int type = which % 2 ? kF32 : kBF16;
    if (which / 2 != 1) {
        a.dx = at(9);
        region("out_dx", kAt * 9, n * dim * 2);
    }
    if (which / 2 != 2) {
        a.dw = at(10);
        region("out_dw", kAt * 10, rows * dim * (type == kF32 ? 4 : 2));
    }
    a.lse = (const float*)at(7);
    a.dloss = (const float*)at(8);
    CHECK(launch_ce_grad(a, T, q8 ? kQ8 : T, type, which % 2, nullptr) == hipSuccess);
#endif
#endif
    return true;
}

}  // namespace

extern "C" {
hipError_t hipLaunchKernel(const void* fn, dim3 grid, dim3 block, void** args, size_t shared, hipStream_t) {
    ++launches;
    CHECK(shared == 0);
    grid_ok(grid, block);
    launch_ok(fn, grid, block, args);
    return hipSuccess;
}
// What the compiler's registration of the kernels calls.
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
hipError_t __hipPopCallConfiguration(dim3*, dim3*, size_t*, hipStream_t*) { return hipSuccess; }
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
}

int main() {
    const uint64_t most_n = (uint64_t)1 << 20, most_dim = (uint64_t)1 << 20, most_rows = (uint64_t)1 << 24,
                   most = (uint64_t)1 << 36;
    auto fits = [&](uint64_t n, uint64_t b, uint64_t c) {
        return n <= most_n && c <= most_dim &&
               (PART == 0 ? b <= most_dim && b * c <= most : b <= most_rows && n * c <= most);
    };
    // Every corner of the accepted sizes, then sizes from all over.
    for (uint64_t n : {(uint64_t)1, (uint64_t)128, (uint64_t)129, (uint64_t)513, (uint64_t)1 << 16, most_n})
        for (uint64_t b : {(uint64_t)1, (uint64_t)257, (uint64_t)50257, most_dim, most_rows - 1, most_rows})
            for (uint64_t c : {(uint64_t)1, (uint64_t)64, (uint64_t)513, (uint64_t)4096, (uint64_t)1 << 16, most_dim})
                for (uint64_t piece : {(uint64_t)0, (uint64_t)1, (uint64_t)1 << 20, UINT64_MAX})
                    if (fits(n, b, c))
                        one(n, b, c, piece, calls & 1, (int)(calls / 2 % 6), 5 + (uint32_t)upto(7), 5000);
    for (int k = 0; k < 20000;) {
        const uint64_t n = size(most_n), b = size(PART ? most_rows : most_dim), c = size(most_dim);
        if (!fits(n, b, c))
            continue;
        const uint64_t piece = upto(2) ? 0 : size(b);
        k += one(n, b, c, piece, upto(1), (int)upto(PART == 0 ? 3 : 5), 5 + (uint32_t)upto(7), 100);
    }
#ifdef ZQ_SANITIZER_CANARY
    std::vector<int> v(4);
    volatile size_t i = 4;
    std::printf("%d\n", v.data()[i]);
#endif
    CHECK(launches > 2 * calls);
    if (failures) {
        std::fprintf(stderr, "%d failures\n", failures);
        return 1;
    }
    std::printf("all checks passed: %llu calls, %llu launches\n", (unsigned long long)calls,
                (unsigned long long)launches);
    return 0;
}
