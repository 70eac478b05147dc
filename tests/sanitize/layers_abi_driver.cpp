// layers_abi_driver.cpp -- the host side of include/zq_layers.h (argument
// validation) under AddressSanitizer and UndefinedBehaviorSanitizer, without a
// GPU: the kernel launchers are stubs that launch nothing.  Every device pointer
// here is a fake address that is never dereferenced.  Random buffers are checked
// against a comparison of every pair of ranges.  Test infrastructure only (built
// and run by tests/test_layers_sanitizers.py).
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../../weight_communication_zero_amd/csrc/zq_layers_launch.h"

static int failures = 0;
static int launches = 0;
#define CHECK(c)                                                                 \
    do {                                                                         \
        if (!(c)) {                                                              \
            std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
            failures++;                                                          \
        }                                                                        \
    } while (0)

namespace zq {
hipError_t launch_swiglu(const SwigluArgs& a, int, uint32_t, hipStream_t) {
    CHECK(a.gate && a.up && a.h && a.gate_codes && a.gate_scales && a.up_codes && a.up_scales);
    launches++;
    return hipSuccess;
}
hipError_t launch_swiglu_grad(const SwigluGradArgs& a, int, hipStream_t) {
    CHECK(a.gate_codes && a.gate_scales && a.up_codes && a.up_scales && a.dh && a.dgate && a.dup);
    launches++;
    return hipSuccess;
}
size_t linear_grad_workspace(uint32_t n, uint32_t, uint32_t) { return 8 * (size_t)n + 256; }
hipError_t launch_linear_grad(const LinearGradArgs& a, int, int, int, hipStream_t) {
    CHECK(a.dy && a.codes && a.scales && a.grad && a.workspace && a.n_tok && a.out_dim && a.in_dim);
    launches++;
    return hipSuccess;
}
size_t ce_loss_workspace(uint32_t n, uint32_t, uint32_t, uint64_t) { return 8 * (size_t)n + 256; }
size_t ce_grad_workspace(uint32_t n, uint32_t, uint32_t, uint64_t) { return 16 * (size_t)n + 256; }
hipError_t launch_ce_loss(const CeArgs& a, int, int w_type, hipStream_t) {
    CHECK(a.x && a.w && a.ids && a.loss && a.lse_out && a.workspace && (w_type != kQ8 || a.w_scales));
    launches++;
    return hipSuccess;
}
hipError_t launch_ce_grad(const CeArgs& a, int, int w_type, int, int, hipStream_t) {
    CHECK(a.x && a.w && a.ids && a.lse && a.dloss && (a.dx || a.dw) && a.workspace &&
          (w_type != kQ8 || a.w_scales));
    launches++;
    return hipSuccess;
}
hipError_t launch_clear(void* p, uint64_t bytes, hipStream_t) {
    CHECK(p && bytes);
    launches++;
    return hipSuccess;
}
}  // namespace zq

struct R {
    uintptr_t lo, hi;
    bool written;
};

static bool any_pair(const std::vector<R>& v) {
    for (size_t i = 0; i < v.size(); ++i)
        for (size_t j = i + 1; j < v.size(); ++j)
            if ((v[i].written || v[j].written) && v[i].lo < v[j].hi && v[j].lo < v[i].hi)
                return true;
    return false;
}

// A buffer at a random multiple of `align` in a span in which some overlap.
struct Draw {
    std::mt19937_64 rng;
    std::vector<R> all;
    explicit Draw(uint64_t seed) : rng(seed) {}
    uint64_t upto(uint64_t n) { return rng() % (n + 1); }
    template <typename T = void>
    T* buffer(size_t bytes, size_t align, bool written) {
        const uintptr_t p = 0x100000 + upto(20000) / align * align;
        all.push_back({p, p + bytes, written});
        return (T*)p;
    }
};

static void outcome(Draw& d, zq_status st, int before) {
    const bool clash = any_pair(d.all);
    CHECK(st == (clash ? ZQ_ERR_ALIAS : ZQ_OK));
    CHECK(launches == before + (clash ? 0 : 1));
}

static void random_buffers() {
    for (uint64_t seed = 0; seed < 20000; ++seed) {
        Draw d(seed);
        const int before = launches;
        const zq_dtype t = (zq_dtype)d.upto(2), half = (zq_dtype)(1 + d.upto(1));
        const size_t e = t == ZQ_FP32 ? 4 : 2;
        const uint32_t block = 32u << d.upto(7);
        const size_t n = 1 + d.upto(300), blocks = (n + block - 1) / block;
        switch (d.upto(4)) {
            case 0: {
                void* g = d.buffer(n * e, 16, false);
                void* u = d.buffer(n * e, 16, false);
                void* h = d.buffer(n * e, 16, true);
                int8_t* gc = d.buffer<int8_t>(n, 16, true);
                float* gs = d.buffer<float>(blocks * 4, 4, true);
                int8_t* uc = d.buffer<int8_t>(n, 16, true);
                float* us = d.buffer<float>(blocks * 4, 4, true);
                outcome(d, zq_swiglu_int8(g, u, t, n, block, h, gc, gs, uc, us, nullptr), before);
                break;
            }
            case 1: {
                int8_t* gc = d.buffer<int8_t>(n, 16, false);
                float* gs = d.buffer<float>(blocks * 4, 4, false);
                int8_t* uc = d.buffer<int8_t>(n, 16, false);
                float* us = d.buffer<float>(blocks * 4, 4, false);
                void* dh = d.buffer(n * e, 16, false);
                void* dg = d.buffer(n * e, 16, true);
                void* du = d.buffer(n * e, 16, true);
                void* h = d.upto(1) ? d.buffer(n * e, 16, true) : nullptr;
                outcome(d, zq_swiglu_grad_int8(gc, gs, uc, us, block, dh, t, n, dg, du, h, nullptr),
                        before);
                break;
            }
            case 2: {
                const size_t tok = 1 + d.upto(20);
                const uint64_t o = 1 + d.upto(20), i = 1 + d.upto(20);
                const size_t need = zq_linear_grad_workspace(tok, o, i);
                void* dy = d.buffer(tok * o * 2, 16, false);
                int8_t* c = d.buffer<int8_t>(tok * i, 16, false);
                float* s = d.buffer<float>((tok * i + block - 1) / block * 4, 4, false);
                void* g = d.buffer(o * i * e, 16, true);
                void* w = d.buffer(need, 16, true);
                outcome(d, zq_linear_grad_int8(dy, half, c, s, block, tok, o, i, g, t, ZQ_GRAD_ADD, w,
                                               need, nullptr), before);
                break;
            }
            default: {
                const bool grad = d.upto(1), q8 = d.upto(1), i64 = d.upto(1);
                const size_t tok = 1 + d.upto(20);
                const uint64_t dim = 1 + d.upto(20), rows = 1 + d.upto(20);
                const size_t need = grad ? zq_ce_grad_workspace(tok, rows, dim, 0)
                                         : zq_ce_loss_workspace(tok, rows, dim, 0);
                const size_t ib = i64 ? 8 : 4;
                const zq_index_type it = i64 ? ZQ_I64 : ZQ_I32;
                void* x = d.buffer(tok * dim * 2, 16, false);
                void* w = d.buffer(rows * dim * (q8 ? 1 : 2), 16, false);
                float* s = q8 ? d.buffer<float>((rows * dim + block - 1) / block * 4, 4, false) : nullptr;
                void* ids = d.buffer(tok * ib, ib, false);
                void* ws = d.buffer(need, 16, true);
                if (grad) {
                    float* lse = d.buffer<float>(tok * 4, 4, false);
                    float* dl = d.buffer<float>(tok * 4, 4, false);
                    const uint64_t which = d.upto(2);
                    void* dx = which != 1 ? d.buffer(tok * dim * 2, 16, true) : nullptr;
                    void* dw = which != 2 ? d.buffer(rows * dim * e, 16, true) : nullptr;
                    const zq_status st =
                        q8 ? zq_ce_grad_int8(x, half, tok, dim, (int8_t*)w, s, block, rows, ids, it, 1.0f,
                                             lse, dl, dx, dw, t, ZQ_GRAD_WRITE, 0, ws, need, nullptr)
                           : zq_ce_grad(x, half, tok, dim, w, rows, ids, it, 1.0f, lse, dl, dx, dw, t,
                                        ZQ_GRAD_WRITE, 0, ws, need, nullptr);
                    outcome(d, st, before);
                } else {
                    float* loss = d.buffer<float>(tok * 4, 4, true);
                    float* lse = d.buffer<float>(tok * 4, 4, true);
                    const zq_status st =
                        q8 ? zq_ce_loss_int8(x, half, tok, dim, (int8_t*)w, s, block, rows, ids, it, 1.0f,
                                             loss, lse, 0, ws, need, nullptr)
                           : zq_ce_loss(x, half, tok, dim, w, rows, ids, it, 1.0f, loss, lse, 0, ws, need,
                                        nullptr);
                    outcome(d, st, before);
                }
            }
        }
    }
}

// Sizes at and past the ends.
static void ends() {
    for (uint64_t big : {(uint64_t)1 << 20, ((uint64_t)1 << 24) + 1, (uint64_t)1 << 60, UINT64_MAX}) {
        (void)zq_linear_grad_workspace((size_t)big, big, big);
        (void)zq_ce_loss_workspace((size_t)big, big, big, big);
        (void)zq_ce_grad_workspace((size_t)big, big, big, big);
        CHECK(zq_swiglu_int8(nullptr, nullptr, ZQ_FP32, (size_t)big, 32, nullptr, nullptr, nullptr, nullptr,
                             nullptr, nullptr) == (big > (uint64_t)1 << 60 ? ZQ_ERR_SIZE : ZQ_ERR_NULL));
    }
}

int main() {
    random_buffers();
    ends();
#ifdef ZQ_SANITIZER_CANARY
    std::vector<int> v(4);
    volatile size_t i = 4;
    std::printf("%d\n", v.data()[i]);
#endif
    CHECK(launches > 1000);
    if (failures)
        return 1;
    std::puts("all checks passed");
    return 0;
}
