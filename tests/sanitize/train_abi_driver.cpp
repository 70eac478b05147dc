// train_abi_driver.cpp -- the host side of include/zq_train.h (argument
// validation, list checks) under AddressSanitizer and
// UndefinedBehaviorSanitizer, without a GPU: the kernel launchers are stubs
// that read what the ABI layer hands them and launch nothing.  Every device
// pointer here is a fake address that is never dereferenced.  Random segment
// lists are checked against a comparison of every pair of ranges.  Test
// infrastructure only (built and run by tests/test_train_sanitizers.py).
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../../weight_communication_zero_amd/csrc/zq_train_launch.h"

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
hipError_t launch_embed_lookup(const LookupArgs& a, int, int, hipStream_t) {
    CHECK(a.table && a.ids && a.out && a.n_tok && a.rows && a.dim);
    launches++;
    return hipSuccess;
}
size_t embed_grad_workspace(uint64_t n_tok, uint64_t, uint64_t) { return 8 * n_tok + 256; }
hipError_t launch_embed_grad(const EmbedGradArgs& a, int, int, int, hipStream_t) {
    CHECK(a.grad && (!a.n_tok || (a.dout && a.ids && a.workspace)));
    launches++;
    return hipSuccess;
}
size_t grad_sumsq_workspace(uint32_t n_seg) { return 16 + 8 * (size_t)n_seg; }
hipError_t launch_grad_sumsq(const GradSegment* segs, uint32_t n_seg, int, bool, double*, double*,
                             hipStream_t) {
    for (uint32_t i = 0; i < n_seg; ++i)
        CHECK(segs[i].n == 0 || segs[i].g);
    launches++;
    return hipSuccess;
}
hipError_t launch_grad_clip(const GradSegment* segs, uint32_t n_seg, int, const double*, float,
                            float, float*, hipStream_t) {
    for (uint32_t i = 0; i < n_seg; ++i)
        CHECK(segs[i].n == 0 || (segs[i].g && segs[i].out));
    launches++;
    return hipSuccess;
}
}  // namespace zq

static void* at(uintptr_t a) { return (void*)a; }

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

static void lists() {
    std::mt19937_64 rng(7);
    int seen[2][2] = {};
    for (int it = 0; it < 40000; ++it) {
        const uint32_t n = (uint32_t)(rng() % 6);
        const bool clip = rng() & 1, ordered = rng() & 1, in_place = rng() & 1;
        const int t = (int)(rng() % 3);
        const uintptr_t esz = t == ZQ_FP32 ? 4 : 2, span = 1 + rng() % 64;
        std::vector<zq_grad_segment> s(n);
        std::vector<R> v;
        uintptr_t g = 0x10000, o = 0x10000 + 16 * (rng() % (4 * span));
        for (auto& x : s) {
            x.n = rng() % 5 ? rng() % 200 : 0;
            if (!ordered) {
                g = 0x10000 + 16 * (rng() % (8 * span));
                o = 0x10000 + 16 * (rng() % (8 * span));
            }
            x.g = at(g);
            x.out = in_place || rng() % 8 == 0 ? at(g) : at(o);
            if (x.n && (!clip || x.out != x.g))
                v.push_back({g, g + x.n * esz, false});
            if (x.n && clip)
                v.push_back({(uintptr_t)x.out, (uintptr_t)x.out + x.n * esz, true});
            g += (x.n * esz + 15) / 16 * 16;
            o += (x.n * esz + 15) / 16 * 16;
        }
        const uintptr_t q = 0x10000 + 8 * (rng() % (32 * span)), w = 0x10000 + 16 * (rng() % (32 * span));
        zq_status st;
        if (clip) {
            const bool norm = rng() & 1;
            const uintptr_t m = 0x10000 + 4 * (rng() % (64 * span));
            v.push_back({q, q + 8, false});
            if (norm)
                v.push_back({m, m + 4, true});
            st = zq_grad_clip_batched(s.data(), n, (zq_dtype)t, (double*)at(q), 1.0f, 0.0f,
                                      norm ? (float*)at(m) : nullptr, nullptr);
        } else {
            v.push_back({q, q + 8, true});
            v.push_back({w, w + 16 + 8 * n, true});
            st = zq_grad_sumsq_batched(s.data(), n, (zq_dtype)t, 0, (double*)at(q), at(w), 1000, nullptr);
        }
        const bool bad = any_pair(v);
        seen[clip][bad]++;
        CHECK(st == (bad ? ZQ_ERR_ALIAS : ZQ_OK));
        if (failures > 5)
            return;
    }
    CHECK(seen[0][0] > 1000 && seen[0][1] > 1000 && seen[1][0] > 1000 && seen[1][1] > 1000);
    std::vector<zq_grad_segment> many(65536);
    for (size_t i = 0; i < many.size(); ++i)
        many[i] = {at(0x100000 + 64 * i), at(0x100000 + 64 * i), i % 3 ? 8u : 0u};
    CHECK(zq_grad_clip_batched(many.data(), 65536, ZQ_FP32, (double*)at(0x1000), 1.0f, 0.0f, nullptr,
                               nullptr) == ZQ_OK);
    many[65535] = many[1];
    CHECK(zq_grad_clip_batched(many.data(), 65536, ZQ_FP32, (double*)at(0x1000), 1.0f, 0.0f, nullptr,
                               nullptr) == ZQ_ERR_ALIAS);
}

int main() {
    const int odd[] = {-1, 3, 1 << 30};
    for (int e : odd) {
        CHECK(zq_embed_lookup(at(64), (zq_dtype)e, 4, 8, at(1024), ZQ_I32, 2, 1.0f, at(4096), ZQ_FP32,
                              nullptr) == ZQ_ERR_DTYPE);
        CHECK(zq_embed_lookup(at(64), ZQ_FP32, 4, 8, at(1024), (zq_index_type)e, 2, 1.0f, at(4096),
                              ZQ_FP32, nullptr) == ZQ_ERR_DTYPE);
        CHECK(zq_embed_grad(at(64), ZQ_FP32, at(1024), ZQ_I32, 2, 4, 8, 1.0f, at(4096), ZQ_FP32,
                            (zq_grad_mode)e, 0, 0, at(8192), 4096, nullptr) == ZQ_ERR_DTYPE);
        CHECK(zq_grad_sumsq_batched(nullptr, 0, (zq_dtype)e, 0, (double*)at(64), at(128), 16, nullptr) ==
              ZQ_ERR_DTYPE);
    }
    CHECK(launches == 0);
    CHECK(zq_embed_lookup(at(64), ZQ_BF16, 4, 8, at(1024), ZQ_I64, 2, 1.0f, at(4096), ZQ_FP16, nullptr) ==
          ZQ_OK);
    CHECK(zq_embed_lookup_int8((int8_t*)at(64), (float*)at(512), 32, 4, 8, at(1024), ZQ_I64, 2, 1.0f,
                               at(4096), ZQ_FP16, nullptr) == ZQ_OK);
    CHECK(zq_embed_grad(at(64), ZQ_FP32, at(1024), ZQ_I32, 2, 4, 8, 1.0f, at(4096), ZQ_BF16, ZQ_GRAD_ADD_SR,
                        0, UINT64_MAX - 32, at(8192), 4096, nullptr) == ZQ_OK);
    CHECK(zq_embed_grad(at(64), ZQ_FP32, at(1024), ZQ_I32, 2, 4, 8, 1.0f, at(4096), ZQ_BF16, ZQ_GRAD_ADD_SR,
                        0, UINT64_MAX - 31, at(8192), 4096, nullptr) == ZQ_ERR_SIZE);
    CHECK(zq_embed_grad(nullptr, ZQ_FP32, nullptr, ZQ_I32, 0, 4, 8, 1.0f, at(4096), ZQ_FP32, ZQ_GRAD_WRITE, 0,
                        0, nullptr, 0, nullptr) == ZQ_OK);
    CHECK(zq_embed_grad_workspace((size_t)-1, 4, 8) == 0 && zq_embed_grad_workspace(4, UINT64_MAX, 8) == 0);
    CHECK(launches == 4);
    lists();
#ifdef ZQ_SANITIZER_CANARY
    std::vector<int> v(4);
    volatile int i = 4;
    std::printf("%d\n", v.data()[i]);
#endif
    if (failures) {
        std::fprintf(stderr, "%d failures\n", failures);
        return 1;
    }
    std::puts("all checks passed");
    return 0;
}
