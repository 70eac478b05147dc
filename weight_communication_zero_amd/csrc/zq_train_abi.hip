// zq_train_abi.hip -- the extern "C" entry points of include/zq_train.h:
// host-side argument validation, then the kernel launches on the caller's
// stream.  Every check runs before anything is enqueued.  No state, no
// device allocation, and no C++ exception leaves an entry point.
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/zq_train.h"
#include "zq_train_launch.h"

namespace {

constexpr uint64_t kMaxElems = (uint64_t)1 << 60;
constexpr uint64_t kMaxListElems = (uint64_t)1 << 40;  // of a norm or clip call
constexpr uint64_t kMaxRows = ((uint64_t)1 << 31) - 2;
constexpr uint64_t kMaxDim = ((uint64_t)1 << 31) - 1;
constexpr uint64_t kMaxTokens = (uint64_t)1 << 30;

bool valid_block(uint32_t b) { return b >= 32 && b <= 4096 && (b & (b - 1)) == 0; }
bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool known_dtype(int d) { return d == ZQ_FP32 || d == ZQ_BF16 || d == ZQ_FP16; }
size_t dtype_bytes(int d) { return d == ZQ_FP32 ? 4 : 2; }
bool known_index(int d) { return d == ZQ_I32 || d == ZQ_I64; }
size_t index_bytes(int d) { return d == ZQ_I64 ? 8 : 4; }
zq_status launched(hipError_t e) { return e == hipSuccess ? ZQ_OK : ZQ_ERR_LAUNCH; }

// The integer a C caller passed for an enum parameter (values outside the
// enumerators are legal in C; they are read as bytes, never as an enum value).
template <typename E>
int raw_enum(const E& e) {
    static_assert(sizeof(E) == sizeof(int), "enums of the ABI are int-sized");
    int v;
    std::memcpy(&v, &e, sizeof v);
    return v;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0)
        return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

bool table_sizes_ok(size_t n_tok, uint64_t rows, uint64_t dim) {
    return rows >= 1 && dim >= 1 && rows <= kMaxRows && dim <= kMaxDim && n_tok <= kMaxTokens &&
           rows <= kMaxElems / dim && n_tok <= kMaxElems / dim;
}

// The checks that both lookups share; `table_bytes` and `scale_bytes` are the
// sizes of what they read.
zq_status lookup(const void* table, int table_type, size_t table_bytes, size_t table_align,
                 const float* scales, size_t scale_bytes, uint32_t log2b, uint64_t rows,
                 uint64_t dim, const void* ids, int id_type, size_t n_tok, float scale, void* out,
                 int out_type, void* stream) {
    if (n_tok == 0)
        return ZQ_OK;
    if (!table || !ids || !out || (table_type == zq::kQ8 && !scales))
        return ZQ_ERR_NULL;
    if (!aligned(table, table_align) || !aligned(scales, 4) || !aligned(ids, index_bytes(id_type)) ||
        !aligned(out, 16))
        return ZQ_ERR_ALIGN;
    const size_t ob = n_tok * dim * dtype_bytes(out_type);
    if (overlap(out, ob, table, table_bytes) || overlap(out, ob, scales, scale_bytes) ||
        overlap(out, ob, ids, n_tok * index_bytes(id_type)))
        return ZQ_ERR_ALIAS;
    zq::LookupArgs a = {};
    a.table = table;
    a.scales = scales;
    a.log2b = log2b;
    a.id64 = id_type == ZQ_I64;
    a.ids = ids;
    a.n_tok = n_tok;
    a.rows = rows;
    a.dim = dim;
    a.scale = scale;
    a.out = out;
    return launched(zq::launch_embed_lookup(a, table_type, out_type, (hipStream_t)stream));
}

struct Range {
    uintptr_t lo, hi;
};

Range range(const void* p, size_t bytes) { return {(uintptr_t)p, (uintptr_t)p + bytes}; }
bool meet(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// Whether a written range overlaps any other one (read ranges may overlap each
// other).
bool alias(std::vector<Range>& read, std::vector<Range>& written) {
    const auto less = [](const Range& a, const Range& b) { return a.lo < b.lo; };
    std::sort(read.begin(), read.end(), less);
    std::sort(written.begin(), written.end(), less);
    uintptr_t end_read = 0, end_written = 0;
    size_t r = 0;
    for (const Range& w : written) {
        for (; r < read.size() && read[r].lo <= w.lo; ++r) {
            if (read[r].lo < end_written)
                return true;
            end_read = std::max(end_read, read[r].hi);
        }
        if (w.lo < end_read || w.lo < end_written)
            return true;
        end_written = w.hi;
    }
    return r < read.size() && read[r].lo < end_written;
}

// What a norm or clip call's segments read (g, where it is not out) and write
// (out): the spans they lie in, and whether the written ones come one after
// the other.  Tensors mostly lie in one buffer in order, and the answer to
// whether anything overlaps then takes no list and no sorting.
struct Spans {
    Range read = {UINTPTR_MAX, 0}, written = {UINTPTR_MAX, 0};
    bool ordered = true;

    void add_read(const Range& r) { read = {std::min(read.lo, r.lo), std::max(read.hi, r.hi)}; }
    void add_written(const Range& r) {
        ordered = ordered && r.lo >= written.hi;
        written = {std::min(written.lo, r.lo), std::max(written.hi, r.hi)};
    }
};

// Checks a list's segments (elements of `esz` bytes; `writes`: out is written).
zq_status check_list(const zq_grad_segment* segs, uint32_t n_seg, size_t esz, bool writes,
                     Spans* spans) {
    uint64_t total = 0;
    for (uint32_t i = 0; i < n_seg; ++i) {
        const zq_grad_segment& s = segs[i];
        if (s.n > kMaxListElems - total)
            return ZQ_ERR_SIZE;
        if (s.n == 0)
            continue;
        total += s.n;
        if (!s.g || (writes && !s.out))
            return ZQ_ERR_NULL;
        if (!aligned(s.g, 16) || (writes && !aligned(s.out, 16)))
            return ZQ_ERR_ALIGN;
        if (!writes || s.out != s.g)
            spans->add_read(range(s.g, s.n * esz));
        if (writes)
            spans->add_written(range(s.out, s.n * esz));
    }
    return ZQ_OK;
}

// Whether a list's written ranges, or one of `more` (of which the first
// `n_written` are written), overlap another range.
bool list_alias(const zq_grad_segment* segs, uint32_t n_seg, size_t esz, bool writes,
                const Spans& spans, const Range* more, uint32_t n_written, uint32_t n_more) {
    bool apart = spans.ordered && !meet(spans.read, spans.written);
    for (uint32_t i = 0; apart && i < n_more; ++i) {
        apart = !meet(more[i], spans.written) && (i >= n_written || !meet(more[i], spans.read));
        for (uint32_t j = 0; apart && j < std::min(i, n_written); ++j)
            apart = !meet(more[i], more[j]);
    }
    if (apart)
        return false;
    std::vector<Range> read(more + n_written, more + n_more), written(more, more + n_written);
    read.reserve(read.size() + n_seg);
    written.reserve(written.size() + n_seg);
    for (uint32_t i = 0; i < n_seg; ++i) {
        const zq_grad_segment& s = segs[i];
        if (s.n && (!writes || s.out != s.g))
            read.push_back(range(s.g, s.n * esz));
        if (s.n && writes)
            written.push_back(range(s.out, s.n * esz));
    }
    return alias(read, written);
}

}  // namespace

extern "C" {

zq_status zq_embed_lookup(const void* table, zq_dtype table_dtype, uint64_t rows, uint64_t dim,
                          const void* ids, zq_index_type id_type_arg, size_t n_tok, float scale,
                          void* out, zq_dtype out_dtype_arg, void* stream) {
    const int t = raw_enum(table_dtype), o = raw_enum(out_dtype_arg), it = raw_enum(id_type_arg);
    if (!known_dtype(t) || !known_dtype(o) || !known_index(it))
        return ZQ_ERR_DTYPE;
    if (!table_sizes_ok(n_tok, rows, dim))
        return ZQ_ERR_SIZE;
    return lookup(table, t, rows * dim * dtype_bytes(t), 16, nullptr, 0, 0, rows, dim, ids, it,
                  n_tok, scale, out, o, stream);
}

zq_status zq_embed_lookup_int8(const int8_t* codes, const float* scales, uint32_t block,
                               uint64_t rows, uint64_t dim, const void* ids,
                               zq_index_type id_type_arg, size_t n_tok, float scale, void* out,
                               zq_dtype out_dtype_arg, void* stream) {
    const int o = raw_enum(out_dtype_arg), it = raw_enum(id_type_arg);
    if (!known_dtype(o) || !known_index(it))
        return ZQ_ERR_DTYPE;
    if (!valid_block(block))
        return ZQ_ERR_BLOCK;
    if (!table_sizes_ok(n_tok, rows, dim))
        return ZQ_ERR_SIZE;
    uint32_t log2b = 0;
    while ((1u << log2b) < block)
        ++log2b;
    return lookup(codes, zq::kQ8, rows * dim, 16, scales, (rows * dim + block - 1) / block * 4,
                  log2b, rows, dim, ids, it, n_tok, scale, out, o, stream);
}

size_t zq_embed_grad_workspace(size_t n_tok, uint64_t rows, uint64_t dim) {
    if (n_tok == 0 || !table_sizes_ok(n_tok, rows, dim))
        return 0;
    return zq::embed_grad_workspace(n_tok, rows, dim);
}

zq_status zq_embed_grad(const void* dout, zq_dtype d_dtype_arg, const void* ids,
                        zq_index_type id_type_arg, size_t n_tok, uint64_t rows, uint64_t dim,
                        float scale, void* grad, zq_dtype grad_dtype_arg, zq_grad_mode mode_arg,
                        uint64_t seed, uint64_t counter_base, void* workspace,
                        size_t workspace_bytes, void* stream) {
    const int d = raw_enum(d_dtype_arg), g = raw_enum(grad_dtype_arg), it = raw_enum(id_type_arg);
    const int mode = raw_enum(mode_arg);
    if (!known_dtype(d) || !known_dtype(g) || !known_index(it) ||
        (mode != ZQ_GRAD_WRITE && mode != ZQ_GRAD_ADD && mode != ZQ_GRAD_ADD_SR) ||
        (mode == ZQ_GRAD_ADD_SR && g != ZQ_BF16))
        return ZQ_ERR_DTYPE;
    if (!table_sizes_ok(n_tok, rows, dim) || counter_base > UINT64_MAX - rows * dim)
        return ZQ_ERR_SIZE;
    if (n_tok == 0 && mode != ZQ_GRAD_WRITE)
        return ZQ_OK;
    if (!grad || (n_tok && (!dout || !ids || !workspace)))
        return ZQ_ERR_NULL;
    if (!aligned(grad, 16))
        return ZQ_ERR_ALIGN;
    zq::EmbedGradArgs a = {};
    a.n_tok = n_tok;
    a.rows = rows;
    a.dim = dim;
    a.scale = scale;
    a.grad = grad;
    a.seed = seed;
    a.cbase = counter_base;
    if (n_tok) {
        if (!aligned(dout, 16) || !aligned(ids, index_bytes(it)) || !aligned(workspace, 16))
            return ZQ_ERR_ALIGN;
        const size_t need = zq::embed_grad_workspace(n_tok, rows, dim);
        if (workspace_bytes < need)
            return ZQ_ERR_SIZE;
        const size_t gb = rows * dim * dtype_bytes(g), db = n_tok * dim * dtype_bytes(d);
        const size_t ib = n_tok * index_bytes(it);
        if (overlap(grad, gb, dout, db) || overlap(grad, gb, ids, ib) ||
            overlap(grad, gb, workspace, need) || overlap(workspace, need, dout, db) ||
            overlap(workspace, need, ids, ib))
            return ZQ_ERR_ALIAS;
        a.dout = dout;
        a.ids = ids;
        a.id64 = it == ZQ_I64;
        a.workspace = workspace;
    }
    return launched(zq::launch_embed_grad(a, d, g, mode, (hipStream_t)stream));
}

size_t zq_grad_sumsq_workspace(uint32_t n_seg) {
    return n_seg > 65536 ? 0 : zq::grad_sumsq_workspace(n_seg);
}

zq_status zq_grad_sumsq_batched(const zq_grad_segment* segs, uint32_t n_seg, zq_dtype g_dtype_arg,
                                int accumulate, double* sumsq, void* workspace,
                                size_t workspace_bytes, void* stream) try {
    const int t = raw_enum(g_dtype_arg);
    if (!known_dtype(t))
        return ZQ_ERR_DTYPE;
    if (n_seg > 65536)
        return ZQ_ERR_SIZE;
    if (!sumsq || !workspace || (n_seg && !segs))
        return ZQ_ERR_NULL;
    const size_t need = zq::grad_sumsq_workspace(n_seg);
    if (workspace_bytes < need)
        return ZQ_ERR_SIZE;
    if (!aligned(sumsq, 8) || !aligned(workspace, 16))
        return ZQ_ERR_ALIGN;
    Spans spans;
    const zq_status st = check_list(segs, n_seg, dtype_bytes(t), false, &spans);
    if (st != ZQ_OK)
        return st;
    const Range more[2] = {range(sumsq, 8), range(workspace, need)};
    if (list_alias(segs, n_seg, dtype_bytes(t), false, spans, more, 2, 2))
        return ZQ_ERR_ALIAS;
    return launched(zq::launch_grad_sumsq(segs, n_seg, t, accumulate != 0, sumsq,
                                          (double*)workspace, (hipStream_t)stream));
} catch (const std::bad_alloc&) {
    return ZQ_ERR_LAUNCH;
}

zq_status zq_grad_clip_batched(const zq_grad_segment* segs, uint32_t n_seg, zq_dtype g_dtype_arg,
                               const double* sumsq, float max_norm, float eps, float* norm,
                               void* stream) try {
    const int t = raw_enum(g_dtype_arg);
    if (!known_dtype(t))
        return ZQ_ERR_DTYPE;
    if (n_seg > 65536 || !(max_norm >= 0.0f) || !(eps >= 0.0f) || std::isinf(max_norm) ||
        std::isinf(eps))
        return ZQ_ERR_SIZE;
    if (!sumsq || (n_seg && !segs))
        return ZQ_ERR_NULL;
    if (!aligned(sumsq, 8) || !aligned(norm, 4))
        return ZQ_ERR_ALIGN;
    Spans spans;
    const zq_status st = check_list(segs, n_seg, dtype_bytes(t), true, &spans);
    if (st != ZQ_OK)
        return st;
    const Range more[2] = {range(norm, norm ? 4 : 0), range(sumsq, 8)};
    const uint32_t skip = norm ? 0 : 1;
    if (list_alias(segs, n_seg, dtype_bytes(t), true, spans, more + skip, 1 - skip, 2 - skip))
        return ZQ_ERR_ALIAS;
    return launched(zq::launch_grad_clip(segs, n_seg, t, sumsq, max_norm, eps, norm,
                                         (hipStream_t)stream));
} catch (const std::bad_alloc&) {
    return ZQ_ERR_LAUNCH;
}

}  // extern "C"
