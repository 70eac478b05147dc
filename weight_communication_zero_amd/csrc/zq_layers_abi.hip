// zq_layers_abi.hip -- the extern "C" entry points of include/zq_layers.h:
// host-side argument validation, then the kernel launches on the caller's stream.
// Every check runs before anything is enqueued.  No state, no allocation, and no
// C++ exception leaves an entry point (nothing here throws).
#include <stdint.h>

#include <cstring>

#include "../../include/zq_layers.h"
#include "zq_layers_launch.h"

namespace {

constexpr uint64_t kMaxElems = (uint64_t)1 << 60;
constexpr uint64_t kMaxTokens = (uint64_t)1 << 20;
constexpr uint64_t kMaxDim = (uint64_t)1 << 20;
constexpr uint64_t kMaxVocab = (uint64_t)1 << 24;
constexpr uint64_t kMaxProduct = (uint64_t)1 << 36;

bool valid_block(uint32_t b) { return b >= 32 && b <= 4096 && (b & (b - 1)) == 0; }
bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool known_dtype(int d) { return d == ZQ_FP32 || d == ZQ_BF16 || d == ZQ_FP16; }
bool half_dtype(int d) { return d == ZQ_BF16 || d == ZQ_FP16; }
size_t dtype_bytes(int d) { return d == ZQ_FP32 ? 4 : 2; }
zq_status launched(hipError_t e) { return e == hipSuccess ? ZQ_OK : ZQ_ERR_LAUNCH; }

uint32_t log2_of(uint32_t block) {
    uint32_t l = 0;
    while ((1u << l) < block)
        ++l;
    return l;
}

size_t scale_bytes(uint64_t n, uint32_t block) { return (n + block - 1) / block * 4; }

// The integer a C caller passed for an enum parameter (values outside the
// enumerators are legal in C; they are read as bytes, never as an enum value).
template <typename E>
int raw_enum(const E& e) {
    static_assert(sizeof(E) == sizeof(int), "enums of the ABI are int-sized");
    int v;
    std::memcpy(&v, &e, sizeof v);
    return v;
}

// A call's buffers: each is there or not (`bytes` 0), aligned, written or read.
struct Buffers {
    struct One {
        uintptr_t lo, hi;
        bool written;
    } list[12];
    int n = 0;
    bool null = false, misaligned = false;

    void add(const void* p, size_t bytes, uintptr_t align, bool written) {
        null = null || !p;
        misaligned = misaligned || !aligned(p, align);
        list[n++] = {(uintptr_t)p, (uintptr_t)p + bytes, written};
    }

    zq_status check() const {
        if (null)
            return ZQ_ERR_NULL;
        if (misaligned)
            return ZQ_ERR_ALIGN;
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((list[i].written || list[j].written) && list[i].lo < list[j].hi &&
                    list[j].lo < list[i].hi)
                    return ZQ_ERR_ALIAS;
        return ZQ_OK;
    }
};

bool ce_sizes_ok(size_t n_tok, uint64_t rows, uint64_t dim) {
    return rows >= 1 && dim >= 1 && rows <= kMaxVocab && dim <= kMaxDim && n_tok <= kMaxTokens &&
           n_tok * dim <= kMaxProduct;
}

// The projection of a cross entropy call: values, or codes and scales.
struct Projection {
    const void* w;
    const float* scales;
    uint32_t block;  // 0: values
};

void add_projection(Buffers& b, const Projection& p, uint64_t n, int type) {
    b.add(p.w, n * (p.block ? 1 : dtype_bytes(type)), 16, false);
    if (p.block)
        b.add(p.scales, scale_bytes(n, p.block), 4, false);
}

zq::CeArgs ce_args(const void* x, size_t n_tok, uint64_t dim, const Projection& p, uint64_t rows,
                   const void* ids, int id_type, float scale, uint64_t piece, void* workspace) {
    zq::CeArgs a = {};
    a.x = x;
    a.n_tok = (uint32_t)n_tok;
    a.dim = (uint32_t)dim;
    a.rows = (uint32_t)rows;
    a.w = p.w;
    a.w_scales = p.scales;
    a.log2b = p.block ? log2_of(p.block) : 0;
    a.ids = ids;
    a.id64 = id_type == ZQ_I64;
    a.scale = scale;
    a.piece = piece;
    a.workspace = workspace;
    return a;
}

zq_status ce_loss(const void* x, zq_dtype dtype, size_t n_tok, uint64_t dim, const Projection& p,
                  uint64_t rows, const void* ids, zq_index_type id_type, float scale, float* loss,
                  float* lse, uint64_t piece, void* workspace, size_t workspace_bytes,
                  void* stream) {
    const int t = raw_enum(dtype), it = raw_enum(id_type);
    if (!half_dtype(t) || (it != ZQ_I32 && it != ZQ_I64))
        return ZQ_ERR_DTYPE;
    if (p.block && !valid_block(p.block))
        return ZQ_ERR_BLOCK;
    if (!ce_sizes_ok(n_tok, rows, dim))
        return ZQ_ERR_SIZE;
    if (n_tok == 0)
        return ZQ_OK;
    const size_t need =
        zq::ce_loss_workspace((uint32_t)n_tok, (uint32_t)rows, (uint32_t)dim, piece);
    if (workspace_bytes < need)
        return ZQ_ERR_SIZE;
    const size_t ib = it == ZQ_I64 ? 8 : 4;
    Buffers b;
    b.add(x, n_tok * dim * 2, 16, false);
    add_projection(b, p, rows * dim, t);
    b.add(ids, n_tok * ib, ib, false);
    b.add(loss, n_tok * 4, 4, true);
    b.add(lse, n_tok * 4, 4, true);
    b.add(workspace, need, 16, true);
    const zq_status st = b.check();
    if (st != ZQ_OK)
        return st;
    zq::CeArgs a = ce_args(x, n_tok, dim, p, rows, ids, it, scale, piece, workspace);
    a.loss = loss;
    a.lse_out = lse;
    return launched(zq::launch_ce_loss(a, t, p.block ? zq::kQ8 : t, (hipStream_t)stream));
}

zq_status ce_grad(const void* x, zq_dtype dtype, size_t n_tok, uint64_t dim, const Projection& p,
                  uint64_t rows, const void* ids, zq_index_type id_type, float scale,
                  const float* lse, const float* dloss, void* dx, void* dw, zq_dtype dw_dtype,
                  zq_grad_mode mode_arg, uint64_t piece, void* workspace, size_t workspace_bytes,
                  void* stream) {
    const int t = raw_enum(dtype), it = raw_enum(id_type), g = raw_enum(dw_dtype);
    const int mode = raw_enum(mode_arg);
    if (!half_dtype(t) || (it != ZQ_I32 && it != ZQ_I64) || !known_dtype(g) ||
        (mode != ZQ_GRAD_WRITE && mode != ZQ_GRAD_ADD))
        return ZQ_ERR_DTYPE;
    if (p.block && !valid_block(p.block))
        return ZQ_ERR_BLOCK;
    if (!ce_sizes_ok(n_tok, rows, dim))
        return ZQ_ERR_SIZE;
    const size_t wb = rows * dim * dtype_bytes(g);
    if (n_tok == 0) {
        if (mode != ZQ_GRAD_WRITE || !dw)
            return ZQ_OK;
        if (!aligned(dw, 16))
            return ZQ_ERR_ALIGN;
        return launched(zq::launch_clear(dw, wb, (hipStream_t)stream));
    }
    const size_t need =
        zq::ce_grad_workspace((uint32_t)n_tok, (uint32_t)rows, (uint32_t)dim, piece);
    if (workspace_bytes < need)
        return ZQ_ERR_SIZE;
    if (!dx && !dw)
        return ZQ_ERR_NULL;
    const size_t ib = it == ZQ_I64 ? 8 : 4;
    Buffers b;
    b.add(x, n_tok * dim * 2, 16, false);
    add_projection(b, p, rows * dim, t);
    b.add(ids, n_tok * ib, ib, false);
    b.add(lse, n_tok * 4, 4, false);
    b.add(dloss, n_tok * 4, 4, false);
    if (dx)
        b.add(dx, n_tok * dim * 2, 16, true);
    if (dw)
        b.add(dw, wb, 16, true);
    b.add(workspace, need, 16, true);
    const zq_status st = b.check();
    if (st != ZQ_OK)
        return st;
    zq::CeArgs a = ce_args(x, n_tok, dim, p, rows, ids, it, scale, piece, workspace);
    a.lse = lse;
    a.dloss = dloss;
    a.dx = dx;
    a.dw = dw;
    return launched(zq::launch_ce_grad(a, t, p.block ? zq::kQ8 : t, g, mode, (hipStream_t)stream));
}

bool linear_sizes_ok(size_t n_tok, uint64_t out_dim, uint64_t in_dim) {
    return out_dim >= 1 && in_dim >= 1 && out_dim <= kMaxDim && in_dim <= kMaxDim &&
           out_dim * in_dim <= kMaxProduct && n_tok <= kMaxTokens;
}

}  // namespace

extern "C" {

zq_status zq_swiglu_int8(const void* gate, const void* up, zq_dtype dtype, size_t n, uint32_t block,
                         void* h, int8_t* gate_codes, float* gate_scales, int8_t* up_codes,
                         float* up_scales, void* stream) {
    const int t = raw_enum(dtype);
    if (!known_dtype(t))
        return ZQ_ERR_DTYPE;
    if (!valid_block(block))
        return ZQ_ERR_BLOCK;
    if (n > kMaxElems)
        return ZQ_ERR_SIZE;
    if (n == 0)
        return ZQ_OK;
    const size_t e = dtype_bytes(t), sb = scale_bytes(n, block);
    Buffers b;
    b.add(gate, n * e, 16, false);
    b.add(up, n * e, 16, false);
    b.add(h, n * e, 16, true);
    b.add(gate_codes, n, 16, true);
    b.add(gate_scales, sb, 4, true);
    b.add(up_codes, n, 16, true);
    b.add(up_scales, sb, 4, true);
    const zq_status st = b.check();
    if (st != ZQ_OK)
        return st;
    const zq::SwigluArgs a = {gate, up, n, h, gate_codes, gate_scales, up_codes, up_scales};
    return launched(zq::launch_swiglu(a, t, block, (hipStream_t)stream));
}

zq_status zq_swiglu_grad_int8(const int8_t* gate_codes, const float* gate_scales,
                              const int8_t* up_codes, const float* up_scales, uint32_t block,
                              const void* dh, zq_dtype dtype, size_t n, void* dgate, void* dup,
                              void* h, void* stream) {
    const int t = raw_enum(dtype);
    if (!known_dtype(t))
        return ZQ_ERR_DTYPE;
    if (!valid_block(block))
        return ZQ_ERR_BLOCK;
    if (n > kMaxElems)
        return ZQ_ERR_SIZE;
    if (n == 0)
        return ZQ_OK;
    const size_t e = dtype_bytes(t), sb = scale_bytes(n, block);
    Buffers b;
    b.add(gate_codes, n, 16, false);
    b.add(gate_scales, sb, 4, false);
    b.add(up_codes, n, 16, false);
    b.add(up_scales, sb, 4, false);
    b.add(dh, n * e, 16, false);
    b.add(dgate, n * e, 16, true);
    b.add(dup, n * e, 16, true);
    if (h)
        b.add(h, n * e, 16, true);
    const zq_status st = b.check();
    if (st != ZQ_OK)
        return st;
    const zq::SwigluGradArgs a = {gate_codes, gate_scales, up_codes, up_scales, log2_of(block),
                                  dh,         n,           dgate,    dup,       h};
    return launched(zq::launch_swiglu_grad(a, t, (hipStream_t)stream));
}

size_t zq_linear_grad_workspace(size_t n_tok, uint64_t out_dim, uint64_t in_dim) {
    if (n_tok == 0 || !linear_sizes_ok(n_tok, out_dim, in_dim))
        return 0;
    return zq::linear_grad_workspace((uint32_t)n_tok, (uint32_t)out_dim, (uint32_t)in_dim);
}

zq_status zq_linear_grad_int8(const void* dy, zq_dtype dtype, const int8_t* codes,
                              const float* scales, uint32_t block, size_t n_tok, uint64_t out_dim,
                              uint64_t in_dim, void* grad, zq_dtype grad_dtype,
                              zq_grad_mode mode_arg, void* workspace, size_t workspace_bytes,
                              void* stream) {
    const int t = raw_enum(dtype), g = raw_enum(grad_dtype), mode = raw_enum(mode_arg);
    if (!half_dtype(t) || !known_dtype(g) || (mode != ZQ_GRAD_WRITE && mode != ZQ_GRAD_ADD))
        return ZQ_ERR_DTYPE;
    if (!valid_block(block))
        return ZQ_ERR_BLOCK;
    if (!linear_sizes_ok(n_tok, out_dim, in_dim))
        return ZQ_ERR_SIZE;
    const size_t gb = out_dim * in_dim * dtype_bytes(g);
    if (n_tok == 0) {
        if (mode != ZQ_GRAD_WRITE)
            return ZQ_OK;
        if (!grad)
            return ZQ_ERR_NULL;
        if (!aligned(grad, 16))
            return ZQ_ERR_ALIGN;
        return launched(zq::launch_clear(grad, gb, (hipStream_t)stream));
    }
    const size_t need =
        zq::linear_grad_workspace((uint32_t)n_tok, (uint32_t)out_dim, (uint32_t)in_dim);
    if (workspace_bytes < need)
        return ZQ_ERR_SIZE;
    Buffers b;
    b.add(dy, n_tok * out_dim * 2, 16, false);
    b.add(codes, n_tok * in_dim, 16, false);
    b.add(scales, scale_bytes(n_tok * in_dim, block), 4, false);
    b.add(grad, gb, 16, true);
    b.add(workspace, need, 16, true);
    const zq_status st = b.check();
    if (st != ZQ_OK)
        return st;
    zq::LinearGradArgs a = {dy, codes, scales, log2_of(block), (uint32_t)n_tok, (uint32_t)out_dim,
                            (uint32_t)in_dim, grad, workspace};
    return launched(zq::launch_linear_grad(a, t, g, mode, (hipStream_t)stream));
}

size_t zq_ce_loss_workspace(size_t n_tok, uint64_t rows, uint64_t dim, uint64_t piece) {
    if (n_tok == 0 || !ce_sizes_ok(n_tok, rows, dim))
        return 0;
    return zq::ce_loss_workspace((uint32_t)n_tok, (uint32_t)rows, (uint32_t)dim, piece);
}

zq_status zq_ce_loss(const void* x, zq_dtype dtype, size_t n_tok, uint64_t dim, const void* w,
                     uint64_t rows, const void* ids, zq_index_type id_type, float scale,
                     float* loss, float* lse, uint64_t piece, void* workspace,
                     size_t workspace_bytes, void* stream) {
    return ce_loss(x, dtype, n_tok, dim, {w, nullptr, 0}, rows, ids, id_type, scale, loss, lse,
                   piece, workspace, workspace_bytes, stream);
}

zq_status zq_ce_loss_int8(const void* x, zq_dtype dtype, size_t n_tok, uint64_t dim,
                          const int8_t* codes, const float* scales, uint32_t block, uint64_t rows,
                          const void* ids, zq_index_type id_type, float scale, float* loss,
                          float* lse, uint64_t piece, void* workspace, size_t workspace_bytes,
                          void* stream) {
    if (block == 0)
        return ZQ_ERR_BLOCK;
    return ce_loss(x, dtype, n_tok, dim, {codes, scales, block}, rows, ids, id_type, scale, loss,
                   lse, piece, workspace, workspace_bytes, stream);
}

size_t zq_ce_grad_workspace(size_t n_tok, uint64_t rows, uint64_t dim, uint64_t piece) {
    if (n_tok == 0 || !ce_sizes_ok(n_tok, rows, dim))
        return 0;
    return zq::ce_grad_workspace((uint32_t)n_tok, (uint32_t)rows, (uint32_t)dim, piece);
}

zq_status zq_ce_grad(const void* x, zq_dtype dtype, size_t n_tok, uint64_t dim, const void* w,
                     uint64_t rows, const void* ids, zq_index_type id_type, float scale,
                     const float* lse, const float* dloss, void* dx, void* dw, zq_dtype dw_dtype,
                     zq_grad_mode mode, uint64_t piece, void* workspace, size_t workspace_bytes,
                     void* stream) {
    return ce_grad(x, dtype, n_tok, dim, {w, nullptr, 0}, rows, ids, id_type, scale, lse, dloss, dx,
                   dw, dw_dtype, mode, piece, workspace, workspace_bytes, stream);
}

zq_status zq_ce_grad_int8(const void* x, zq_dtype dtype, size_t n_tok, uint64_t dim,
                          const int8_t* codes, const float* scales, uint32_t block, uint64_t rows,
                          const void* ids, zq_index_type id_type, float scale, const float* lse,
                          const float* dloss, void* dx, void* dw, zq_dtype dw_dtype,
                          zq_grad_mode mode, uint64_t piece, void* workspace,
                          size_t workspace_bytes, void* stream) {
    if (block == 0)
        return ZQ_ERR_BLOCK;
    return ce_grad(x, dtype, n_tok, dim, {codes, scales, block}, rows, ids, id_type, scale, lse,
                   dloss, dx, dw, dw_dtype, mode, piece, workspace, workspace_bytes, stream);
}

}  // extern "C"
