// norm_api.cu -- C ABI of layer norm (include/layernorm.h) and of the norm
// backward passes: validation, kernel choice and launch.  Shares the library's
// per-device state (device.h) and status conventions with the other entry
// points.
#include "layernorm.h"
#include "checks.h"
#include "device.h"
#include "norm_launch.h"

#include <cmath>
#include <cstdio>
#include <cstring>

namespace rmsnorm {
namespace {

constexpr int64_t kMaxHidden = 0x7FFFFFFFll;

struct NormCall {
    int sz = 0;
    bool layer = false;
    int vb = 0;                 // widest vector of the arrays and the row pitch
    NormParams p;
    rmsnorm_options_t opt;
    DeviceView dv;
};

rmsnorm_status_t check_shape(int32_t dtype, int64_t rows, int64_t hidden, NormCall* c) {
    if (dtype != RMSNORM_DTYPE_F32 && dtype != RMSNORM_DTYPE_BF16) return RMSNORM_ERR_INVALID_ARG;
    std::memset(&c->p, 0, sizeof(c->p));
    std::memset(&c->opt, 0, sizeof(c->opt));
    c->sz = dtype == RMSNORM_DTYPE_F32 ? 4 : 2;
    if (rows < 0 || hidden <= 0 || hidden > kMaxHidden) return RMSNORM_ERR_INVALID_ARG;
    // every array of this shape, the fp32 pair of each row included, has a size in 63 bits
    if (rows > (INT64_MAX / 8) / hidden) return RMSNORM_ERR_INVALID_ARG;
    c->p.rows = rows;
    c->p.hidden = static_cast<int32_t>(hidden);
    c->p.inv_hidden = 1.0f / static_cast<float>(hidden);
    return RMSNORM_OK;
}

// Options these operators take: a path, and nothing else.
rmsnorm_status_t check_options(const rmsnorm_options_t* opt, NormCall* c) {
    if (!opt) return RMSNORM_OK;
    const rmsnorm_options_t& o = *opt;
    if (o.cluster || o.threads || o.grid || o.vec_bytes || o.chunk_bytes || o.stages || o.weights ||
        o.reserved || o.epilogue)
        return RMSNORM_ERR_INVALID_ARG;
    if (o.fault_inject) return o.fault_inject < 0 || o.fault_inject > 2 ? RMSNORM_ERR_INVALID_ARG
                                                                        : RMSNORM_ERR_UNSUPPORTED;
    if (o.path != RMSNORM_PATH_AUTO && o.path != RMSNORM_PATH_TWOPASS) return RMSNORM_ERR_INVALID_ARG;
    c->opt = o;
    return RMSNORM_OK;
}

void count_vectors(NormCall* c, uintptr_t bits) {
    c->vb = widest_vector(bits, static_cast<int64_t>(c->p.hidden) * c->sz, c->sz);
    c->p.nvec = c->p.hidden / (c->vb / c->sz);
}

rmsnorm_status_t launch(const NormCall& c, NormFn fn, const LaunchShape& s, cudaStream_t stream) {
    return note(launch_ex(fn, s, stream, c.p)) == cudaSuccess ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

int clamp_grid(int64_t want, int64_t most) { return static_cast<int>(want < most ? want : most); }

// ------------------------------------------------------ layer norm forward --

rmsnorm_status_t layernorm_run(int32_t dtype, const void* x, const void* w, const void* b, void* y,
                               float* mean, float* rstd, int64_t rows, int64_t hidden, float eps,
                               const rmsnorm_options_t* opt, cudaStream_t stream) {
    NormCall c;
    rmsnorm_status_t st = check_shape(dtype, rows, hidden, &c);
    if (st != RMSNORM_OK) return st;
    if (!x || !y || !std::isfinite(eps) || eps < 0.f) return RMSNORM_ERR_INVALID_ARG;
    const uintptr_t sz = static_cast<uintptr_t>(c.sz);
    if (!aligned(x, sz) || !aligned(w, sz) || !aligned(b, sz) || !aligned(y, sz) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return RMSNORM_ERR_INVALID_ARG;
    const uint64_t n = static_cast<uint64_t>(rows) * hidden * sz;
    const uint64_t nh = static_cast<uint64_t>(hidden) * sz, nr = static_cast<uint64_t>(rows) * 4;
    const Span in[] = {span(x, n), span(w, nh), span(b, nh), span(y, n), span(mean, nr)};
    if (clashes(in[3], in, 3, 1) || clashes(in[4], in, 4, 0) || clashes(span(rstd, nr), in, 5, 0))
        return RMSNORM_ERR_INVALID_ARG;
    st = check_options(opt, &c);
    if (st != RMSNORM_OK) return st;
    if (rows == 0) return RMSNORM_OK;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    c.p.x = x;
    c.p.w = w;
    c.p.b = b;
    c.p.out = y;
    c.p.mean = mean;
    c.p.rstd = rstd;
    c.p.eps = eps;
    count_vectors(&c, in[0].p | in[1].p | in[2].p | in[3].p);
    const LaunchShape s{clamp_grid(rows, 8ll * c.dv.sms), layernorm_twopass_block(), 1, 0};
    return launch(c, layernorm_twopass_ptr(dtype, c.vb), s, stream);
}

// --------------------------------------------------------- backward passes --

constexpr int64_t kBwdPartsWaves = 8;      // CTAs per SM the column kernel aims at
constexpr int64_t kBwdMaxParts = 512;

// Parts of the three-kernel backward pass: enough CTAs to fill the GPU, at
// least four rows each.  Independent of the vector width, so that the
// workspace is too.
int64_t bwd_parts(const DeviceView& dv, int64_t rows, int64_t hidden, int sz) {
    const int64_t col_ctas = div_up(hidden * sz, 16ll * norm_bwd_cols_block());
    int64_t parts = div_up(kBwdPartsWaves * dv.sms, col_ctas);
    if (parts > kBwdMaxParts) parts = kBwdMaxParts;
    if (parts > div_up(rows, 4)) parts = div_up(rows, 4);
    return parts < 1 ? 1 : parts;
}

struct BwdSpace {
    int64_t parts;
    uint64_t row_stats, part_w, part_b, bytes;    // offsets, and the size
};

BwdSpace bwd_space(const DeviceView& dv, int64_t rows, int64_t hidden, int sz, bool layer) {
    BwdSpace s;
    auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
    s.parts = bwd_parts(dv, rows, hidden, sz);
    s.row_stats = 0;
    s.part_w = up(static_cast<uint64_t>(rows) * 8);
    s.part_b = s.part_w + up(static_cast<uint64_t>(s.parts) * hidden * 4);
    s.bytes = layer ? s.part_b + up(static_cast<uint64_t>(s.parts) * hidden * 4) : s.part_b;
    return s;
}

rmsnorm_status_t bwd_workspace(int32_t dtype, int64_t rows, int64_t hidden, bool layer,
                               size_t* bytes) {
    NormCall c;
    if (!bytes) return RMSNORM_ERR_INVALID_ARG;
    const rmsnorm_status_t st = check_shape(dtype, rows, hidden, &c);
    if (st != RMSNORM_OK) return st;
    *bytes = 0;
    if (rows == 0) return RMSNORM_OK;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    *bytes = bwd_space(c.dv, rows, hidden, c.sz, layer).bytes;
    return RMSNORM_OK;
}

rmsnorm_status_t bwd_run(int32_t dtype, bool layer, const void* dy, const void* x, const void* w,
                         const float* mean, const float* rstd, void* dx, float* dw, float* db,
                         int64_t rows, int64_t hidden, float eps, void* workspace,
                         size_t workspace_bytes, const rmsnorm_options_t* opt,
                         cudaStream_t stream) {
    NormCall c;
    rmsnorm_status_t st = check_shape(dtype, rows, hidden, &c);
    if (st != RMSNORM_OK) return st;
    if (!dy || !x || !dx || (layer && (!mean || !rstd))) return RMSNORM_ERR_INVALID_ARG;
    if (!layer && (!std::isfinite(eps) || eps < 0.f)) return RMSNORM_ERR_INVALID_ARG;
    const uintptr_t sz = static_cast<uintptr_t>(c.sz);
    if (!aligned(dy, sz) || !aligned(x, sz) || !aligned(w, sz) || !aligned(dx, sz) ||
        !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dw, 4) || !aligned(db, 4) ||
        !aligned(workspace, 16))
        return RMSNORM_ERR_INVALID_ARG;
    const uint64_t n = static_cast<uint64_t>(rows) * hidden * sz;
    const uint64_t nh = static_cast<uint64_t>(hidden), nr = static_cast<uint64_t>(rows) * 4;
    const Span a[] = {span(dy, n), span(x, n), span(w, nh * sz), span(mean, nr), span(rstd, nr),
                      span(dx, n), span(dw, nh * 4), span(db, nh * 4)};
    if (clashes(a[5], a, 5, 2) || clashes(a[6], a, 6, 0) || clashes(a[7], a, 7, 0) ||
        clashes(span(workspace, workspace_bytes), a, 8, 0))
        return RMSNORM_ERR_INVALID_ARG;
    st = check_options(opt, &c);
    if (st != RMSNORM_OK) return st;
    if (rows == 0) {            // sums over no rows
        if (dw && note(cudaMemsetAsync(dw, 0, nh * 4, stream)) != cudaSuccess) return RMSNORM_ERR_CUDA;
        if (db && note(cudaMemsetAsync(db, 0, nh * 4, stream)) != cudaSuccess) return RMSNORM_ERR_CUDA;
        return RMSNORM_OK;
    }
    if (!workspace) return RMSNORM_ERR_INVALID_ARG;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    const BwdSpace ws = bwd_space(c.dv, rows, hidden, c.sz, layer);
    if (workspace_bytes < ws.bytes) return RMSNORM_ERR_INVALID_ARG;
    char* base = static_cast<char*>(workspace);
    c.p.x = x;
    c.p.dy = dy;
    c.p.w = w;
    c.p.out = dx;
    c.p.mean = const_cast<float*>(mean);
    c.p.rstd = const_cast<float*>(rstd);
    c.p.eps = eps;
    c.p.row_stats = reinterpret_cast<float2*>(base + ws.row_stats);
    c.p.part_w = dw ? reinterpret_cast<float*>(base + ws.part_w) : nullptr;
    c.p.part_b = db ? reinterpret_cast<float*>(base + ws.part_b) : nullptr;
    c.p.dw = dw;
    c.p.db = db;
    count_vectors(&c, a[0].p | a[1].p | a[2].p | a[5].p);
    c.p.rows_per_part = div_up(rows, ws.parts);
    c.p.parts = static_cast<int32_t>(div_up(rows, c.p.rows_per_part));
    const LaunchShape rs{clamp_grid(rows, 8ll * c.dv.sms), norm_bwd_rows_block(), 1, 0};
    st = launch(c, norm_bwd_rows_ptr(dtype, c.vb, layer), rs, stream);
    if (st != RMSNORM_OK) return st;
    LaunchShape cs{static_cast<int>(div_up(c.p.nvec, norm_bwd_cols_block())), norm_bwd_cols_block(), 1, 0};
    cs.grid_y = c.p.parts;
    st = launch(c, norm_bwd_cols_ptr(dtype, c.vb, layer), cs, stream);
    if (st != RMSNORM_OK || (!dw && !db)) return st;
    LaunchShape ds{static_cast<int>(div_up(hidden, kNormReduceCols)),
                   kNormReduceCols * kNormReduceLanes, 1, 0};
    ds.grid_y = db ? 2 : 1;
    return launch(c, norm_bwd_reduce_ptr(), ds, stream);
}

}  // namespace
}  // namespace rmsnorm

using namespace rmsnorm;

extern "C" {

rmsnorm_status_t layernorm_fwd_f32(const float* x, const float* w, const float* b, float* y,
                                   float* mean, float* rstd, int64_t rows, int64_t hidden,
                                   float eps, rmsnorm_stream_t stream) {
    return layernorm_run(RMSNORM_DTYPE_F32, x, w, b, y, mean, rstd, rows, hidden, eps, nullptr,
                         reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t layernorm_fwd_bf16(const uint16_t* x, const uint16_t* w, const uint16_t* b,
                                    uint16_t* y, float* mean, float* rstd, int64_t rows,
                                    int64_t hidden, float eps, rmsnorm_stream_t stream) {
    return layernorm_run(RMSNORM_DTYPE_BF16, x, w, b, y, mean, rstd, rows, hidden, eps, nullptr,
                         reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t layernorm_fwd_ex(int32_t dtype, const void* x, const void* w, const void* b,
                                  void* y, float* mean, float* rstd, int64_t rows, int64_t hidden,
                                  float eps, const rmsnorm_options_t* opt,
                                  rmsnorm_stream_t stream) {
    return layernorm_run(dtype, x, w, b, y, mean, rstd, rows, hidden, eps, opt,
                         reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t layernorm_bwd_workspace(int32_t dtype, int64_t rows, int64_t hidden,
                                         size_t* bytes) {
    return bwd_workspace(dtype, rows, hidden, true, bytes);
}

rmsnorm_status_t layernorm_bwd_f32(const float* dy, const float* x, const float* w,
                                   const float* mean, const float* rstd, float* dx, float* dw,
                                   float* db, int64_t rows, int64_t hidden, void* workspace,
                                   size_t workspace_bytes, rmsnorm_stream_t stream) {
    return bwd_run(RMSNORM_DTYPE_F32, true, dy, x, w, mean, rstd, dx, dw, db, rows, hidden, 0.f,
                   workspace, workspace_bytes, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t layernorm_bwd_bf16(const uint16_t* dy, const uint16_t* x, const uint16_t* w,
                                    const float* mean, const float* rstd, uint16_t* dx, float* dw,
                                    float* db, int64_t rows, int64_t hidden, void* workspace,
                                    size_t workspace_bytes, rmsnorm_stream_t stream) {
    return bwd_run(RMSNORM_DTYPE_BF16, true, dy, x, w, mean, rstd, dx, dw, db, rows, hidden, 0.f,
                   workspace, workspace_bytes, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t layernorm_bwd_ex(int32_t dtype, const void* dy, const void* x, const void* w,
                                  const float* mean, const float* rstd, void* dx, float* dw,
                                  float* db, int64_t rows, int64_t hidden, void* workspace,
                                  size_t workspace_bytes, const rmsnorm_options_t* opt,
                                  rmsnorm_stream_t stream) {
    return bwd_run(dtype, true, dy, x, w, mean, rstd, dx, dw, db, rows, hidden, 0.f, workspace,
                   workspace_bytes, opt, reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_bwd_workspace(int32_t dtype, int64_t rows, int64_t hidden,
                                       size_t* bytes) {
    return bwd_workspace(dtype, rows, hidden, false, bytes);
}

rmsnorm_status_t rmsnorm_bwd_f32(const float* dy, const float* x, const float* w, float* dx,
                                 float* dw, int64_t rows, int64_t hidden, float eps,
                                 void* workspace, size_t workspace_bytes,
                                 rmsnorm_stream_t stream) {
    return bwd_run(RMSNORM_DTYPE_F32, false, dy, x, w, nullptr, nullptr, dx, dw, nullptr, rows,
                   hidden, eps, workspace, workspace_bytes, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_bwd_bf16(const uint16_t* dy, const uint16_t* x, const uint16_t* w,
                                  uint16_t* dx, float* dw, int64_t rows, int64_t hidden, float eps,
                                  void* workspace, size_t workspace_bytes,
                                  rmsnorm_stream_t stream) {
    return bwd_run(RMSNORM_DTYPE_BF16, false, dy, x, w, nullptr, nullptr, dx, dw, nullptr, rows,
                   hidden, eps, workspace, workspace_bytes, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_bwd_ex(int32_t dtype, const void* dy, const void* x, const void* w,
                                void* dx, float* dw, int64_t rows, int64_t hidden, float eps,
                                void* workspace, size_t workspace_bytes,
                                const rmsnorm_options_t* opt, rmsnorm_stream_t stream) {
    return bwd_run(dtype, false, dy, x, w, nullptr, nullptr, dx, dw, nullptr, rows, hidden, eps,
                   workspace, workspace_bytes, opt, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
