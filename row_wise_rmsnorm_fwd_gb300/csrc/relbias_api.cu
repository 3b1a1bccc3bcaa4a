// relbias_api.cu -- C ABI of the row softmax with a learned relative position
// bias (include/rowsoftmax.h): validation, the bucket rule, kernel choice and
// launch.
#include "rowsoftmax.h"
#include "checks.h"
#include "device.h"
#include "relbias_launch.h"

#include <cmath>
#include <cstring>
#include <limits>

namespace rmsnorm {
namespace {

constexpr int64_t kMaxOffset = 1ll << 40;
constexpr int64_t kMaxHeadRows = 1ll << 30;    // a row's number plus a grid's stride is a 32-bit int
constexpr int64_t kWindowBudget = 64 << 10;    // shared memory of a CTA's windows, about
constexpr int64_t kBwdStatic = 4 << 10;        // of a backward CTA, other than windows, at most

// Smallest distance of each bucket of one direction (half of them): one by one
// up to half / 2 =: near, then where
//     near + log(n / near) / log(max_distance / near) * (half - near)
// reaches the bucket's number, for real logarithms: an edge that is a whole
// number (near * (max_distance / near)^(k / (half - near)) often is) belongs to
// the upper bucket.  Long doubles of 64 bits and more put an edge within 1e-18 of
// its value, relatively; over all rules that check_rule lets pass (half up to 256,
// max_distance up to 4096) no edge that is not whole lies within 4e-12 of a whole
// number, so what is within 1e-16 of one is one.
static_assert(std::numeric_limits<long double>::digits >= 64,
              "bucket edges: a long double of 64 bits or more");
void bucket_edges(int half, int max_distance, int32_t* edges) {
    const int near = half / 2;
    for (int k = 0; k < near; ++k) edges[k] = k;
    const long double ratio = static_cast<long double>(max_distance) / near;
    for (int k = near; k < half; ++k) {
        const long double e =
            near * powl(ratio, static_cast<long double>(k - near) / (half - near));
        const long double whole = roundl(e);
        edges[k] = static_cast<int32_t>(fabsl(e - whole) <= 1e-16L * e ? whole : ceill(e));
    }
}

rmsnorm_status_t check_rule(int num_buckets, int max_distance, int both, int* half) {
    if (both != 0 && both != 1) return RMSNORM_ERR_INVALID_ARG;
    if (num_buckets < 2 || num_buckets > kBiasMaxBuckets) return RMSNORM_ERR_INVALID_ARG;
    if (both && (num_buckets < 4 || num_buckets % 2 != 0)) return RMSNORM_ERR_INVALID_ARG;
    *half = both ? num_buckets / 2 : num_buckets;
    if (max_distance <= *half / 2 || max_distance > kBiasMaxDistance) return RMSNORM_ERR_INVALID_ARG;
    return RMSNORM_OK;
}

// The edges cost some powl calls; a thread keeps those of its last rule.
void fill_edges(BiasParams* p, int max_distance) {
    struct Last {
        int half = 0, max_distance = 0;
        int32_t edges[kBiasMaxBuckets];
    };
    static thread_local Last last;
    if (last.half != p->half || last.max_distance != max_distance) {
        bucket_edges(p->half, max_distance, last.edges);
        last.half = p->half;
        last.max_distance = max_distance;
    }
    std::memcpy(p->edges, last.edges, sizeof(int32_t) * p->half);
}

struct BiasCall {
    int sz = 0;
    int vb = 0;
    int64_t elems = 0;
    int64_t window = 0;         // the last edge
    BiasParams p;
    DeviceView dv;
};

rmsnorm_status_t check_call(int32_t dtype, int64_t batch, int64_t heads, int64_t q_len,
                            int64_t k_len, const rowsoftmax_relbias_t* a,
                            const rmsnorm_options_t* opt, BiasCall* c) {
    if (dtype != RMSNORM_DTYPE_F32 && dtype != RMSNORM_DTYPE_BF16) return RMSNORM_ERR_INVALID_ARG;
    if (!a || a->reserved != 0 || (a->causal != 0 && a->causal != 1)) return RMSNORM_ERR_INVALID_ARG;
    if (!std::isfinite(a->scale)) return RMSNORM_ERR_INVALID_ARG;
    if (batch < 0 || q_len < 0 || heads <= 0 || k_len <= 0) return RMSNORM_ERR_INVALID_ARG;
    if (heads > 65535 || k_len > kBiasMaxKeys) return RMSNORM_ERR_INVALID_ARG;
    if (q_len > kMaxHeadRows || batch > kMaxHeadRows || (q_len > 0 && batch > kMaxHeadRows / q_len))
        return RMSNORM_ERR_INVALID_ARG;
    if (a->q_offset > kMaxOffset || a->q_offset < -kMaxOffset) return RMSNORM_ERR_INVALID_ARG;
    if (!aligned(a->q_start, 4) || !aligned(a->kv_len, 4)) return RMSNORM_ERR_INVALID_ARG;
    std::memset(&c->p, 0, sizeof(c->p));
    BiasParams& p = c->p;
    const rmsnorm_status_t st = check_rule(a->num_buckets, a->max_distance, a->bidirectional, &p.half);
    if (st != RMSNORM_OK) return st;
    c->sz = dtype == RMSNORM_DTYPE_F32 ? 4 : 2;
    // batch * q_len <= 2^30 and heads * k_len < 2^46: the product may pass 63 bits
    if (batch * q_len > 0 && heads * k_len > (INT64_MAX / 8) / (batch * q_len))
        return RMSNORM_ERR_INVALID_ARG;
    c->elems = batch * q_len * heads * k_len;
    if (opt) {
        const rmsnorm_options_t& o = *opt;
        if (o.cluster || o.threads || o.grid || o.vec_bytes || o.chunk_bytes || o.stages ||
            o.weights || o.reserved || o.epilogue || o.fault_inject)
            return RMSNORM_ERR_INVALID_ARG;
        if (o.path != RMSNORM_PATH_AUTO && o.path != RMSNORM_PATH_ROWREG &&
            o.path != RMSNORM_PATH_TWOPASS)
            return RMSNORM_ERR_INVALID_ARG;
    }
    p.elems = c->elems;
    p.q_start = a->q_start;
    p.kv_len = a->kv_len;
    p.q_offset = a->q_offset;
    p.scale = a->scale;
    p.head_rows = static_cast<int32_t>(batch * q_len);
    p.q_len = static_cast<int32_t>(q_len);
    p.k_len = static_cast<int32_t>(k_len);
    p.heads = static_cast<int32_t>(heads);
    p.causal = a->causal;
    p.both = a->bidirectional;
    p.num_buckets = a->num_buckets;
    fill_edges(&p, a->max_distance);
    c->window = p.edges[p.half - 1];
    return RMSNORM_OK;
}

int path(const rmsnorm_options_t* opt) { return opt ? opt->path : RMSNORM_PATH_AUTO; }

// CTAs per head: at most `per_sm` CTAs per SM over all heads (one wave), at
// most one per row block, at least one.
int parts_per_head(const BiasCall& c, int64_t row_blocks, int64_t per_sm) {
    int64_t n = per_sm * c.dv.sms / c.p.heads;
    if (n > row_blocks) n = row_blocks;
    return static_cast<int>(n < 1 ? 1 : n);
}

constexpr int64_t kCtasPerSm = 8;           // at most, over all heads

int most_parts(const BiasCall& c) { return parts_per_head(c, c.p.head_rows, kCtasPerSm); }

rmsnorm_status_t launch(const BiasCall& c, BiasFn fn, const LaunchShape& s, cudaStream_t stream) {
    if (ensure_prepared(c.dv.dev, reinterpret_cast<KernelFn>(fn), c.dv.smem_optin) != cudaSuccess)
        return RMSNORM_ERR_CUDA;
    return note(launch_ex(fn, s, stream, c.p)) == cudaSuccess ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

void count_vectors(BiasCall* c, uintptr_t bits) {
    c->vb = widest_vector(bits, static_cast<int64_t>(c->p.k_len) * c->sz, c->sz);
    c->p.nvec = c->p.k_len / (c->vb / c->sz);
}

int window_bytes(const BiasCall& c) {
    const int lo = static_cast<int>(c.window);
    return 4 * bias_window_slots(lo, c.p.both ? lo : 0, c.vb / c.sz);
}

// Rows in registers, if they fit and the arrays start on 16-byte boundaries:
// the launch shape and the kernel; else leaves *fn null, status OK.
rmsnorm_status_t plan_rowreg(int32_t dtype, BiasCall* c, uintptr_t bases, bool bwd, bool forced,
                             LaunchShape* s, BiasFn* fn) {
    if (bases % 16 != 0) return RMSNORM_OK;
    const int64_t epv = 16 / c->sz;
    const bool shift = c->p.k_len % epv != 0;
    // vectors a row touches, wherever it starts
    const int64_t nvec = shift ? (c->p.k_len + 2 * (epv - 1)) / epv : c->p.k_len / epv;
    // Threads per row, of nv vectors each: whole warps, or a power of two.
    auto threads_of = [&](int64_t nv) {
        const int64_t n = div_up(nvec, nv);
        if (n > 32) return div_up(n, 32) * 32;
        int64_t g = 1;
        while (g < n) g <<= 1;
        return g;
    };
    // A row's time hardly depends on how many of its threads' vectors are in use,
    // so 6 vectors per thread where that takes fewer threads without room for more
    // vectors: up to two warps per row, forward bf16 at any width.  Measured (us,
    // 4 / 6): forward fp32 rows of 640 150 / 102, of 260 69 / 55, bf16 rows of 1536
    // 179 / 140, of 2056 156 / 131, of 6000 336 / 282, of 12000 101 / 74; backward
    // bf16 rows of 1536 226 / 182, of 2056 187 / 167, fp32 rows of 516 168 / 143.
    // Not below half a warp (backward, fp32 rows of 160: 60 / 62), nor with room for
    // more (forward, fp32 rows of 2048: 168 / 219; backward, bf16 rows of 3100: 246 /
    // 301), nor with more than two warps otherwise (forward, fp32 rows of 3000: 246 /
    // 260; backward, bf16 rows of 12000: 100 / 107).  And where 4 would need more
    // than the largest block, against the kernels that read rows twice (bf16 rows
    // of 24000, causal: forward 293 / 153, backward 294 / 214).
    int nv = 4;
    int64_t group = threads_of(nv);
    const int64_t six = threads_of(6);
    const bool fewer = 6 * six <= 4 * group && six >= 16 && (six <= 64 || (c->sz == 2 && !bwd));
    if (fewer || group > kBiasMaxThreads) {
        nv = 6;
        group = six;
    }
    if (group > kBiasMaxThreads) return RMSNORM_OK;
    const int lo = static_cast<int>(c->window);
    const BiasVecWindow vw = bias_vec_window(lo, c->p.both ? lo : 0, static_cast<int>(epv));
    const int window = 4 * vw.copies * vw.copy;
    const bool sums = bwd && c->p.part;
    // CTAs of 256 threads; forward bf16 and backward rows of two warps and more
    // 128.  Measured (us, 128 / 256 threads): forward bf16 rows of 2048 360 /
    // 411, fp32 rows of 1024 181 / 170; backward bf16 rows of 2048 509 / 532,
    // causal 427 / 460, rows of 512 (16 lanes) 99 / 75.
    const int64_t threads = bwd ? (group >= 64 ? 128 : 256) : (c->sz == 2 ? 128 : 256);
    int64_t rpc = group < threads ? threads / group : 1;
    int64_t windows = rpc, turns = 0;
    // Windows of sums: one for each row group that is a warp or more, as the budget
    // allows.  Where a warp has several rows, a window for each would leave an SM one
    // to six warps, so its rows add to one or two windows in turn (two where three CTAs
    // of them fit an SM, as many as their registers allow), and CTAs are halved until
    // two fit.  Measured (us, 2^25 scores, a window per row / in turn), 32 buckets up to
    // 128: bf16 rows of 8 keys 1058 / 115, of 32 266 / 62, of 128 80 / 47, fp32 of 64 140 /
    // 75; 64 buckets up to 500: bf16 of 8 8617 / 248, of 32 2276 / 123, of 128 303 / 68, of
    // 512 95 / 61, fp32 of 64 547 / 105.  One window a warp against two: bf16 of 32 keys 87
    // / 62, of 256 46 / 46; CTAs of one per SM against two, 64 buckets up to 1000: bf16 of
    // 64 172 / 150.
    if (sums && group < 32) {
        const int64_t per = 32 / group;                      // rows of a warp
        const int64_t sm = c->dv.smem_optin + 1024;          // an SM's
        auto bytes = [&](int64_t n) { return n * window + 4 * vw.size + kBwdStatic; };
        int64_t warps = threads / 32;
        while (warps > 1 && 2 * bytes(warps) > sm) warps /= 2;
        const int64_t each = 3 * bytes(2 * warps) <= sm ? 2 : 1;
        windows = warps * each;
        turns = per / each;
        rpc = warps * per;
    } else if (sums) {
        if (rpc > kWindowBudget / window) rpc = kWindowBudget / window;
        if (rpc < 1) rpc = 1;
        windows = rpc;
    }
    const int64_t smem = bwd ? (sums ? windows * window + 4 * vw.size : 0) : window;
    if (smem > c->dv.smem_optin - 8192) return RMSNORM_OK;
    const int block = static_cast<int>(rpc * group);
    const BiasFn f = relbias_rowreg_ptr(dtype, nv, shift, bwd, turns > 1);
    int occ = 0;
    if (cached_occupancy(c->dv.dev, c->dv.smem_optin, reinterpret_cast<KernelFn>(f), block,
                         static_cast<int>(smem), 1, &occ) != cudaSuccess)
        return RMSNORM_ERR_CUDA;
    if (occ < 1) return RMSNORM_OK;
    // Windows so large that an SM holds few warps beside them: the kernel that reads
    // rows twice, whose CTAs of 256 threads keep one of a quarter of the size.  Measured
    // (us, 2^25 scores, in registers / read twice), 64 buckets up to 2000, 128 threads: bf16
    // rows of 64 keys 357 / 1209, fp32 of 384 252 / 199; 128 buckets up to 4096: fp32 rows of 512 (32
    // threads) 1714 / 205, bf16 of 2048 (64) 417 / 91, fp32 of 8192 (512) 111 / 121.
    if (sums && !forced && occ * block < (turns > 1 ? 128 : 256)) return RMSNORM_OK;
    c->p.nvec = static_cast<int32_t>(nvec);
    c->p.group = static_cast<int32_t>(group);
    c->p.rows_per_cta = static_cast<int32_t>(rpc);
    c->p.turns = static_cast<int32_t>(turns);
    c->p.parts = parts_per_head(*c, div_up(c->p.head_rows, rpc), occ > kCtasPerSm ? kCtasPerSm : occ);
    *s = LaunchShape{c->p.parts * c->p.heads, block, 1, static_cast<int>(smem)};
    *fn = f;
    return RMSNORM_OK;
}

rmsnorm_status_t fwd_run(int32_t dtype, const void* x, const void* table, void* y, int64_t batch,
                         int64_t heads, int64_t q_len, int64_t k_len,
                         const rowsoftmax_relbias_t* a, const rmsnorm_options_t* opt,
                         cudaStream_t stream) {
    BiasCall c;
    const rmsnorm_status_t st = check_call(dtype, batch, heads, q_len, k_len, a, opt, &c);
    if (st != RMSNORM_OK) return st;
    if (!x || !table || !y) return RMSNORM_ERR_INVALID_ARG;
    const uintptr_t sz = static_cast<uintptr_t>(c.sz);
    if (!aligned(x, sz) || !aligned(table, sz) || !aligned(y, sz)) return RMSNORM_ERR_INVALID_ARG;
    const uint64_t n = static_cast<uint64_t>(c.elems) * sz;
    const uint64_t nb = static_cast<uint64_t>(batch) * 4;
    const Span in[] = {span(x, n), span(table, static_cast<uint64_t>(a->num_buckets) * heads * sz),
                       span(a->q_start, nb), span(a->kv_len, nb)};
    if (clashes(span(y, n), in, 4, 1)) return RMSNORM_ERR_INVALID_ARG;
    if (c.elems == 0) return RMSNORM_OK;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    c.p.x = x;
    c.p.table = table;
    c.p.out = y;
    const uintptr_t bases = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y);
    LaunchShape s{0, 0, 1, 0};
    BiasFn fn = nullptr;
    if (path(opt) != RMSNORM_PATH_TWOPASS &&
        plan_rowreg(dtype, &c, bases, false, path(opt) == RMSNORM_PATH_ROWREG, &s, &fn) != RMSNORM_OK)
        return RMSNORM_ERR_CUDA;
    if (!fn) {
        if (path(opt) == RMSNORM_PATH_ROWREG) return RMSNORM_ERR_UNSUPPORTED;
        count_vectors(&c, bases);
        c.p.parts = most_parts(c);
        s = LaunchShape{c.p.parts * c.p.heads, relbias_wide_block(), 1, window_bytes(c)};
        fn = relbias_fwd_wide_ptr(dtype, c.vb);
    }
    return launch(c, fn, s, stream);
}

// The parts never exceed most_parts for any vector width or alignment.
uint64_t space_needed(const BiasCall& c) {
    return static_cast<uint64_t>(most_parts(c)) * c.p.heads * c.p.num_buckets * 8;
}

rmsnorm_status_t bwd_run(int32_t dtype, const void* dy, const void* y, void* dx, float* dtable,
                         int64_t batch, int64_t heads, int64_t q_len, int64_t k_len,
                         const rowsoftmax_relbias_t* a, void* workspace, size_t workspace_bytes,
                         const rmsnorm_options_t* opt, cudaStream_t stream) {
    BiasCall c;
    rmsnorm_status_t st = check_call(dtype, batch, heads, q_len, k_len, a, opt, &c);
    if (st != RMSNORM_OK) return st;
    if (!dy || !y || !dx) return RMSNORM_ERR_INVALID_ARG;
    const uintptr_t sz = static_cast<uintptr_t>(c.sz);
    if (!aligned(dy, sz) || !aligned(y, sz) || !aligned(dx, sz) || !aligned(dtable, 4) ||
        !aligned(workspace, 16))
        return RMSNORM_ERR_INVALID_ARG;
    const uint64_t n = static_cast<uint64_t>(c.elems) * sz;
    const uint64_t nb = static_cast<uint64_t>(batch) * 4;
    const uint64_t nt = static_cast<uint64_t>(a->num_buckets) * heads * 4;
    const Span s[] = {span(dy, n), span(y, n), span(a->q_start, nb), span(a->kv_len, nb),
                      span(dx, n), span(dtable, nt)};
    if (clashes(s[4], s, 4, 2) || clashes(s[5], s, 5, 0) ||
        clashes(span(workspace, workspace_bytes), s, 6, 0))
        return RMSNORM_ERR_INVALID_ARG;
    if (c.elems == 0) {          // sums over no rows
        if (dtable && note(cudaMemsetAsync(dtable, 0, nt, stream)) != cudaSuccess)
            return RMSNORM_ERR_CUDA;
        return RMSNORM_OK;
    }
    if (dtable && !workspace) return RMSNORM_ERR_INVALID_ARG;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    if (dtable && workspace_bytes < space_needed(c)) return RMSNORM_ERR_INVALID_ARG;
    c.p.x = dy;
    c.p.y = y;
    c.p.out = dx;
    c.p.part = dtable ? static_cast<double*>(workspace) : nullptr;
    c.p.dtable = dtable;
    const uintptr_t bases = s[0].p | s[1].p | s[4].p;
    LaunchShape ls{0, 0, 1, 0};
    BiasFn fn = nullptr;
    if (path(opt) != RMSNORM_PATH_TWOPASS &&
        plan_rowreg(dtype, &c, bases, true, path(opt) == RMSNORM_PATH_ROWREG, &ls, &fn) != RMSNORM_OK)
        return RMSNORM_ERR_CUDA;
    if (!fn) {
        if (path(opt) == RMSNORM_PATH_ROWREG) return RMSNORM_ERR_UNSUPPORTED;
        count_vectors(&c, bases);
        c.p.parts = most_parts(c);
        ls = LaunchShape{c.p.parts * c.p.heads, relbias_wide_block(), 1, window_bytes(c)};
        fn = relbias_bwd_wide_ptr(dtype, c.vb);
    }
    st = launch(c, fn, ls, stream);
    if (st != RMSNORM_OK || !dtable) return st;
    LaunchShape rs{c.p.heads, relbias_reduce_block(), 1, 0};
    rs.grid_y = static_cast<int>(div_up(32ll * c.p.num_buckets, relbias_reduce_block()));
    return launch(c, relbias_reduce_ptr(), rs, stream);
}

}  // namespace
}  // namespace rmsnorm

using namespace rmsnorm;

extern "C" {

rmsnorm_status_t rowsoftmax_relbias_fwd_f32(const float* x, const float* table, float* y,
                                            int64_t batch, int64_t heads, int64_t q_len,
                                            int64_t k_len, const rowsoftmax_relbias_t* bias,
                                            rmsnorm_stream_t stream) {
    return fwd_run(RMSNORM_DTYPE_F32, x, table, y, batch, heads, q_len, k_len, bias, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rowsoftmax_relbias_fwd_bf16(const uint16_t* x, const uint16_t* table, uint16_t* y,
                                             int64_t batch, int64_t heads, int64_t q_len,
                                             int64_t k_len, const rowsoftmax_relbias_t* bias,
                                             rmsnorm_stream_t stream) {
    return fwd_run(RMSNORM_DTYPE_BF16, x, table, y, batch, heads, q_len, k_len, bias, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rowsoftmax_relbias_fwd_ex(int32_t dtype, const void* x, const void* table,
                                           void* y, int64_t batch, int64_t heads, int64_t q_len,
                                           int64_t k_len, const rowsoftmax_relbias_t* bias,
                                           const rmsnorm_options_t* opt,
                                           rmsnorm_stream_t stream) {
    return fwd_run(dtype, x, table, y, batch, heads, q_len, k_len, bias, opt,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rowsoftmax_relbias_bwd_workspace(int32_t dtype, int64_t batch, int64_t heads,
                                                  int64_t q_len, int64_t k_len,
                                                  const rowsoftmax_relbias_t* bias,
                                                  size_t* bytes) {
    BiasCall c;
    if (!bytes) return RMSNORM_ERR_INVALID_ARG;
    const rmsnorm_status_t st = check_call(dtype, batch, heads, q_len, k_len, bias, nullptr, &c);
    if (st != RMSNORM_OK) return st;
    *bytes = 0;
    if (c.elems == 0) return RMSNORM_OK;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    *bytes = space_needed(c);
    return RMSNORM_OK;
}

rmsnorm_status_t rowsoftmax_relbias_bwd_f32(const float* dy, const float* y, float* dx,
                                            float* dtable, int64_t batch, int64_t heads,
                                            int64_t q_len, int64_t k_len,
                                            const rowsoftmax_relbias_t* bias, void* workspace,
                                            size_t workspace_bytes, rmsnorm_stream_t stream) {
    return bwd_run(RMSNORM_DTYPE_F32, dy, y, dx, dtable, batch, heads, q_len, k_len, bias,
                   workspace, workspace_bytes, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rowsoftmax_relbias_bwd_bf16(const uint16_t* dy, const uint16_t* y, uint16_t* dx,
                                             float* dtable, int64_t batch, int64_t heads,
                                             int64_t q_len, int64_t k_len,
                                             const rowsoftmax_relbias_t* bias, void* workspace,
                                             size_t workspace_bytes, rmsnorm_stream_t stream) {
    return bwd_run(RMSNORM_DTYPE_BF16, dy, y, dx, dtable, batch, heads, q_len, k_len, bias,
                   workspace, workspace_bytes, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rowsoftmax_relbias_bwd_ex(int32_t dtype, const void* dy, const void* y, void* dx,
                                           float* dtable, int64_t batch, int64_t heads,
                                           int64_t q_len, int64_t k_len,
                                           const rowsoftmax_relbias_t* bias, void* workspace,
                                           size_t workspace_bytes, const rmsnorm_options_t* opt,
                                           rmsnorm_stream_t stream) {
    return bwd_run(dtype, dy, y, dx, dtable, batch, heads, q_len, k_len, bias, workspace,
                   workspace_bytes, opt, reinterpret_cast<cudaStream_t>(stream));
}

int32_t rowsoftmax_relbias_bucket(int64_t relative, int32_t num_buckets, int32_t max_distance,
                                  int32_t bidirectional) {
    int half;
    if (check_rule(num_buckets, max_distance, bidirectional, &half) != RMSNORM_OK) return -1;
    int32_t edges[kBiasMaxBuckets];
    bucket_edges(half, max_distance, edges);
    int64_t n = relative < 0 ? (relative == INT64_MIN ? INT64_MAX : -relative)
                             : (bidirectional ? relative : 0);
    int32_t k = half - 1;
    while (edges[k] > n) --k;
    return k + (bidirectional && relative > 0 ? half : 0);
}

}  // extern "C"
