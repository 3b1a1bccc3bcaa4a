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

// Options these operators take: a path, the limit of its waits and, in the
// test build of the library, the staged path's fault.
rmsnorm_status_t check_options(const rmsnorm_options_t* opt, NormCall* c) {
    if (!opt) return RMSNORM_OK;
    const rmsnorm_options_t& o = *opt;
    if (o.cluster || o.threads || o.grid || o.vec_bytes || o.chunk_bytes || o.stages || o.weights ||
        o.reserved || o.epilogue || o.fault_inject < 0 || o.fault_inject > 2)
        return RMSNORM_ERR_INVALID_ARG;
    if (o.path != RMSNORM_PATH_AUTO && o.path != RMSNORM_PATH_STAGED &&
        o.path != RMSNORM_PATH_TWOPASS)
        return RMSNORM_ERR_INVALID_ARG;
    if (o.fault_inject &&
        (!RMSNORM_FAULT_INJECT || o.fault_inject != 1 || o.path != RMSNORM_PATH_STAGED))
        return RMSNORM_ERR_UNSUPPORTED;
    c->opt = o;
    return RMSNORM_OK;
}

void set_waits(NormCall* c) {
    c->p.status = c->dv.status;
    c->p.fault = c->opt.fault_inject;
    c->p.timeout_ns = c->opt.wait_timeout_ns ? c->opt.wait_timeout_ns : kDefaultTimeoutNs;
}

void count_vectors(NormCall* c, uintptr_t bits) {
    c->vb = widest_vector(bits, static_cast<int64_t>(c->p.hidden) * c->sz, c->sz);
    c->p.nvec = c->p.hidden / (c->vb / c->sz);
}

rmsnorm_status_t launch(const NormCall& c, NormFn fn, const LaunchShape& s, cudaStream_t stream) {
    return note(launch_ex(fn, s, stream, c.p)) == cudaSuccess ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

int pow2_ceil(int64_t v) {
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

int clamp_grid(int64_t want, int64_t most) { return static_cast<int>(want < most ? want : most); }

// ------------------------------------------------------ layer norm forward --

// How rows are staged (k_blockring.cuh): as they are where they, the arrays and
// the weights are on 16-byte boundaries, else shifted, which wants the arrays on
// one and rows of 32 bytes at least.
struct StagedRows {
    bool shift;
    int period;             // rows after which their alignment repeats
    int64_t nvec;           // whole vectors of a row, at most
    int64_t row_slot;       // bytes of a row in shared memory: the vectors it touches
};

bool staged_rows(const NormCall& c, uintptr_t more_weights, StagedRows* r) {
    const NormParams& p = c.p;
    const int64_t row_bytes = static_cast<int64_t>(p.hidden) * c.sz;
    if (!aligned(p.x, 16) || !aligned(p.dy, 16) || !aligned(p.out, 16)) return false;
    const int epv = 16 / c.sz;
    r->shift = row_bytes % 16 != 0 || !aligned(p.w, 16) || more_weights % 16 != 0;
    r->period = 1;
    r->nvec = row_bytes / 16;
    r->row_slot = row_bytes;
    if (!r->shift) return true;
    if (row_bytes < 32 || row_bytes > (1 << 20)) return false;
    while (r->period * p.hidden % epv != 0) r->period *= 2;
    r->nvec = p.hidden / epv;
    r->row_slot = (static_cast<int64_t>(p.hidden) + 2 * (epv - 1)) / epv * 16;
    return true;
}

// CTAs for blocks of `block_rows` rows: one wave, at least one per alignment.
int staged_grid(const NormCall& c, const StagedRows& r, int64_t block_rows, int64_t resident) {
    const int64_t blocks = r.period * div_up(div_up(c.p.rows, r.period), block_rows);
    const int64_t n = blocks < resident ? blocks : resident;
    return static_cast<int>(n < r.period ? r.period : n);
}

// Rows staged in shared memory: 64 bytes of a row per thread, CTAs of 256 threads
// or one row, a ring of two blocks, one wave of resident CTAs.  Measured (% of
// the HBM copy peak), 65536 rows of 4096 fp32 / 4096 bf16 / 8192 bf16: 32 bytes a
// thread 75 / 70 / 68, 64 bytes 99 / 91 / 92, 128 bytes (fewer, longer threads)
// 89 / 87 / 88; rings of three blocks (fewer CTAs) 92 / 87 / 88; CTAs of about
// four blocks each instead of one wave 92 / 85 / 81 (each CTA starts with an
// empty ring).  Leaves *fn null, status OK, where rows cannot be staged or two
// blocks do not fit shared memory.
constexpr int64_t kStagedRowBytesPerThread = 64;
constexpr int64_t kStagedBlock = 256;
constexpr int64_t kStagedSlots = 2;

int group_of(int64_t nvec, int64_t vecs_per_thread, int least) {
    int64_t g = div_up(nvec, vecs_per_thread);
    if (g > 1024) return 1024;
    if (g < least) g = least;
    return g <= 32 ? pow2_ceil(g) : static_cast<int>(div_up(g, 32) * 32);
}

rmsnorm_status_t plan_staged(int32_t dtype, NormCall* c, LaunchShape* s, NormFn* fn) {
    StagedRows r;
    if (!staged_rows(*c, reinterpret_cast<uintptr_t>(c->p.b), &r)) return RMSNORM_OK;
    const int group = group_of(r.nvec, kStagedRowBytesPerThread / 16, 1);
    const int64_t rpc = group < kStagedBlock ? kStagedBlock / group : 1;
    const int block = static_cast<int>(rpc * group);
    const int64_t bytes = kStagedSlots * rpc * r.row_slot + (r.shift ? 2 * r.row_slot : 0);
    if (bytes > c->dv.smem_optin - 2048) return RMSNORM_OK;
    const int smem = static_cast<int>(bytes);
    const NormFn f = layernorm_staged_ptr(dtype, r.shift);
    int occ = 0;
    if (cached_occupancy(c->dv.dev, c->dv.smem_optin, reinterpret_cast<KernelFn>(f), block, smem, 1,
                         &occ) != cudaSuccess)
        return RMSNORM_ERR_CUDA;
    if (occ < 1) return RMSNORM_OK;
    *s = LaunchShape{staged_grid(*c, r, rpc, static_cast<int64_t>(c->dv.sms) * occ), block, 1, smem};
    *fn = f;
    c->p.group = group;
    c->p.rows_per_cta = static_cast<int32_t>(rpc);
    c->p.nslots = static_cast<int32_t>(kStagedSlots);
    c->p.row_slot = static_cast<int32_t>(r.row_slot);
    c->p.period = r.period;
    set_waits(c);
    return RMSNORM_OK;
}

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
    LaunchShape s{0, 0, 1, 0};
    NormFn fn = nullptr;
    if (c.opt.path != RMSNORM_PATH_TWOPASS) {
        st = plan_staged(dtype, &c, &s, &fn);
        if (st == RMSNORM_ERR_CUDA) return st;
    }
    if (!fn) {
        if (c.opt.path == RMSNORM_PATH_STAGED) return RMSNORM_ERR_UNSUPPORTED;
        s = LaunchShape{clamp_grid(rows, 8ll * c.dv.sms), layernorm_twopass_block(), 1, 0};
        fn = layernorm_twopass_ptr(dtype, c.vb);
    }
    return launch(c, fn, s, stream);
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

// Rows staged in shared memory, read once: 16 elements of a row per thread, 32
// where a row needs more than 512 threads otherwise; CTAs of 256 threads or one
// row, a ring of three blocks, one wave of resident CTAs.  Two rows between
// barriers (16 elements; rows that fill their threads, in layer norm bf16 others
// too) for RMSNorm, unless in bf16 that halves the resident CTAs, and for layer
// norm, whose kernel then starts more slowly, where it leaves every CTA a dozen
// such blocks.  Measured (us, one row / two):
//   layer norm fp32 65536 x 1024 132 / 125, 16384 x 4096 131 / 131, 8192 x 4096 72 /
//     73, 4096 x 4096 42 / 45, bf16 65536 x 8192 539 / 531, 4096 x 4096 30 / 34
//   RMSNorm bf16 65536 x 8192 581 / 496, 131072 x 512 80 / 67, 4096 x 512 9.9 / 7.1,
//     128 x 2048 6.5 / 5.6, fp32 32768 x 4096 258 / 246, 1024 x 4096 18.3 / 18.1
//   half as many CTAs: bf16 30000 x 5120 152 / 181, fp32 15000 x 5120 146 / 150
//   rows that leave threads idle: layer norm bf16 65536 x 1280 128 / 114, 30000 x
//     5568 249 / 232, but fp32 65536 x 768 102 / 153, RMSNorm bf16 65536 x 1280 95 / 107
// Rings of two blocks, % of the HBM copy peak: 80 against 89 (layer norm bf16,
// 8192), 84 against 97 (fp32), 61 against 95 (RMSNorm bf16, 4096); of four the same
// as three or, where they cost a CTA per SM, 65 (layer norm bf16, 4096).  8
// elements per thread: bf16 rows of 4096 68, fp32 99.  32 elements against two
// reads of the row: bf16 rows of 16384, layer norm 86 / 50, RMSNorm 98 / 52.
constexpr int64_t kBwdBlock = 256;
constexpr int64_t kBwdSlots = 3;
constexpr int64_t kBwdMaxHidden = 32ll * kNormBwdMaxThreads;
constexpr int64_t kBwdTwoRowBlocks = 12;    // layer norm: blocks per CTA from which two rows pay

// Most CTAs of the one-pass kernel, and so its most parts: four per SM, fewer
// for rows that take a large share of an SM's threads, none for rows that it
// cannot hold.
int64_t bwd_staged_ctas(const DeviceView& dv, int64_t hidden) {
    if (hidden > kBwdMaxHidden) return 0;
    const int64_t per_sm = 16384 / hidden;
    return dv.sms * (per_sm < 1 ? 1 : (per_sm > 4 ? 4 : per_sm));
}

rmsnorm_status_t plan_bwd_staged(int32_t dtype, NormCall* c, LaunchShape* s, NormFn* fn) {
    StagedRows r;
    if (c->p.hidden > kBwdMaxHidden || !staged_rows(*c, 0, &r)) return RMSNORM_OK;
    const int epv = 16 / c->sz;
    const int elems = r.nvec * epv > 16 * kNormBwdMaxThreads ? 32 : 16;
    const int64_t vecs = elems / epv;
    const int group = group_of(r.nvec, vecs, r.shift ? 16 : 1);     // shifted: a thread per edge element
    const int64_t rpc = group < kBwdBlock ? kBwdBlock / group : 1;
    const int block = static_cast<int>(rpc * group);
    const bool bf16 = dtype == RMSNORM_DTYPE_BF16;
    const bool fills = c->p.w && r.nvec == group * vecs && !(elems == 32 && c->layer);
    const int mode = r.shift ? 2 : (fills ? 0 : 1);
    const int64_t weights = r.shift ? r.row_slot : 0;
    const int64_t budget = c->dv.smem_optin - 2048 - weights;
    const int64_t ctas_most = bwd_staged_ctas(c->dv, c->p.hidden);
    struct Form {            // rows between barriers, and what a launch of them takes
        int rows;
        int64_t slots;
        int smem, occ;
        NormFn fn;
    };
    // false: a CUDA error; occ 0: does not fit
    auto form = [&](int rows, Form* o) {
        const int64_t slot = rows * rpc * r.row_slot;       // of one array
        *o = Form{rows, kBwdSlots, 0, 0, nullptr};
        while (o->slots > 2 && 2 * o->slots * slot > budget) --o->slots;
        if (2 * o->slots * slot > budget) return true;
        o->smem = static_cast<int>(2 * o->slots * slot + weights);
        o->fn = bf16 ? norm_bwd_staged_ptr_bf16(elems, c->layer, rows, mode)
                     : norm_bwd_staged_ptr_f32(elems, c->layer, rows, mode);
        return cached_occupancy(c->dv.dev, c->dv.smem_optin, reinterpret_cast<KernelFn>(o->fn),
                                block, o->smem, 1, &o->occ) == cudaSuccess;
    };
    Form f, two;
    if (!form(1, &f)) return RMSNORM_ERR_CUDA;
    const bool whole = mode == 0 || (mode == 1 && c->layer && bf16);
    if (whole && elems == 16 &&
        (!c->layer || c->p.rows >= 2 * rpc * kBwdTwoRowBlocks * ctas_most)) {
        if (!form(2, &two)) return RMSNORM_ERR_CUDA;
        if (two.occ > 0 && (c->layer || !bf16 || f.occ < 2 * two.occ)) f = two;
    }
    if (f.occ < 1) return RMSNORM_OK;
    int64_t ctas = static_cast<int64_t>(c->dv.sms) * f.occ;
    if (ctas > ctas_most) ctas = ctas_most;
    *s = LaunchShape{staged_grid(*c, r, f.rows * rpc, ctas), block, 1, f.smem};
    *fn = f.fn;
    c->p.group = group;
    c->p.rows_per_cta = static_cast<int32_t>(rpc);
    c->p.nslots = static_cast<int32_t>(f.slots);
    c->p.row_slot = static_cast<int32_t>(r.row_slot);
    c->p.period = r.period;
    c->p.parts = s->grid;
    set_waits(c);
    return RMSNORM_OK;
}

struct BwdSpace {
    int64_t parts;
    uint64_t row_stats, part_w, part_b, bytes;    // offsets, and the size
};

BwdSpace bwd_space(const DeviceView& dv, int64_t rows, int64_t hidden, int sz, bool layer) {
    BwdSpace s;
    auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
    s.parts = bwd_parts(dv, rows, hidden, sz);
    int64_t staged = bwd_staged_ctas(dv, hidden);
    if (staged > rows + 8) staged = rows + 8;     // a block more per alignment at most
    if (s.parts < staged) s.parts = staged;
    s.row_stats = 0;
    s.part_w = up(static_cast<uint64_t>(rows) * 8);
    s.part_b = s.part_w + up(static_cast<uint64_t>(s.parts) * hidden * 4);
    s.bytes = layer ? s.part_b + up(static_cast<uint64_t>(s.parts) * hidden * 4) : s.part_b;
    return s;
}

rmsnorm_status_t launch_reduce(const NormCall& c, cudaStream_t stream) {
    const int width = c.p.hidden % 4 == 0 ? 4 : 1;
    LaunchShape s{static_cast<int>(div_up(c.p.hidden, kNormReduceCols * width)), kNormReduceThreads,
                  1, 0};
    s.grid_y = c.p.db ? 2 : 1;
    return launch(c, norm_bwd_reduce_ptr(width), s, stream);
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
    c.layer = layer;
    if (c.opt.path != RMSNORM_PATH_TWOPASS) {
        LaunchShape s{0, 0, 1, 0};
        NormFn fn = nullptr;
        st = plan_bwd_staged(dtype, &c, &s, &fn);
        if (st == RMSNORM_ERR_CUDA) return st;
        if (fn) {
            st = launch(c, fn, s, stream);
            if (st != RMSNORM_OK || (!dw && !db)) return st;
            return launch_reduce(c, stream);
        }
        if (c.opt.path == RMSNORM_PATH_STAGED) return RMSNORM_ERR_UNSUPPORTED;
    }
    c.p.rows_per_part = div_up(rows, bwd_parts(c.dv, rows, hidden, c.sz));
    c.p.parts = static_cast<int32_t>(div_up(rows, c.p.rows_per_part));
    const LaunchShape rs{clamp_grid(rows, 8ll * c.dv.sms), norm_bwd_rows_block(), 1, 0};
    st = launch(c, norm_bwd_rows_ptr(dtype, c.vb, layer), rs, stream);
    if (st != RMSNORM_OK) return st;
    LaunchShape cs{static_cast<int>(div_up(c.p.nvec, norm_bwd_cols_block())), norm_bwd_cols_block(), 1, 0};
    cs.grid_y = c.p.parts;
    st = launch(c, norm_bwd_cols_ptr(dtype, c.vb, layer), cs, stream);
    if (st != RMSNORM_OK || (!dw && !db)) return st;
    return launch_reduce(c, stream);
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
