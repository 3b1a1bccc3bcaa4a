// blocknorm_api.cu -- C ABI of the boundary between two blocks
// (include/rmsnorm_block.h): validation, kernel choice and launch.  Shares the
// library's per-device state (device.h) and status conventions with the other entry
// points.
#include "rmsnorm_block.h"
#include "blocknorm_launch.h"
#include "checks.h"
#include "device.h"

#include <cmath>
#include <cstring>

namespace rmsnorm {
namespace {

constexpr int64_t kMaxHidden = 1 << 20;
constexpr int kMaxCluster = 16;
constexpr int kLastFault = RMSNORM_FAULT_INJECT ? kFaultClusterLateThread : 2;

struct BlockCall {
    int dtype = 0;
    int sz = 0;
    BlockParams p;
    int32_t path = RMSNORM_PATH_AUTO;
    int32_t cluster = 0;         // forced; 0: automatic
    DeviceView dv;
};

rmsnorm_status_t check_shape(int32_t dtype, int64_t rows, int64_t hidden, const rmsnorm_block_t* b,
                             BlockCall* c) {
    if (dtype != RMSNORM_DTYPE_F32 && dtype != RMSNORM_DTYPE_BF16) return RMSNORM_ERR_INVALID_ARG;
    if (!b) return RMSNORM_ERR_INVALID_ARG;
    std::memset(&c->p, 0, sizeof(c->p));
    c->dtype = dtype;
    c->sz = dtype == RMSNORM_DTYPE_F32 ? 4 : 2;
    if (rows < 0 || hidden <= 0 || hidden > kMaxHidden) return RMSNORM_ERR_INVALID_ARG;
    // every array, the fp32 sums of each row and gate row included, has a size in 63 bits
    if (rows > (INT64_MAX / 64) / (hidden + 16)) return RMSNORM_ERR_INVALID_ARG;
    if (b->gate && b->gate_rows < 1) return RMSNORM_ERR_INVALID_ARG;
    BlockParams& p = c->p;
    p.rows = rows;
    p.hidden = static_cast<int32_t>(hidden);
    p.inv_hidden = 1.0f / static_cast<float>(hidden);
    p.gate_rows = b->gate && b->gate_rows < rows ? b->gate_rows : (rows > 0 ? rows : 1);
    p.gates = rows > 0 ? div_up(rows, p.gate_rows) : 1;
    return RMSNORM_OK;
}

// The rule and the options, once the shape is known to be good.
rmsnorm_status_t check_rule(const rmsnorm_block_t& b, const rmsnorm_options_t* opt, bool back, BlockCall* c) {
    if (b.post_norm < 0 || b.post_norm > 1 || b.pre_norm < 0 || b.pre_norm > 1 ||
        !std::isfinite(b.residual_scale) || !std::isfinite(b.branch_scale) ||
        !std::isfinite(b.post_eps) || b.post_eps < 0.f || !std::isfinite(b.pre_eps) || b.pre_eps < 0.f)
        return RMSNORM_ERR_INVALID_ARG;
    const uintptr_t sz = static_cast<uintptr_t>(c->sz);
    if (!aligned(b.post_w, sz) || !aligned(b.pre_w, sz) || !aligned(b.gate, sz))
        return RMSNORM_ERR_INVALID_ARG;
    BlockParams& p = c->p;
    p.post_w = b.post_norm ? b.post_w : nullptr;
    p.pre_w = b.pre_norm ? b.pre_w : nullptr;
    p.gate = b.gate;
    p.post = b.post_norm;
    p.pre = b.pre_norm;
    p.residual_scale = b.residual_scale;
    p.branch_scale = b.branch_scale;
    p.post_eps = b.post_eps;
    p.pre_eps = b.pre_eps;
    p.timeout_ns = wait_limit(0);
    if (!opt) return RMSNORM_OK;
    const rmsnorm_options_t& o = *opt;
    if (o.cluster < 0 || o.cluster > kMaxCluster || (o.cluster & (o.cluster - 1)) || o.threads || o.grid ||
        o.vec_bytes || o.chunk_bytes || o.stages || o.weights || o.reserved || o.epilogue ||
        o.fault_inject < 0 || o.fault_inject > kLastFault)
        return RMSNORM_ERR_INVALID_ARG;
    if (o.path != RMSNORM_PATH_AUTO && o.path != RMSNORM_PATH_STAGED && o.path != RMSNORM_PATH_TWOPASS &&
        !(o.path == RMSNORM_PATH_ROWREG && !back))
        return RMSNORM_ERR_INVALID_ARG;
    if (o.cluster && o.path != RMSNORM_PATH_STAGED) return RMSNORM_ERR_INVALID_ARG;
    if (o.fault_inject && (!RMSNORM_FAULT_INJECT || o.path != RMSNORM_PATH_STAGED ||
                           (o.fault_inject >= 2 && o.cluster < 2)))
        return RMSNORM_ERR_UNSUPPORTED;
    c->path = o.path;
    c->cluster = o.cluster;
    p.fault = o.fault_inject;
    p.timeout_ns = wait_limit(o.wait_timeout_ns);
    return RMSNORM_OK;
}

uintptr_t bits(const void* a) { return reinterpret_cast<uintptr_t>(a); }

rmsnorm_status_t launch(const BlockCall& c, BlockFn fn, const LaunchShape& s, cudaStream_t stream) {
    return note(launch_ex(fn, s, stream, c.p)) == cudaSuccess ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

int at_most(int64_t want, int64_t most) { return static_cast<int>(want < most ? want : most); }

// --------------------------------------------------------------- staged rows --

constexpr int64_t kBlockThreads = 256;        // threads that narrow rows share a CTA of
constexpr int64_t kBwdCtasPerSm = 4;          // CTAs, or clusters, at most: few parts

int64_t pow2_ceil(int64_t v) {
    int64_t p = 1;
    while (p < v) p <<= 1;
    return p;
}

// Threads for a row, or a slice, of nvec vectors.
int64_t group_of(int64_t nvec) {
    const int64_t g = div_up(nvec, kBlockStagedBytes / 16);
    return g <= 32 ? pow2_ceil(g) : div_up(g, 32) * 32;
}

BlockFn staged_ptr(const BlockVariant& v) {
    if (v.vb < 16) {
        if (v.dtype == RMSNORM_DTYPE_F32) return v.back ? blocknorm_bwd_ragged_f32(v) : blocknorm_fwd_ragged_f32(v);
        return v.back ? blocknorm_bwd_ragged_bf16(v) : blocknorm_fwd_ragged_bf16(v);
    }
    if (v.dtype == RMSNORM_DTYPE_F32) return v.back ? blocknorm_bwd_staged_f32(v) : blocknorm_fwd_staged_f32(v);
    return v.back ? blocknorm_bwd_staged_bf16(v) : blocknorm_fwd_staged_bf16(v);
}

// Rows staged in shared memory.  read_bits: of the addresses of the arrays that are staged;
// other_bits: of the outputs, weights and gate; narr: arrays with a place in a slot.  Leaves
// s->grid 0, status OK, where rows cannot be staged.
rmsnorm_status_t plan_staged(BlockCall* c, uintptr_t read_bits, uintptr_t other_bits, int narr, bool back,
                             LaunchShape* s, BlockFn* fn) {
    BlockParams& p = c->p;
    const int64_t row_bytes = static_cast<int64_t>(p.hidden) * c->sz;
    s->grid = 0;
    if (read_bits % 16) return RMSNORM_OK;
    const int vb = widest_vector(other_bits, row_bytes, c->sz);
    // what lies behind a ragged array's last boundary has to be within its last row
    if (vb < 16 && (c->cluster > 1 || row_bytes < 16)) return RMSNORM_OK;
    const int64_t nvec = div_up(row_bytes, 16);
    const int64_t max_threads = back ? kBlockBwdMaxThreads
                                : vb < 16 ? kBlockFwdRaggedMaxThreads : kBlockFwdMaxThreads;
    const int64_t budget = c->dv.smem_optin - 6 * 1024;             // static shared memory beside it
    // fp32 backward rows that would take all the threads of an SM (3844 to 4096 elements) are split
    // in two, so that two CTAs share it.  Measured (us, split / not): 16384 rows of 3844 235 / 263, 3968
    // 257 / 265, 4096 273 / 273, with the post norm alone 164 / 183, with the pre norm alone 274 / 266;
    // 2048 rows of 3844 37.8 / 36.5, 4096 38.2 / 38.1.
    int64_t least = 1;
    if (back && c->sz == 4 && vb == 16 && group_of(nvec) == kBlockBwdMaxThreads) least = 2;
    // Forward rows that have to be split, which costs two exchanges a row, are split into slices of
    // at most 256 threads, so that an SM has several CTAs: fp32 8192 x 16384 with clusters of 2 /
    // 4 / 8 461 / 443 / 414 us, 8192 x 12288 379 / 357 / 350, bf16 8192 x 32768 508 / 501 / 475.
    if (!back && vb == 16 && group_of(nvec) > max_threads)
        while (least < kMaxCluster && group_of(div_up(nvec, least)) > kBlockThreads) least *= 2;
    for (int64_t cluster = c->cluster ? c->cluster : least; cluster <= (vb < 16 ? 1 : kMaxCluster); cluster *= 2) {
        const int64_t slice = div_up(nvec, cluster);
        // a split row's CTA is one group of whole warps, with a thread for each rank to send to
        const int64_t narrow = group_of(slice), group = cluster > 1 && narrow < 32 ? 32 : narrow;
        const bool last = c->cluster != 0;
        // every rank has at least one vector
        if (group <= max_threads && (cluster == 1 || (cluster - 1) * slice < nvec)) {
            // Several narrow rows to a CTA, fewer where that leaves SMs without one or
            // more than a gate row has.
            int64_t rows = cluster == 1 && group < kBlockThreads ? kBlockThreads / group : 1;
            while (rows > 1 && rows * group > 32 &&
                   (div_up(p.rows, rows) < c->dv.sms || rows / 2 >= p.gate_rows))
                rows /= 2;
            const int block = static_cast<int>(rows * group);
            // a ragged row's window starts less than 16 bytes before it
            const int64_t row_slot = vb < 16 ? div_up(row_bytes + 16 - vb, 16) * 16 : slice * 16;
            const int64_t slot = narr * rows * row_slot;
            const int64_t scratch = back && rows > 1 ? rows * row_bytes * 4 / c->sz : 0;
            // Kernels without predicates or filled-in weights, measured (us, with / without, no gate):
            // both norms fp32 16384 x 8192 328 / 339, backward 497 / 505, bf16 65536 x 4096 352 / 340,
            // backward 503 / 512; pre norm alone bf16 131072 x 1024 183 / 190, fp32 16384 x 4096 175 /
            // 181, backward 16384 x 8192 527 / 539; post norm alone fp32 8192 x 12288 211 / 234, 8192 x
            // 16384 backward 360 / 375, bf16 8192 x 32768 280 / 302, but 32768 x 8192 273 / 261, backward
            // 331 / 321, 16384 x 16384 260 / 226.
            const bool whole = vb == 16 && nvec == cluster * group * (kBlockStagedBytes / 16) && (!p.post || p.post_w) &&
                               (!p.pre || p.pre_w) && (p.post || p.pre);
            *fn = staged_ptr({c->dtype, vb, back, p.post != 0, p.pre != 0, cluster > 1, whole, p.gate != nullptr});
            int best = 0;
            for (int64_t slots = 3; slots >= 2; --slots) {
                const int64_t smem = slots * slot + scratch;
                if (smem > budget) continue;
                int occ = 0;
                if (cached_occupancy(c->dv.dev, c->dv.smem_optin, reinterpret_cast<KernelFn>(*fn), block,
                                     static_cast<int>(smem), static_cast<int>(cluster), &occ) != cudaSuccess)
                    return RMSNORM_ERR_CUDA;
                if (occ <= best) continue;
                best = occ;
                s->smem = static_cast<int>(smem);
                p.nslots = static_cast<int32_t>(slots);
            }
            if (best > 0) {
                const int64_t last_rows = p.rows - (p.gates - 1) * p.gate_rows;
                p.block_rows = static_cast<int32_t>(rows);
                p.blocks_per_gate = div_up(p.gate_rows, rows);
                p.blocks = (p.gates - 1) * p.blocks_per_gate + div_up(last_rows, rows);
                p.group = static_cast<int32_t>(group);
                p.cluster = static_cast<int32_t>(cluster);
                p.slice_vecs = static_cast<int32_t>(slice);
                p.row_slot = static_cast<int32_t>(row_slot);
                p.status = c->dv.status;
                int64_t units = cluster > 1 ? best : static_cast<int64_t>(c->dv.sms) * best;
                // what the workspace has parts for
                if (back && units > kBwdCtasPerSm * c->dv.sms) units = kBwdCtasPerSm * c->dv.sms;
                if (units > p.blocks) units = p.blocks;
                p.units = units;
                s->grid = static_cast<int>(units * cluster);
                s->block = block;
                s->cluster = static_cast<int>(cluster);
                return RMSNORM_OK;
            }
        }
        if (last) break;
    }
    return RMSNORM_OK;
}

// ------------------------------------------------------------------- forward --

constexpr int64_t kRegsRowBytes = 512;        // narrower rows share a CTA, staged in pieces
constexpr int64_t kRegsBf16Threads = 768;     // wider bf16 rows: twice as much to a thread

// Rows of vectors of less than 16 bytes held in registers, a CTA to a row.  Leaves s->grid 0,
// status OK, where they are wider or a CTA cannot hold one.
rmsnorm_status_t plan_regs(BlockCall* c, int vb, LaunchShape* s, BlockFn* fn) {
    s->grid = 0;
    int nv = kBlockRegsVecs;
    int64_t block = div_up(div_up(c->p.nvec, nv), 32) * 32;
    if (block > (c->sz == 2 ? kRegsBf16Threads : kBlockRegsMaxThreads)) {
        nv *= 2;
        block = div_up(div_up(c->p.nvec, nv), 32) * 32;
    }
    if (vb == 16 || block > kBlockRegsMaxThreads) return RMSNORM_OK;
    // odd bf16 rows of most of an SM's threads: 32768 x 8191 1008 us, read for each sum 846
    if (c->path == RMSNORM_PATH_AUTO && vb == 2 && block > kRegsBf16Threads) return RMSNORM_OK;
    *fn = blocknorm_fwd_regs_ptr(c->dtype, vb, nv);
    int occ = 0;
    if (cached_occupancy(c->dv.dev, c->dv.smem_optin, reinterpret_cast<KernelFn>(*fn),
                         static_cast<int>(block), 0, 1, &occ) != cudaSuccess)
        return RMSNORM_ERR_CUDA;
    if (occ < 1) return RMSNORM_OK;
    s->grid = at_most(c->p.rows, static_cast<int64_t>(c->dv.sms) * occ);
    s->block = static_cast<int>(block);
    return RMSNORM_OK;
}

rmsnorm_status_t fwd_run(int32_t dtype, const void* x, const void* residual, void* h, void* y,
                         int64_t rows, int64_t hidden, const rmsnorm_block_t* b,
                         const rmsnorm_options_t* opt, cudaStream_t stream) {
    BlockCall c;
    rmsnorm_status_t st = check_shape(dtype, rows, hidden, b, &c);
    if (st != RMSNORM_OK) return st;
    if (!x || !residual || !h) return RMSNORM_ERR_INVALID_ARG;
    st = check_rule(*b, opt, false, &c);
    if (st != RMSNORM_OK) return st;
    const uintptr_t sz = static_cast<uintptr_t>(c.sz);
    if ((c.p.pre != 0) != (y != nullptr) || !aligned(x, sz) || !aligned(residual, sz) ||
        !aligned(h, sz) || !aligned(y, sz))
        return RMSNORM_ERR_INVALID_ARG;
    const uint64_t n = static_cast<uint64_t>(rows) * hidden * sz, nh = static_cast<uint64_t>(hidden) * sz;
    const Span a[] = {span(x, n), span(residual, n), span(b->post_w, nh), span(b->pre_w, nh),
                      span(b->gate, static_cast<uint64_t>(c.p.gates) * nh), span(h, n)};
    if (clashes(a[5], a, 5, 2) || clashes(span(y, n), a, 5, 2) || overlaps(span(y, n), a[5]))
        return RMSNORM_ERR_INVALID_ARG;
    if (rows == 0) return RMSNORM_OK;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    c.p.x = x;
    c.p.residual = residual;
    c.p.h = h;
    c.p.y = y;
    const uintptr_t read = bits(x) | bits(residual);
    const uintptr_t other = bits(h) | bits(y) | bits(c.p.post_w) | bits(c.p.pre_w) | bits(c.p.gate);
    const int vb = widest_vector(read | other, hidden * c.sz, c.sz);
    c.p.nvec = static_cast<int32_t>(hidden / (vb / c.sz));
    if (c.path == RMSNORM_PATH_ROWREG || (c.path == RMSNORM_PATH_AUTO && vb < 16 && hidden * c.sz >= kRegsRowBytes)) {
        LaunchShape s{0, 0, 1, 0};
        BlockFn fn = nullptr;
        st = plan_regs(&c, vb, &s, &fn);
        if (st != RMSNORM_OK) return st;
        if (s.grid) return launch(c, fn, s, stream);
        if (c.path == RMSNORM_PATH_ROWREG) return RMSNORM_ERR_UNSUPPORTED;
    }
    if (c.path == RMSNORM_PATH_STAGED ||
        (c.path == RMSNORM_PATH_AUTO && (vb == 16 || hidden * c.sz < kRegsRowBytes))) {
        LaunchShape s{0, 0, 1, 0};
        BlockFn fn = nullptr;
        st = plan_staged(&c, read, other, 2, false, &s, &fn);
        if (st != RMSNORM_OK) return st;
        if (s.grid) return launch(c, fn, s, stream);
        if (c.path == RMSNORM_PATH_STAGED) return RMSNORM_ERR_UNSUPPORTED;
    }
    const LaunchShape s{at_most(rows, 8ll * c.dv.sms), blocknorm_rows_block(), 1, 0};
    return launch(c, blocknorm_fwd_any_ptr(dtype, vb), s, stream);
}

// ------------------------------------------------------------------ backward --

constexpr int64_t kColsWaves = 8;      // CTAs per SM the column kernel aims at
constexpr int64_t kMaxGridParts = 512; // of them side by side in the rows' direction

struct BwdSpace {
    int64_t parts_per_gate, parts, grid_parts;     // any-width kernels
    uint64_t row_stats, part_pre, part_gate, gate_sums, bytes;
};

// Parts of the any-width kernels: enough CTAs to fill the GPU, at least four rows
// each, none across gate rows.  Whatever the vectors' width, so that the workspace is
// the same.
BwdSpace bwd_space(const BlockCall& c) {
    const BlockParams& p = c.p;
    BwdSpace s;
    auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
    const int64_t col_ctas = div_up(static_cast<int64_t>(p.hidden) * c.sz, 16ll * blocknorm_cols_block());
    int64_t want = div_up(kColsWaves * c.dv.sms, col_ctas);
    if (want > kMaxGridParts) want = kMaxGridParts;
    s.parts_per_gate = div_up(want, p.gates);
    const int64_t most = div_up(p.gate_rows, 4);
    if (s.parts_per_gate > most) s.parts_per_gate = most;
    s.parts = p.gates * s.parts_per_gate;
    s.grid_parts = s.parts < kMaxGridParts ? s.parts : kMaxGridParts;
    // the staged kernel's: a part for each unit, and one more for each gate row but the first
    const int64_t units = p.rows < kBwdCtasPerSm * c.dv.sms ? p.rows : kBwdCtasPerSm * c.dv.sms;
    const int64_t gate_parts = units + p.gates - 1;
    const uint64_t row = static_cast<uint64_t>(p.hidden) * 4;
    s.row_stats = 0;
    s.part_pre = up(static_cast<uint64_t>(p.rows) * sizeof(float4));
    s.part_gate = s.part_pre + up((s.grid_parts > units ? s.grid_parts : units) * row);
    s.gate_sums = s.part_gate + up((s.parts > gate_parts ? s.parts : gate_parts) * row);
    s.bytes = s.gate_sums + (p.gates > 1 ? up(p.gates * row) : 0);
    return s;
}

constexpr int64_t kFewParts = 16;

rmsnorm_status_t launch_reduce(BlockCall& c, cudaStream_t stream) {
    BlockParams& p = c.p;
    p.few_parts = p.gates > 1 && (p.units ? p.units / p.gates + 2 : p.parts_per_gate) <= kFewParts;
    const int width = p.hidden % 4 == 0 ? 4 : 1;
    LaunchShape s{static_cast<int>(div_up(p.hidden, kBlockReduceCols * width)), kBlockReduceThreads, 1, 0};
    if (p.part_pre || p.part_gate) {
        s.grid_y = p.part_gate ? 1 + at_most(p.gates, 65534) : 1;
        if (p.part_gate && p.few_parts) {      // as many CTAs as there are tasks
            const int64_t tasks = p.gates * div_up(p.hidden, kBlockReduceThreads * width);
            s.grid_y = 1 + at_most(div_up(tasks, s.grid), 65534);
        }
        const rmsnorm_status_t st = launch(c, blocknorm_reduce_ptr(c.dtype, width, true), s, stream);
        if (st != RMSNORM_OK) return st;
    }
    if (!p.gate_sums) return RMSNORM_OK;
    s.grid_y = 1;
    return launch(c, blocknorm_reduce_ptr(c.dtype, width, false), s, stream);
}

rmsnorm_status_t bwd_workspace(int32_t dtype, int64_t rows, int64_t hidden, const rmsnorm_block_t* b,
                               size_t* bytes) {
    BlockCall c;
    if (!bytes) return RMSNORM_ERR_INVALID_ARG;
    const rmsnorm_status_t st = check_shape(dtype, rows, hidden, b, &c);
    if (st != RMSNORM_OK) return st;
    *bytes = 0;
    if (rows == 0) return RMSNORM_OK;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    *bytes = bwd_space(c).bytes;
    return RMSNORM_OK;
}

rmsnorm_status_t bwd_run(int32_t dtype, const void* dy, const void* dh, const void* x, const void* h,
                         void* dx, void* dres, float* dpost_w, float* dpre_w, float* dgate,
                         int64_t rows, int64_t hidden, const rmsnorm_block_t* b, void* workspace,
                         size_t workspace_bytes, const rmsnorm_options_t* opt, cudaStream_t stream) {
    BlockCall c;
    rmsnorm_status_t st = check_shape(dtype, rows, hidden, b, &c);
    if (st != RMSNORM_OK) return st;
    if (!x || !dx || !dres) return RMSNORM_ERR_INVALID_ARG;
    st = check_rule(*b, opt, true, &c);
    if (st != RMSNORM_OK) return st;
    if (c.p.pre ? !dy || !h : dy != nullptr) return RMSNORM_ERR_INVALID_ARG;
    if ((dpost_w && !c.p.post) || (dpre_w && !c.p.pre) || (dgate && !b->gate))
        return RMSNORM_ERR_INVALID_ARG;
    if (!c.p.pre) h = nullptr;                   // not read
    const uintptr_t sz = static_cast<uintptr_t>(c.sz);
    if (!aligned(dy, sz) || !aligned(dh, sz) || !aligned(x, sz) || !aligned(h, sz) || !aligned(dx, sz) ||
        !aligned(dres, sz) || !aligned(dpost_w, 4) || !aligned(dpre_w, 4) || !aligned(dgate, 4) ||
        !aligned(workspace, 16))
        return RMSNORM_ERR_INVALID_ARG;
    const uint64_t n = static_cast<uint64_t>(rows) * hidden * sz, nh = static_cast<uint64_t>(hidden);
    const uint64_t ng = static_cast<uint64_t>(c.p.gates) * nh;
    const Span a[] = {span(dy, n),  span(dh, n),           span(x, n),           span(h, n),
                      span(b->post_w, nh * sz), span(b->pre_w, nh * sz), span(b->gate, ng * sz),
                      span(dx, n),  span(dres, n),         span(dpost_w, nh * 4), span(dpre_w, nh * 4),
                      span(dgate, ng * 4)};
    if (clashes(a[7], a, 7, 4) || clashes(a[8], a, 7, 4) || overlaps(a[7], a[8]) ||
        clashes(a[9], a, 9, 0) || clashes(a[10], a, 10, 0) || clashes(a[11], a, 11, 0) ||
        clashes(span(workspace, workspace_bytes), a, 12, 0))
        return RMSNORM_ERR_INVALID_ARG;
    if (rows == 0) {            // sums over no rows
        float* sums[] = {dpost_w, dpre_w, dgate};
        for (float* d : sums)
            if (d && note(cudaMemsetAsync(d, 0, nh * 4, stream)) != cudaSuccess) return RMSNORM_ERR_CUDA;
        return RMSNORM_OK;
    }
    if (!workspace) return RMSNORM_ERR_INVALID_ARG;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    const BwdSpace ws = bwd_space(c);
    if (workspace_bytes < ws.bytes) return RMSNORM_ERR_INVALID_ARG;
    char* base = static_cast<char*>(workspace);
    BlockParams& p = c.p;
    p.x = x;
    p.dy = dy;
    p.dh = dh;
    p.h_in = h;
    p.dx = dx;
    p.dres = dres;
    p.dpost_w = dpost_w;
    p.dpre_w = dpre_w;
    p.dgate = dgate;
    p.row_stats = reinterpret_cast<float4*>(base + ws.row_stats);
    p.part_pre = dpre_w ? reinterpret_cast<float*>(base + ws.part_pre) : nullptr;
    p.part_gate = dpost_w || dgate ? reinterpret_cast<float*>(base + ws.part_gate) : nullptr;
    p.gate_sums = dpost_w && p.gates > 1 ? reinterpret_cast<float*>(base + ws.gate_sums) : nullptr;
    const uintptr_t read = bits(dy) | bits(dh) | bits(x) | bits(h);
    const uintptr_t other = bits(dx) | bits(dres) | bits(p.post_w) | bits(p.pre_w) | bits(p.gate);
    if (c.path != RMSNORM_PATH_TWOPASS) {
        LaunchShape s{0, 0, 1, 0};
        BlockFn fn = nullptr;
        st = plan_staged(&c, read, other, p.pre ? 4 : 2, true, &s, &fn);
        if (st != RMSNORM_OK) return st;
        if (s.grid) {
            p.pre_parts = static_cast<int32_t>(p.units);
            st = launch(c, fn, s, stream);
            return st == RMSNORM_OK ? launch_reduce(c, stream) : st;
        }
        if (c.path == RMSNORM_PATH_STAGED) return RMSNORM_ERR_UNSUPPORTED;
    }
    p.parts_per_gate = ws.parts_per_gate;
    p.parts = ws.parts;
    p.rows_per_part = div_up(p.gate_rows, ws.parts_per_gate);
    p.pre_parts = static_cast<int32_t>(ws.grid_parts);
    const int vb = widest_vector(read | other, hidden * c.sz, c.sz);
    p.nvec = static_cast<int32_t>(hidden / (vb / c.sz));
    const LaunchShape rs{at_most(rows, 8ll * c.dv.sms), blocknorm_rows_block(), 1, 0};
    st = launch(c, blocknorm_bwd_rows_ptr(dtype, vb), rs, stream);
    if (st != RMSNORM_OK) return st;
    LaunchShape cs{static_cast<int>(div_up(p.nvec, blocknorm_cols_block())), blocknorm_cols_block(), 1, 0};
    cs.grid_y = static_cast<int>(ws.grid_parts);
    st = launch(c, blocknorm_bwd_cols_ptr(dtype, vb), cs, stream);
    if (st != RMSNORM_OK) return st;
    return launch_reduce(c, stream);
}

}  // namespace
}  // namespace rmsnorm

using namespace rmsnorm;

extern "C" {

rmsnorm_status_t rmsnorm_block_fwd_f32(const float* x, const float* residual, float* h, float* y,
                                       int64_t rows, int64_t hidden, const rmsnorm_block_t* block,
                                       rmsnorm_stream_t stream) {
    return fwd_run(RMSNORM_DTYPE_F32, x, residual, h, y, rows, hidden, block, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_block_fwd_bf16(const uint16_t* x, const uint16_t* residual, uint16_t* h,
                                        uint16_t* y, int64_t rows, int64_t hidden,
                                        const rmsnorm_block_t* block, rmsnorm_stream_t stream) {
    return fwd_run(RMSNORM_DTYPE_BF16, x, residual, h, y, rows, hidden, block, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_block_fwd_ex(int32_t dtype, const void* x, const void* residual, void* h,
                                      void* y, int64_t rows, int64_t hidden,
                                      const rmsnorm_block_t* block, const rmsnorm_options_t* opt,
                                      rmsnorm_stream_t stream) {
    return fwd_run(dtype, x, residual, h, y, rows, hidden, block, opt,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_block_bwd_workspace(int32_t dtype, int64_t rows, int64_t hidden,
                                             const rmsnorm_block_t* block, size_t* bytes) {
    return bwd_workspace(dtype, rows, hidden, block, bytes);
}

rmsnorm_status_t rmsnorm_block_bwd_f32(const float* dy, const float* dh, const float* x,
                                       const float* h, float* dx, float* dresidual, float* dpost_w,
                                       float* dpre_w, float* dgate, int64_t rows, int64_t hidden,
                                       const rmsnorm_block_t* block, void* workspace,
                                       size_t workspace_bytes, rmsnorm_stream_t stream) {
    return bwd_run(RMSNORM_DTYPE_F32, dy, dh, x, h, dx, dresidual, dpost_w, dpre_w, dgate, rows,
                   hidden, block, workspace, workspace_bytes, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_block_bwd_bf16(const uint16_t* dy, const uint16_t* dh, const uint16_t* x,
                                        const uint16_t* h, uint16_t* dx, uint16_t* dresidual,
                                        float* dpost_w, float* dpre_w, float* dgate, int64_t rows,
                                        int64_t hidden, const rmsnorm_block_t* block,
                                        void* workspace, size_t workspace_bytes,
                                        rmsnorm_stream_t stream) {
    return bwd_run(RMSNORM_DTYPE_BF16, dy, dh, x, h, dx, dresidual, dpost_w, dpre_w, dgate, rows,
                   hidden, block, workspace, workspace_bytes, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_block_bwd_ex(int32_t dtype, const void* dy, const void* dh, const void* x,
                                      const void* h, void* dx, void* dresidual, float* dpost_w,
                                      float* dpre_w, float* dgate, int64_t rows, int64_t hidden,
                                      const rmsnorm_block_t* block, void* workspace,
                                      size_t workspace_bytes, const rmsnorm_options_t* opt,
                                      rmsnorm_stream_t stream) {
    return bwd_run(dtype, dy, dh, x, h, dx, dresidual, dpost_w, dpre_w, dgate, rows, hidden, block,
                   workspace, workspace_bytes, opt, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
