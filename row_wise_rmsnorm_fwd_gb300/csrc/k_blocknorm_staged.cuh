// k_blocknorm_staged.cuh -- the boundary between two blocks (formulas in
// include/rmsnorm_block.h): rows staged in shared memory and read from HBM once.
//
// A group of p.group threads takes a row (with a cluster: a slice of it), 32 bytes of
// each array to a thread, which it holds in registers, packed, from the sums to the
// outputs.  The ring's slot is free again behind the block barrier of the sums.
//
// Rows that are not whole 16-byte vectors, or weights or outputs off the boundaries: a
// thread's 16 bytes are pieces of VB bytes each, taken G pieces apart, so that accesses stay
// side by side; everything between load and store is the same.
//
// What bounds it: HBM, where rows fill their threads.  32 bytes a thread and up to 64
// registers keep 32 warps to an SM forward; backward the column sums take a thread's 128
// registers and 16 warps are all there are, so the instructions of a pass count, and the
// blocks under way while it runs: a ring of three slots refilled as early as can be.  One
// pass ahead with fewer blocks under way (the sums of the next row between the same barriers
// as the outputs of this one, rows read again from shared memory) was slower: fp32 16384 x 8192
// 658 us against 478.  Measured (calls back to back, us and % of the HBM copy peak):
//   forward bf16 65536 x 4096 342 (92), 32768 x 8192 344 (92), 131072 x 1024 181 (87), 65536 x
//     1280 136 (73), fp32 16384 x 4096 167 (95), 16384 x 8192 349 (91)
//   backward bf16 65536 x 8192 951 (100), 32768 x 4096 259 (92), 131072 x 1024 249 (95), 32768 x
//     5120 398 (75), 65536 x 1280 204 (73), fp32 16384 x 4096 273 (87), 16384 x 8192 495 (96)
//   the sum and the norm before the next block alone: forward bf16 65536 x 4096 359 (88), 32768 x 8192 355
//     (89), 131072 x 1024 184 (86), 65536 x 1280 118 (84), fp32 16384 x 4096 176 (90), 16384 x 8192 340
//     (93); backward 545 (87), 543 (87), 269 (88), 164 (91), 274 (87), 528 (90)
//   with a gate row for 512 rows backward bf16 32768 x 8192 486 (98), for 16 rows 638 (74), for 4 1056
//     (45), for one 2777 (17): a part in fp32 for each, read twice by the sums' two launches; forward 349
//     (91), 352 (90), 360 (88), 400 (79)
//   split rows: forward fp32 8192 x 16384 410 (77), 8192 x 12288 349 (68), backward 479 (99), 429 (83),
//     bf16 16384 x 16384 697 (68), 16384 x 12288 555 (64)
//   in pieces: forward bf16 262144 x 110 88 (39), fp32 262144 x 66 110 (37), backward 131072 x 130
//     163 (37), 65536 x 1027 367 (65), bf16 65536 x 2050 884 (27), 65536 x 1027 587 (20)
// The kernels for any width instead: forward bf16 65536 x 4096 524, backward 65536 x 8192 2275.
#pragma once
#include "k_blocknorm.cuh"
#include "k_blockring.cuh"
#include "k_rowblocks.cuh"
#include "pairs.cuh"

namespace rmsnorm {

// A cluster's exchange of N sums per row: two sets of slots and two mbarriers, used in
// turn.  A phase takes one local arrival, which expects the bytes of all ranks.  A peer
// sends a row's sums only behind its block barrier of that row, by when all its threads have
// read the row before: it is never two rows ahead of a slot that is still read.
struct BlockExchange {
    alignas(16) float slot[2][16][8];
    alignas(8) uint64_t bar[2];
};

// Sums of all ranks in rank order; false once the bounded wait has run out, which the thread that
// it ran out for reports.  Every thread has a clock of its own, so where the sums arrive close to
// the limit some may get them and some not: what the result decides for the CTA is first agreed on.
template <int N>
__device__ __forceinline__ bool exchange_sums(BlockExchange* ex, float (&v)[8], int ncta, uint32_t rank,
                                              uint32_t it, const BlockParams& p) {
    const uint32_t b = it & 1u;
    const uint32_t bar = smem_addr(&ex->bar[b]);
    const int tid = threadIdx.x;
    if (tid == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(ncta * N * 4));
    bool send = tid < ncta;
#if RMSNORM_FAULT_INJECT
    if (p.fault == kFaultClusterWithholdPartial && rank == 0 && it == 0) send = false;
#endif
    if (send) {
        const uint32_t to = map_to_rank(smem_addr(&ex->slot[b][rank][0]), static_cast<uint32_t>(tid));
        const uint32_t peer_bar = map_to_rank(bar, static_cast<uint32_t>(tid));
        if constexpr (N == 1) {
            st_async_f32(to, v[0], peer_bar);
        } else {
#pragma unroll
            for (int k = 0; k < N; k += 2) st_async_v2_f32(to + 4 * k, v[k], v[k + 1], peer_bar);
        }
    }
    bool ok = mbar_wait_bounded<true>(bar, (it >> 1) & 1u, p.timeout_ns);
#if RMSNORM_FAULT_INJECT
    if (p.fault == kFaultClusterLateThread && rank == 0 && it == 0 && tid == static_cast<int>(blockDim.x) - 1)
        ok = false;
#endif
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = 0.f;
    if (ok) {
        for (int c = 0; c < ncta; ++c) {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += ex->slot[b][c][k];
        }
    } else {
        report_timeout(p.status, kSiteClusterExchange);
    }
    return ok;
}

__device__ __forceinline__ void exchange_init(BlockExchange* ex) {
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&ex->bar[0]), 1);
        mbar_init(smem_addr(&ex->bar[1]), 1);
        fence_mbarrier_init_cluster();
    }
    __syncthreads();
    cluster_sync_all();
}

// A thread's place: its row of a block and its vectors.
struct RowPlace {
    int g, t, G, width, wpg, gw0;
    __device__ __forceinline__ explicit RowPlace(int group) : G(group) {
        width = G < 32 ? G : 32;
        g = static_cast<int>(threadIdx.x) / G;
        t = static_cast<int>(threadIdx.x) - g * G;
        wpg = G >> 5;
        gw0 = g * wpg;
    }
};

constexpr int kBlockVecs = kBlockStagedBytes / 16;

// What a kernel may take for granted of its rows and weights.
//   kBlockSome: nothing: a thread may lack vectors, and weights may be absent (ones)
//   kBlockPlain: every thread has all its vectors, the norms' weights are there, no gate
//   kBlockGated: the same with a gate
enum : int { kBlockSome, kBlockPlain, kBlockGated };

// Pieces of VB bytes that make up 16.
template <int VB>
constexpr int kPieces = 16 / VB;
template <int VB>
constexpr uint32_t kAllPieces = (1u << kPieces<VB>) - 1;

// Piece j of a vector put in, and taken out.
template <int VB>
__device__ __forceinline__ void put_piece(Vec<16>& v, int j, const Vec<VB>& w) {
    if constexpr (VB == 2) {
        const uint32_t h = w.h;
        v.u[j / 2] = j % 2 ? (v.u[j / 2] & 0xFFFFu) | (h << 16) : h;
    } else {
#pragma unroll
        for (int k = 0; k < VB / 4; ++k) v.u[j * (VB / 4) + k] = w.u[k];
    }
}
template <int VB>
__device__ __forceinline__ Vec<VB> take_piece(const Vec<16>& v, int j) {
    Vec<VB> w;
    if constexpr (VB == 2) {
        w.h = static_cast<uint16_t>(j % 2 ? v.u[j / 2] >> 16 : v.u[j / 2]);
    } else {
#pragma unroll
        for (int k = 0; k < VB / 4; ++k) w.u[k] = v.u[j * (VB / 4) + k];
    }
    return w;
}

// FAST: a branch for threads that have all pieces (all of a row but its last ones).  Measured
// (us, with / without): forward bf16 262144 x 110 88 / 101, 131072 x 251 119 / 192, fp32 262144 x
// 101 131 / 154, but with 8-byte pieces 262144 x 66 118 / 110, 131072 x 126 65 / 59; backward fp32 32768
// x 2050 500 / 464.
//
// A vector of a slot; zeros where (bit j of `on`: piece j) it is missing.  apart: bytes from
// piece to piece.
template <int VB, int MODE, bool FAST>
__device__ __forceinline__ Vec<16> slot_vec(uint32_t at, int apart, uint32_t on) {
    if constexpr (VB == 16) {
        return MODE == kBlockSome ? ld_slot_if(at, on) : ld_slot(at);
    } else {
        Vec<16> v;
        auto piece = [&](int j, bool yes) {
            Vec<VB> w;
            const uint32_t q = yes, a = at + j * apart;
            if constexpr (VB == 8) {
                asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
                             "@p ld.shared.v2.u32 {%0,%1}, [%2];\n\t}"
                             : "=&r"(w.u[0]), "=&r"(w.u[1]) : "r"(a), "r"(q));
            } else if constexpr (VB == 4) {
                asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t"
                             "@p ld.shared.u32 %0, [%1];\n\t}" : "=&r"(w.u[0]) : "r"(a), "r"(q));
            } else {
                asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t"
                             "@p ld.shared.u16 %0, [%1];\n\t}" : "=&h"(w.h) : "r"(a), "r"(q));
            }
            put_piece<VB>(v, j, w);
        };
        auto whole_piece = [&](int j) {
            Vec<VB> w;
            const uint32_t a = at + j * apart;
            if constexpr (VB == 8)
                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w.u[0]), "=r"(w.u[1]) : "r"(a));
            else if constexpr (VB == 4)
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w.u[0]) : "r"(a));
            else
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w.h) : "r"(a));
            put_piece<VB>(v, j, w);
        };
        if (FAST && on == kAllPieces<VB>) {
#pragma unroll
            for (int j = 0; j < kPieces<VB>; ++j) whole_piece(j);
        } else {
#pragma unroll
            for (int j = 0; j < kPieces<VB>; ++j) piece(j, on >> j & 1u);
        }
        return v;
    }
}

// A vector of weights.  Volatile: read where it stands, from L1, and not kept.
template <typename T, int VB, int MODE, bool FAST>
__device__ __forceinline__ Vec<16> weight_vec(const char* from, int apart, uint32_t on) {
    Vec<16> v;
    if (MODE == kBlockSome) {
        v = ones_vec<T>();
        if (!from) return v;
    }
    if constexpr (VB == 16) {
        if (MODE == kBlockSome && !on) return v;
        asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.u[0]), "=r"(v.u[1]), "=r"(v.u[2]), "=r"(v.u[3]) : "l"(from));
    } else if (FAST && on == kAllPieces<VB>) {
#pragma unroll
        for (int j = 0; j < kPieces<VB>; ++j) put_piece<VB>(v, j, ld_ro<VB>(from + j * apart));
    } else {
#pragma unroll
        for (int j = 0; j < kPieces<VB>; ++j)
            if (on >> j & 1u) put_piece<VB>(v, j, ld_ro<VB>(from + j * apart));
    }
    return v;
}

// A vector stored, the pieces that there are.
template <int VB, bool FAST>
__device__ __forceinline__ void store_vec(char* to, int apart, uint32_t on, const Vec<16>& v) {
    if constexpr (VB == 16) {
        if (on) st_stream<16>(to, v);
    } else if (FAST && on == kAllPieces<VB>) {
#pragma unroll
        for (int j = 0; j < kPieces<VB>; ++j) st_stream<VB>(to + j * apart, take_piece<VB>(v, j));
    } else {
#pragma unroll
        for (int j = 0; j < kPieces<VB>; ++j)
            if (on >> j & 1u) st_stream<VB>(to + j * apart, take_piece<VB>(v, j));
    }
}

// The pieces that a thread has of a row of `bytes`: column of its vector i (bytes from the
// row's start on) and the bits.
template <int VB, int MODE>
__device__ __forceinline__ void row_columns(const RowPlace& at, int first, int bytes, int (&col)[kBlockVecs],
                                            uint32_t (&valid)[kBlockVecs]) {
#pragma unroll
    for (int i = 0; i < kBlockVecs; ++i) {
        const int c = (i * kPieces<VB> * at.G + at.t) * VB;
        col[i] = first + c;
        valid[i] = 0;
#pragma unroll
        for (int j = 0; j < kPieces<VB>; ++j)
            if (MODE != kBlockSome || c + j * at.G * VB < bytes) valid[i] |= 1u << j;
    }
}

// Pair k of two vectors' product: for bf16 the mixed-precision product, which widens its
// operands by itself (added to -0, which changes no product).
template <typename T>
__device__ __forceinline__ Lanes product(const Vec<16>& a, const Vec<16>& b, int k) {
    if constexpr (sizeof(T) == 2) {
        float c, d;
        asm("{\n\t.reg .b16 l, h, m, n;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 {m, n}, %3;\n\t"
            "fma.rn.f32.bf16 %0, l, m, %4;\n\tfma.rn.f32.bf16 %1, h, n, %4;\n\t}"
            : "=f"(c), "=f"(d) : "r"(a.u[k]), "r"(b.u[k]), "f"(-0.0f));
        return {pack_x2(c, d)};
    } else {
        return lanes<T>(a, k) * lanes<T>(b, k);
    }
}

// The same of a vector with itself, added to a pair.
template <typename T>
__device__ __forceinline__ Lanes add_square(const Vec<16>& a, int k, Lanes to) {
    if constexpr (sizeof(T) == 2) {
        float c, d, e, f;
        unpack_x2(to.v, e, f);
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "fma.rn.f32.bf16 %0, l, l, %3;\n\tfma.rn.f32.bf16 %1, h, h, %4;\n\t}"
            : "=f"(c), "=f"(d) : "r"(a.u[k]), "f"(e), "f"(f));
        return {pack_x2(c, d)};
    } else {
        return fma(lanes<T>(a, k), lanes<T>(a, k), to);
    }
}

// Keep vectors packed from here on: widened before, they would be held widened.
template <int N>
__device__ __forceinline__ void stay_packed(Vec<16> (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) opaque(v[i].u[k]);
    }
}

// ------------------------------------------------------------------- forward --

template <typename T, bool POST, bool PRE, bool CL, int MODE, int VB>
__global__ void __launch_bounds__(VB == 16 ? kBlockFwdMaxThreads : kBlockFwdRaggedMaxThreads, 1)
blocknorm_fwd_staged_kernel(const BlockParams p) {
    constexpr int NV = kBlockVecs, PN = kPairs<T>, EPV = VecTraits<T, 16>::kElems;
    constexpr bool GATE = MODE != kBlockPlain;
    using L = Lanes;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ alignas(8) uint64_t bars[kRowBlocksMaxSlots];
    __shared__ float red[2][2][32 * 8];
    __shared__ BlockExchange ex[CL ? 2 : 1];
    pdl_trigger();
    const RowPlace at(p.group);
    const uint32_t rank = CL ? cluster_ctarank() : 0;
    const void* const arrays[2] = {p.x, p.residual};
    const RowBlocks<2, VB != 16> ring(p, arrays, sizeof(T), rank, static_cast<int>(CL ? cluster_id_x() : blockIdx.x),
                            static_cast<int>(CL ? cluster_count_x() : gridDim.x), smem, bars);
    if constexpr (CL) {
        exchange_init(&ex[0]);
        exchange_init(&ex[1]);
    } else {
        __syncthreads();
    }
    pdl_wait();
    auto now = ring.start(), ahead = now;        // the block at work, and the next to be copied
    if (threadIdx.x < 32) ring.prologue(ahead);
    uint32_t valid[NV];
    int col[NV];
    row_columns<VB, MODE>(at, ring.at, ring.bytes, col, valid);
    const int apart = at.G * VB;           // bytes from piece to piece, kPieces of them a vector
    const uint32_t in_slot = static_cast<uint32_t>(at.g * ring.slot_row + at.t * VB);
    const char* post_w = static_cast<const char*>(p.post_w);
    const char* pre_w = static_cast<const char*>(p.pre_w);
    const L rs = L::all(p.residual_scale);
    int slot = 0;
    uint32_t use = 0;
    bool bad = false;
    int64_t n = 0;
    for (; n < ring.count; ++n) {
        const int64_t gate_row = now.gate, row0 = now.row;
        const int rows = now.rows;
        ring.advance(now);
        const int64_t row = row0 + at.g;
        // rows that the block lacks: sums of what the slot held before, not used
        const bool here = at.g < rows;
        Vec<16> x[NV], r[NV], w[NV], g[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (POST)
                w[i] = weight_vec<T, VB, MODE, (VB < 8)>(post_w ? post_w + col[i] : nullptr, apart, valid[i]);
            if constexpr (GATE)
                g[i] = weight_vec<T, VB, MODE, (VB < 8)>(at_or_null(p.gate, gate_row * ring.row_bytes + col[i]), apart,
                                               valid[i]);
        }
        const bool ok = ring.wait(slot, use) && !bad;
        ring.template finish<T>(slot, row0, rows);
        RowSums<1> s;
        L acc = L::all(0.f);
        const uint32_t in = in_slot + static_cast<uint32_t>(ring.skip(row));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = slot_vec<VB, MODE, (VB < 8)>(ring.base(slot, 0) + in + i * kPieces<VB> * apart, apart, valid[i]);
            r[i] = slot_vec<VB, MODE, (VB < 8)>(ring.base(slot, 1) + in + i * kPieces<VB> * apart, apart, valid[i]);
            if constexpr (POST) {
#pragma unroll
                for (int k = 0; k < PN; ++k) acc = add_square<T>(x[i], k, acc);
            }
        }
        float scale = p.branch_scale;
        if constexpr (POST) {
            s.v[0] = acc.total();
            s.gather(red[0][n & 1], at.width);
        }
        if (__syncthreads_or(!ok)) break;                     // uniform
        if (threadIdx.x < 32 && n + p.nslots < ring.count) ring.issue(slot, n + p.nslots, ahead);
        if constexpr (POST) {
            s.totals(red[0][n & 1], at.width, at.gw0, at.wpg);
            if (CL && !exchange_sums<1>(&ex[0], s.v, p.cluster, rank, static_cast<uint32_t>(n), p)) bad = true;
            scale *= rsqrtf(fmaf(s.v[0], p.inv_hidden, p.post_eps));
        }
        L h[NV * PN];
        acc = L::all(0.f);
        const L sc = L::all(scale);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float o[EPV];
#pragma unroll
            for (int k = 0; k < PN; ++k) {
                L b = lanes<T>(x[i], k) * sc;
                if constexpr (POST && GATE) b = b * product<T>(w[i], g[i], k);
                else if constexpr (POST) b = b * lanes<T>(w[i], k);
                else if constexpr (GATE) b = b * lanes<T>(g[i], k);
                const L v = fma(rs, lanes<T>(r[i], k), b);
                h[i * PN + k] = v;
                if constexpr (PRE) acc = fma(v, v, acc);
                v.put(o + 2 * k);
            }
            if (here)
                store_vec<VB, (VB < 8)>(static_cast<char*>(p.h) + row * ring.row_bytes + col[i], apart, valid[i],
                              pack<T, 16>(o));
        }
        if constexpr (PRE) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                w[i] = weight_vec<T, VB, MODE, (VB < 8)>(pre_w ? pre_w + col[i] : nullptr, apart, valid[i]);
            s.v[0] = acc.total();
            s.gather(red[1][n & 1], at.width);
            if (at.wpg > 1) __syncthreads();
            else __syncwarp();
            s.totals(red[1][n & 1], at.width, at.gw0, at.wpg);
            if (CL && !exchange_sums<1>(&ex[1], s.v, p.cluster, rank, static_cast<uint32_t>(n), p)) bad = true;
            const L rh = L::all(rsqrtf(fmaf(s.v[0], p.inv_hidden, p.pre_eps)));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float o[EPV];
#pragma unroll
                for (int k = 0; k < PN; ++k) (h[i * PN + k] * rh * lanes<T>(w[i], k)).put(o + 2 * k);
                if (here)
                    store_vec<VB, (VB < 8)>(static_cast<char*>(p.y) + row * ring.row_bytes + col[i], apart, valid[i],
                                  pack<T, 16>(o));
            }
        }
        if (++slot == p.nslots) {
            slot = 0;
            ++use;
        }
    }
    if constexpr (CL) bad = __syncthreads_or(bad);      // after the last row nothing else says so
    if (n < ring.count && threadIdx.x == 0) {
        if (!bad) report_timeout(p.status, kSiteStagedFull);
        ring.drain(n, slot, use);
    }
    if constexpr (CL) {
        __syncthreads();
        cluster_sync_all();
    }
}

// ------------------------------------------------------------------ backward --

// N floats (a power of two) at a time.
template <int N>
__device__ __forceinline__ void put_floats(float* to, const float* f) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int k = 0; k < N; k += 4) *reinterpret_cast<float4*>(to + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
    } else if constexpr (N == 2) {
        *reinterpret_cast<float2*>(to) = make_float2(f[0], f[1]);
    } else {
        *to = *f;
    }
}

// Column sums of a CTA's vectors, written to `to` (one row of a part).  Several row groups:
// added in order through shared memory.
template <typename T, int VB>
__device__ __forceinline__ void write_part(const Lanes (&acc)[kBlockVecs * kPairs<T>], float* to,
                                           const RowPlace& at, int groups, const int (&col)[kBlockVecs],
                                           const uint32_t (&valid)[kBlockVecs], float* scratch, int slice_elems,
                                           int first_elem) {
    constexpr int EPV = VecTraits<T, 16>::kElems, PN = kPairs<T>, SZ = static_cast<int>(sizeof(T));
    constexpr int EPP = VB / SZ;                          // elements of a piece
    auto put = [&](float* row, int i) {                   // row: of column 0
        float f[EPV];
#pragma unroll
        for (int k = 0; k < PN; ++k) acc[i * PN + k].put(f + 2 * k);
#pragma unroll
        for (int j = 0; j < kPieces<VB>; ++j)
            if (valid[i] >> j & 1u) put_floats<EPP>(row + (col[i] + j * at.G * VB) / SZ, f + j * EPP);
    };
    if (groups == 1) {
#pragma unroll
        for (int i = 0; i < kBlockVecs; ++i) put(to, i);
        return;
    }
#pragma unroll
    for (int i = 0; i < kBlockVecs; ++i) put(scratch + at.g * slice_elems - first_elem, i);
    __syncthreads();
    constexpr int W = EPP < 4 ? EPP : 4;
    for (int c = threadIdx.x * W; c < slice_elems; c += blockDim.x * W) {
        float v[W];
#pragma unroll
        for (int k = 0; k < W; ++k) v[k] = 0.f;
        for (int g = 0; g < groups; ++g) {
            const float* from = scratch + g * slice_elems + c;
            float f[W];
            if constexpr (W == 4) {
                const float4 q = *reinterpret_cast<const float4*>(from);
                f[0] = q.x;
                f[1] = q.y;
                f[2] = q.z;
                f[3] = q.w;
            } else if constexpr (W == 2) {
                const float2 q = *reinterpret_cast<const float2*>(from);
                f[0] = q.x;
                f[1] = q.y;
            } else {
                f[0] = *from;
            }
#pragma unroll
            for (int k = 0; k < W; ++k) v[k] += f[k];
        }
        put_floats<W>(to + first_elem + c, v);
    }
    __syncthreads();
}

template <typename T, bool POST, bool PRE, bool CL, int MODE, int VB>
__global__ void __launch_bounds__(kBlockBwdMaxThreads, 1) blocknorm_bwd_staged_kernel(const BlockParams p) {
    constexpr int NV = kBlockVecs, PN = kPairs<T>, EPV = VecTraits<T, 16>::kElems;
    constexpr int NARR = PRE ? 4 : 2;
    constexpr bool GATE = MODE != kBlockPlain;
    // With both norms in bf16 not all weights fit beside the column sums: pre_w is read again in
    // each pass.  post_w and the gate are kept, their product in fp32: the ring leaves L1 too
    // little for all three.  Measured (us, bf16 32768 x 8192 with a gate, all three read again /
    // so): 577 / 505.
    constexpr bool REREAD = PRE && POST && sizeof(T) == 2;
    constexpr int NS = PRE && POST ? 6 : (PRE || POST ? 2 : 0);
    using L = Lanes;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ alignas(8) uint64_t bars[kRowBlocksMaxSlots];
    __shared__ float red[2][32 * 8];
    __shared__ BlockExchange ex[1];
    pdl_trigger();
    const RowPlace at(p.group);
    const uint32_t rank = CL ? cluster_ctarank() : 0;
    const int unit = static_cast<int>(CL ? cluster_id_x() : blockIdx.x);
    const int units = static_cast<int>(CL ? cluster_count_x() : gridDim.x);
    auto make_ring = [&]() {
        if constexpr (PRE) {
            const void* const arrays[4] = {p.x, p.dh, p.dy, p.h_in};
            return RowBlocks<4, VB != 16>(p, arrays, sizeof(T), rank, unit, units, smem, bars);
        } else {
            const void* const arrays[2] = {p.x, p.dh};
            return RowBlocks<2, VB != 16>(p, arrays, sizeof(T), rank, unit, units, smem, bars);
        }
    };
    const RowBlocks<NARR, VB != 16> ring = make_ring();
    if constexpr (CL) exchange_init(ex);
    else __syncthreads();
    pdl_wait();
    auto now = ring.start(), ahead = now;        // the block at work, and the next to be copied
    if (threadIdx.x < 32) ring.prologue(ahead);
    uint32_t valid[NV];
    int col[NV];
    row_columns<VB, MODE>(at, ring.at, ring.bytes, col, valid);
    const int apart = at.G * VB;
    float* scratch = reinterpret_cast<float*>(smem + (ring.base(p.nslots, 0) - ring.base(0, 0)));
    const int slice_elems = ring.bytes / static_cast<int>(sizeof(T));
    const int first_elem = ring.at / static_cast<int>(sizeof(T));
    const char* post_w = static_cast<const char*>(p.post_w);
    const char* pre_w = static_cast<const char*>(p.pre_w);
    const bool have_dh = p.dh != nullptr;
    const uint32_t in_slot = static_cast<uint32_t>(at.g * ring.slot_row + at.t * VB);
    // pre_w and, without the post norm, the gate of the rows at hand, packed; post_w times the
    // gate in fp32
    Vec<16> pw[NV], gt[NV];
    L u[POST ? NV * PN : 1];
    auto read_pre = [&](int i) {
        if constexpr (PRE)
            pw[i] = weight_vec<T, VB, MODE, false>(pre_w ? pre_w + col[i] : nullptr, apart, valid[i]);
    };
    auto read_post = [&](int64_t gate_row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (GATE)
                gt[i] = weight_vec<T, VB, MODE, false>(at_or_null(p.gate, gate_row * ring.row_bytes + col[i]),
                                                       apart, valid[i]);
            if constexpr (POST) {
                const Vec<16> w =
                    weight_vec<T, VB, MODE, false>(post_w ? post_w + col[i] : nullptr, apart, valid[i]);
#pragma unroll
                for (int k = 0; k < PN; ++k)
                    u[i * PN + k] = GATE ? product<T>(w, gt[i], k) : lanes<T>(w, k);
            }
        }
    };
    if constexpr (!REREAD) {
#pragma unroll
        for (int i = 0; i < NV; ++i) read_pre(i);
    }
    if constexpr (!GATE) read_post(0);
    L acc[NV * PN], pre[PRE ? NV * PN : 1];     // sums of D * xh and of dy * h * rh
#pragma unroll
    for (int k = 0; k < NV * PN; ++k) acc[k] = L::all(0.f);
#pragma unroll
    for (int k = 0; k < (PRE ? NV * PN : 1); ++k) pre[k] = L::all(0.f);
    // The CTA's sums of gate row s are part unit + s: both only grow along the units'
    // ranges of blocks, and one of them does from each part to the next.
    auto write_gate = [&](int64_t s) {
        if (p.part_gate)
            write_part<T, VB>(acc, p.part_gate + (unit + s) * p.hidden, at, p.block_rows, col, valid, scratch,
                              slice_elems, first_elem);
    };
    int slot = 0;
    uint32_t use = 0;
    bool bad = false;
    int64_t n = 0, last_gate = -1;
    for (; n < ring.count; ++n) {
        const int64_t gate_row = now.gate, row0 = now.row;
        const int rows = now.rows;
        ring.advance(now);
        if (gate_row != last_gate) {
            if (last_gate >= 0) {
                write_gate(last_gate);
#pragma unroll
                for (int k = 0; k < NV * PN; ++k) acc[k] = L::all(0.f);
            }
            last_gate = gate_row;
            if constexpr (GATE) read_post(gate_row);
        }
        if constexpr (GATE && !POST) stay_packed(gt);
        if constexpr (PRE && !REREAD) stay_packed(pw);
        const int64_t row = row0 + at.g;
        const bool here = at.g < rows;
        const bool ok = ring.wait(slot, use) && !bad;
        ring.template finish<T>(slot, row0, rows);
        const uint32_t in_row = in_slot + static_cast<uint32_t>(ring.skip(row));
        Vec<16> x[NV], d[NV], y[PRE ? NV : 1], h[PRE ? NV : 1];
        RowSums<NS> s;
        L a[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) a[k] = L::all(0.f);
        // post_w * gate
        auto factor = [&](int i, int k) {
            if constexpr (POST) return u[i * PN + k];
            else if constexpr (GATE) return lanes<T>(gt[i], k);
            else return L::all(1.f);
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t in = in_row + i * kPieces<VB> * apart;
            if constexpr (REREAD) read_pre(i);
            x[i] = slot_vec<VB, MODE, false>(ring.base(slot, 0) + in, apart, valid[i]);
            d[i] = have_dh ? slot_vec<VB, MODE, false>(ring.base(slot, 1) + in, apart, valid[i]) : zero_vec();
            if constexpr (PRE) {
                y[i] = slot_vec<VB, MODE, false>(ring.base(slot, 2) + in, apart, valid[i]);
                h[i] = slot_vec<VB, MODE, false>(ring.base(slot, 3) + in, apart, valid[i]);
            }
#pragma unroll
            for (int k = 0; k < PN; ++k) {
                L q, gy;
                if constexpr (POST) {
                    q = factor(i, k) * lanes<T>(x[i], k);
                    const L xk = lanes<T>(x[i], k);
                    a[2] = fma(xk, xk, a[2]);
                    a[3] = fma(q, lanes<T>(d[i], k), a[3]);
                }
                if constexpr (PRE) {
                    const L hk = lanes<T>(h[i], k);
                    gy = product<T>(y[i], pw[i], k);
                    a[0] = fma(hk, hk, a[0]);
                    a[1] = fma(gy, hk, a[1]);
                    if constexpr (POST) {
                        a[4] = fma(q, gy, a[4]);
                        a[5] = fma(q, hk, a[5]);
                    }
                }
            }
        }
        // the sums that there are, in the order of block_factors
        constexpr int FIRST = PRE ? 0 : 2;
#pragma unroll
        for (int k = 0; k < NS; ++k) s.v[k] = a[FIRST + k].total();
        if constexpr (NS > 0) s.gather(red[n & 1], at.width);
        if (__syncthreads_or(!ok)) break;                     // uniform
        if (threadIdx.x < 32 && n + p.nslots < ring.count) ring.issue(slot, n + p.nslots, ahead);
        if constexpr (NS > 0) {
            s.totals(red[n & 1], at.width, at.gw0, at.wpg);
            if (CL && !exchange_sums<NS>(ex, s.v, p.cluster, rank, static_cast<uint32_t>(n), p)) bad = true;
        }
        stay_packed(x);
        stay_packed(d);
        if constexpr (PRE) {
            stay_packed(y);
            stay_packed(h);
        }
        float six[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NS; ++k) six[FIRST + k] = s.v[k];
        const BlockFactors f = block_factors(six, p);
        const L rh = L::all(f.rh), kh = L::all(-f.kh), rx = L::all(f.rx), kx = L::all(-f.kx);
        const L bs = L::all(p.branch_scale), rs = L::all(p.residual_scale);
        // rows that the block lacks have sums of what the slot held before, and add nothing
        if (here) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float ox[EPV], od[EPV];
                if constexpr (REREAD) read_pre(i);
#pragma unroll
                for (int k = 0; k < PN; ++k) {
                    const L xk = lanes<T>(x[i], k);
                    L D = lanes<T>(d[i], k);
                    if constexpr (PRE) {
                        const L hk = lanes<T>(h[i], k);
                        D = fma(rh, fma(hk, kh, product<T>(y[i], pw[i], k)), D);
                        pre[i * PN + k] = fma(lanes<T>(y[i], k), hk * rh, pre[i * PN + k]);
                    }
                    (D * rs).put(od + 2 * k);
                    const L e = D * bs * factor(i, k);
                    if constexpr (POST) {
                        acc[i * PN + k] = fma(D, xk * rx, acc[i * PN + k]);
                        (fma(xk, kx, e) * rx).put(ox + 2 * k);
                    } else {
                        acc[i * PN + k] = fma(D, xk, acc[i * PN + k]);
                        e.put(ox + 2 * k);
                    }
                }
                const int64_t to = row * ring.row_bytes + col[i];
                store_vec<VB, false>(static_cast<char*>(p.dx) + to, apart, valid[i], pack<T, 16>(ox));
                store_vec<VB, false>(static_cast<char*>(p.dres) + to, apart, valid[i], pack<T, 16>(od));
            }
        }
        if (++slot == p.nslots) {
            slot = 0;
            ++use;
        }
    }
    if constexpr (CL) bad = __syncthreads_or(bad);      // after the last row nothing else says so
    if (n < ring.count || bad) {
        if (threadIdx.x == 0) {
            if (!bad) report_timeout(p.status, kSiteStagedFull);
            ring.drain(n, slot, use);
        }
        __syncthreads();
    } else if (ring.count > 0) {
        write_gate(last_gate);
        if constexpr (PRE) {
            if (p.part_pre)
                write_part<T, VB>(pre, p.part_pre + static_cast<int64_t>(unit) * p.hidden, at, p.block_rows, col,
                                  valid, scratch, slice_elems, first_elem);
        }
    }
    if constexpr (CL) {
        __syncthreads();
        cluster_sync_all();
    }
}

}  // namespace rmsnorm
