// k_rowblocks.cuh -- blocks of consecutive rows of several arrays brought into shared
// memory by 1-D bulk copies, a ring of them in flight, for kernels that take a block
// into registers at once: its slot is refilled behind the block barrier that every
// kernel has for the rows' sums, so a ring of two keeps a whole block under way at all
// times.
//
// Arrays are on 16-byte boundaries.  Rows of whole 16-byte vectors come many to a copy; RAGGED,
// rows of any length, each by itself, from the boundary at or before its start to the one at
// or after its end (the bytes around it belong to its neighbours).  Behind the arrays'
// last boundary nothing may be read by such copies: what the last row has there is copied by
// threads (finish).  With one gate row the blocks are dealt out in turn, so that the CTAs
// read side by side; else they lie within the rows of a gate row and are dealt out in
// contiguous ranges, so that a CTA meets few gate rows, in order.  With a cluster each CTA
// takes its slice of every row (one row to a block).
#pragma once
#include "blocknorm_launch.h"
#include "common.cuh"
#include "integers.cuh"

namespace rmsnorm {

constexpr int kRowBlocksMaxSlots = 4;

template <int NARR, bool RAGGED>
struct RowBlocks {
    const BlockParams& p;
    const char* src[NARR];       // null: absent
    int narr;                    // arrays present
    uint32_t slots, bars;        // shared-memory addresses
    int64_t first, step, count;  // the unit's blocks
    int unit;                    // number of the CTA, or of the cluster
    int row_bytes, at, bytes;    // a row, and the CTA's slice of it
    int slot_row;                // bytes of a row in a slot

    __device__ __forceinline__ RowBlocks(const BlockParams& p_, const void* const (&arrays)[NARR],
                                         int sz, uint32_t rank, int unit_, int units,
                                         unsigned char* smem, uint64_t* barriers)
        : p(p_), narr(0), slots(smem_addr(smem)), bars(smem_addr(barriers)), unit(unit_) {
#pragma unroll
        for (int a = 0; a < NARR; ++a) {
            src[a] = static_cast<const char*>(arrays[a]);
            narr += src[a] != nullptr;
        }
        if (p.gates == 1) {
            first = unit;
            step = units;
            count = (p.blocks - unit + units - 1) / units;
        } else {
            first = p.blocks * unit / units;
            step = 1;
            count = p.blocks * (unit + 1) / units - first;
        }
        row_bytes = p.hidden * sz;
        slot_row = RAGGED ? p.row_slot : p.slice_vecs * 16;
        at = RAGGED ? 0 : static_cast<int>(rank) * slot_row;
        bytes = row_bytes - at;
        if (!RAGGED && bytes > slot_row) bytes = slot_row;
        if (threadIdx.x == 0) {
            for (int k = 0; k < p.nslots; ++k) mbar_init(bars + 8 * k, 1);
            fence_mbarrier_init_cluster();
        }
    }

    // The unit's blocks in order: gate row, block within it, first row and number of rows.
    struct Cursor {
        int64_t gate, j, row;
        int rows;
    };
    __device__ __forceinline__ void locate(Cursor& c) const {
        c.row = c.gate * p.gate_rows + c.j * p.block_rows;
        int64_t end = (c.gate + 1) * p.gate_rows;
        if (end > p.rows) end = p.rows;
        c.rows = static_cast<int>(end - c.row < p.block_rows ? end - c.row : p.block_rows);
    }
    __device__ __forceinline__ Cursor start() const {
        Cursor c;
        c.gate = p.gates == 1 ? 0 : div_nonneg(first, p.blocks_per_gate);
        c.j = first - c.gate * p.blocks_per_gate;
        locate(c);
        return c;
    }
    __device__ __forceinline__ void advance(Cursor& c) const {
        c.j += step;
        if (p.gates > 1 && c.j == p.blocks_per_gate) {     // step is 1 then
            c.j = 0;
            ++c.gate;
        }
        locate(c);
    }

    // Shared-memory address of array a (counted with the absent ones) in a slot.
    __device__ __forceinline__ uint32_t base(int slot, int a) const {
        return slots + static_cast<uint32_t>((slot * NARR + a) * p.block_rows * slot_row);
    }

    // Bytes of an array before its last boundary.
    __device__ __forceinline__ int64_t inside() const { return p.rows * row_bytes / 16 * 16; }
    // Bytes of a row's slot before the row.
    __device__ __forceinline__ int skip(int64_t row) const {
        return RAGGED ? static_cast<int>(row * row_bytes % 16) : 0;
    }

    // One warp: start the copies of the n-th block, at `c`, into `slot`, and go on to the next.
    __device__ __forceinline__ void issue(int slot, int64_t n, Cursor& c) const {
        const int lane = threadIdx.x & 31;
        const uint32_t bar = bars + 8 * slot;
#if RMSNORM_FAULT_INJECT
        if (p.fault == kFaultStagedWithholdCopy && n == 0) {   // armed for bytes that never come
            if (lane == 0) mbar_arrive_expect_tx(bar, 16);
            advance(c);
            return;
        }
#endif
        const int64_t row = c.row;
        const int rows = c.rows;
        advance(c);
        if constexpr (!RAGGED) {
            if (lane != 0) return;
            // one row of a slice, or whole rows, which follow one another
            const uint32_t n_bytes = static_cast<uint32_t>(p.cluster > 1 ? bytes : rows * row_bytes);
            mbar_arrive_expect_tx(bar, n_bytes * narr);
            const int64_t from = row * row_bytes + at;
#pragma unroll
            for (int a = 0; a < NARR; ++a)
                if (src[a]) bulk_g2s_plain(base(slot, a), src[a] + from, n_bytes, bar);
        } else {
            // a row's window: as large as any row needs, but not past the last boundary
            auto window = [&](int r, int64_t& from) {
                from = (row + r) * row_bytes / 16 * 16;
                const int64_t left = inside() - from;
                return static_cast<uint32_t>(left < slot_row ? left : slot_row);
            };
            uint32_t total = 0;
            int64_t from;
            for (int r = lane; r < rows; r += 32) total += window(r, from);
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) total += __shfl_xor_sync(0xffffffffu, total, m);
            if (lane == 0) mbar_arrive_expect_tx(bar, total * narr);
            __syncwarp();
            for (int r = lane; r < rows; r += 32) {
                const uint32_t n_bytes = window(r, from);
                if (n_bytes == 0) continue;                 // a last row of less than 16 bytes
#pragma unroll
                for (int a = 0; a < NARR; ++a)
                    if (src[a])
                        bulk_g2s_plain(base(slot, a) + static_cast<uint32_t>(r * slot_row), src[a] + from,
                                       n_bytes, bar);
            }
        }
    }

    __device__ __forceinline__ void prologue(Cursor& c) const {
        for (int k = 0; k < p.nslots && k < count; ++k) issue(k, k, c);
    }

    // All threads, after a block has landed: what the arrays' last row, if it is the
    // block's last, has behind their last boundary.  Ends with a barrier if there is any.
    template <typename T>
    __device__ __forceinline__ void finish(int slot, int64_t row0, int rows) const {
        if constexpr (RAGGED) {
            const int64_t end = inside();
            const int tail = static_cast<int>((p.rows * row_bytes - end) / static_cast<int>(sizeof(T)));
            if (tail == 0 || row0 + rows != p.rows) return;      // uniform
            const int64_t from = (p.rows - 1) * row_bytes / 16 * 16;
            if (static_cast<int>(threadIdx.x) < tail) {
                const uint32_t to = static_cast<uint32_t>((rows - 1) * slot_row) +
                                    static_cast<uint32_t>(end - from) + threadIdx.x * static_cast<uint32_t>(sizeof(T));
#pragma unroll
                for (int a = 0; a < NARR; ++a) {
                    if (!src[a]) continue;
                    const char* v = src[a] + end + threadIdx.x * sizeof(T);
                    if constexpr (sizeof(T) == 4)
                        asm volatile("st.shared.u32 [%0], %1;" :: "r"(base(slot, a) + to),
                                     "r"(*reinterpret_cast<const uint32_t*>(v)) : "memory");
                    else
                        asm volatile("st.shared.u16 [%0], %1;" :: "r"(base(slot, a) + to),
                                     "h"(*reinterpret_cast<const uint16_t*>(v)) : "memory");
                }
            }
            __syncthreads();
        }
    }

    // Wait (bounded) for block n.
    __device__ __forceinline__ bool wait(int slot, uint32_t use) const {
        return mbar_wait_bounded<false>(bars + 8 * slot, use & 1u, p.timeout_ns);
    }

    // One thread, after the wait for block n has run out and every thread has left the
    // loop: wait (bounded) for what is under way.
    __device__ __forceinline__ void drain(int64_t n, int slot, uint32_t use) const {
        for (int k = 0; k < p.nslots && n + k < count; ++k) {
            wait(slot, use);
            if (++slot == p.nslots) {
                slot = 0;
                ++use;
            }
        }
    }
};

// ------------------------------------------------------------ sums of a row --

// Eight values summed over a warp in nine exchanges: lanes hand over the half of the values
// that they do not keep.  Lane L ends with the sum of value L / 4.
__device__ __forceinline__ float warp_sum8(const float (&v)[8]) {
    const int lane = threadIdx.x & 31;
    float a[4], b[2], c;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float keep = lane & 16 ? v[k + 4] : v[k], give = lane & 16 ? v[k] : v[k + 4];
        a[k] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float keep = lane & 8 ? a[k + 2] : a[k], give = lane & 8 ? a[k] : a[k + 2];
        b[k] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
    }
    {
        const float keep = lane & 4 ? b[1] : b[0], give = lane & 4 ? b[0] : b[1];
        c = keep + __shfl_xor_sync(0xffffffffu, give, 4);
    }
    c += __shfl_xor_sync(0xffffffffu, c, 2);
    return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

// N sums of each row group, in three steps around the block barrier of an iteration.
// red: [2][32][8] floats, the halves used in turn.
//   gather: before the barrier; group_totals: behind it.  Groups of less than a warp need no
//   shared memory: `width` lanes hold their totals already.
template <int N>
struct RowSums {
    float v[8];
    __device__ __forceinline__ RowSums() {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
    }
    __device__ __forceinline__ void gather(float* red, int width) {
        const int lane = threadIdx.x & 31;
        if (width < 32) {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = group_allreduce_sum(v[k], width);
        } else if constexpr (N > 2) {
            const float s = warp_sum8(v);
            if ((lane & 3) == 0) red[(threadIdx.x >> 5) * 8 + (lane >> 2)] = s;
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float s = warp_allreduce_sum(v[k]);
                if (lane == 0) red[(threadIdx.x >> 5) * 8 + k] = s;
            }
        }
    }
    // warps first .. first + n - 1 are the group's
    __device__ __forceinline__ void totals(const float* red, int width, int first, int n) {
        if (width < 32) return;
        const int lane = threadIdx.x & 31, k = lane & 7;
        float s = 0.f;
        if (k < N)
            for (int w = lane >> 3; w < n; w += 4) s += red[(first + w) * 8 + k];
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = __shfl_sync(0xffffffffu, s, j);
    }
};

}  // namespace rmsnorm
