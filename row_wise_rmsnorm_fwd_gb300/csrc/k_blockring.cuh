// k_blockring.cuh -- row blocks brought into shared memory by 1-D bulk copies,
// a ring of them in flight.
//
// A CTA works on blocks of `block_rows` rows of one or two arrays of the same
// layout.  Bulk copies and vector accesses want 16-byte boundaries:
//
// Aligned rows (a multiple of 16 bytes): a block is consecutive rows, one copy
// per array.
//
// SHIFT, rows of any length (from 32 bytes): row r begins r * H mod EPV elements
// behind a boundary, which has a period of `period` (1, 2, 4 or 8) rows.  A CTA
// takes rows r = its number mod period only, so all its rows have the same
// shift, and every column the same place in a vector: row by row its vectors,
// weights and column sums line up as for aligned rows, `shift` elements later.
// Each row is copied by itself, from the boundary at or before its start to the
// one at or after its end; the bytes around it belong to the neighbouring
// rows (the arrays start on a boundary).  Only behind the arrays' last boundary
// nothing may be read: what the arrays' last row has there, less than 16 bytes,
// is copied by threads (finish).
//
// Slots are handed back without "empty" barriers: a kernel has one block-wide
// barrier in each iteration, and behind the one of iteration n every thread is
// done with iteration n - 1, whose slot one warp then refills.  Proxy rule as in
// k_ring.cuh: a slot that the async proxy writes is read by generic loads only
// behind the mbarrier wait, and refilled behind the block barrier; finish's
// generic writes go to a CTA's last block, which nothing overwrites.
#pragma once
#include "common.cuh"
#include "norm_launch.h"

namespace rmsnorm {

constexpr int kBlockRingMaxSlots = 8;

// Slot and use number of consecutive blocks.
struct RingStep {
    int slot = 0;
    uint32_t use = 0;
    __device__ __forceinline__ void next(int nslots) {
        if (++slot == nslots) {
            slot = 0;
            ++use;
        }
    }
};

// The kernel's parameters are read where they are needed (they are in constant
// memory) rather than kept in registers; NARR arrays (x, and dy).
template <typename T, bool SHIFT, int NARR>
struct RowRing {
    static constexpr int EPV = 16 / static_cast<int>(sizeof(T));
    const NormParams& p;
    const int block_rows;
    uint32_t slots;              // shared-memory address of p.nslots * NARR * block_rows * row slots
    uint32_t bars;               // of p.nslots mbarriers
    int shift;                   // elements of a row's first vector before the row
    int64_t first, step;         // the CTA's first row, and rows from block to block
    int count;                   // blocks of this CTA

    __device__ __forceinline__ int period() const { return SHIFT ? p.period : 1; }
    __device__ __forceinline__ int row_bytes() const { return p.hidden * static_cast<int>(sizeof(T)); }
    __device__ __forceinline__ int row_slot() const { return SHIFT ? p.row_slot : row_bytes(); }
    // Bytes of an array before its last boundary.
    __device__ __forceinline__ int64_t inside() const { return p.rows * row_bytes() / 16 * 16; }
    // Shared-memory address of array a's part of a slot.
    __device__ __forceinline__ uint32_t base(int slot, int a) const {
        return slots + static_cast<uint32_t>((slot * NARR + a) * block_rows * row_slot());
    }

    // All threads; then a barrier before the first issue.
    __device__ __forceinline__ RowRing(const NormParams& p_, int block_rows_, unsigned char* smem,
                                       uint64_t* barriers)
        : p(p_), block_rows(block_rows_), slots(smem_addr(smem)), bars(smem_addr(barriers)) {
        const int cls = static_cast<int>(blockIdx.x) % period();
        const int mine = static_cast<int>(blockIdx.x) / period();
        // CTAs of the class, and its blocks
        const int64_t ctas = (static_cast<int>(gridDim.x) - cls + period() - 1) / period();
        const int64_t class_rows = p.rows > cls ? (p.rows - cls + period() - 1) / period() : 0;
        const int64_t blocks = (class_rows + block_rows - 1) / block_rows;
        count = mine < blocks ? static_cast<int>((blocks - mine + ctas - 1) / ctas) : 0;
        first = cls + static_cast<int64_t>(mine) * block_rows * period();
        step = ctas * block_rows * period();
        shift = SHIFT ? static_cast<int>(static_cast<int64_t>(cls) * p.hidden % EPV) : 0;
        if (threadIdx.x == 0) {
            for (int k = 0; k < p.nslots; ++k) mbar_init(bars + 8 * k, 1);
            fence_mbarrier_init_cluster();
        }
    }

    // One warp: start the copies of the CTA's n-th block into `slot`.
    __device__ __forceinline__ void issue(int slot, int n) const {
        const int lane = threadIdx.x & 31;
        const uint32_t bar = bars + 8 * slot;
        const char* x = static_cast<const char*>(p.x);
        const char* dy = static_cast<const char*>(p.dy);
        const int64_t row0 = first + n * step;
        const int64_t left = (p.rows - row0 + period() - 1) / period();  // rows of the class from there
        const int nrows = static_cast<int>(left < block_rows ? left : block_rows);
#if RMSNORM_FAULT_INJECT
        if (p.fault == kFaultStagedWithholdCopy && n == 0) {   // armed for bytes that never come
            if (lane == 0) mbar_arrive_expect_tx(bar, 16);
            return;
        }
#endif
        if constexpr (!SHIFT) {
            if (lane == 0) {
                const uint32_t bytes = static_cast<uint32_t>(nrows * row_bytes());
                const int64_t at = row0 * row_bytes();
                mbar_arrive_expect_tx(bar, bytes * NARR);
                bulk_g2s_plain(base(slot, 0), x + at, bytes, bar);
                if (NARR == 2) bulk_g2s_plain(base(slot, 1), dy + at, bytes, bar);
            }
        } else {
            // a row's window is the same size for all rows of the class but the arrays' last
            const uint32_t whole = static_cast<uint32_t>((shift * static_cast<int>(sizeof(T)) +
                                                          row_bytes() + 15) / 16 * 16);
            const int64_t from = row0 * row_bytes() / 16 * 16;
            const int64_t stride = static_cast<int64_t>(period()) * row_bytes();
            const int64_t end = from + (nrows - 1) * stride + whole;     // of the last row's window
            const uint32_t over = end > inside() ? static_cast<uint32_t>(end - inside()) : 0u;
            if (lane == 0) mbar_arrive_expect_tx(bar, (whole * nrows - over) * NARR);
            __syncwarp();
            for (int r = lane; r < nrows; r += 32) {
                const uint32_t bytes = r == nrows - 1 ? whole - over : whole;
                const uint32_t to = static_cast<uint32_t>(r * row_slot());
                bulk_g2s_plain(base(slot, 0) + to, x + from + r * stride, bytes, bar);
                if (NARR == 2) bulk_g2s_plain(base(slot, 1) + to, dy + from + r * stride, bytes, bar);
            }
        }
    }

    // One warp: the CTA's first blocks.
    __device__ __forceinline__ void prologue() const {
        for (int k = 0; k < p.nslots && k < count; ++k) issue(k, k);
    }

    // One warp, behind the barrier of iteration n: refill the slot of n - 1.
    __device__ __forceinline__ void refill(const RingStep& s, int n) const {
        if (n > 0 && n - 1 + p.nslots < count)
            issue(s.slot ? s.slot - 1 : p.nslots - 1, n - 1 + p.nslots);
    }

    // All threads, after the CTA's last block has landed: what the arrays' last
    // row, if it is among its rows, has behind their last boundary.  Ends with a
    // barrier if there is any.
    __device__ __forceinline__ void finish(int slot, int n) const {
        if (!SHIFT || n != count - 1) return;
        const int64_t total = p.rows * row_bytes();
        const int64_t row0 = first + n * step;
        const int64_t last = p.rows - 1;
        const int tail = static_cast<int>((total - inside()) / static_cast<int>(sizeof(T)));
        if (tail == 0 || last < row0 || (last - row0) % period() != 0 ||
            (last - row0) / period() >= block_rows)
            return;                                          // uniform
        if (static_cast<int>(threadIdx.x) < tail) {
            const int r = static_cast<int>((last - row0) / period());
            const int64_t at = last * row_bytes() / 16 * 16;   // the row's window starts there
            const uint32_t to = static_cast<uint32_t>(r * row_slot()) +
                                static_cast<uint32_t>(inside() - at) +
                                threadIdx.x * static_cast<uint32_t>(sizeof(T));
            copy_elem(base(slot, 0) + to, static_cast<const char*>(p.x) + inside());
            if (NARR == 2) copy_elem(base(slot, 1) + to, static_cast<const char*>(p.dy) + inside());
        }
        __syncthreads();
    }
    __device__ __forceinline__ void copy_elem(uint32_t to, const char* from) const {
        const T v = reinterpret_cast<const T*>(from)[threadIdx.x];
        if constexpr (sizeof(T) == 4) {
            asm volatile("st.shared.u32 [%0], %1;" :: "r"(to), "r"(__float_as_uint(v)) : "memory");
        } else {
            asm volatile("st.shared.u16 [%0], %1;" :: "r"(to), "h"(__bfloat16_as_ushort(v))
                         : "memory");
        }
    }

    // Wait (bounded) for the block at `s`.
    __device__ __forceinline__ bool wait(const RingStep& s) const {
        return mbar_wait_bounded<false>(bars + 8 * s.slot, s.use & 1u, p.timeout_ns);
    }

    // One thread, after the wait for block n, at `s`, has run out and every
    // thread has left the loop before its refill: wait (bounded) for what is
    // under way.
    __device__ __forceinline__ void drain(RingStep s, int n) const {
        const int issued = n == 0 ? p.nslots : p.nslots - 1;   // blocks n, n + 1, ...
        for (int k = 0; k < issued && n + k < count; ++k) {
            wait(s);
            s.next(p.nslots);
        }
    }
};

// 16 bytes of shared memory.  Volatile: a kernel that passes over its rows
// several times reads them again instead of keeping them, widened, in registers.
__device__ __forceinline__ Vec<16> ld_slot(uint32_t a) {
    Vec<16> v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.u[0]), "=r"(v.u[1]), "=r"(v.u[2]), "=r"(v.u[3]) : "r"(a));
    return v;
}

// The same where `on`, else zeros: one predicated load, no branch.
__device__ __forceinline__ Vec<16> ld_slot_if(uint32_t a, bool on) {
    Vec<16> v;
    const uint32_t q = on;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                 "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
                 "@p ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
                 : "=&r"(v.u[0]), "=&r"(v.u[1]), "=&r"(v.u[2]), "=&r"(v.u[3]) : "r"(a), "r"(q));
    return v;
}

// A row in its slot: whole vectors, and with SHIFT up to EPV - 1 elements before
// the first and behind the last of them (its edges), which threads take one
// by one, so that the loops over vectors stay those of aligned rows.
template <typename T, bool SHIFT>
struct RowVecs {
    static constexpr int EPV = 16 / static_cast<int>(sizeof(T));
    int nvec, hidden;
    int head, edges;         // elements before the vectors, and on both sides
    int skip;                // of the slot's first vector, elements before the row
    __device__ __forceinline__ RowVecs(int shift, int hidden_) : hidden(hidden_) {
        skip = SHIFT ? shift : 0;
        head = SHIFT ? min((EPV - skip) % EPV, hidden) : 0;
        nvec = (hidden - head) / EPV;
        edges = SHIFT ? hidden - nvec * EPV : 0;
    }
    // column of vector v's first element, and its bytes from the slot's row on
    __device__ __forceinline__ int col(int v) const { return head + v * EPV; }
    __device__ __forceinline__ int vec_at() const { return SHIFT && skip > 0 ? 16 : 0; }
    // the same for edge element e
    __device__ __forceinline__ int edge_col(int e) const { return e < head ? e : e + nvec * EPV; }
    __device__ __forceinline__ int edge_at(int e) const {
        return (skip + edge_col(e)) * static_cast<int>(sizeof(T));
    }
};

// One element of shared memory, widened; stored to global memory.
template <typename T>
__device__ __forceinline__ float ld_elem(uint32_t a) {
    if constexpr (sizeof(T) == 4) {
        float v;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
        return v;
    } else {
        Vec<2> v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v.h) : "r"(a));
        return get<T, 2>(v, 0);
    }
}
template <typename T>
__device__ __forceinline__ void st_elem(void* base, int64_t at, float v) {
    constexpr int sz = static_cast<int>(sizeof(T));
    const float f[1] = {v};
    st_stream<sz>(static_cast<char*>(base) + at * sz, pack<T, sz>(f));
}

// Weights laid out like a row in its slot, in shared memory; size = elements of
// a row's slot.
template <typename T>
__device__ __forceinline__ void copy_shifted(T* to, const void* from, int skip, int hidden, int size,
                                             float fill) {
    const T* w = static_cast<const T*>(from);
    for (int j = threadIdx.x; j < size; j += blockDim.x) {
        const bool in = j >= skip && j < skip + hidden;
        to[j] = w && in ? w[j - skip] : static_cast<T>(fill);
    }
}

// The vectors t, t + G, ... of a row of nvec: `full` of them (nvec / G) every
// thread has, one more those with `more`.
template <typename F>
__device__ __forceinline__ void for_vectors(int t, int G, int full, bool more, F f) {
    int i = full;
    for (; i >= 4; i -= 4, t += 4 * G) {
        f(t);
        f(t + G);
        f(t + 2 * G);
        f(t + 3 * G);
    }
    if (i & 2) {
        f(t);
        f(t + G);
        t += 2 * G;
    }
    if (i & 1) {
        f(t);
        t += G;
    }
    if (more) f(t);
}

// Sum over the lanes of a share: a warp, or fewer than 32 lanes (a power of two).
__device__ __forceinline__ float share_sum(float v, int width) {
    return width == 32 ? warp_allreduce_sum(v) : group_allreduce_sum(v, width);
}

}  // namespace rmsnorm
