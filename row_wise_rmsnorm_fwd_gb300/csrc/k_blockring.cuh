// k_blockring.cuh -- row blocks brought into shared memory by 1-D bulk copies,
// a ring of them in flight.
//
// A CTA works on row blocks first, first + stride, ...; a block is
// `block_bytes` of consecutive rows of one or two arrays of the same layout.
// Rows may have any length: a bulk copy wants 16-byte boundaries, so a block is
// copied from the boundary at or before its start to the one at or after its
// end, and its rows begin `shift` bytes into the slot.  The bytes around it
// belong to the neighbouring rows (the arrays start on a boundary); only
// behind the arrays' last boundary nothing may be read, so what a block has
// there, less than 16 bytes, is copied by threads (finish_block).
//
// Slots are handed back without "empty" barriers: a kernel has one block-wide
// barrier in each iteration, and behind the one of iteration n every thread is
// done with iteration n - 1, whose slot one thread then refills.  Proxy rule
// as in k_ring.cuh: a slot that the async proxy writes is read by generic loads
// only behind the mbarrier wait, and refilled behind the block barrier;
// finish_block's generic writes go to a CTA's last block, which nothing
// overwrites.
#pragma once
#include "common.cuh"

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

struct BlockRing {
    const char* src[2];          // src[1] null: one array
    uint32_t slots;              // shared-memory address of nslots * narrays * slot_bytes
    uint32_t bars;               // of nslots mbarriers
    int nslots;
    int slot_bytes;              // one array's share of a slot
    int narrays;
    int64_t block_bytes;
    int64_t total_bytes;         // of one array
    int count;                   // blocks of this CTA
    int tail_from;               // of those, the first that reaches behind the arrays' last boundary

    static __device__ __forceinline__ int64_t down(int64_t v) { return v - (v & 15); }
    __device__ __forceinline__ int64_t start(int n) const {
        return (blockIdx.x + static_cast<int64_t>(n) * gridDim.x) * block_bytes;
    }

    // `units` blocks in all; all threads, then a barrier before the first issue.
    __device__ __forceinline__ void init(const void* a0, const void* a1, unsigned char* smem,
                                         uint64_t* barriers, int64_t units) {
        src[0] = static_cast<const char*>(a0);
        src[1] = static_cast<const char*>(a1);
        narrays = a1 ? 2 : 1;
        slots = smem_addr(smem);
        bars = smem_addr(barriers);
        const int64_t grid = gridDim.x, mine = blockIdx.x;
        count = mine < units ? static_cast<int>((units - mine + grid - 1) / grid) : 0;
        tail_from = count;
        while (tail_from > 0 && start(tail_from - 1) + block_bytes > down(total_bytes)) --tail_from;
        if (threadIdx.x == 0) {
            for (int k = 0; k < nslots; ++k) mbar_init(bars + 8 * k, 1);
            fence_mbarrier_init_cluster();
        }
    }

    // Shared-memory address of array a's part of a slot; the n-th block's rows
    // begin start(n) & 15 bytes into it.
    __device__ __forceinline__ uint32_t base(int slot, int a) const {
        return slots + static_cast<uint32_t>((slot * narrays + a) * slot_bytes);
    }

    // One thread: start the copies of the CTA's n-th block into `slot`.
    __device__ __forceinline__ void issue(int slot, int n, int fault) const {
        const int64_t from = down(start(n));
        const int64_t to = min(down(start(n) + block_bytes + 15), down(total_bytes));
        const uint32_t bytes = to > from ? static_cast<uint32_t>(to - from) : 0u;
        const uint32_t bar = bars + 8 * slot;
#if RMSNORM_FAULT_INJECT
        if (fault == kFaultStagedWithholdCopy && n == 0) {   // armed for bytes that never come
            mbar_arrive_expect_tx(bar, 16);
            return;
        }
#else
        (void)fault;
#endif
        mbar_arrive_expect_tx(bar, bytes * narrays);
        if (bytes == 0) return;
        for (int a = 0; a < narrays; ++a) bulk_g2s_plain(base(slot, a), src[a] + from, bytes, bar);
    }

    // One thread: the CTA's first blocks.
    __device__ __forceinline__ void prologue(int fault) const {
        for (int k = 0; k < nslots && k < count; ++k) issue(k, k, fault);
    }

    // One thread, behind the barrier of iteration n: refill the slot of n - 1.
    __device__ __forceinline__ void refill(const RingStep& step, int n, int fault) const {
        if (n > 0 && n - 1 + nslots < count)
            issue(step.slot ? step.slot - 1 : nslots - 1, n - 1 + nslots, fault);
    }

    // All threads, after block n >= tail_from has landed: its bytes behind the
    // arrays' last boundary.  Ends with a barrier.
    template <typename T>
    __device__ __forceinline__ void finish(int slot, int n) const {
        const int64_t at = start(n);
        const int64_t end = min(at + block_bytes, total_bytes);
        const int64_t from = max(down(total_bytes), at);
        const int tail = static_cast<int>((end - from) / static_cast<int>(sizeof(T)));
        if (static_cast<int>(threadIdx.x) < tail) {
            for (int a = 0; a < narrays; ++a) {
                const T v = reinterpret_cast<const T*>(src[a] + from)[threadIdx.x];
                const uint32_t to = base(slot, a) + static_cast<uint32_t>(from - down(at)) +
                                    threadIdx.x * static_cast<uint32_t>(sizeof(T));
                if constexpr (sizeof(T) == 4) {
                    asm volatile("st.shared.u32 [%0], %1;" :: "r"(to), "r"(__float_as_uint(v))
                                 : "memory");
                } else {
                    asm volatile("st.shared.u16 [%0], %1;" :: "r"(to), "h"(__bfloat16_as_ushort(v))
                                 : "memory");
                }
            }
        }
        __syncthreads();
    }

    // Wait (bounded) for the block in `slot` on the slot's `use`-th use.
    __device__ __forceinline__ bool wait(const RingStep& step, uint64_t timeout_ns) const {
        return mbar_wait_bounded<false>(bars + 8 * step.slot, step.use & 1u, timeout_ns);
    }

    // One thread, after the wait for block n, at `step`, has run out and every
    // thread has left the loop before its refill: wait (bounded) for what is
    // under way.
    __device__ __forceinline__ void drain(RingStep step, int n, uint64_t timeout_ns) const {
        const int issued = n == 0 ? nslots : nslots - 1;     // blocks n, n + 1, ...
        for (int k = 0; k < issued && n + k < count; ++k) {
            wait(step, timeout_ns);
            step.next(nslots);
        }
    }
};

// A vector of shared memory.  Volatile: a kernel that passes over its rows
// several times reads them again instead of keeping them, widened, in registers.
template <int VB>
__device__ __forceinline__ Vec<VB> ld_slot(uint32_t a) {
    Vec<VB> v;
    if constexpr (VB == 16) {
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.u[0]), "=r"(v.u[1]), "=r"(v.u[2]), "=r"(v.u[3]) : "r"(a));
    } else if constexpr (VB == 8) {
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.u[0]), "=r"(v.u[1]) : "r"(a));
    } else if constexpr (VB == 4) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v.u[0]) : "r"(a));
    } else {
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v.h) : "r"(a));
    }
    return v;
}

// The same where `on`, else zeros: one predicated load, no branch.
template <int VB>
__device__ __forceinline__ Vec<VB> ld_slot_if(uint32_t a, bool on) {
    Vec<VB> v;
    const uint32_t q = on;
    if constexpr (VB == 16) {
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                     "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
                     "@p ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
                     : "=&r"(v.u[0]), "=&r"(v.u[1]), "=&r"(v.u[2]), "=&r"(v.u[3]) : "r"(a), "r"(q));
    } else if constexpr (VB == 8) {
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                     "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
                     "@p ld.shared.v2.u32 {%0,%1}, [%2];\n\t}"
                     : "=&r"(v.u[0]), "=&r"(v.u[1]) : "r"(a), "r"(q));
    } else if constexpr (VB == 4) {
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t"
                     "@p ld.shared.u32 %0, [%1];\n\t}" : "=&r"(v.u[0]) : "r"(a), "r"(q));
    } else {
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t"
                     "@p ld.shared.u16 %0, [%1];\n\t}" : "=&h"(v.h) : "r"(a), "r"(q));
    }
    return v;
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
