// Device helpers shared by the serving operators (prompt attention, key weights, the 8-bit
// key/value cache): work items of a packed batch, block reductions.
#pragma once

#include "common.cuh"

namespace energon {

// A bounded wait ran out earlier: no more work.  (The other bits concern single sequences; a
// launch that stopped at them would compute what its blocks happened to start before.)
__device__ __forceinline__ bool stopped(const int32_t* st) {
    return st != nullptr && (*reinterpret_cast<const volatile int32_t*>(st) & ENERGON_DEVICE_TIMEOUT) != 0;
}

// The same for a whole block at once: another kernel may set the bit while this one starts, and warps that
// meet at barriers, or take each other's counts, must not part.
__device__ __forceinline__ bool block_stopped(const int32_t* st) { return __syncthreads_or(stopped(st)) != 0; }

// Rows of sequence b of a packed batch; false (and n = 0) when they do not lie in [0, rows].
__device__ __forceinline__ bool seq_rows(const int32_t* __restrict__ cu, int b, int rows, int& start, int& n) {
    start = cu[b];
    const int end = cu[b + 1];
    n = end - start;
    if (start >= 0 && end >= start && end <= rows) return true;
    n = 0;
    return false;
}

// Passes over the sequences of a packed batch, 32 at a time (a lane each), and tells which are good: rows in
// [0, rows], none of them between the first and the last row of the sequences before.  Good sequences then
// share no row, so that none is written twice and the launches' bounds on the work hold whatever the
// offsets are.  (Where all offsets ascend in [0, rows] all sequences are good.)
struct RowWalk {
    int lo = 0x7fffffff, hi = -1;  // first and last + 1 of the rows passed so far
    // Sequence base + lane: its first row, and how many rows; n = 0 where it is not good, and behind the last one.
    __device__ __forceinline__ void step(const int32_t* __restrict__ cu, int batch, int base, int rows, int& start, int& n) {
        constexpr unsigned ALL = 0xffffffffu;
        const int lane = threadIdx.x & 31;
        start = n = 0;
        if (base + lane < batch) seq_rows(cu, base + lane, rows, start, n);
        int a = n > 0 ? start : 0x7fffffff, z = n > 0 ? start + n : -1;  // of this sequence and those before
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(ALL, a, o), y = __shfl_up_sync(ALL, z, o);
            if (lane >= o) a = min(a, x), z = max(z, y);
        }
        a = min(a, lo), z = max(z, hi);
        int before_lo = __shfl_up_sync(ALL, a, 1), before_hi = __shfl_up_sync(ALL, z, 1);
        if (lane == 0) before_lo = lo, before_hi = hi;
        lo = __shfl_sync(ALL, a, 31), hi = __shfl_sync(ALL, z, 31);
        if (start < before_hi && start + n > before_lo) n = 0;
    }
};

// The item among 32 sequences, this lane's with n items, `before` items before them: the lane, or -1, and the
// item's index inside its sequence.
__device__ __forceinline__ int item_lane(int item, int n, int& before, int& j) {
    const int lane = threadIdx.x & 31;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, item < before + x);
    if (past) {
        const int l = __ffs(past) - 1;
        j = item - before - __shfl_sync(0xffffffffu, x - n, l);
        return l;
    }
    before += __shfl_sync(0xffffffffu, x, 31);
    return -1;
}
// find_item where some sequence's rows are not in [0, rows]; -1 when there are fewer items.  (Apart: in line this
// code, hardly ever run, cost the kernels around it 2 to 4 %.)
template <typename F>
__device__ __noinline__ int2 find_item_walk(const int32_t* __restrict__ cu, int batch, int rows, int item, F count) {
    RowWalk walk;
    int before = 0, j = 0;
    for (int base = 0; base < batch; base += 32) {
        int start, len;
        walk.step(cu, batch, base, rows, start, len);
        const int b = base + (threadIdx.x & 31);
        const int l = item_lane(item, b < batch ? count(b, len) : 0, before, j);
        if (l >= 0) return make_int2(base + l, j);
    }
    return make_int2(-1, 0);
}
// Work item `item` of a packed batch in which good sequence b, of n rows, has count(b, n) items (>= 0; none
// of n = 0): the sequence and the item's index inside it.  Every warp computes it for itself, 32 sequences at
// a time; the result is the same in every thread.  False when there are fewer items.
template <typename F>
__device__ __forceinline__ bool find_item(const int32_t* __restrict__ cu, int batch, int rows, int item, F count, int& b, int& j) {
    int before = 0;
    for (int base = 0; base < batch; base += 32) {
        const int i = base + (threadIdx.x & 31);
        int start, len = 0;
        const bool inside = i >= batch || seq_rows(cu, i, rows, start, len);
        const int l = item_lane(item, i < batch ? count(i, len) : 0, before, j);
        if (__any_sync(0xffffffffu, !inside)) {
            const int2 at = find_item_walk(cu, batch, rows, item, count);
            b = at.x, j = at.y;
            return b >= 0;
        }
        if (l >= 0) {
            b = base + l;
            return true;
        }
    }
    return false;
}

// Records ENERGON_DEVICE_BAD_LENGTH if some sequence is not good; called by one warp of one block of a
// launch.  (Only a step back of the offsets, itself a sequence of less than 0 rows, makes sequences meet.)
__device__ __forceinline__ void check_rows(const int32_t* __restrict__ cu, int batch, int rows, int32_t* status) {
    bool bad = false;
    for (int b = threadIdx.x & 31; b < batch; b += 32) {
        int s, n;
        bad |= !seq_rows(cu, b, rows, s, n);
    }
    if (bad) status_or(status, ENERGON_DEVICE_BAD_LENGTH);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Bounded wait for the phase of `parity`, in line: a call would make its caller hold its registers
// in the call's order.  Gives up like mbar_wait_bounded.
__device__ __forceinline__ bool wait_in_line(uint64_t* bar, uint32_t parity, const volatile int* abort_flag,
                                             uint64_t timeout_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    const uint32_t tries = tries_between_looks(timeout_ns);
    for (uint32_t it = 1; it < (1u << 30); ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & tries) == 0 && (*abort_flag || global_ns() - t0 > timeout_ns)) return false;
    }
    return false;
}

// One lane of a converged warp, the same one each time.  Work that a single thread issues is issued
// by a warp whose control flow is uniform: its operands then live in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// Limit of the waits for copies and products that are in flight when a block ends: they must not land
// in the shared memory of the next block, however short the limit that a caller set for other waits.
__device__ __forceinline__ uint64_t landing_limit(uint64_t timeout_ns) { return timeout_ns > 1000000000ull ? timeout_ns : 1000000000ull; }

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 one_by_one(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// 2^x; results below the normal range are 0 (they would be lost in 16 bits, and in a sum >= 1).
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 2^x of a pair without the special function unit (16 results per cycle and SM, where the FMA pipe
// makes 128 operations): x = j + f with j whole and |f| <= 1/2 (the reduction of W. J. Cody, W. Waite, Software
// Manual for the Elementary Functions, 1980), 2^f by a polynomial of degree 5 with constant term 1 fitted for the smallest relative error (1.7e-7), times 2^j from j's bits.
// x <= 126; below -126 the result is 0 or next to it; NaN stays NaN.
__device__ __forceinline__ float2 exp2_poly(float2 x) {
    constexpr float MAGIC = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.x) : "f"(-127.0f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.y) : "f"(-127.0f));
    const uint64_t t = two(x.x, x.y);
    const uint64_t r = add2(t, two(MAGIC, MAGIC));
    const uint64_t f = fma2(add2(r, two(-MAGIC, -MAGIC)), two(-1.0f, -1.0f), t);
    uint64_t y = fma2(f, two(0.001326472033f, 0.001326472033f), two(0.009671512991f, 0.009671512991f));
    y = fma2(y, f, two(0.055507339537f, 0.055507339537f));
    y = fma2(y, f, two(0.240222424269f, 0.240222424269f));
    y = fma2(y, f, two(0.693147003651f, 0.693147003651f));
    y = fma2(y, f, two(1.0f, 1.0f));
    // the low bits of r are those of j
    const float2 j = one_by_one(r);
    const float a = __uint_as_float(__float_as_uint(j.x) * 0x800000u + 0x3f800000u);
    const float b = __uint_as_float(__float_as_uint(j.y) * 0x800000u + 0x3f800000u);
    return one_by_one(mul2(y, two(a, b)));
}

// Chained launches: a kernel may start while the one before it ends; it waits before it reads.
__device__ __forceinline__ void wait_for_earlier_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Launch that may start while the kernel before it ends (it waits for it itself).
template <typename... P, typename... A>
static cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace energon
