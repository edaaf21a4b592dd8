// The attention weight that each key of the packed prompts receives, on the 5th-generation
// tensor cores (fp16, bf16).
//
//   w_h(t) = sum_{j in group h} sum_{s >= t, s in window} exp(c q_j(s) . k_h(t) - lse_j(s))
//
// The products are taken transposed, X = K Q^T with 128 keys as the rows: a key is then a lane of
// TMEM and a thread, its sum never leaves a register, and the sums lse_j(s) are one number per
// column, read from shared memory by all lanes at once.  Per 128 x 128 tile the tensor cores need
// 512 cycles (d = 128) and the exponentials 1024 (16 per cycle and SM), which bound the call: the
// products of one tile run while the exponentials of the tile before are taken (two buffers in
// TMEM), and two blocks share an SM.
//
// One block = 128 keys of one (sequence, kv head) and a part of the query heads that share them;
// the blocks of a group form a cluster, whose first block adds their sums in a fixed order.  With few
// queries per key (a window of up to 256) one block takes all heads: a block's start costs more than
// the steps that the others would take from it (the last 64 queries of 8 prompts: 18.6 us, with
// clusters of 4, and a head per step, it took 68).
//
// One prompt of 4096 tokens, all queries, 32 heads of 128, 8 kv heads, fp16: 100 us, 687 TFLOP/s; its 268 million
// exponentials alone would take the special function units 60 us.
#include <cudaTypedefs.h>
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "serving.cuh"

namespace energon {

namespace {
constexpr int BK = 128;            // keys per block
constexpr int BQ = 128;            // queries per step
constexpr int BOX = 128 * 128;     // bytes of 128 rows x 64 columns of 16 bits
constexpr int EXP_WARPS = 8;       // two threads per key, each with half of a step's queries
constexpr int THREADS = EXP_WARPS * 32 + 96;  // and loader, products, sums
// One pair of columns in four takes its exponentials from the FMA pipe (2^x by a polynomial): on
// one prompt of 4096 tokens with 32 heads 6 % faster than none and 8 % faster than every second.
constexpr int POLY = 8;
constexpr float LOG2E = 1.4426950408889634f;

template <int HD>
struct WCfg {
    static constexpr int TILE = HD / 64 * BOX;
    static constexpr int SMEM = 3 * TILE + 1024;  // keys, two buffers of queries
};
}  // namespace

// Adds the exponentials of 32 columns of a key's row; with EDGE only columns lo .. hi - 1 count.
template <bool EDGE>
__device__ __forceinline__ void add_exponentials(const uint32_t* r, const float* neg_lse, uint64_t c2, int lo, int hi,
                                                 uint64_t (&sum)[2]) {
    const float4* l4 = reinterpret_cast<const float4*>(neg_lse);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        const float4 l = l4[e / 4];
        float2 u = one_by_one(fma2(two(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), c2, two(l.x, l.y)));
        float2 v = one_by_one(fma2(two(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])), c2, two(l.z, l.w)));
        if (EDGE) {
            if (e < lo || e >= hi) u.x = -INFINITY;
            if (e + 1 < lo || e + 1 >= hi) u.y = -INFINITY;
            if (e + 2 < lo || e + 2 >= hi) v.x = -INFINITY;
            if (e + 3 < lo || e + 3 >= hi) v.y = -INFINITY;
        }
        sum[0] = add2(sum[0], two(exp2_fast(u.x), exp2_fast(u.y)));
        v = e % POLY == 0 ? exp2_poly(v) : make_float2(exp2_fast(v.x), exp2_fast(v.y));
        sum[1] = add2(sum[1], two(v.x, v.y));
    }
}

struct KeyWeightArgs {
    PromptArgs p;
    float c;      // scale * log2(e)
    int cluster;  // blocks that share the heads of a group
};

// QW: queries of a head in a step.  A window of at most 64 (32) leaves room for two (four) heads in it.
template <typename T, int HD, int QW>
__global__ void __launch_bounds__(THREADS, 2)
key_weights_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const KeyWeightArgs a) {
    using C = WCfg<HD>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t k_full, q_full[2], q_empty[2], s_full[2], s_empty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead;
    __shared__ __align__(16) float neg_lse[2][BQ];  // -lse in units of log2
    __shared__ float part[2][BK];
    const PromptArgs& p = a.p;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    // blocks of a cluster share the item; items of all kv heads pass by before the next tile of keys
    const int64_t lin = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) / a.cluster;
    const int rank = blockIdx.x % a.cluster, kvh = (int)(lin % p.n_kv);
    // What needs no length comes first: it runs under the loads of the lengths.
    const bool stop = stopped(p.status);
    if (warp == EXP_WARPS && lane == 0) {
        mbar_init(&k_full, 1), mbar_init(&drain, 1);
        for (int i = 0; i < 2; ++i)
            mbar_init(&q_full[i], 1), mbar_init(&q_empty[i], 1), mbar_init(&s_full[i], 33), mbar_init(&s_empty[i], EXP_WARPS * 32);
        dead = stop;  // the blocks of a cluster must not part: no early return
        fence_mbar_init();
        tma_prefetch_desc(&tm_k), tma_prefetch_desc(&tm_q);
    }
    if (warp == EXP_WARPS + 1) {
        tmem_alloc(&tmem_slot, 2 * BQ);
        tmem_relinquish();
    }
    if (lin == 0 && rank == 0 && tid < 32 && !stopped(p.status)) check_rows(p.cu, p.batch, p.rows, p.status);
    int b, blk, start, n;
    auto count = [](int, int len) { return (len + BK - 1) / BK; };
    if (!find_item(p.cu, p.batch, p.rows, (int)(lin / p.n_kv), count, b, blk)) {
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == EXP_WARPS + 1) tmem_dealloc(__shfl_sync(0xffffffffu, tmem_slot, 0), 2 * BQ);
        return;
    }
    seq_rows(p.cu, b, p.rows, start, n);
    const int t0 = blk * BK, group = p.n_heads / p.n_kv, heads = group / a.cluster;
    const int head0 = kvh * group + rank * heads;
    const int begin = max(t0, n - min(p.window, n));  // first query that counts for these keys
    constexpr int PACK = BQ / QW;                               // heads of a step
    const int per_head = PACK > 1 ? 1 : (n - begin + BQ - 1) / BQ;  // (PACK > 1: n - begin <= window <= QW)
    const int steps = PACK > 1 ? (heads + PACK - 1) / PACK : per_head * heads;
    // column c of step x: head `head_of` of this block (may be behind the last), query `query_of`
    auto head_of = [&](int x, int c) { return PACK > 1 ? x * PACK + c / QW : x / per_head; };
    auto query_of = [&](int x, int c) { return PACK > 1 ? begin + c % QW : begin + x % per_head * BQ + c; };

    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sq = base + C::TILE;
    auto load_queries = [&](int x) {
        const int live = min(PACK, heads - head_of(x, 0));
        mbar_arrive_expect_tx(&q_full[x & 1], C::TILE / PACK * live);
        for (int i = 0; i < live; ++i)
            for (int h = 0; h < HD / 64; ++h)
                tma_load_2d(sq + (x & 1) * C::TILE + h * BOX + i * QW * 128, &tm_q, &q_full[x & 1],
                            (head0 + head_of(x, i * QW)) * HD + 64 * h, start + query_of(x, 0));
    };
    if (warp == EXP_WARPS && lane == 0 && !stop) {  // (this thread made the barriers)
        mbar_arrive_expect_tx(&k_full, C::TILE);
        for (int h = 0; h < HD / 64; ++h) tma_load_2d(base + h * BOX, &tm_k, &k_full, kvh * HD + 64 * h, start + t0);
        for (int x = 0; x < min(steps, 2); ++x) load_queries(x);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
    const bool was_stopped = dead != 0;
    __syncthreads();
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (wait_in_line(bar, parity, &dead, p.timeout_ns)) return true;
        *reinterpret_cast<volatile int*>(&dead) = 1;
        return false;
    };
    // TMEM is read, and work is issued, by whole warps: their lanes give up together
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };

    if (was_stopped) {
        // no work
    } else if (warp == EXP_WARPS) {
        if (lane == 0) {
            // ---- loader
            int x = min(steps, 2);
            for (; x < steps; ++x) {
                if (!wait(&q_empty[x & 1], ((x >> 1) - 1) & 1)) break;
                load_queries(x);
            }
            // all copies have landed before the block ends, also where a wait ran out
            mbar_wait_bounded(&k_full, 0, nullptr, landing_limit(p.timeout_ns));
            for (int y = max(0, x - 2); y < x; ++y) mbar_wait_bounded(&q_full[y & 1], (y >> 1) & 1, nullptr, landing_limit(p.timeout_ns));
        }
    } else if (warp == EXP_WARPS + 1) {
        // ---- products: the whole warp follows, one lane issues
        constexpr uint32_t idesc = idesc_f16(std::is_same<T, __half>::value ? 0u : 1u, BK, BQ, 0);
        bool ok = wait_warp(&k_full, 0);
        for (int x = 0; ok && x < steps; ++x) {
            ok = wait_warp(&q_full[x & 1], (x >> 1) & 1) && (x < 2 || wait_warp(&s_empty[x & 1], ((x >> 1) - 1) & 1));
            tc_fence_after();
            if (ok && elect_one()) {
                const uint32_t k = smem_u32(base), q = smem_u32(sq + (x & 1) * C::TILE);
#pragma unroll
                for (int s = 0; s < HD / 16; ++s)
                    umma_f16(tmem + (x & 1) * BQ, smem_desc_k128(k + (s >> 2) * BOX) + 2 * (s & 3),
                             smem_desc_k128(q + (s >> 2) * BOX) + 2 * (s & 3), idesc, s > 0);
                umma_commit(&s_full[x & 1]);
                umma_commit(&q_empty[x & 1]);
            }
        }
        if (elect_one()) umma_commit(&drain);  // all products are done before the block ends
        mbar_wait_bounded(&drain, 0, nullptr, landing_limit(p.timeout_ns));
    } else if (warp == EXP_WARPS + 2) {
        // ---- sums of the queries
        for (int x = 0; x < steps; ++x) {
            if (x >= 2 && !wait(&s_empty[x & 1], ((x >> 1) - 1) & 1)) break;
#pragma unroll
            for (int i = 0; i < BQ; i += 32) {
                const int head = head_of(x, i), s = query_of(x, i) + lane;  // (32 columns are of one head)
                neg_lse[x & 1][i + lane] = head < heads && s < n ? -p.lse[(int64_t)(head0 + head) * p.rows + start + s] * LOG2E : 0.0f;
            }
            mbar_arrive(&s_full[x & 1]);  // with the products of this step
        }
    } else {
        // ---- exponentials
        // (a thread's columns are the even or the odd groups of 32, so that few queries occupy both)
        const int half = warp >> 2, t = t0 + (tid & 127);
        const uint32_t S = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 32;
        const uint64_t c2 = two(a.c, a.c);
        uint64_t sum[2] = {two(0.0f, 0.0f), two(0.0f, 0.0f)};
        for (int x = 0; x < steps; ++x) {
            const int at = x & 1;
            if (!wait_warp(&s_full[at], (x >> 1) & 1)) break;
            tc_fence_after();
            const int s0 = query_of(x, half * 32);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int s1 = PACK > 1 ? query_of(x, half * 32 + 64 * h) : s0 + 64 * h;  // queries s1 .. s1 + 31
                if (s1 >= n || (PACK > 1 && head_of(x, half * 32 + 64 * h) >= heads)) continue;
                uint32_t r[32];
                tmem_ld_x32(S + at * BQ + 64 * h, r);
                tmem_wait_ld_regs(r);
                const float* l = &neg_lse[at][half * 32 + 64 * h];
                if (s1 < t0 + BK - 1 || s1 + 32 > n) add_exponentials<true>(r, l, c2, t - s1, n - s1, sum);
                else add_exponentials<false>(r, l, c2, 0, 0, sum);
            }
            tc_fence_before();
            mbar_arrive(&s_empty[at]);
        }
        const float2 u = one_by_one(add2(sum[0], sum[1]));
        part[half][tid & 127] = u.x + u.y;
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == EXP_WARPS + 1) tmem_dealloc(tmem, 2 * BQ);
    if (tid == 0 && dead) status_or(p.status, ENERGON_DEVICE_TIMEOUT);
    if (tid < BK) part[0][tid] += part[1][tid];
    float w = tid < BK ? part[0][tid] : 0.0f;
    bool good = dead == 0;
    if (a.cluster > 1) {
        cluster_sync();
        if (rank == 0 && tid < BK) {
            w = 0.0f;
            for (int r = 0; r < a.cluster; ++r) {
                float y;
                int d;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(y) : "r"(mapa_shared(smem_u32(&part[0][tid]), r)) : "memory");
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(d) : "r"(mapa_shared(smem_u32(&dead), r)) : "memory");
                w += y;
                good = good && d == 0;
            }
        }
        cluster_sync();  // no block leaves while its sums are read
    }
    if (rank == 0 && good && tid < BK && t0 + tid < n) p.weights[(int64_t)kvh * p.rows + start + t0 + tid] = w;
}

template <typename T, int HD, int QW>
static cudaError_t key_weights_tc(const PromptArgs& p, cudaStream_t st) {
    using C = WCfg<HD>;
    CUtensorMap q, k;
    cudaError_t e = rows_map(&q, p.dtype, p.q, (int64_t)p.n_heads * HD, p.rows, p.ld_q, QW);
    if (e == cudaSuccess) e = rows_map(&k, p.dtype, p.k, (int64_t)p.n_kv * HD, p.rows, p.ld_k, BK);
    if (e == cudaSuccess) e = prepare_smem((const void*)key_weights_tc_kernel<T, HD, QW>, C::SMEM);
    if (e != cudaSuccess) return e;
    KeyWeightArgs a;
    a.p = p;
    a.c = p.scale * LOG2E;
    const int group = p.n_heads / p.n_kv;
    a.cluster = 1;
    for (int i = 2; i <= 8 && p.window > 256; ++i)
        if (group % i == 0) a.cluster = i;
    const int64_t most = p.rows / BK + (p.batch < p.rows ? p.batch : p.rows);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(most * a.cluster), p.n_kv), cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM, cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.cluster, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
    cfg.attrs = at, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, key_weights_tc_kernel<T, HD, QW>, q, k, a);
}

template <typename T, int HD>
static cudaError_t key_weights_tc_w(const PromptArgs& p, cudaStream_t st) {
    // heads share a step where the window leaves room: on the last 64 queries of 8 prompts 18.6 us
    // instead of 22.3, on the last 32 14.9
    const bool share = p.n_heads > p.n_kv;
    if (share && p.window <= 32) return key_weights_tc<T, HD, 32>(p, st);
    if (share && p.window <= 64) return key_weights_tc<T, HD, 64>(p, st);
    return key_weights_tc<T, HD, 128>(p, st);
}

cudaError_t launch_key_weights_tc(const PromptArgs& p, cudaStream_t st) {
    if (p.dtype == ENERGON_BF16)
        return p.head_dim == 64 ? key_weights_tc_w<__nv_bfloat16, 64>(p, st) : key_weights_tc_w<__nv_bfloat16, 128>(p, st);
    return p.head_dim == 64 ? key_weights_tc_w<__half, 64>(p, st) : key_weights_tc_w<__half, 128>(p, st);
}

}  // namespace energon
