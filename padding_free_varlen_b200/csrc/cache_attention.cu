// Attention of one new token per sequence over the paged 8-bit cache.
//
//   x_t = c sum_d q_d K(t)_d,  K(t) = code * scale(page, head);  o = sum_t exp(x_t - lse) V(t)
//
// The cache's codes are read once: 2 d bytes per token and kv head, which bounds the call.  The
// query heads of a kv head therefore pass over a token together, on the tensor cores
// (mma m16n8k16, fp16 in, fp32 sums; at most 16 queries meet a tile, so that the wide
// tcgen05 tiles would stand empty, and the codes have to pass the registers anyway to become
// 16-bit numbers).  A code is exact in fp16.  A query row is scaled by a power of two to
// below 2^15: fp16 and bf16 queries are then exact (bf16 elements below 2^-28 of the row's largest
// lose bits below 2^-39 of it), fp32 queries are held as two fp16 terms (2^-22 of the element).
// The scales stay outside the sums over d: one factor per (page, head) for the scores, and the values'
// factor belongs to the probability: p * scale is rounded to fp16 (two terms for fp32 outputs) in a unit of the
// query's own, a power of two that the largest product p * scale met so far reaches 2^5 to 2^15 of.  A unit
// from the scales alone would round away tokens of small scales beside a page of a large scale without weight.
//
// A warp takes 32 tokens at a time: K and V rows land in its own ring of STAGES buffers by
// TMA (the box of a page's tokens, swizzled so that the 16-byte reads of the fragments hit
// different banks), and it keeps its own running maximum, sum and output; the maximum may lag behind
// by 2^GROW, so that the output is seldom rescaled.  The block's warps are joined in shared memory; the
// splits of a long sequence by a second kernel, which also adds the weights from the scores that the
// first one left (they need the sums over all splits).
//
// 64 sequences of 1 to 8192 tokens (261 thousand in all), 64 heads of 128, 8 kv heads, bf16: 104 us without
// weights, 5.2 TB/s (0.79 of the measured copy rate), 134 us with them.  What bounds it: turning
// a step's 8 KB of codes into fp16 takes 350 of the about 650 instructions of a step and warp (3 warps per
// scheduler, 0.58 instructions a cycle); the scores cost 17 us to write and 20 us in the
// second kernel, although they stay in L2.  Tried: four blocks per SM with
// one buffer for V (143 us), splits of 512, 1024 and 4096 tokens (159, 140, 152 us) instead of 2048, queries
// as the rows of the first product (half of a tile empty, 156 us).
#include <cudaTypedefs.h>
#include <math.h>

#include "internal.h"
#include "serving.cuh"

namespace energon {

namespace {
constexpr int STEP = 32;     // tokens a warp takes at a time
constexpr int CW = 4;        // warps per block
constexpr int STAGES = 2;    // buffers per warp
constexpr int BLOCK_STEP = STEP * CW;
constexpr int MAX_SPLITS = 148;
constexpr int SUPER = 32;    // steps whose page entries a warp holds (one per lane)
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float GROW = 8.0f;      // log2 of the growth that a running maximum may lag behind
// Probability times value scale is held in units of 2^(unit - P_UP): at most 2^(P_UP + GROW) of them, the range
// of fp16.  A unit lies in [UNIT_MIN, UNIT_MAX] (it and its reciprocal are normal numbers) and at most 2^UNIT_SPAN
// below the largest scale (scale / unit does not overflow).
constexpr float P_UP = 7.0f, UNIT_MIN = -119.0f, UNIT_MAX = 133.0f, UNIT_SPAN = 112.0f;

template <int HD>
struct DCfg {
    static constexpr int TILE = STEP * HD;  // bytes of K, and of V, per buffer
    static constexpr int WARP = STAGES * 2 * TILE;
    static constexpr int SMEM = CW * WARP + 1024;
};

// What a call keeps between its launches: per split a maximum and sum, with more than one split an
// unnormalised output; the scores (accumulate only).
struct AttnWs {
    float2* ml;     // [batch][heads][splits]
    float* part;    // [batch][heads][splits][d]
    float* scores;  // [batch][kv heads][stride][group], in units of log2
    int stride, splits, chunk, group;  // group: query heads per kv head
    size_t bytes;
};
inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
AttnWs attn_ws(void* ws, int batch, int max_len, int n_heads, int n_kv, int head_dim, int accumulate) {
    AttnWs w;
    const int64_t rows = (int64_t)batch * n_heads;
    const int tiles = cdiv(n_heads / n_kv, 16);
    // Enough blocks for two per SM where the lengths give them: a split is at least one step of
    // every warp, and at most MAX_SPLITS are joined.
    const int64_t blocks = (int64_t)batch * n_kv * tiles;
    int64_t want = blocks > 0 ? cdiv(2 * 148, blocks) : 1;
    // tokens per split are bounded too: with many sequences of different lengths short splits even out the SMs
    const int64_t fine = cdiv(max_len, 2048);
    if (want < fine) want = fine < 64 ? fine : 64;
    if (want > MAX_SPLITS) want = MAX_SPLITS;
    w.chunk = cdiv(cdiv(max_len > 0 ? max_len : 1, want), BLOCK_STEP) * BLOCK_STEP;
    w.splits = cdiv(max_len > 0 ? max_len : 1, w.chunk);
    w.stride = cdiv(max_len, 16) * 16;
    w.group = n_heads / n_kv;
    size_t at = 0;
    char* base = static_cast<char*>(ws);
    auto take = [&](size_t n) {
        char* p = base + at;
        at += (n + 255) / 256 * 256;
        return p;
    };
    const size_t parts = w.splits > 1 ? (size_t)rows * w.splits : 0;
    w.ml = reinterpret_cast<float2*>(take((size_t)rows * w.splits * sizeof(float2)));
    w.part = reinterpret_cast<float*>(take(parts * head_dim * sizeof(float)));
    w.scores = reinterpret_cast<float*>(take(accumulate ? (size_t)rows * w.stride * sizeof(float) : 0));
    w.bytes = at;
    return w;
}
__device__ __forceinline__ int cached_len(const CacheArgs& c, int b, bool& bad) {
    const int n = c.lens[b];
    bad = n < 0 || n > c.max_len || (int64_t)n > (int64_t)c.max_pages * c.page_len;
    return bad ? 0 : n;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with a zero sum before it.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// An 8 x 8 matrix of 16-bit elements (lane 4 g + c: row g, columns 2c and 2c + 1) transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// Two biased codes (bytes LO and HI of w, each code + 128) as a pair of fp16: 0x6400 | byte is
// 1024 + byte, less 1152.
template <int LO, int HI>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
    const uint32_t x = __byte_perm(w, 0x64646464u, LO | 0x40 | (HI << 8) | 0x4000);
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), bias);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^k for -126 <= k <= 127.
__device__ __forceinline__ float power_of_two(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }
// The same of a float that holds a whole number (the low bits of 1.5 * 2^23 + 127 + k are those of 127 + k).
__device__ __forceinline__ float power_of_two(float k) { return __uint_as_float(__float_as_uint(12582912.0f + 127.0f + k) << 23); }
// The smallest whole number l with |x| < 2^l (-126 below the normal range, 129 for infinity and NaN).
__device__ __forceinline__ float log2_above(float x) { return (float)(int)(__float_as_uint(x) << 1 >> 24) - 126.0f; }
__device__ __forceinline__ uint32_t pair_f16(float a, float b) { return pack2<__half>(a, b); }
// What fp16 leaves of a pair.
__device__ __forceinline__ uint32_t rest_f16(float a, float b, uint32_t hi) {
    const float2 h = unpack2<__half>(hi);
    return pack2<__half>(a - h.x, b - h.y);
}
// The codes stream through L2 without displacing the scores, which are read again.
__device__ __forceinline__ uint64_t streaming() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}
// Elements [0, N) of a row at p as floats.
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* p, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N * (int)sizeof(T) / 16; ++i) {
        const uint4 w = reinterpret_cast<const uint4*>(p)[i];
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) {
                x[4 * i + j] = __uint_as_float(u[j]);
            } else {
                const float2 f = unpack2<T>(u[j]);
                x[8 * i + 2 * j] = f.x, x[8 * i + 2 * j + 1] = f.y;
            }
        }
    }
}
}  // namespace

struct SplitArgs {
    AttnWs ws;
    int q_tiles;
    uint64_t timeout_ns;
};

// One block = one split of one sequence, for up to QT query heads of one kv head.  Fragment
// layout of a warp's lane (g = lane / 4, c = lane % 4): scores have tokens g, g + 8 of each 16 as
// rows and queries 2c, 2c + 1 (+ 8 r) as columns; the contraction over d takes the elements of lane
// c from its own d / 4 consecutive ones, for queries and keys alike.  The output is held transposed,
// rows d = (d / 8) g + j, columns queries 2c, 2c + 1: the lane that holds a query's maximum and sum
// also holds its outputs, and the probabilities become the second product's operand by
// transposing 8 x 8 blocks.
template <typename T, int HD, int QT>
__global__ void __launch_bounds__(CW * 32, QT == 8 && sizeof(T) == 2 ? 3 : 2) cache_attn_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                             const __grid_constant__ CUtensorMap tm_v,
                                                             const CacheAttnArgs a, const SplitArgs sp) {
    using C = DCfg<HD>;
    constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;
    constexpr int R = QT / 8;          // query rows per lane
    constexpr int KS = HD / 16;        // mma steps over d
    constexpr int ND = HD / 8;         // outputs of a query per lane
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[CW][STAGES];
    __shared__ float sh_m[CW][QT], sh_l[CW][QT];
    const CacheArgs& c = a.c;
    if (block_stopped(c.status)) return;
    let_next_grid_start();
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cc = lane & 3;
    const int split = blockIdx.z, b = blockIdx.y, P = c.page_len;
    const int kvh = blockIdx.x / sp.q_tiles, qt = blockIdx.x % sp.q_tiles, group = a.n_heads / c.n_kv;
    const int head0 = kvh * group + qt * QT, n_q = min(QT, group - qt * QT);
    bool bad;
    const int n = cached_len(c, b, bad);
    if (bad && split == 0 && blockIdx.x == 0 && tid == 0) status_or(c.status, ENERGON_DEVICE_BAD_LENGTH);
    const int t_begin = split * sp.ws.chunk, t_end = min(n, t_begin + sp.ws.chunk);
    if (split > 0 && t_begin >= n) return;

    if (lane == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(&bars[warp][s], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    __syncwarp();

    // this lane's part of the queries
    uint32_t qf[TERMS][KS][R][2];
    float qs[R][2];  // of queries 8 r + 2c, + 1
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float x[HD / 4], most = 0.0f;
        const bool have = g + 8 * r < n_q;
        if (have) {
            load_row<T, HD / 4>(static_cast<const T*>(a.q) + b * a.ld_q + (int64_t)(head0 + g + 8 * r) * HD + cc * (HD / 4), x);
        } else {
#pragma unroll
            for (int i = 0; i < HD / 4; ++i) x[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < HD / 4; ++i) most = fmaxf(most, fabsf(x[i]));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // most < 2^e; what lies below the normal range is held to 2^-149
        const int e = most > 0.0f ? max((int)(__float_as_uint(most) >> 23), 1) - 126 : 0;
        const float q_unit = ldexpf(a.scale * LOG2E, e - 15);
        qs[r][0] = __shfl_sync(0xffffffffu, q_unit, 8 * cc), qs[r][1] = __shfl_sync(0xffffffffu, q_unit, 8 * cc + 4);
        // 2^(15 - e) in two factors: alone it may lie outside the range of fp32.  An infinite element makes all
        // scores infinite or NaN; the softmax of such a row is NaN, also where all of them are -infinity.
        const float up0 = most < INFINITY ? power_of_two((15 - e) / 2) : NAN, up1 = power_of_two(15 - e - (15 - e) / 2);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float u = x[4 * s + 2 * h] * up0 * up1, v = x[4 * s + 2 * h + 1] * up0 * up1;
                qf[0][s][r][h] = pair_f16(u, v);
                if constexpr (TERMS == 2) qf[1][s][r][h] = rest_f16(u, v, qf[0][s][r][h]);
            }
    }

    // Exponentials refer to m and the outputs to m + unit (in log2); both are whole, so that rescaling is exact.
    float m[R][2], l[R][2], unit[R][2], acc[R][ND / 2][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r][0] = m[r][1] = -INFINITY, l[r][0] = l[r][1] = 0.0f, unit[r][0] = unit[r][1] = UNIT_MIN;
#pragma unroll
        for (int i = 0; i < ND / 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[r][i][e] = 0.0f;
    }
    // scores are kept as [token][query of the group]; this lane's place for its sequence's token g
    float* const scores = sp.ws.scores + (((int64_t)b * c.n_kv + kvh) * sp.ws.stride + g) * sp.ws.group + qt * QT + 2 * cc;
    const int log_p = __ffs(P) - 1;
    float lowest = UNIT_MIN;  // the least unit that the scales met so far allow
    bool ok = true;
    uint8_t* mine = ring + warp * C::WARP;
    const uint64_t policy = streaming();
    // Where this lane's pieces begin in a buffer: keys of token g (16-byte pieces 2c and 2c + 1, or c), values
    // of tokens 2c and 2c + 1 (piece g, or half of piece g / 2).  The swizzle repeats after 8 rows.
    const int k_at[2] = {g * HD + ((HD == 128 ? (2 * cc) ^ g : cc ^ ((g >> 1) & 3)) << 4), g * HD + (((2 * cc + 1) ^ g) << 4)};
    int v_at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = 2 * cc + h;
        v_at[h] = C::TILE + row * HD + (HD == 128 ? (g ^ row) << 4 : (((g >> 1) ^ ((row >> 1) & 3)) << 4) + 8 * (g & 1));
    }
    const int total = max(0, (t_end - t_begin + STEP - 1) / STEP);
    const int steps = total > warp ? (total - warp + CW - 1) / CW : 0;  // of this warp
    int used = 0;  // buffers filled so far: buffer used % STAGES, parity used / STAGES
    for (int s0 = 0; s0 < steps; s0 += SUPER) {
        // lane i: pages and scales of step s0 + i (two pages where they have 16 tokens)
        const int now = min(SUPER, steps - s0);
        int tile[2] = {-1, -1};  // page * heads + head
        float ks[2] = {0.0f, 0.0f}, vs[2] = {0.0f, 0.0f};
        if (lane < now) {
            const int t = t_begin + ((s0 + lane) * CW + warp) * STEP;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (t + 16 * h >= t_end) break;
                const int p = c.table[(int64_t)b * c.max_pages + ((t + 16 * h) >> log_p)];
                if ((unsigned)p < (unsigned)c.n_pages) {
                    tile[h] = p * c.n_kv + kvh;
                    ks[h] = c.k_scale[(int64_t)p * c.n_kv + kvh];
                    vs[h] = c.v_scale[(int64_t)p * c.n_kv + kvh];
                } else {
                    status_or(c.status, ENERGON_DEVICE_BAD_PAGE);
                }
            }
        }
        const float v_top = warp_max(fmaxf(log2_above(vs[0]), log2_above(vs[1])));
        if (v_top - UNIT_SPAN > lowest) {
            lowest = v_top - UNIT_SPAN;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float by = exp2_fast(fminf(unit[r][e] - lowest, 0.0f));
                    unit[r][e] = fmaxf(unit[r][e], lowest);
#pragma unroll
                    for (int y = 0; y < ND / 2; ++y) acc[r][y][e] *= by, acc[r][y][2 + e] *= by;
                }
        }

        auto fetch = [&](int i) {
            const int p0 = __shfl_sync(0xffffffffu, tile[0], i), p1 = __shfl_sync(0xffffffffu, tile[1], i);
            const int at = (used + i) % STAGES;
            if (lane == 0) {
                const int t = t_begin + ((s0 + i) * CW + warp) * STEP;
                uint64_t* bar = &bars[warp][at];
                uint8_t* k = mine + at * 2 * C::TILE;
                uint8_t* v = k + C::TILE;
                if (P == 16) {
                    const int live = (p0 >= 0) + (p1 >= 0);
                    if (live) mbar_arrive_expect_tx(bar, live * C::TILE);
                    else mbar_arrive(bar);
                    if (p0 >= 0) {
                        tma_load_3d(k, &tm_k, bar, 0, 0, p0, policy);
                        tma_load_3d(v, &tm_v, bar, 0, 0, p0, policy);
                    }
                    if (p1 >= 0) {
                        tma_load_3d(k + C::TILE / 2, &tm_k, bar, 0, 0, p1, policy);
                        tma_load_3d(v + C::TILE / 2, &tm_v, bar, 0, 0, p1, policy);
                    }
                } else if (p0 >= 0) {
                    mbar_arrive_expect_tx(bar, 2 * C::TILE);
                    tma_load_3d(k, &tm_k, bar, 0, t & (P - 1), p0, policy);
                    tma_load_3d(v, &tm_v, bar, 0, t & (P - 1), p0, policy);
                } else {
                    mbar_arrive(bar);
                }
            }
        };
        for (int i = 0; i < min(STAGES, now); ++i) fetch(i);
        for (int i = 0; i < now; ++i) {
            const int at = (used + i) % STAGES;
            if (ok) ok = mbar_wait_bounded(&bars[warp][at], ((used + i) / STAGES) & 1, nullptr, sp.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                // let the copies that are still in flight land before the block may end
                for (int j = i; j < min(i + STAGES, now); ++j)
                    mbar_wait_bounded(&bars[warp][(used + j) % STAGES], ((used + j) / STAGES) & 1, nullptr,
                                      landing_limit(sp.timeout_ns));
                break;
            }
            const uint8_t* buf = mine + at * 2 * C::TILE;
            const uint8_t *const k0 = buf + k_at[0], *const k1 = buf + k_at[1], *const v0 = buf + v_at[0], *const v1 = buf + v_at[1];
            const int t0 = t_begin + ((s0 + i) * CW + warp) * STEP;

            float x[2][R][4];  // [16 tokens][queries 8 r ..][token g: queries 2c, 2c + 1; token g + 8: the same]
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t w[2][KS];  // this lane's codes of tokens g, g + 8
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    *reinterpret_cast<uint4*>(&w[j][0]) = *reinterpret_cast<const uint4*>(k0 + (16 * u + 8 * j) * HD);
                    if constexpr (HD == 128) *reinterpret_cast<uint4*>(&w[j][4]) = *reinterpret_cast<const uint4*>(k1 + (16 * u + 8 * j) * HD);
                }
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const uint32_t y0 = w[0][s] ^ 0x80808080u, y1 = w[1][s] ^ 0x80808080u;
                    const uint32_t a0 = codes_f16<0, 1>(y0), a1 = codes_f16<0, 1>(y1), a2 = codes_f16<2, 3>(y0), a3 = codes_f16<2, 3>(y1);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int y = 0; y < TERMS; ++y)
                            if (s == 0 && y == 0) mma_f16_first(x[u][r], a0, a1, a2, a3, qf[y][s][r][0], qf[y][s][r][1]);
                            else mma_f16(x[u][r], a0, a1, a2, a3, qf[y][s][r][0], qf[y][s][r][1]);
                }
            }

            // scores in units of log2, masked; the maxima that the exponentials refer to
            const int p0 = __shfl_sync(0xffffffffu, tile[0], i), p1 = __shfl_sync(0xffffffffu, tile[1], i);
            const float ks0 = __shfl_sync(0xffffffffu, ks[0], i), ks1 = __shfl_sync(0xffffffffu, ks[1], i);
            const float vs0 = __shfl_sync(0xffffffffu, vs[0], i), vs1 = __shfl_sync(0xffffffffu, vs[1], i);
            const bool whole = t0 + STEP <= t_end && p0 >= 0 && p1 >= 0;
            bool grown = false;  // beyond what the maximum, or the unit, may lag behind
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[u][r][e] *= (u ? ks1 : ks0) * qs[r][e & 1];
            }
            if (!whole) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if ((u ? p1 : p0) < 0 || t0 + 16 * u + 8 * h + g >= t_end) {
#pragma unroll
                            for (int r = 0; r < R; ++r) x[u][r][2 * h] = x[u][r][2 * h + 1] = -INFINITY;
                        }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    grown |= max3(fmaxf(x[0][r][e], x[0][r][2 + e]), x[1][r][e], x[1][r][2 + e]) - m[r][e] >
                             fminf(GROW, unit[r][e] + (GROW - v_top));
            }
            if (a.accumulate) {
                float* to = scores + (int64_t)t0 * sp.ws.group;
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!whole && t0 + 16 * u + 8 * h + g >= t_end) continue;
                            float* y = to + (16 * u + 8 * h) * sp.ws.group + 8 * r;
                            const int q = 8 * r + 2 * cc;  // an even group keeps pairs aligned
                            if (q + 1 < n_q && (sp.ws.group & 1) == 0) {
                                *reinterpret_cast<float2*>(y) = make_float2(x[u][r][2 * h], x[u][r][2 * h + 1]);
                            } else {
                                if (q < n_q) y[0] = x[u][r][2 * h];
                                if (q + 1 < n_q) y[1] = x[u][r][2 * h + 1];
                            }
                        }
            }
            if (__any_sync(0xffffffffu, grown)) {
                const float v0 = log2_above(vs0), v1 = log2_above(vs1);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x0 = fmaxf(x[0][r][e], x[0][r][2 + e]), x1 = fmaxf(x[1][r][e], x[1][r][2 + e]);
                        float mx = fmaxf(x0, x1);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const bool up = mx - m[r][e] > GROW;
                        const float top = up ? ceilf(mx) : m[r][e], ref = top == -INFINITY ? 0.0f : top;
                        float most = fmaxf(x0 - ref + v0, x1 - ref + v1);  // log2 of probability times scale
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                        const float now = up ? unit[r][e] + (m[r][e] - top) : unit[r][e];  // the same unit, from the new maximum
                        const float next = fminf(fmaxf(most - now > GROW ? ceilf(most) : now, lowest), UNIT_MAX);
                        if (up || next != now) {
                            const float by = exp2_fast(now - next);
                            if (up) l[r][e] *= exp2_fast(m[r][e] - top);
                            m[r][e] = top, unit[r][e] = next;
#pragma unroll
                            for (int y = 0; y < ND / 2; ++y) acc[r][y][e] *= by, acc[r][y][2 + e] *= by;
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float vf = u ? vs1 : vs0;
                uint32_t pf[TERMS][R][2];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float ms0 = m[r][0] == -INFINITY ? 0.0f : m[r][0], ms1 = m[r][1] == -INFINITY ? 0.0f : m[r][1];
                    const float f0 = vf * power_of_two(P_UP - unit[r][0]), f1 = vf * power_of_two(P_UP - unit[r][1]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float e0 = exp2_fast(x[u][r][2 * h] - ms0), e1 = exp2_fast(x[u][r][2 * h + 1] - ms1);
                        l[r][0] += e0, l[r][1] += e1;
                        const uint32_t hi = pair_f16(e0 * f0, e1 * f1);
                        pf[0][r][h] = transposed(hi);
                        if constexpr (TERMS == 2) pf[1][r][h] = transposed(rest_f16(e0 * f0, e1 * f1, hi));
                    }
                }
                uint32_t w[4][ND / 4];  // [tokens 2c, 2c + 1, 2c + 8, 2c + 9][this lane's d / 8 codes]
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint8_t* from = (h & 1 ? v1 : v0) + (16 * u + 8 * (h >> 1)) * HD;
                    if constexpr (HD == 128) *reinterpret_cast<uint4*>(&w[h][0]) = *reinterpret_cast<const uint4*>(from);
                    else *reinterpret_cast<uint2*>(&w[h][0]) = *reinterpret_cast<const uint2*>(from);
#pragma unroll
                    for (int y = 0; y < ND / 4; ++y) w[h][y] ^= 0x80808080u;
                }
#pragma unroll
                for (int y = 0; y < ND / 4; ++y)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t ab = __byte_perm(w[0][y], w[1][y], half ? 0x7362 : 0x5140);
                        const uint32_t cd = __byte_perm(w[2][y], w[3][y], half ? 0x7362 : 0x5140);
                        const uint32_t a0 = codes_f16<0, 1>(ab), a1 = codes_f16<2, 3>(ab);
                        const uint32_t a2 = codes_f16<0, 1>(cd), a3 = codes_f16<2, 3>(cd);
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int z = 0; z < TERMS; ++z)
                                mma_f16(acc[r][2 * y + half], a0, a1, a2, a3, pf[z][r][0], pf[z][r][1]);
                    }
            }
            __syncwarp();  // every lane has read the buffer
            if (i + STAGES < now) fetch(i + STAGES);
        }
        used += now;
        if (!ok) break;
    }
    if (!ok && lane == 0) status_or(c.status, ENERGON_DEVICE_TIMEOUT);

    // ---- the block's warps joined: o[w][query][d] in the ring, relative to the common maximum
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], o);
            if (g == 0) sh_m[warp][8 * r + 2 * cc + e] = m[r][e], sh_l[warp][8 * r + 2 * cc + e] = l[r][e];
        }
    if (!__syncthreads_and(ok)) return;
    constexpr int LD = HD + 4;
    float* out = reinterpret_cast<float*>(ring);
    static_assert(CW * QT * LD * 4 <= CW * C::WARP, "the joined outputs fit in the ring");
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int q = 2 * cc + e + 8 * r;
            float top = sh_m[0][q];
#pragma unroll
            for (int w = 1; w < CW; ++w) top = fmaxf(top, sh_m[w][q]);
            const float mw = sh_m[warp][q];
            const float f = mw == -INFINITY ? 0.0f : exp2_fast(mw - top) * power_of_two(unit[r][e] - P_UP);
            float* to = out + (warp * QT + q) * LD + ND * g;
#pragma unroll
            for (int y = 0; y < ND / 4; ++y)
                *reinterpret_cast<float4*>(to + 4 * y) = make_float4(acc[r][2 * y][e] * f, acc[r][2 * y][2 + e] * f,
                                                                     acc[r][2 * y + 1][e] * f, acc[r][2 * y + 1][2 + e] * f);
        }
    __syncthreads();
    for (int i = tid; i < n_q * (HD / 4); i += CW * 32) {
        const int q = i / (HD / 4), d = i % (HD / 4) * 4;
        float top = sh_m[0][q], sum = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 1; w < CW; ++w) top = fmaxf(top, sh_m[w][q]);
#pragma unroll
        for (int w = 0; w < CW; ++w) {
            const float mw = sh_m[w][q];
            // where no maximum was met the sum is 0, or NaN: a NaN score counts in no maximum
            sum += mw == -INFINITY ? sh_l[w][q] : sh_l[w][q] * exp2_fast(mw - top);
            const float4 y = *reinterpret_cast<const float4*>(out + (w * QT + q) * LD + d);
            o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
        }
        const int64_t row = (int64_t)b * a.n_heads + head0 + q;
        if (d == 0) sp.ws.ml[row * sp.ws.splits + split] = make_float2(top, sum);
        if (sp.ws.splits > 1) {
            *reinterpret_cast<float4*>(sp.ws.part + (row * sp.ws.splits + split) * HD + d) = o;
        } else {
            T* to = static_cast<T*>(a.o) + b * a.ld_o + (int64_t)(head0 + q) * HD + d;
            const float y[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) to[e] = from_f<T>(sum == 0.0f ? 0.0f : y[e] / sum);
            if (d == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : top * LN2 + logf(sum);
        }
    }
}

// What remains when the splits are done, per (sequence, kv head).  With more than one split the first
// blocks join the outputs of `per_block` query heads each, 8 / per_block warps to a head; the others
// add the probabilities of FIN_TOKENS tokens to their weights,
//     weight(t) += sum over the heads of the group of exp2(score - lse).
constexpr int FIN = 256, FIN_TOKENS = 2048;
struct FinishArgs {
    CacheAttnArgs a;
    AttnWs ws;
    int joins, per_block;
};
// Maximum and sum (relative to it) of a query head over its splits; weights of the splits to f.
__device__ __forceinline__ float2 join_sums(const AttnWs& ws, int64_t row, int live, float* f) {
    const int lane = threadIdx.x & 31;
    float top = -INFINITY, l = 0.0f;
    for (int s = lane; s < live; s += 32) top = fmaxf(top, ws.ml[row * ws.splits + s].x);
    top = warp_max(top);
    for (int s = lane; s < live; s += 32) {
        const float2 ml = ws.ml[row * ws.splits + s];
        const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - top);
        if (f) f[s] = w;
        l += ml.x == -INFINITY ? ml.y : ml.y * w;  // (0, or NaN)
    }
    return make_float2(top, warp_sum(l));
}
template <typename T, int HD>
__global__ void __launch_bounds__(FIN) cache_finish_kernel(const FinishArgs fa) {
    const CacheAttnArgs& a = fa.a;
    const AttnWs& ws = fa.ws;
    const CacheArgs& c = a.c;
    wait_for_earlier_grid();
    if (block_stopped(c.status)) return;
    const int b = blockIdx.z, kvh = blockIdx.y, group = ws.group, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad;
    const int n = cached_len(c, b, bad);
    const int live = max(1, (n + ws.chunk - 1) / ws.chunk);
    const int64_t row0 = (int64_t)b * a.n_heads + kvh * group;
    if ((int)blockIdx.x < fa.joins) {
        constexpr int E = HD / 32;
        __shared__ float f[FIN / 32][MAX_SPLITS], sums[FIN / 32][HD];
        const int warps = FIN / 32 / fa.per_block, sub = warp % warps;
        const int h = blockIdx.x * fa.per_block + warp / warps;
        const int64_t row = row0 + h;
        float2 ml = make_float2(0.0f, 0.0f);
        if (h < group) {
            ml = join_sums(ws, row, live, f[warp]);
            __syncwarp();
            const float* part = ws.part + row * ws.splits * HD + lane * E;
            float o[E] = {};
#pragma unroll 4
            for (int s = sub; s < live; s += warps) {
                const float w = f[warp][s];
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] += part[(int64_t)s * HD + e] * w;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = o[e];
        }
        __syncthreads();
        if (h < group && sub == 0) {
            T* to = static_cast<T*>(a.o) + b * a.ld_o + (int64_t)(kvh * group + h) * HD;
            for (int d = lane; d < HD; d += 32) {
                float y = 0.0f;
                for (int w = 0; w < warps; ++w) y += sums[warp + w][d];
                to[d] = from_f<T>(ml.y == 0.0f ? 0.0f : y / ml.y);
            }
            if (lane == 0 && a.lse) a.lse[row] = ml.y == 0.0f ? -INFINITY : ml.x * LN2 + logf(ml.y);
        }
        return;
    }
    const int t0 = ((int)blockIdx.x - fa.joins) * FIN_TOKENS;
    if (t0 >= n) return;
    const int end = min(n, t0 + FIN_TOKENS), log_p = __ffs(c.page_len) - 1;
    __shared__ float lse2[32];
    for (int h0 = 0; h0 < group; h0 += 32) {
        const int some = min(32, group - h0);
        if (h0 > 0) __syncthreads();
        for (int h = warp; h < some; h += FIN / 32) {
            const float2 ml = join_sums(ws, row0 + h0 + h, live, nullptr);
            if (lane == 0) lse2[h] = ml.x + log2f(ml.y);
        }
        __syncthreads();
        const float* x = ws.scores + ((int64_t)b * c.n_kv + kvh) * ws.stride * group + h0;
        constexpr int K = 4;  // tokens of a thread at a time: their loads are on their way together
        for (int t = t0 + tid; t < end; t += K * FIN) {
            int page[K];
            float sum[K] = {};
#pragma unroll
            for (int k = 0; k < K; ++k) page[k] = t + k * FIN < end ? c.table[(int64_t)b * c.max_pages + ((t + k * FIN) >> log_p)] : -1;
            if (group % 4 == 0) {  // 16-byte aligned: h0 and the group are multiples of 4
#pragma unroll 2
                for (int h = 0; h < some; h += 4) {
                    float4 z[K];
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        z[k] = t + k * FIN < end ? *reinterpret_cast<const float4*>(x + (int64_t)(t + k * FIN) * group + h) : make_float4(0, 0, 0, 0);
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        sum[k] += exp2_fast(z[k].x - lse2[h]) + exp2_fast(z[k].y - lse2[h + 1]) + exp2_fast(z[k].z - lse2[h + 2]) + exp2_fast(z[k].w - lse2[h + 3]);
                }
            } else {
                for (int h = 0; h < some; ++h)
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (t + k * FIN < end) sum[k] += exp2_fast(x[(int64_t)(t + k * FIN) * group + h] - lse2[h]);
            }
            // a page named once has one writer per call; sequences that share a page add in any order
#pragma unroll
            for (int k = 0; k < K; ++k)
                if ((unsigned)page[k] < (unsigned)c.n_pages)
                    atomicAdd(c.weight + ((int64_t)page[k] * c.n_kv + kvh) * c.page_len + ((t + k * FIN) & (c.page_len - 1)), sum[k]);
        }
    }
}

size_t cache_attention_ws_bytes(int batch, int max_len, int n_heads, int n_kv, int head_dim, bool accumulate) {
    return attn_ws(nullptr, batch, max_len, n_heads, n_kv, head_dim, accumulate).bytes;
}

// The codes as a [pages * heads][page_len][d] tensor of bytes, boxes of up to 32 tokens.
static cudaError_t codes_map(CUtensorMap* m, const CacheArgs& c, const int8_t* codes) {
    const auto encode = tensor_map_encoder();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_len, (cuuint64_t)c.n_pages * c.n_kv};
    const cuuint64_t strides[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.head_dim * c.page_len};
    const cuuint32_t box[3] = {(cuuint32_t)c.head_dim, (cuuint32_t)(c.page_len < STEP ? c.page_len : STEP), 1};
    const cuuint32_t one[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(codes), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <typename T, int HD, int QT>
static cudaError_t cache_attn(const CacheAttnArgs& a, cudaStream_t st) {
    CUtensorMap tm_k, tm_v;
    cudaError_t e = codes_map(&tm_k, a.c, a.c.k_codes);
    if (e == cudaSuccess) e = codes_map(&tm_v, a.c, a.c.v_codes);
    if (e == cudaSuccess) e = prepare_smem((const void*)cache_attn_kernel<T, HD, QT>, DCfg<HD>::SMEM);
    if (e != cudaSuccess) return e;
    SplitArgs sp;
    sp.ws = attn_ws(a.ws, a.c.batch, a.c.max_len, a.n_heads, a.c.n_kv, HD, a.accumulate);
    sp.q_tiles = cdiv(a.n_heads / a.c.n_kv, QT);
    sp.timeout_ns = a.timeout_ns;
    const dim3 grid(a.c.n_kv * sp.q_tiles, a.c.batch, sp.ws.splits);
    cache_attn_kernel<T, HD, QT><<<grid, CW * 32, DCfg<HD>::SMEM, st>>>(tm_k, tm_v, a, sp);
    e = cudaGetLastError();
    FinishArgs f;
    f.a = a, f.ws = sp.ws;
    // few heads: all warps of a block to each; many: a warp each, which has fewer blocks to start
    f.per_block = (int64_t)a.c.batch * a.n_heads <= 4 * 148 ? 1 : FIN / 32;
    f.joins = sp.ws.splits > 1 ? cdiv(sp.ws.group, f.per_block) : 0;
    const int blocks = f.joins + (a.accumulate ? cdiv(a.c.max_len, FIN_TOKENS) : 0);
    if (e == cudaSuccess && blocks > 0)
        e = launch_early(cache_finish_kernel<T, HD>, dim3(blocks, a.c.n_kv, a.c.batch), FIN, st, f);
    return e;
}

template <typename T>
static cudaError_t cache_attn_t(const CacheAttnArgs& a, cudaStream_t st) {
    const bool wide = a.n_heads / a.c.n_kv > 8;  // more than 8 queries per kv head: 16 of them meet a tile
    if (a.c.head_dim == 64) return wide ? cache_attn<T, 64, 16>(a, st) : cache_attn<T, 64, 8>(a, st);
    return wide ? cache_attn<T, 128, 16>(a, st) : cache_attn<T, 128, 8>(a, st);
}

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t st) {
    if (a.c.batch <= 0) return cudaSuccess;
    switch (a.dtype) {
    case ENERGON_F32: return cache_attn_t<float>(a, st);
    case ENERGON_F16: return cache_attn_t<__half>(a, st);
    case ENERGON_BF16: return cache_attn_t<__nv_bfloat16>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace energon
