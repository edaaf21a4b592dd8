// Causal attention of packed prompts with grouped heads, and the attention weight their keys
// receive, on CUDA cores: the fp32 path (the 16-bit types run on the tensor cores).
//
//   o_j(s) = sum_{t <= s} exp(c q_j(s) . k(t) - lse_j(s)) v(t),  lse_j(s) = log sum_{t <= s} exp(c q . k)
//   w_h(t) = sum_{j in group h} sum_{s >= t, s in window} exp(c q_j(s) . k_h(t) - lse_j(s))
//
// Both multiply 64 x 64 tiles: 256 threads, each 4 x 4 scores (rows 4 ty + i, columns tx + 16 j)
// from shared memory with 16-byte loads, so that 8 loads feed 64 multiply-adds.  Rows of a tile
// are padded by 4 floats: the 16 columns' loads then fall into different banks.
#include <math.h>

#include "internal.h"
#include "serving.cuh"

namespace energon {

namespace {
constexpr int PT = 64;  // tile edge: queries and keys

template <int HD>
struct PCfg {
    static constexpr int LD = HD + 4;  // floats per row of a Q or K tile
    static constexpr int LP = PT + 4;  // floats per row of the probabilities
    static constexpr int SMEM = (2 * PT * LD + PT * HD + PT * LP) * (int)sizeof(float);
    static constexpr int SMEM_W = 2 * PT * LD * (int)sizeof(float);
};

// Rows row0 .. of a packed tensor (head offset applied) to a [64][ld] tile of floats times
// `mul`; rows from `rows` on become 0.
template <int HD>
__device__ __forceinline__ void load_tile(float* dst, int ld, const float* __restrict__ src, int64_t ld_src, int rows,
                                          float mul) {
    constexpr int PIECES = HD / 4, PER = PT * PIECES / 256;  // 16-byte pieces of a row, and per thread
    float4 x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x + i * 256, r = e / PIECES;
        x[i] = r < rows ? *reinterpret_cast<const float4*>(src + r * ld_src + e % PIECES * 4) : make_float4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x + i * 256;
        *reinterpret_cast<float4*>(dst + e / PIECES * ld + e % PIECES * 4) = make_float4(x[i].x * mul, x[i].y * mul, x[i].z * mul, x[i].w * mul);
    }
}

// x[i][j] = Q row (4 ty + i) . K row (tx + 16 j)
template <int HD>
__device__ __forceinline__ void tile_scores(const float* Q, const float* K, int ty, int tx, float (&x)[4][4]) {
    constexpr int LD = PCfg<HD>::LD;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0.0f;
#pragma unroll 4
    for (int d = 0; d < HD; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(Q + (4 * ty + i) * LD + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(K + (tx + 16 * j) * LD + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = fmaf(a[i].x, b[j].x, x[i][j]);
                x[i][j] = fmaf(a[i].y, b[j].y, x[i][j]);
                x[i][j] = fmaf(a[i].z, b[j].z, x[i][j]);
                x[i][j] = fmaf(a[i].w, b[j].w, x[i][j]);
            }
    }
}

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
}  // namespace

// One block = 64 queries of one (sequence, head).  Scores are kept times log2(e), so that
// the exponentials are exp2.
template <int HD>
__global__ void __launch_bounds__(256) prompt_simt_kernel(const PromptArgs p) {
    using C = PCfg<HD>;
    extern __shared__ float sm[];
    float *Q = sm, *K = Q + PT * C::LD, *V = K + PT * C::LD, *P = V + PT * HD;
    if (block_stopped(p.status)) return;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) check_rows(p.cu, p.batch, p.rows, p.status);
    int b, blk, start, n;
    auto count = [](int, int len) { return (len + PT - 1) / PT; };
    if (!find_item(p.cu, p.batch, p.rows, blockIdx.x, count, b, blk)) return;
    seq_rows(p.cu, b, p.rows, start, n);
    const int head = blockIdx.y, kvh = head / (p.n_heads / p.n_kv), q0 = blk * PT;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const float* q = static_cast<const float*>(p.q) + (int64_t)(start + q0) * p.ld_q + (int64_t)head * HD;
    const float* k = static_cast<const float*>(p.k) + (int64_t)start * p.ld_k + (int64_t)kvh * HD;
    const float* v = static_cast<const float*>(p.v) + (int64_t)start * p.ld_v + (int64_t)kvh * HD;
    load_tile<HD>(Q, C::LD, q, p.ld_q, n - q0, p.scale * LOG2E);

    float m[4], l[4], acc[4][HD / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) acc[i][c] = 0.0f;
    }
    const int k_end = min(n, q0 + PT);
    for (int k0 = 0; k0 < k_end; k0 += PT) {
        __syncthreads();
        load_tile<HD>(K, C::LD, k + (int64_t)k0 * p.ld_k, p.ld_k, n - k0, 1.0f);
        load_tile<HD>(V, HD, v + (int64_t)k0 * p.ld_v, p.ld_v, n - k0, 1.0f);
        __syncthreads();
        if (q0 + (ty & ~1) * 4 >= n) continue;  // none of this warp's 8 queries is there
        float x[4][4];
        tile_scores<HD>(Q, K, ty, tx, x);
        const bool diag = k0 == q0;  // the only tile with keys after a query
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = 4 * ty + i;
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (diag && tx + 16 * j > s) x[i][j] = -INFINITY;
                mx = fmaxf(mx, x[i][j]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_new = fmaxf(m[i], mx);
            // every score -inf (an infinite input): subtract 0, the exponentials are 0
            const float ms = m_new == -INFINITY ? 0.0f : m_new;
            const float alpha = exp2f(m[i] - ms);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = exp2f(x[i][j] - ms);
                sum += e;
                P[s * C::LP + tx + 16 * j] = e;
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[i] = l[i] * alpha + sum;
            m[i] = m_new;
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) acc[i][c] *= alpha;
        }
        __syncwarp();  // a row of P is written and read by the same half warp
        // O rows 4 ty + i, columns 4 tx + 64 c + 0..3
        const int t_end = diag ? 4 * ty + 4 : PT;  // keys after the warp's last query are never read
        for (int t = 0; t < t_end; t += 4) {
            float pr[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = *reinterpret_cast<const float4*>(P + (4 * ty + i) * C::LP + t);
                pr[i][0] = f.x, pr[i][1] = f.y, pr[i][2] = f.z, pr[i][3] = f.w;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int c = 0; c < HD / 64; ++c) {
                    const float4 w = *reinterpret_cast<const float4*>(V + (t + u) * HD + 64 * c + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (diag && t + u > 4 * ty + i) continue;  // 0 * NaN of a later value stays out
                        acc[i][4 * c + 0] = fmaf(pr[i][u], w.x, acc[i][4 * c + 0]);
                        acc[i][4 * c + 1] = fmaf(pr[i][u], w.y, acc[i][4 * c + 1]);
                        acc[i][4 * c + 2] = fmaf(pr[i][u], w.z, acc[i][4 * c + 2]);
                        acc[i][4 * c + 3] = fmaf(pr[i][u], w.w, acc[i][4 * c + 3]);
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int s = q0 + 4 * ty + i;
        if (s >= n) continue;
        const float inv = 1.0f / l[i];
        float* o = static_cast<float*>(p.o) + (int64_t)(start + s) * p.ld_o + (int64_t)head * HD + 4 * tx;
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) o[(c >> 2) * 64 + (c & 3)] = acc[i][c] * inv;
        if (p.lse != nullptr && tx == 0) p.lse[(int64_t)head * p.rows + start + s] = m[i] * LN2 + logf(l[i]);
    }
}

// One block = 64 keys of one (sequence, kv head); the queries that see them pass by in tiles
// of 64, head after head.  Thread columns are keys: each thread sums over its rows, the 16
// threads of a column are joined at the end in a fixed order.
template <int HD>
__global__ void __launch_bounds__(256) key_weights_simt_kernel(const PromptArgs p) {
    using C = PCfg<HD>;
    extern __shared__ float sm[];
    float *Q = sm, *K = Q + PT * C::LD;
    __shared__ float part[16][PT];
    if (block_stopped(p.status)) return;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) check_rows(p.cu, p.batch, p.rows, p.status);
    int b, blk, start, n;
    auto count = [](int, int len) { return (len + PT - 1) / PT; };
    if (!find_item(p.cu, p.batch, p.rows, blockIdx.x, count, b, blk)) return;
    seq_rows(p.cu, b, p.rows, start, n);
    const int kvh = blockIdx.y, group = p.n_heads / p.n_kv, t0 = blk * PT;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int first = max(t0, n - min(p.window, n));  // first query that counts for these keys
    load_tile<HD>(K, C::LD, static_cast<const float*>(p.k) + (int64_t)(start + t0) * p.ld_k + (int64_t)kvh * HD, p.ld_k,
                     n - t0, 1.0f);
    float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int g = 0; g < group; ++g) {
        const int head = kvh * group + g;
        for (int s0 = first; s0 < n; s0 += PT) {
            __syncthreads();
            load_tile<HD>(Q, C::LD, static_cast<const float*>(p.q) + (int64_t)(start + s0) * p.ld_q + (int64_t)head * HD,
                             p.ld_q, n - s0, p.scale * LOG2E);
            __syncthreads();
            if (s0 + (ty & ~1) * 4 >= n) continue;  // none of this warp's 8 queries is there
            float x[4][4];
            tile_scores<HD>(Q, K, ty, tx, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = s0 + 4 * ty + i;
                if (s >= n) continue;
                const float l2 = p.lse[(int64_t)head * p.rows + start + s] * LOG2E;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (t0 + tx + 16 * j <= s) w[j] += exp2f(x[i][j] - l2);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) part[ty][tx + 16 * j] = w[j];
    __syncthreads();
    if (tid < PT && t0 + tid < n) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += part[i][tid];
        p.weights[(int64_t)kvh * p.rows + start + t0 + tid] = sum;
    }
}

// Upper bound of the tiles of `tile` rows that `batch` sequences of `rows` rows in all have.
static unsigned max_tiles(int rows, int batch, int tile) {
    return (unsigned)(rows / tile + (batch < rows ? batch : rows));
}

template <int HD>
static cudaError_t prompt_simt(const PromptArgs& a, bool weights, cudaStream_t st) {
    using C = PCfg<HD>;
    const void* kernel = weights ? (const void*)key_weights_simt_kernel<HD> : (const void*)prompt_simt_kernel<HD>;
    const int smem = weights ? C::SMEM_W : C::SMEM;
    cudaError_t e = prepare_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    const dim3 grid(max_tiles(a.rows, a.batch, PT), weights ? a.n_kv : a.n_heads);
    if (weights) key_weights_simt_kernel<HD><<<grid, 256, smem, st>>>(a);
    else prompt_simt_kernel<HD><<<grid, 256, smem, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_prompt(const PromptArgs& a, bool weights, cudaStream_t st) {
    if (a.batch <= 0 || a.rows <= 0) return cudaSuccess;
    if (a.dtype != ENERGON_F32) return weights ? launch_key_weights_tc(a, st) : launch_prompt_tc(a, st);
    return a.head_dim == 64 ? prompt_simt<64>(a, weights, st) : prompt_simt<128>(a, weights, st);
}

}  // namespace energon
