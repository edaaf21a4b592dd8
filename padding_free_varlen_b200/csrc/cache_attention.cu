// Attention of one new token per sequence over the paged 8-bit cache.
//
//   x_t = c sum_d q_d K(t)_d,  K(t) = code * scale(page, head);  o = sum_t exp(x_t - lse) V(t)
//
// Simple form: one block per (sequence, query head) walks over the tokens, 128 at a time.
#include <math.h>

#include "internal.h"
#include "serving.cuh"

namespace energon {

namespace {
constexpr int DT = 128;  // tokens per step, threads per block
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

struct AttnWs {
    float* scores;  // [batch][heads][stride], in units of log2 (accumulate only)
    float* lse2;    // [batch][heads]
    int stride;
};
__host__ __device__ inline AttnWs attn_ws(void* ws, int batch, int max_len, int n_heads) {
    AttnWs w;
    w.stride = (max_len + 15) / 16 * 16;
    w.lse2 = static_cast<float*>(ws);
    w.scores = w.lse2 + ((size_t)batch * n_heads + 63) / 64 * 64;
    return w;
}
__device__ __forceinline__ int cached_len(const CacheArgs& c, int b, bool& bad) {
    const int n = c.lens[b];
    bad = n < 0 || n > c.max_len || (int64_t)n > (int64_t)c.max_pages * c.page_len;
    return bad ? 0 : n;
}
}  // namespace

template <typename T, int HD>
__global__ void __launch_bounds__(DT) cache_attn_kernel(const CacheAttnArgs a) {
    const CacheArgs& c = a.c;
    if (stopped(c.status)) return;
    __shared__ float q[HD], pr[DT], red[DT / 32];
    __shared__ int64_t tile[DT];  // page * n_kv + head of each token of the step, -1: masked
    const int tid = threadIdx.x, b = blockIdx.y, head = blockIdx.x, P = c.page_len;
    const int kvh = head / (a.n_heads / c.n_kv);
    bool bad;
    const int n = cached_len(c, b, bad);
    if (bad && head == 0 && tid == 0) status_or(c.status, ENERGON_DEVICE_BAD_LENGTH);
    const AttnWs ws = attn_ws(a.ws, c.batch, c.max_len, a.n_heads);
    for (int i = tid; i < HD; i += DT)
        q[i] = to_f(static_cast<const T*>(a.q)[b * a.ld_q + (int64_t)head * HD + i]) * (a.scale * LOG2E);
    float m = -INFINITY, l = 0.0f, acc = 0.0f;
    for (int t0 = 0; t0 < n; t0 += DT) {
        __syncthreads();
        const int t = t0 + tid;
        float x = -INFINITY;
        tile[tid] = -1;
        if (t < n) {
            const int page = c.table[(int64_t)b * c.max_pages + t / P];
            if ((unsigned)page < (unsigned)c.n_pages) {
                tile[tid] = (int64_t)page * c.n_kv + kvh;
                const int8_t* k = c.k_codes + (tile[tid] * P + t % P) * HD;
                float s = 0.0f;
                for (int i = 0; i < HD; i += 4) {
                    const char4 e = *reinterpret_cast<const char4*>(k + i);
                    s = fmaf(q[i], (float)e.x, s), s = fmaf(q[i + 1], (float)e.y, s);
                    s = fmaf(q[i + 2], (float)e.z, s), s = fmaf(q[i + 3], (float)e.w, s);
                }
                x = s * c.k_scale[tile[tid]];
            } else {
                status_or(c.status, ENERGON_DEVICE_BAD_PAGE);
            }
        }
        if (a.accumulate && t < n) ws.scores[((int64_t)b * a.n_heads + head) * ws.stride + t] = x;
        float mx = warp_max(x);
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        float m_new = m;
#pragma unroll
        for (int w = 0; w < DT / 32; ++w) m_new = fmaxf(m_new, red[w]);
        const float ms = m_new == -INFINITY ? 0.0f : m_new;
        const float alpha = exp2f(m - ms);
        pr[tid] = exp2f(x - ms);
        __syncthreads();
        l *= alpha, acc *= alpha;
        for (int i = 0; i < min(DT, n - t0); ++i) {
            l += pr[i];
            if (tid < HD && tile[i] >= 0)
                acc = fmaf(pr[i] * c.v_scale[tile[i]], (float)c.v_codes[(tile[i] * P + (t0 + i) % P) * HD + tid], acc);
        }
        m = m_new;
    }
    if (tid < HD)
        static_cast<T*>(a.o)[b * a.ld_o + (int64_t)head * HD + tid] = from_f<T>(l > 0.0f || isnan(l) ? acc / l : 0.0f);
    if (tid == 0) {
        const float lse2 = l == 0.0f ? -INFINITY : m + log2f(l);
        ws.lse2[b * a.n_heads + head] = lse2;
        if (a.lse) a.lse[b * a.n_heads + head] = l == 0.0f ? -INFINITY : m * LN2 + logf(l);
    }
}

// weight(t) += sum over the heads of the group of exp2(score - lse)
__global__ void __launch_bounds__(256) cache_weight_kernel(const CacheAttnArgs a) {
    const CacheArgs& c = a.c;
    if (stopped(c.status)) return;
    const int b = blockIdx.z, kvh = blockIdx.y, group = a.n_heads / c.n_kv, P = c.page_len;
    bool bad;
    const int n = cached_len(c, b, bad), t = blockIdx.x * 256 + threadIdx.x;
    if (t >= n) return;
    const int page = c.table[(int64_t)b * c.max_pages + t / P];
    if ((unsigned)page >= (unsigned)c.n_pages) return;
    const AttnWs ws = attn_ws(a.ws, c.batch, c.max_len, a.n_heads);
    float sum = 0.0f;
    for (int g = 0; g < group; ++g) {
        const int64_t r = (int64_t)b * a.n_heads + kvh * group + g;
        sum += exp2f(ws.scores[r * ws.stride + t] - ws.lse2[r]);
    }
    // a page of one sequence has one writer per call; sequences that share a page add in any order
    atomicAdd(c.weight + ((int64_t)page * c.n_kv + kvh) * P + t % P, sum);
}

size_t cache_attention_ws_bytes(int batch, int max_len, int n_heads, int n_kv, int head_dim, bool accumulate) {
    (void)n_kv, (void)head_dim;
    const size_t rows = (size_t)batch * n_heads;
    return ((rows + 63) / 64 * 64 + (accumulate ? rows * (size_t)(((int64_t)max_len + 15) / 16 * 16) : 0)) * sizeof(float);
}

template <typename T>
static cudaError_t cache_attn(const CacheAttnArgs& a, cudaStream_t st) {
    const dim3 grid(a.n_heads, a.c.batch);
    if (a.c.head_dim == 64) cache_attn_kernel<T, 64><<<grid, DT, 0, st>>>(a);
    else cache_attn_kernel<T, 128><<<grid, DT, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.accumulate || a.c.max_len == 0) return e;
    cache_weight_kernel<<<dim3((unsigned)((a.c.max_len + 255) / 256), a.c.n_kv, a.c.batch), 256, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t st) {
    if (a.c.batch <= 0) return cudaSuccess;
    switch (a.dtype) {
    case ENERGON_F32: return cache_attn<float>(a, st);
    case ENERGON_F16: return cache_attn<__half>(a, st);
    case ENERGON_BF16: return cache_attn<__nv_bfloat16>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace energon
