// The paged 8-bit key/value cache: writing new tokens to it, and cutting it down to the tokens
// that received most attention weight.
//
// Element = code * scale with one fp32 scale per (page, kv head) for keys and one for values, so
// that a page's scale leaves every sum over its tokens: the attention kernel multiplies codes.
#include <float.h>
#include <math.h>

#include "internal.h"
#include "serving.cuh"

namespace energon {

namespace {

__device__ __forceinline__ bool page_ok(int page, int n_pages) { return (unsigned)page < (unsigned)n_pages; }
__device__ __forceinline__ bool len_ok(int len, const CacheArgs& c) {
    return len >= 0 && len <= c.max_len && (int64_t)len <= (int64_t)c.max_pages * c.page_len;
}

// ------------------------------------------------------------------ append

// 8 consecutive elements of a row as floats.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T>(u[i]);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The nearest code to x / scale (fp32 quotient, ties to even).
__device__ __forceinline__ int encode(float x, float scale) {
    if (isnan(x)) return 0;
    if (isinf(x)) return x > 0.0f ? 127 : -127;
    if (!(scale > 0.0f)) return 0;
    return __float2int_rn(fminf(fmaxf(__fdiv_rn(x, scale), -127.0f), 127.0f));
}

// New tokens of sequence b: rows start .. start + n - 1 at positions len - n .. len - 1.
__device__ __forceinline__ bool append_span(const AppendArgs& a, int b, int& start, int& n, int& len) {
    len = a.c.lens[b];
    if (seq_rows(a.cu, b, a.rows, start, n) && len_ok(len, a.c) && n <= len) return true;
    n = 0;
    return false;
}

constexpr int APPEND_THREADS = 256;
}  // namespace

// One block = the new tokens of one page of one kv head, keys or values.  The rows are read once
// for the largest magnitude and again (from the cache next to the SM) to be encoded.
template <typename T>
__global__ void __launch_bounds__(APPEND_THREADS) kv_append_kernel(const AppendArgs a) {
    const CacheArgs& c = a.c;
    if (stopped(c.status)) return;
    const int tid = threadIdx.x, P = c.page_len, d = c.head_dim;
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid < 32) {
        bool bad = false;
        int s, n, len;
        for (int i = tid; i < c.batch; i += 32) bad |= !append_span(a, i, s, n, len);
        if (bad) status_or(c.status, ENERGON_DEVICE_BAD_LENGTH);
    }
    int b, j, start, n, len;
    auto count = [&](int i) {
        int s, m, l;
        append_span(a, i, s, m, l);
        return m > 0 ? (l - 1) / P - (l - m) / P + 1 : 0;
    };
    if (!find_item(c.batch, blockIdx.x, count, b, j)) return;
    append_span(a, b, start, n, len);
    const int head = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    const int at = (len - n) / P + j;                                      // page of the sequence
    const int s0 = max(len - n - at * P, 0), s1 = min(len - at * P, P);    // its slots that receive tokens
    const int row0 = start + at * P + s0 - (len - n);
    const int page = c.table[(int64_t)b * c.max_pages + at];
    if (!page_ok(page, c.n_pages)) {
        if (tid == 0) status_or(c.status, ENERGON_DEVICE_BAD_PAGE);
        return;
    }
    const T* x = static_cast<const T*>(values ? a.v : a.k) + (int64_t)head * d;
    const int64_t ld = values ? a.ld_v : a.ld_k;
    const int64_t tile = (int64_t)page * c.n_kv + head;
    int8_t* codes = (values ? c.v_codes : c.k_codes) + tile * P * d;
    float* scale_at = (values ? c.v_scale : c.k_scale) + tile;

    const int per_row = d / 8, chunks = (s1 - s0) * per_row;
    float amax = 0.0f;
    bool odd = false;
    for (int i = tid; i < chunks; i += APPEND_THREADS) {
        float f[8];
        load8<T>(x + (row0 + i / per_row) * ld + (i % per_row) * 8, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (isfinite(f[e])) amax = fmaxf(amax, fabsf(f[e]));
            else odd = true;
        }
    }
    __shared__ float warp_amax[APPEND_THREADS / 32];
    const float old = *scale_at;  // before any thread may write it
    amax = warp_max(amax);
    if ((tid & 31) == 0) warp_amax[tid >> 5] = amax;
    if (__syncthreads_or(odd) && tid == 0) status_or(c.status, ENERGON_DEVICE_NONFINITE);
#pragma unroll
    for (int w = 0; w < APPEND_THREADS / 32; ++w) amax = fmaxf(amax, warp_amax[w]);
    float need = amax * (1.0f / 127.0f);
    if (need < FLT_MIN) need = 0.0f;
    float scale = need;
    if (s0 > 0) {  // the page holds earlier tokens
        int up = 0;
        if (old > 0.0f) {
            if (need > old) {
                int e_old, e_need;
                const float m_old = frexpf(old, &e_old), m_need = frexpf(need, &e_need);
                up = e_need - e_old + (m_need > m_old ? 1 : 0);
            }
            scale = ldexpf(old, up);
        }
        if (up > 0) {
            const float by = ldexpf(1.0f, -up);
            for (int i = tid; i < P * d / 4; i += APPEND_THREADS) {
                const int slot = i * 4 / d;
                if (slot >= s0 && slot < s1) continue;
                char4 q = reinterpret_cast<char4*>(codes)[i];
                q.x = (signed char)__float2int_rn(q.x * by), q.y = (signed char)__float2int_rn(q.y * by);
                q.z = (signed char)__float2int_rn(q.z * by), q.w = (signed char)__float2int_rn(q.w * by);
                reinterpret_cast<char4*>(codes)[i] = q;
            }
        }
    }
    if (tid == 0) *scale_at = scale;
    for (int i = tid; i < chunks; i += APPEND_THREADS) {
        float f[8];
        load8<T>(x + (row0 + i / per_row) * ld + (i % per_row) * 8, f);
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[h] |= (uint32_t)(encode(f[4 * h + e], scale) & 0xff) << (8 * e);
        }
        *reinterpret_cast<uint2*>(codes + (int64_t)(s0 + i / per_row) * d + (i % per_row) * 8) = make_uint2(w[0], w[1]);
    }
    if (!values && c.weight != nullptr)
        for (int s = s0 + tid; s < s1; s += APPEND_THREADS)
            c.weight[tile * P + s] = a.weights ? a.weights[(int64_t)head * a.rows + row0 + s - s0] : 0.0f;
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st) {
    if (a.c.batch <= 0 || a.rows <= 0) return cudaSuccess;
    const int some = a.c.batch < a.rows ? a.c.batch : a.rows;
    const dim3 grid((unsigned)(a.rows / a.c.page_len) + 2u * (unsigned)some, 2 * a.c.n_kv);
    switch (a.dtype) {
    case ENERGON_F32: kv_append_kernel<float><<<grid, APPEND_THREADS, 0, st>>>(a); break;
    case ENERGON_F16: kv_append_kernel<__half><<<grid, APPEND_THREADS, 0, st>>>(a); break;
    case ENERGON_BF16: kv_append_kernel<__nv_bfloat16><<<grid, APPEND_THREADS, 0, st>>>(a); break;
    default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

// ------------------------------------------------------------------ evict

namespace {
constexpr int SEL_THREADS = 1024;
constexpr int MOVE_THREADS = 256;

// What the selection leaves for the move, per (sequence, kv head): a header and, per kept
// token, its old position and the factors of its key and value codes.
struct EvictWs {
    int4* head;       // {tokens kept, pages at a time, unused, unused}
    int32_t* src;     // [stride]
    float *by_k, *by_v;
    int stride;
};
__host__ __device__ inline EvictWs evict_ws(void* ws, int items, int budget) {
    EvictWs w;
    w.stride = (budget + 31) / 32 * 32;
    w.head = static_cast<int4*>(ws);
    w.src = reinterpret_cast<int32_t*>(w.head + items);
    w.by_k = reinterpret_cast<float*>(w.src + (size_t)items * w.stride);
    w.by_v = w.by_k + (size_t)items * w.stride;
    return w;
}

// Order-preserving key of a weight; NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block of two 16-bit counts in one word; the total goes to `total`.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the previous use of warp_sums is over
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    uint32_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < SEL_THREADS / 32; ++w) {
        if (w == warp) before = sum;
        sum += warp_sums[w];
    }
    total = sum;
    return before + x - v;
}
}  // namespace

// One block = one (sequence, kv head): the kept positions, in order; their weights moved; the
// new pages' scales.  The smallest kept weight is found digit by digit (8 bits at a time from
// the top) from counts of the keys that share the digits found so far.
__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(const EvictArgs a) {
    const CacheArgs& c = a.c;
    if (stopped(c.status)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.y, h = blockIdx.x, P = c.page_len;
    const int item = b * c.n_kv + h;
    const EvictWs ws = evict_ws(a.ws, c.batch * c.n_kv, a.budget);
    __shared__ uint32_t sums[32];
    __shared__ int hist[256];
    __shared__ uint32_t found;
    __shared__ int left;
    const int32_t* old_row = c.table + (int64_t)b * c.max_pages;
    const int32_t* new_row = a.new_table + (int64_t)b * a.new_max_pages;

    const int n = c.lens[b];
    const bool good = len_ok(n, c);
    const int keep = good ? min(n, a.budget) : 0;
    bool bad = false;
    if (good) {
        for (int i = tid; i < (n + P - 1) / P; i += SEL_THREADS) bad |= !page_ok(old_row[i], c.n_pages);
        for (int i = tid; i < (keep + P - 1) / P; i += SEL_THREADS) bad |= !page_ok(new_row[i], c.n_pages);
    }
    bad = __syncthreads_or(bad);
    if (!good || bad || keep == 0) {
        if (tid == 0) {
            ws.head[item] = make_int4(0, 0, 0, 0);
            if (h == 0 && (!good || bad)) status_or(c.status, good ? ENERGON_DEVICE_BAD_PAGE : ENERGON_DEVICE_BAD_LENGTH);
        }
        return;
    }
    const bool in_place = new_row[0] == old_row[0], cut = n > a.budget;
    if (tid == 0) ws.head[item] = make_int4(keep, cut || !in_place, in_place, 0);
    if (in_place && !cut) return;
    int32_t* src = ws.src + (int64_t)item * ws.stride;
    auto weight_at = [&](const int32_t* row, int t) -> float* {
        return c.weight + (((int64_t)row[t / P] * c.n_kv + h) * P + t % P);
    };

    // tokens 0 .. m-1 compete for `want` places; kept are keys above thr and the first `ties` equal to it
    const int m = cut ? n - a.recent : 0, want = a.budget - a.recent;
    uint32_t thr = 0xffffffffu;
    int ties = 0;
    if (cut && want > 0) {
        uint32_t prefix = 0;
        int rest = want;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += SEL_THREADS) hist[i] = 0;
            __syncthreads();
            for (int t = tid; t < m; t += SEL_THREADS) {
                const uint32_t k = order_key(*weight_at(old_row, t));
                if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int d = 255, r = rest;
                while (d > 0 && hist[d] < r) r -= hist[d--];
                found = (uint32_t)d, left = r;
            }
            __syncthreads();
            prefix |= found << shift;
            rest = left;
        }
        thr = prefix, ties = rest;
    }
    uint32_t above = 0, equal = 0;  // kept outright / equal to thr so far
    for (int t0 = 0; t0 < n; t0 += SEL_THREADS) {
        const int t = t0 + tid;
        float w = 0.0f;
        bool gt = false, eq = false;
        if (t < n) {
            w = *weight_at(old_row, t);
            if (t >= m) gt = true;
            else if (want > 0) {
                const uint32_t k = order_key(w);
                gt = k > thr, eq = k == thr;
            }
        }
        uint32_t total;
        const uint32_t x = block_scan((gt ? 1u : 0u) | (eq ? 0x10000u : 0u), sums, total);
        const uint32_t e = equal + (x >> 16);
        // in place: the slot is at or before t, and later rounds read behind it only
        if (gt || (eq && e < (uint32_t)ties)) {
            const int slot = (int)(above + (x & 0xffffu) + min(e, (uint32_t)ties));
            src[slot] = t;
            *weight_at(new_row, slot) = w;
        }
        above += total & 0xffffu, equal += total >> 16;
    }
    __syncthreads();
    // Scales: a warp per new page.  In place a page's scale is an input of its own and of earlier
    // pages only, so that a round's scales are written when the round has read.
    const int pages = (keep + P - 1) / P;
    for (int p0 = 0; p0 < pages; p0 += SEL_THREADS / 32) {
        const int p = p0 + warp;
        float mk = 0.0f, mv = 0.0f;
        if (p < pages) {
            for (int i = lane; i < P && p * P + i < keep; i += 32) {
                const int64_t at = (int64_t)old_row[src[p * P + i] / P] * c.n_kv + h;
                mk = fmaxf(mk, c.k_scale[at]), mv = fmaxf(mv, c.v_scale[at]);
            }
            mk = warp_max(mk), mv = warp_max(mv);
            for (int i = lane; i < P && p * P + i < keep; i += 32) {
                const int64_t at = (int64_t)old_row[src[p * P + i] / P] * c.n_kv + h;
                const float sk = c.k_scale[at], sv = c.v_scale[at];
                ws.by_k[(int64_t)item * ws.stride + p * P + i] = sk > 0.0f ? __fdiv_rn(sk, mk) : 0.0f;
                ws.by_v[(int64_t)item * ws.stride + p * P + i] = sv > 0.0f ? __fdiv_rn(sv, mv) : 0.0f;
            }
        }
        __syncthreads();
        if (p < pages && lane == 0) {
            const int64_t at = (int64_t)new_row[p] * c.n_kv + h;
            c.k_scale[at] = mk, c.v_scale[at] = mv;
        }
        __syncthreads();
    }
}

// One block = one new page of one (sequence, kv head), keys or values; in place one block does
// all pages in order: a page is written after everything that is read from it was read (a kept
// token's slot is never behind its old position).
__global__ void __launch_bounds__(MOVE_THREADS) evict_move_kernel(const EvictArgs a) {
    const CacheArgs& c = a.c;
    if (stopped(c.status)) return;
    const int tid = threadIdx.x, P = c.page_len, d = c.head_dim;
    const int b = blockIdx.z, h = blockIdx.y >> 1, item = b * c.n_kv + h;
    const bool values = blockIdx.y & 1;
    const EvictWs ws = evict_ws(a.ws, c.batch * c.n_kv, a.budget);
    const int4 head = ws.head[item];
    const int keep = head.x, pages = (keep + P - 1) / P;
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) a.new_lens[b] = keep;
    if (head.y == 0) return;
    const bool in_place = head.z != 0;
    if (in_place && blockIdx.x != 0) return;
    const int32_t* old_row = c.table + (int64_t)b * c.max_pages;
    const int32_t* new_row = a.new_table + (int64_t)b * a.new_max_pages;
    const int32_t* src = ws.src + (int64_t)item * ws.stride;
    const float* by = (values ? ws.by_v : ws.by_k) + (int64_t)item * ws.stride;
    int8_t* codes = values ? c.v_codes : c.k_codes;
    const int per_row = d / 16;
    for (int p = in_place ? 0 : blockIdx.x; p < pages; p += in_place ? 1 : gridDim.x) {
        const int rows = min(P, keep - p * P);
        uint4 x[4];  // at most 128 rows x 128 bytes = 4 x 16 bytes per thread
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = tid + r * MOVE_THREADS;
            if (i < rows * per_row) {
                const int t = src[p * P + i / per_row];
                x[r] = *reinterpret_cast<const uint4*>(
                    codes + (((int64_t)old_row[t / P] * c.n_kv + h) * P + t % P) * d + (i % per_row) * 16);
            }
        }
        if (in_place) __syncthreads();
        int8_t* to = codes + ((int64_t)new_row[p] * c.n_kv + h) * P * d;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = tid + r * MOVE_THREADS;
            if (i < rows * per_row) {
                const float f = by[p * P + i / per_row];
                uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t y = 0;
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int q = (int)(int8_t)(w[e] >> (8 * s));
                        y |= (uint32_t)(__float2int_rn(__fmul_rn((float)q, f)) & 0xff) << (8 * s);
                    }
                    w[e] = y;
                }
                *reinterpret_cast<uint4*>(to + (int64_t)(i / per_row) * d + (i % per_row) * 16) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (in_place) __syncthreads();
    }
}

size_t cache_evict_ws_bytes(int batch, int n_kv, int budget) {
    const size_t items = (size_t)batch * n_kv, stride = ((size_t)budget + 31) / 32 * 32;
    return items * (sizeof(int4) + 12 * stride);
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t st) {
    if (a.c.batch <= 0) return cudaSuccess;
    evict_select_kernel<<<dim3(a.c.n_kv, a.c.batch), SEL_THREADS, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int most = a.budget < a.c.max_len ? a.budget : a.c.max_len;
    const unsigned pages = (unsigned)((most + a.c.page_len - 1) / a.c.page_len);
    evict_move_kernel<<<dim3(pages > 0 ? pages : 1, 2 * a.c.n_kv, a.c.batch), MOVE_THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace energon
