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

// 8 consecutive elements of a row as they are, and as floats.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void floats8(const Raw8<T>& r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const uint32_t u[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) {
                x[4 * i + j] = __uint_as_float(u[j]);
            } else {
                const float2 f = unpack2<T>(u[j]);
                x[2 * j] = f.x, x[2 * j + 1] = f.y;
            }
        }
    }
}

// The nearest code to x / scale (fp32 quotient, ties to even), any x and scale.
__device__ __noinline__ int encode_any(float x, float scale) {
    if (isnan(x)) return 0;
    if (isinf(x)) return x > 0.0f ? 127 : -127;
    if (!(scale > 0.0f)) return 0;
    return __float2int_rn(fminf(fmaxf(__fdiv_rn(x, scale), -127.0f), 127.0f));
}
// Codes of 8 finite elements with |x| <= 127 scale (1 + 2^-22), 2^-90 < scale < 2^120, from
// inv = 1 / scale rounded to nearest.  The quotient is made exact in its last place by two residual
// corrections q + (x - q scale) inv (P. Markstein, Computation of elementary functions on the IBM RISC
// System/6000 processor, 1990: the second one rounds a quotient that is good to its last place
// correctly).  A test of nearness to the middle of two codes would not do: bf16 elements over a page's
// largest lie there once in some hundred.  Adding 1.5 * 2^23 rounds to the code, left in the low byte.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], uint64_t neg_scale, uint64_t inv) {
    constexpr float MAGIC = 12582912.0f;
    uint32_t byte[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint64_t v = two(x[e], x[e + 1]);
        uint64_t q = mul2(v, inv);
        q = fma2(fma2(q, neg_scale, v), inv, q);
        q = fma2(fma2(q, neg_scale, v), inv, q);
        const float2 f = one_by_one(add2(q, two(MAGIC, MAGIC)));
        byte[e] = __float_as_uint(f.x), byte[e + 1] = __float_as_uint(f.y);
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = __byte_perm(__byte_perm(byte[4 * h], byte[4 * h + 1], 0x0040), __byte_perm(byte[4 * h + 2], byte[4 * h + 3], 0x0040), 0x5410);
    return make_uint2(w[0], w[1]);
}

constexpr int APPEND_THREADS = 256;
constexpr int APPEND_HELD = 128 * 128 / 8 / APPEND_THREADS;  // pieces of 8 elements per thread of the largest page
}  // namespace

// One block = the new tokens of one page of one kv head, keys or values.  The rows are read once, into
// registers: for the largest magnitude, then to be encoded.
template <typename T>
__global__ void __launch_bounds__(APPEND_THREADS, sizeof(T) == 4 ? 2 : 4) kv_append_kernel(const AppendArgs a) {
    const CacheArgs& c = a.c;
    if (block_stopped(c.status)) return;
    const int tid = threadIdx.x, P = c.page_len, d = c.head_dim, log_p = __ffs(P) - 1;
    const int32_t* const lens = c.lens;
    const int64_t room = (int64_t)c.max_pages * P;
    // A sequence of l tokens that ends with m new ones has to hold them and to fit in its pages.
    auto fits = [room](int l, int m) { return m <= l && l <= room; };
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid < 32) {
        bool bad = false;
        int s, m;
        for (int i = tid; i < c.batch; i += 32) bad |= !seq_rows(a.cu, i, a.rows, s, m) || !fits(lens[i], m);
        if (bad) status_or(c.status, ENERGON_DEVICE_BAD_LENGTH);
    }
    int b, j, start, n;
    auto count = [lens, fits, log_p](int i, int m) {
        const int l = lens[i];
        return m > 0 && fits(l, m) ? ((l - 1) >> log_p) - ((l - m) >> log_p) + 1 : 0;
    };
    if (!find_item(a.cu, c.batch, a.rows, blockIdx.x, count, b, j)) return;
    seq_rows(a.cu, b, a.rows, start, n);
    // new tokens: rows start .. start + n - 1 at positions len - n .. len - 1
    const int len = lens[b];
    const int at = ((len - n) >> log_p) + j;                               // page of the sequence
    const int s0 = max(len - n - at * P, 0), s1 = min(len - at * P, P);    // its slots that receive tokens
    const int row0 = start + at * P + s0 - (len - n);
    const int page = c.table[(int64_t)b * c.max_pages + at];
    if (!page_ok(page, c.n_pages)) {
        if (tid == 0) status_or(c.status, ENERGON_DEVICE_BAD_PAGE);
        return;
    }
    __shared__ float warp_amax[2][APPEND_THREADS / 32];
    int round = 0;
    for (int part = blockIdx.y; part < 2 * c.n_kv; part += gridDim.y, ++round) {  // keys and values of every head
        const int head = part >> 1;
        const bool values = part & 1;
        const T* x = static_cast<const T*>(values ? a.v : a.k) + (int64_t)head * d;
        const int64_t ld = values ? a.ld_v : a.ld_k;
        const int64_t tile = (int64_t)page * c.n_kv + head;
        int8_t* codes = (values ? c.v_codes : c.k_codes) + tile * P * d;
        float* scale_at = (values ? c.v_scale : c.k_scale) + tile;

        const int per_row = d / 8, log_q = __ffs(per_row) - 1, chunks = (s1 - s0) * per_row;
        Raw8<T> held[APPEND_HELD];
#pragma unroll
        for (int r = 0; r < APPEND_HELD; ++r) {
            const int i = tid + r * APPEND_THREADS;
            if (i >= chunks) break;
            const uint4* from = reinterpret_cast<const uint4*>(x + (row0 + (i >> log_q)) * ld + (i & (per_row - 1)) * 8);
#pragma unroll
            for (int y = 0; y < (int)sizeof(T) / 2; ++y) held[r].w[y] = from[y];
        }
        const float old = *scale_at;  // before any thread may write it
        // Magnitudes compare like their bits; of 16-bit types two at a time.
        uint32_t most[2] = {0, 0};
#pragma unroll
        for (int r = 0; r < APPEND_HELD; ++r) {
            if (tid + r * APPEND_THREADS >= chunks) break;
#pragma unroll
            for (int y = 0; y < (int)sizeof(T) / 2; ++y) {
                const uint32_t u[4] = {held[r].w[y].x, held[r].w[y].y, held[r].w[y].z, held[r].w[y].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (sizeof(T) == 4) most[e & 1] = max(most[e & 1], u[e] & 0x7fffffffu);
                    else most[e & 1] = __vmaxu2(most[e & 1], u[e] & 0x7fff7fffu);
                }
            }
        }
        float amax;
        if constexpr (sizeof(T) == 4) {
            amax = __uint_as_float(max(most[0], most[1]));
        } else {
            const float2 f = unpack2<T>(__vmaxu2(most[0], most[1]));
            amax = isnan(f.x) || isnan(f.y) ? NAN : fmaxf(f.x, f.y);
        }
        const bool odd = !isfinite(amax);
        if (odd) {  // a value that is not finite does not count
            amax = 0.0f;
#pragma unroll
            for (int r = 0; r < APPEND_HELD; ++r) {
                if (tid + r * APPEND_THREADS >= chunks) break;
                float f[8];
                floats8<T>(held[r], f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (isfinite(f[e])) amax = fmaxf(amax, fabsf(f[e]));
            }
        }
        amax = warp_max(amax);
        if ((tid & 31) == 0) warp_amax[round & 1][tid >> 5] = amax;
        const bool any_odd = __syncthreads_or(odd);
        if (any_odd && tid == 0) status_or(c.status, ENERGON_DEVICE_NONFINITE);
#pragma unroll
        for (int w = 0; w < APPEND_THREADS / 32; ++w) amax = fmaxf(amax, warp_amax[round & 1][w]);
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
        const bool plain = !any_odd && scale > 0x1p-90f && scale < 0x1p120f;
        const float inv = plain ? __frcp_rn(scale) : 0.0f;
#pragma unroll
        for (int r = 0; r < APPEND_HELD; ++r) {
            const int i = tid + r * APPEND_THREADS;
            if (i >= chunks) break;
            float f[8];
            floats8<T>(held[r], f);
            uint2 w;
            if (plain) {
                w = encode8(f, two(-scale, -scale), two(inv, inv));
            } else {
                uint32_t y[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e >> 2] |= (uint32_t)(encode_any(f[e], scale) & 0xff) << (8 * (e & 3));
                w = make_uint2(y[0], y[1]);
            }
            *reinterpret_cast<uint2*>(codes + (int64_t)(s0 + (i >> log_q)) * d + (i & (per_row - 1)) * 8) = w;
        }
        if (!values && c.weight != nullptr)
            for (int s = s0 + tid; s < s1; s += APPEND_THREADS)
                c.weight[tile * P + s] = a.weights ? a.weights[(int64_t)head * a.rows + row0 + s - s0] : 0.0f;
    }
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st) {
    if (a.c.batch <= 0 || a.rows <= 0) return cudaSuccess;
    const int some = a.c.batch < a.rows ? a.c.batch : a.rows;
    // a sequence's tokens begin and end inside a page at most, and no page receives less than one
    const int64_t most = (int64_t)a.rows / a.c.page_len + 2 * (int64_t)some;
    const int64_t pages = most < a.rows ? most : a.rows;
    // A block finds its page by a chain of loads; where pages are many it takes several heads of it (about two
    // rounds of blocks on the SMs).  16 prompts, 15 thousand tokens in all: 35 us, of which memory would
    // take 15; 48 single tokens: 7 us, a block for each page and head.
    int64_t parts = (4 * 148 * 2 + pages - 1) / pages;
    if (parts > 2 * a.c.n_kv) parts = 2 * a.c.n_kv;
    const dim3 grid((unsigned)pages, (unsigned)parts);
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
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int HELD = 8;                        // weights that a thread of the selection holds
constexpr int SPAN = HELD * SEL_THREADS;       // tokens that the block takes at a time
constexpr int SEL_SMEM = 192 * 1024;           // weights behind the first SPAN wait in shared memory up to here
constexpr int MOVE_THREADS = 256;
constexpr int SLICES = 4;                      // blocks that share the rows of a sequence cut in place

// What the selection leaves for the move, per (sequence, kv head): a header and, per kept
// token, its old position and the factors of its key and value codes.
struct EvictWs {
    int4* head;       // {tokens kept, anything to move, in place, unused}
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
}  // namespace

// One block = one (sequence, kv head): the kept positions, in order; their weights moved; the
// new pages' scales.  The smallest kept weight is the largest key T that at least `want` keys
// reach; it is found two bits at a time from the counts of keys at or above three candidates.
// Counting needs no histogram, whose bins collide where weights are alike: 3 compares per token and
// step, from registers.  8 weights per thread are held there; more wait in shared memory.  16 caches of up
// to 8192 tokens, 8 kv heads, cut to 2048 each: 26 us (with a histogram of 8 bits a step 48 us); the
// chain of 17 counts, a barrier in each, bounds it.
__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(const EvictArgs a, int smem_floats) {
    const CacheArgs& c = a.c;
    extern __shared__ float more[];  // weights SPAN .. SPAN + smem_floats - 1
    __shared__ int counts[2][3][SEL_WARPS];
    __shared__ uint32_t taken[HELD][SEL_WARPS];
    let_next_grid_start();
    if (block_stopped(c.status)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.y, h = blockIdx.x, P = c.page_len, log_p = __ffs(P) - 1;
    const int item = b * c.n_kv + h;
    const EvictWs ws = evict_ws(a.ws, c.batch * c.n_kv, a.budget);
    const int32_t* old_row = c.table + (int64_t)b * c.max_pages;
    const int32_t* new_row = a.new_table + (int64_t)b * a.new_max_pages;

    const int n = c.lens[b];
    const bool good = len_ok(n, c);
    const int keep = good ? min(n, a.budget) : 0;
    bool bad = false;
    if (good) {
        for (int i = tid; i < (n + P - 1) >> log_p; i += SEL_THREADS) bad |= !page_ok(old_row[i], c.n_pages);
        for (int i = tid; i < (keep + P - 1) >> log_p; i += SEL_THREADS) bad |= !page_ok(new_row[i], c.n_pages);
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
        return c.weight + (((int64_t)row[t >> log_p] * c.n_kv + h) << log_p) + (t & (P - 1));
    };
    float held[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int t = i * SEL_THREADS + tid;
        held[i] = t < n ? *weight_at(old_row, t) : 0.0f;
    }
    for (int t = SPAN + tid; t < min(n, SPAN + smem_floats); t += SEL_THREADS) more[t - SPAN] = *weight_at(old_row, t);
    // (a thread reads back its own weights only)
    auto weight_of = [&](int t) { return t - SPAN < smem_floats ? more[t - SPAN] : *weight_at(old_row, t); };

    // tokens 0 .. m-1 compete for `want` places; kept are keys above thr and the first `ties` equal to it
    const int m = cut ? n - a.recent : 0, want = a.budget - a.recent;
    uint32_t thr = 0xffffffffu;
    int ties = 0;
    if (cut && want > 0) {
        uint32_t key[HELD];
#pragma unroll
        for (int i = 0; i < HELD; ++i) key[i] = order_key(held[i]);
        uint32_t prefix = 0;
        // steps 0 .. 15 settle two bits each; step 16 counts the keys above the threshold
        for (int step = 0; step <= 16; ++step) {
            const int shift = 30 - 2 * step;
            uint32_t at[3];
#pragma unroll
            for (int d = 0; d < 3; ++d) at[d] = step < 16 ? prefix | (uint32_t)(d + 1) << shift : prefix + 1;
            int x[3];
            uint32_t three = 0;  // at most HELD * 32 a warp: 10 bits each
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                if (i * SEL_THREADS + tid >= m) break;
                three += (key[i] >= at[0] ? 1u : 0u) + (key[i] >= at[1] ? 1u << 10 : 0u) + (key[i] >= at[2] ? 1u << 20 : 0u);
            }
            three = __reduce_add_sync(0xffffffffu, three);
#pragma unroll
            for (int d = 0; d < 3; ++d) x[d] = lane == 0 ? (int)(three >> 10 * d & 1023u) : 0;
            for (int t = SPAN + tid; t < m; t += SEL_THREADS) {
                const uint32_t k = order_key(weight_of(t));
#pragma unroll
                for (int d = 0; d < 3; ++d) x[d] += k >= at[d];
            }
            int(*part)[SEL_WARPS] = counts[step & 1];
#pragma unroll
            for (int d = 0; d < 3; ++d) {
                const int y = m > SPAN ? __reduce_add_sync(0xffffffffu, x[d]) : x[d];
                if (lane == 0) part[d][warp] = y;
            }
            __syncthreads();  // the other half of `counts` is written next: nobody reads it any more
#pragma unroll
            for (int d = 0; d < 3; ++d) x[d] = __reduce_add_sync(0xffffffffu, part[d][lane]);
            if (step < 16) prefix |= (uint32_t)((x[0] >= want) + (x[1] >= want) + (x[2] >= want)) << shift;
            else ties = prefix == 0xffffffffu ? want : want - x[0];
        }
        thr = prefix;
    }
    int above = 0, equal = 0;  // kept outright / equal to thr so far
    for (int s0 = 0; s0 < n; s0 += SPAN) {
        if (s0 > 0) {
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                const int t = s0 + i * SEL_THREADS + tid;
                held[i] = t < n ? weight_of(t) : 0.0f;
            }
        }
        uint32_t gts[HELD], eqs[HELD];
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int t = s0 + i * SEL_THREADS + tid;
            bool gt = false, eq = false;
            if (t < n) {
                if (t >= m) gt = true;
                else if (want > 0) {
                    const uint32_t k = order_key(held[i]);
                    gt = k > thr, eq = k == thr;
                }
            }
            gts[i] = __ballot_sync(0xffffffffu, gt), eqs[i] = __ballot_sync(0xffffffffu, eq);
            if (lane == 0) taken[i][warp] = __popc(gts[i]) | __popc(eqs[i]) << 16;
        }
        __syncthreads();  // also: this span is read
        const uint32_t below = (1u << lane) - 1;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const uint32_t v = taken[i][lane];
            const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0u), all = __reduce_add_sync(0xffffffffu, v);
            const bool gt = gts[i] >> lane & 1, eq = eqs[i] >> lane & 1;
            const int e = equal + (int)(before >> 16) + __popc(eqs[i] & below);
            // in place: the slot is at or before t, and later spans read behind it only
            if (gt || (eq && e < ties)) {
                const int slot = above + (int)(before & 0xffffu) + __popc(gts[i] & below) + min(e, ties);
                src[slot] = s0 + i * SEL_THREADS + tid;
                *weight_at(new_row, slot) = held[i];
            }
            above += (int)(all & 0xffffu), equal += (int)(all >> 16);
        }
        __syncthreads();
    }
    // Scales: a warp per new page.  In place a page's scale is an input of its own and of earlier
    // pages only, so that a round's scales are written when the round has read.
    const int pages = (keep + P - 1) >> log_p;
    for (int p0 = 0; p0 < pages; p0 += SEL_WARPS) {
        const int p = p0 + warp;
        float sk[4], sv[4], mk = 0.0f, mv = 0.0f;  // at most 128 tokens a page
        if (p < pages) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int slot = p * P + i * 32 + lane;
                const bool live = i * 32 + lane < P && slot < keep;
                const int64_t at = live ? (int64_t)old_row[src[slot] >> log_p] * c.n_kv + h : 0;
                sk[i] = live ? c.k_scale[at] : 0.0f, sv[i] = live ? c.v_scale[at] : 0.0f;
                mk = fmaxf(mk, sk[i]), mv = fmaxf(mv, sv[i]);
            }
            mk = warp_max(mk), mv = warp_max(mv);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int slot = p * P + i * 32 + lane;
                if (i * 32 + lane >= P || slot >= keep) continue;
                ws.by_k[(int64_t)item * ws.stride + slot] = sk[i] > 0.0f ? __fdiv_rn(sk[i], mk) : 0.0f;
                ws.by_v[(int64_t)item * ws.stride + slot] = sv[i] > 0.0f ? __fdiv_rn(sv[i], mv) : 0.0f;
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

// Codes times the token's factor, rounded.  (Adding 1.5 * 2^23 to the product instead of converting it
// gained nothing, and lost exactness where the two became one fused operation.)
__device__ __forceinline__ uint4 scaled_codes(uint4 x, float f) {
    if (f == 1.0f) return x;
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
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
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Moves 134 MB for the caches above in 31 us, of which memory would take 20.
//
// One block = one new page of one (sequence, kv head), keys and values; in place SLICES blocks do
// all pages in order, each its part of the rows' bytes: a page is written after everything that is read
// from it was read (a kept token's slot is never behind its old position).
__global__ void __launch_bounds__(MOVE_THREADS) evict_move_kernel(const EvictArgs a) {
    const CacheArgs& c = a.c;
    wait_for_earlier_grid();
    if (block_stopped(c.status)) return;
    const int tid = threadIdx.x, P = c.page_len, d = c.head_dim, log_p = __ffs(P) - 1;
    const int b = blockIdx.z, h = blockIdx.y, item = b * c.n_kv + h;
    const EvictWs ws = evict_ws(a.ws, c.batch * c.n_kv, a.budget);
    const int4 head = ws.head[item];
    const int keep = head.x, pages = (keep + P - 1) >> log_p;
    if (blockIdx.x == 0 && h == 0 && tid == 0) a.new_lens[b] = keep;
    if (head.y == 0) return;
    const bool in_place = head.z != 0;
    if (in_place ? blockIdx.x >= SLICES : (int)blockIdx.x >= pages) return;
    const int32_t* old_row = c.table + (int64_t)b * c.max_pages;
    const int32_t* new_row = a.new_table + (int64_t)b * a.new_max_pages;
    const int32_t* src = ws.src + (int64_t)item * ws.stride;
    const float *by_k = ws.by_k + (int64_t)item * ws.stride, *by_v = ws.by_v + (int64_t)item * ws.stride;
    const int pieces = d / 16 / (in_place ? SLICES : 1);          // 16-byte pieces of a row for this block
    const int first = in_place ? (int)blockIdx.x * pieces : 0, log_q = __ffs(pieces) - 1;
    for (int p = in_place ? 0 : blockIdx.x; p < pages; p += in_place ? 1 : gridDim.x) {
        const int n = min(P, keep - p * P) * pieces;
        uint4 k[4], v[4];  // at most 128 rows x 128 bytes = 4 x 16 bytes per thread
        float fk[4], fv[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = tid + r * MOVE_THREADS;
            if (i < n) {
                const int slot = p * P + (i >> log_q), t = src[slot];
                const int64_t at = ((((int64_t)old_row[t >> log_p] * c.n_kv + h) << log_p) + (t & (P - 1))) * d + (first + (i & (pieces - 1))) * 16;
                k[r] = *reinterpret_cast<const uint4*>(c.k_codes + at), v[r] = *reinterpret_cast<const uint4*>(c.v_codes + at);
                fk[r] = by_k[slot], fv[r] = by_v[slot];
            }
        }
        if (in_place) __syncthreads();
        const int64_t to = (((int64_t)new_row[p] * c.n_kv + h) << log_p) * d;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = tid + r * MOVE_THREADS;
            if (i < n) {
                const int64_t at = to + (int64_t)(i >> log_q) * d + (first + (i & (pieces - 1))) * 16;
                *reinterpret_cast<uint4*>(c.k_codes + at) = scaled_codes(k[r], fk[r]);
                *reinterpret_cast<uint4*>(c.v_codes + at) = scaled_codes(v[r], fv[r]);
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
    // weights behind the first SPAN tokens, as far as shared memory holds them
    const int behind = a.c.max_len > SPAN ? a.c.max_len - SPAN : 0;
    const int floats = behind < SEL_SMEM / 4 ? behind : SEL_SMEM / 4;
    cudaError_t e = floats * 4 > 40 * 1024 ? prepare_smem((const void*)evict_select_kernel, SEL_SMEM) : cudaSuccess;
    if (e != cudaSuccess) return e;
    evict_select_kernel<<<dim3(a.c.n_kv, a.c.batch), SEL_THREADS, floats * 4, st>>>(a, floats);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int most = a.budget < a.c.max_len ? a.budget : a.c.max_len;
    const int pages = (most + a.c.page_len - 1) / a.c.page_len;
    return launch_early(evict_move_kernel, dim3(pages > SLICES ? pages : SLICES, a.c.n_kv, a.c.batch), MOVE_THREADS, st, a);
}

}  // namespace energon
