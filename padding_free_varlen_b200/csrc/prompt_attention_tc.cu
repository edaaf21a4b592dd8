// Causal attention of packed prompts with grouped heads on the 5th-generation tensor cores
// (fp16, bf16).
//
//   o_j(s) = sum_{t <= s} exp(c q_j(s) . k(t) - lse_j(s)) v(t)
//
// A block holds NT tiles of 128 queries that read the same keys: two query heads of one kv head
// where a kv head has an even number of them, else neighbouring tiles of one head.  Keys and
// values pass by in blocks of BN, one pass with a running maximum and sum:
//   loader     one thread: Q tiles, then K and V blocks into a ring of buffers by TMA
//   products   one thread: S_i = Q_i K^T into TMEM, O_i += P_i V with P_i read from TMEM (over the
//              columns of S_i).  Tile 1's products run while tile 0's softmax does, and the other
//              way round.
//   softmax    four warps per tile, a thread per query: row of S to registers, maximum,
//              exponentials, P rounded to 16 bits back to TMEM.  O is rescaled only when the
//              maximum grew by more than 2^8: until then the exponentials are at most 2^8, in
//              range of both types, and the common factor leaves with the sum.
//   scan       two warps: rows of V behind the sequence and values that are not finite are
//              zeroed in the blocks that cross the diagonal (there 0 * NaN would reach earlier
//              rows); the latter are noted and added to the rows that see them at the end.
#include <cudaTypedefs.h>
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "serving.cuh"

namespace energon {

namespace {
constexpr int BM = 128;                 // queries per tile
constexpr int QBOX = BM * 128;          // bytes of 128 rows x 64 columns of 16 bits
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float GROW = 8.0f;            // log2 of the growth that the running maximum may lag behind

constexpr int BN = 64;                  // keys per block

template <int HD, int NT>
struct TCfg {
    static constexpr int QT = HD / 64 * QBOX;                // bytes of a Q tile
    static constexpr int KT = HD * BN * 2;                   // bytes of a K or V block
    static constexpr int RING = NT == 2 ? (HD == 128 ? 5 : 8) : 2;  // buffers of K, and of V
    static constexpr int SMEM = NT * QT + 2 * RING * KT + 1024;
    static constexpr int THREADS = NT * 128 + 128;
    static constexpr int SCAN = NT == 2 ? 32 : 64;           // threads that scan V
    static constexpr int O_COL = NT * 2 * BN;                // S takes two buffers per tile
    static constexpr int TMEM = NT == 2 ? 512 : 256;
    static constexpr int CTAS = NT == 2 ? 1 : 2;
    static constexpr int SCANS = NT * BM / BN;               // most blocks that cross a diagonal
};

// O (or S) += A B with A (M = 128 rows, 16-bit, two per 32-bit column) read from TMEM.
__device__ __forceinline__ void umma_f16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void wg_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
}  // namespace

// Maximum of N scores.
template <int N>
__device__ __forceinline__ float max_of(const uint32_t* x) {
    float m[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        m[y] = fmaxf(__uint_as_float(x[2 * y]), __uint_as_float(x[2 * y + 1]));
#pragma unroll
        for (int e = 8; e < N; e += 8) m[y] = max3(m[y], __uint_as_float(x[e + 2 * y]), __uint_as_float(x[e + 2 * y + 1]));
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

struct PromptTcArgs {
    PromptArgs p;
    int pair_heads;  // NT == 2: the tiles are two heads of one kv head
    int head_steps;  // heads, or pairs of them
    float c;         // scale * log2(e)
};

template <typename T, int HD, int NT>
__global__ void __launch_bounds__(TCfg<HD, NT>::THREADS, TCfg<HD, NT>::CTAS)
prompt_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                 const PromptTcArgs a) {
    using C = TCfg<HD, NT>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t q_full[NT], s_full[NT][2], p_full[NT][2], o_done[NT], o_full[NT], drain[NT];
    __shared__ uint64_t k_full[C::RING], k_empty[C::RING], v_full[C::RING], v_empty[C::RING];
    __shared__ uint64_t v_in[C::SCANS], v_ok[C::SCANS];  // blocks that are scanned: landed, scanned (used once each)
    __shared__ uint32_t tmem_slot;
    __shared__ int dead, odd;
    __shared__ int first[3][HD];  // first key whose value in this column is +inf, -inf, NaN
    const PromptArgs& p = a.p;
    if (stopped(p.status)) return;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int64_t item = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;  // heads pass by first
    if (item == 0 && tid < 32) check_rows(p.cu, p.batch, p.rows, p.status);

    // ---- which queries
    const int tile_rows = NT == 2 && !a.pair_heads ? 2 * BM : BM;
    int b, blk, start, n;
    auto count = [&](int i) {
        int s, len;
        seq_rows(p.cu, i, p.rows, s, len);
        return (len + tile_rows - 1) / tile_rows;
    };
    if (!find_item(p.batch, (int)(item / a.head_steps), count, b, blk)) return;
    seq_rows(p.cu, b, p.rows, start, n);
    blk = (n + tile_rows - 1) / tile_rows - 1 - blk;  // the longest rows first
    const int head0 = (int)(item % a.head_steps) * (a.pair_heads ? 2 : 1);
    const int kvh = head0 / (p.n_heads / p.n_kv);
    auto q0_of = [&](int i) { return blk * tile_rows + (a.pair_heads ? 0 : i * BM); };
    auto head_of = [&](int i) { return head0 + (a.pair_heads ? i : 0); };
    // key blocks of tile i (0: the tile has no queries)
    auto blocks_of = [&](int i) { return q0_of(i) < n ? (min(n, q0_of(i) + BM) + BN - 1) / BN : 0; };
    const int nb0 = blocks_of(0), nb1 = NT == 2 ? blocks_of(NT - 1) : 0, nb = max(nb0, nb1);
    const int scan0 = q0_of(0) / BN;  // first block with keys behind a query

    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring_k = base + NT * C::QT;
    uint8_t* ring_v = ring_k + C::RING * C::KT;
    for (int i = tid; i < 3 * HD; i += C::THREADS) (&first[0][0])[i] = 0x7fffffff;
    if (tid == 0) {
        for (int i = 0; i < NT; ++i) {
            mbar_init(&q_full[i], 1), mbar_init(&o_done[i], 1), mbar_init(&o_full[i], 1), mbar_init(&drain[i], 1);
            for (int y = 0; y < 2; ++y) mbar_init(&s_full[i][y], 1), mbar_init(&p_full[i][y], 128);
        }
        for (int i = 0; i < C::RING; ++i)
            mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], NT), mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], NT);
        for (int i = 0; i < C::SCANS; ++i) mbar_init(&v_in[i], 1), mbar_init(&v_ok[i], C::SCAN);
        dead = 0, odd = 0;
        fence_mbar_init();
    }
    if (warp == NT * 4) {
        tmem_alloc(&tmem_slot, C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (wait_in_line(bar, parity, &dead, p.timeout_ns)) return true;
        *reinterpret_cast<volatile int*>(&dead) = 1;
        return false;
    };

    if (warp == NT * 4) {
        if (lane == 0) {
            // ---- loader: Q, then K(0), K(1), V(0), K(2), V(1), ...
            for (int i = 0; i < NT; ++i) {
                if (i > 0 && nb1 == 0) break;
                mbar_arrive_expect_tx(&q_full[i], C::QT);
                for (int h = 0; h < HD / 64; ++h)
                    tma_load_2d(base + i * C::QT + h * QBOX, &tm_q, &q_full[i], head_of(i) * HD + 64 * h, start + q0_of(i));
            }
            int nk = 0, nv = 0;  // blocks asked for
            for (int x = 0; x < 2 * nb; ++x) {
                const bool keys = nk < nb && nk - nv < 2;
                const int kb = keys ? nk : nv, at = kb % C::RING;
                if (kb >= C::RING && !wait(keys ? &k_empty[at] : &v_empty[at], (kb / C::RING - 1) & 1)) break;
                uint64_t* bar = keys ? &k_full[at] : &v_full[at];
                if (!keys && kb >= scan0) {  // the scan waits for this one alone
                    mbar_arrive(bar);
                    bar = &v_in[kb - scan0];
                }
                mbar_arrive_expect_tx(bar, C::KT);
                for (int h = 0; h < HD / 64; ++h)
                    tma_load_2d((keys ? ring_k : ring_v) + at * C::KT + h * BN * 128, keys ? &tm_k : &tm_v, bar,
                                kvh * HD + 64 * h, start + kb * BN);
                (keys ? nk : nv) += 1;
            }
            // All copies have landed before the block ends, also where a wait ran out.
            for (int i = 0; i < NT; ++i)
                if (i == 0 || nb1 > 0) mbar_wait_bounded(&q_full[i], 0, nullptr, p.timeout_ns);
            for (int y = max(0, nk - C::RING); y < nk; ++y)
                mbar_wait_bounded(&k_full[y % C::RING], (y / C::RING) & 1, nullptr, p.timeout_ns);
            for (int y = max(0, nv - C::RING); y < nv; ++y)
                mbar_wait_bounded(&v_full[y % C::RING], (y / C::RING) & 1, nullptr, p.timeout_ns);
            for (int kb = scan0; kb < nv; ++kb) mbar_wait_bounded(&v_in[kb - scan0], 0, nullptr, p.timeout_ns);
        }
    } else if (warp > NT * 4 && warp <= NT * 4 + NT) {
        // ---- products of tile i: the whole warp follows, one lane issues.  A warp per tile: one's
        // products fill the time in which the other looks at its barriers.
        constexpr uint32_t fmt = std::is_same<T, __half>::value ? 0u : 1u;
        constexpr uint32_t idesc_s = idesc_f16(fmt, BM, BN, 0), idesc_o = idesc_f16(fmt, BM, HD, 1);
        const int i = warp - NT * 4 - 1, mine = i == 0 ? nb0 : nb1;
        auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
        auto have_k = [&](int kb) { return wait_warp(&k_full[kb % C::RING], (kb / C::RING) & 1); };
        auto scores = [&](int kb) {  // and K's buffer is free once they are done
            if (kb < mine) {
                const uint32_t q = smem_u32(base + i * C::QT), k = smem_u32(ring_k + kb % C::RING * C::KT);
#pragma unroll
                for (int s = 0; s < HD / 16; ++s)
                    umma_f16(tmem + (2 * i + (kb & 1)) * BN, smem_desc_k128(q + (s >> 2) * QBOX) + 2 * (s & 3),
                             smem_desc_k128(k + (s >> 2) * BN * 128) + 2 * (s & 3), idesc_s, s > 0);
                umma_commit(&s_full[i][kb & 1]);
            }
            umma_commit(&k_empty[kb % C::RING]);
        };
        // the scores run two blocks ahead of the products with V
        bool ok = mine == 0 || wait_warp(&q_full[i], 0);
        for (int kb = 0; ok && kb < 2 && kb < nb; ++kb) {
            ok = have_k(kb);
            tc_fence_after();
            if (ok && elect_one()) scores(kb);
        }
        for (int kb = 0; ok && kb < nb; ++kb) {
            const int at = kb % C::RING;
            ok = wait_warp(&v_full[at], (kb / C::RING) & 1) && (kb + 2 >= nb || have_k(kb + 2)) &&
                 (kb < scan0 || (wait_warp(&v_in[kb - scan0], 0) && wait_warp(&v_ok[kb - scan0], 0))) &&
                 (kb >= mine || wait_warp(&p_full[i][kb & 1], (kb >> 1) & 1));
            tc_fence_after();
            if (ok && elect_one()) {
                if (kb < mine) {
                    const uint32_t v = smem_u32(ring_v + at * C::KT);
#pragma unroll
                    for (int s = 0; s < BN / 16; ++s)
                        umma_f16_tmem_a(tmem + C::O_COL + i * HD, tmem + (2 * i + (kb & 1)) * BN + s * 8,
                                        smem_desc_mn128(v + s * 2048, BN * 128, 1024), idesc_o, kb > 0 || s > 0);
                    umma_commit(kb + 1 < mine ? &o_done[i] : &o_full[i]);
                }
                umma_commit(&v_empty[at]);
                if (kb + 2 < nb) scores(kb + 2);  // over the scores of block kb: these products come first
            }
        }
        if (elect_one()) umma_commit(&drain[i]);  // all products are done before the block ends
        mbar_wait_bounded(&drain[i], 0, nullptr, p.timeout_ns);
    } else if (warp > NT * 4 + NT) {
        // ---- scan of V
        constexpr uint32_t INF = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
        const int me = tid - (NT * 4 + NT + 1) * 32;
        for (int kb = scan0; kb < nb; ++kb) {
            if (!wait(&v_in[kb - scan0], 0)) break;
            uint8_t* v = ring_v + kb % C::RING * C::KT;
            for (int r = me; r < BN; r += C::SCAN) {
                const int t = kb * BN + r;
                uint32_t most = 0;
                if (t < n) {
#pragma unroll
                    for (int ch = 0; ch < HD / 8; ++ch) {
                        const uint4 w = *reinterpret_cast<const uint4*>(v + (ch >> 3) * BN * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
                        most = __vmaxu2(__vmaxu2(__vmaxu2(most, w.x & 0x7fff7fffu), __vmaxu2(w.y & 0x7fff7fffu, w.z & 0x7fff7fffu)),
                                        w.w & 0x7fff7fffu);
                    }
                    if ((most & 0xffffu) < INF && (most >> 16) < INF) continue;
                    for (int d = 0; d < HD; ++d) {
                        uint16_t* e = reinterpret_cast<uint16_t*>(v + (d >> 6) * BN * 128 + r * 128 +
                                                                  (((d >> 3 & 7) ^ (r & 7)) << 4)) + (d & 7);
                        const uint32_t w = *e;
                        if ((w & 0x7fffu) < INF) continue;
                        atomicMin(&first[(w & 0x7fffu) > INF ? 2 : w >> 15][d], t);
                        *e = 0;
                    }
                    odd = 1;
                } else {
#pragma unroll
                    for (int ch = 0; ch < HD / 8; ++ch)
                        *reinterpret_cast<uint4*>(v + (ch >> 3) * BN * 128 + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&v_ok[kb - scan0]);
        }
    } else {
        // ---- softmax of tile i, one query per thread
        const int i = NT == 2 ? warp >> 2 : 0, row = tid & 127, q0 = q0_of(i), s = q0 + row;
        const int mine = i == 0 ? nb0 : nb1;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t S0 = tmem + lanes + 2 * i * BN, O = tmem + lanes + C::O_COL + i * HD;
        float m = -INFINITY, mc = 0.0f;  // the maximum that the exponentials refer to, and times c (0 for -infinity)
        uint64_t sum[4] = {0, 0, 0, 0};  // pairs of partial sums (+0.0)
        // TMEM is read and written by whole warps: their lanes give up together
        auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
        bool ok = true;
        for (int kb = 0; kb < mine; ++kb) {
            const uint32_t S = S0 + (kb & 1) * BN;
            ok = wait_warp(&s_full[i][kb & 1], (kb >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            uint32_t x[BN];
            tmem_ld_x32(S, x);
            tmem_ld_x32(S + 32, x + 32);
            tmem_wait_ld_regs(x);
            tmem_wait_ld_regs(x + 32);
            if (kb >= q0 / BN) {
                const int see = s - kb * BN;  // keys up to here
#pragma unroll
                for (int e = 0; e < BN; ++e)
                    if (e > see) x[e] = 0xff800000u;
            }
            const float mx = max_of<BN>(x);
            if (kb == 0) {
                m = mx;
                mc = m == -INFINITY ? 0.0f : m * a.c;
            } else if (__any_sync(0xffffffffu, (mx - m) * a.c > GROW)) {
                // O is at rest once the products of block kb - 1 are done; those of kb - 2 were before S,
                // those of kb wait for this thread: the phase is the barrier's current or last one
                ok = wait_warp(&o_done[i], (kb - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                float by = 1.0f;
                if ((mx - m) * a.c > GROW) {
                    by = m == -INFINITY ? 0.0f : exp2_fast(mc - mx * a.c);
                    m = mx, mc = mx * a.c;
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) sum[y] = mul2(sum[y], two(by, by));
#pragma unroll 1
                for (int h = 0; h < HD / 32; ++h) {
                    uint32_t o[32];
                    tmem_ld_x32(O + 32 * h, o);
                    tmem_wait_ld_regs(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                    tmem_st_x32(O + 32 * h, o);
                }
            }
            const uint64_t c2 = two(a.c, a.c), m2 = two(-mc, -mc);
#pragma unroll
            for (int h = 0; h < BN / 32; ++h) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t* y = x + 32 * h + 2 * e;
                    const float2 z = one_by_one(fma2(two(__uint_as_float(y[0]), __uint_as_float(y[1])), c2, m2));
                    const float e0 = exp2_fast(z.x), e1 = exp2_fast(z.y);
                    sum[e & 3] = add2(sum[e & 3], two(e0, e1));
                    w[e] = pack2<T>(e0, e1);
                }
                tmem_st_x16(S + 16 * h, w);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_full[i][kb & 1]);
        }
        if (mine > 0 && ok) ok = wait_warp(&o_full[i], 0);
        // values that are not finite, as noted for the blocks that this tile reads
        for (int kb = scan0; ok && kb < mine; ++kb) ok = wait_warp(&v_ok[kb - scan0], 0);
        if (mine > 0 && ok) {
            tc_fence_after();
            const float2 l2 = one_by_one(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
            const float l = l2.x + l2.y, inv = 1.0f / l;
            const bool fix = *reinterpret_cast<volatile int*>(&odd) != 0;
            // O / l, rounded, over the Q tile (no product reads it any more), 128-byte swizzle
            uint8_t* out = base + i * C::QT;
#pragma unroll 1
            for (int h = 0; h < HD / 32; ++h) {
                uint32_t o[32];
                tmem_ld_x32(O + 32 * h, o);
                tmem_wait_ld_regs(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float f = __uint_as_float(o[e]) * inv;
                    if (fix) {
                        if (s >= first[0][32 * h + e]) f += INFINITY;
                        if (s >= first[1][32 * h + e]) f -= INFINITY;
                        if (s >= first[2][32 * h + e]) f = NAN;
                    }
                    o[e] = __float_as_uint(f);
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint4 w;
                    w.x = pack2<T>(__uint_as_float(o[8 * g]), __uint_as_float(o[8 * g + 1]));
                    w.y = pack2<T>(__uint_as_float(o[8 * g + 2]), __uint_as_float(o[8 * g + 3]));
                    w.z = pack2<T>(__uint_as_float(o[8 * g + 4]), __uint_as_float(o[8 * g + 5]));
                    w.w = pack2<T>(__uint_as_float(o[8 * g + 6]), __uint_as_float(o[8 * g + 7]));
                    const int ch = (h & 1) * 4 + g;
                    *reinterpret_cast<uint4*>(out + (h >> 1) * QBOX + row * 128 + ((ch ^ (row & 7)) << 4)) = w;
                }
            }
            if (s < n && p.lse != nullptr) p.lse[(int64_t)head_of(i) * p.rows + start + s] = (mc + log2f(l)) * LN2;
            fence_proxy_async_smem();
        }
        // (all threads of the tile agree on `mine`; a wait that ran out lets none of them store)
        wg_sync(1 + i);
        if (mine > 0 && *reinterpret_cast<volatile int*>(&dead) == 0) {
            uint8_t* out = base + i * C::QT;
            const int rows = min(BM, n - q0);
            if (rows == BM) {
                if (row == 0) {
                    for (int h = 0; h < HD / 64; ++h) tma_store_2d(&tm_o, out + h * QBOX, head_of(i) * HD + 64 * h, start + q0);
                    bulk_commit();
                    bulk_wait_read<0>();
                }
            } else {
                constexpr int PER = HD / 8;  // 16-byte pieces of a row
                for (int y = row; y < rows * PER; y += 128) {
                    const int r = y / PER, ch = y % PER;
                    const uint4 w = *reinterpret_cast<const uint4*>(out + (ch >> 3) * QBOX + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
                    *reinterpret_cast<uint4*>(static_cast<T*>(p.o) + (int64_t)(start + q0 + r) * p.ld_o + (int64_t)head_of(i) * HD + ch * 8) = w;
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && dead) status_or(p.status, ENERGON_DEVICE_TIMEOUT);
    if (warp == NT * 4) tmem_dealloc(tmem, C::TMEM);
}

// ------------------------------------------------------------------ host side

// A [rows, cols] 16-bit tensor with rows ld elements apart, boxes of 64 columns.
cudaError_t rows_map(CUtensorMap* m, int dtype, const void* ptr, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
    const auto encode = tensor_map_encoder();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, one[2] = {1, 1};
    const auto type = dtype == ENERGON_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return encode(m, type, 2, const_cast<void*>(ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <typename T, int HD, int NT>
static cudaError_t prompt_tc(const PromptArgs& p, cudaStream_t st) {
    using C = TCfg<HD, NT>;
    CUtensorMap q, k, v, o;
    const int64_t wq = (int64_t)p.n_heads * HD, wk = (int64_t)p.n_kv * HD;
    cudaError_t e = rows_map(&q, p.dtype, p.q, wq, p.rows, p.ld_q, BM);
    if (e == cudaSuccess) e = rows_map(&k, p.dtype, p.k, wk, p.rows, p.ld_k, BN);
    if (e == cudaSuccess) e = rows_map(&v, p.dtype, p.v, wk, p.rows, p.ld_v, BN);
    if (e == cudaSuccess) e = rows_map(&o, p.dtype, p.o, wq, p.rows, p.ld_o, BM);
    if (e == cudaSuccess) e = prepare_smem((const void*)prompt_tc_kernel<T, HD, NT>, C::SMEM);
    if (e != cudaSuccess) return e;
    PromptTcArgs a;
    a.p = p;
    a.pair_heads = NT == 2 && p.n_heads / p.n_kv % 2 == 0;
    a.c = p.scale * LOG2E;
    const int tile = NT == 2 && !a.pair_heads ? 2 * BM : BM;
    const int most = p.rows / tile + (p.batch < p.rows ? p.batch : p.rows);
    a.head_steps = a.pair_heads ? p.n_heads / 2 : p.n_heads;
    const dim3 grid(most, a.head_steps);
    prompt_tc_kernel<T, HD, NT><<<grid, C::THREADS, C::SMEM, st>>>(q, k, v, o, a);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t prompt_tc_t(const PromptArgs& p, cudaStream_t st) {
    const bool two_tiles = p.rows / p.batch > 256;
    if (p.head_dim == 64) return two_tiles ? prompt_tc<T, 64, 2>(p, st) : prompt_tc<T, 64, 1>(p, st);
    return two_tiles ? prompt_tc<T, 128, 2>(p, st) : prompt_tc<T, 128, 1>(p, st);
}

cudaError_t launch_prompt_tc(const PromptArgs& p, cudaStream_t st) {
    return p.dtype == ENERGON_BF16 ? prompt_tc_t<__nv_bfloat16>(p, st) : prompt_tc_t<__half>(p, st);
}

}  // namespace energon
