// Causal attention of packed prompts with grouped heads on the 5th-generation tensor cores
// (fp16, bf16).
//
//   o_j(s) = sum_{t <= s} exp(c q_j(s) . k(t) - lse_j(s)) v(t)
//
// An item is a tile of 128 queries of one (sequence, head).  Its keys and values pass by once in blocks
// of 64, with a running maximum and sum (M. Milakov, N. Gimelshein, Online normalizer calculation for softmax,
// 2018):
//   loader     one warp: announces the items, loads Q tiles and K and V blocks by TMA
//   products   one warp: S = Q K^T into TMEM (two buffers, up to two blocks ahead), O += P V with P
//              read from TMEM (over the columns of S)
//   softmax    four warps, a thread per query: row of S to registers, maximum, exponentials, P rounded to
//              16 bits back to TMEM.  O is rescaled only when the maximum grew by more than 2^8:
//              until then the exponentials are at most 2^8 (fp16: times 2^7), in range of both types, and
//              the common factor leaves with the sum.
//   scan       two warps: rows of V behind the sequence and values that are not finite are
//              zeroed in the blocks that cross the diagonal (there 0 * NaN would reach earlier
//              rows); the latter are noted and added to the rows that see them at the end.
// Two blocks share an SM, so that one's softmax runs under the other's products.  A block that is done with
// an item takes the next one of a block that has not started (cluster launch control): the loads
// and scores of the next item overlap the end of this one, and the hardware keeps balancing the load.
// On 64 requests of 1 to 256 tokens that took 172 us where a block per item took 277.
//
// One prompt of 8192 tokens, 32 heads of 128, 8 kv heads, bf16: 455 us, 1210 TFLOP/s, 0.88 of the
// sustained rate of a library matrix product here.  A step of 64 keys needs 640
// cycles of the tensor cores (384 for the scores, which read both operands from shared memory, 256 for the
// products with V) and 512 of the special function units (64 x 128 exponentials at 16 a cycle); taking a quarter of
// the exponentials on the FMA pipe measured slower.  Tried and slower: 128 keys per block with one buffer of
// scores (528 us), two tiles per block that share K and V (448 us there and 6 % faster with 96 kv heads, but 10 to
// 70 % slower on prompts below 128 tokens).
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
// log2 of the factor of fp16 probabilities: with GROW they fill its range, and those down to 2^-21 of the
// largest keep all their bits (without it many small ones together could vanish).  It leaves with the sum.
template <typename T>
constexpr float P_UP = std::is_same<T, __half>::value ? 7.0f : 0.0f;

constexpr int BN = 64;                  // keys per block

constexpr int SOFT = 4;                 // softmax warps; then the loader's, the products' and those that scan
constexpr int SCAN = 64;                // threads that scan V
constexpr int THREADS = SOFT * 32 + 64 + SCAN;
constexpr int READERS = SOFT + 1 + SCAN / 32;  // warps that follow the items
constexpr int SCANS = BM / BN;          // most blocks that cross the diagonal
constexpr int O_COL = 2 * BN;           // TMEM: two buffers of S, then O
constexpr int OUT = 32 * 128;           // bytes of a softmax warp's outputs on their way out

template <int HD>
struct TCfg {
    static constexpr int QT = HD / 64 * QBOX;         // bytes of a Q tile
    static constexpr int KT = HD * BN * 2;            // bytes of a K or V block
    static constexpr int RING = HD == 128 ? 2 : 4;    // buffers of K, and of V
    static constexpr int TILES = QT + 2 * RING * KT + SOFT * OUT;
    static constexpr int TMEM = 256;
};
constexpr int ITEMS = 4;  // items that the loader announces ahead

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
// Barrier of the softmax threads; true in all of them if `ok` is in all.
__device__ __forceinline__ bool softmax_sync(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok), "n"(SOFT * 32)
        : "memory");
    return r != 0;
}
// Barrier of the threads that scan; true in all of them if `ok` is in all.
template <int N>
__device__ __forceinline__ bool scan_sync(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 8, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok), "n"(N)
        : "memory");
    return r != 0;
}
// Three positions below 256 of 9 bits each; 256: none.  note_bad lowers one of them.
constexpr uint32_t NONE_BAD = 256u | 256u << 9 | 256u << 18;
__device__ __forceinline__ void note_bad(uint32_t* word, int kind, int at) {
    uint32_t old = *reinterpret_cast<volatile uint32_t*>(word);
    while ((int)(old >> 9 * kind & 511u) > at) {
        const uint32_t want = (old & ~(511u << 9 * kind)) | (uint32_t)at << 9 * kind;
        const uint32_t was = atomicCAS(word, old, want);
        if (was == old) break;
        old = was;
    }
}
// Asks for the place of a block that has not started (it will not start any more if granted): the
// hardware's own order of blocks, without their start.
__device__ __forceinline__ void ask_next_block(uint4* answer, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ bool next_block(const uint4* answer, int& x, int& y) {
    uint32_t got;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 r, [%3];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::y.b32.b128 %2, r;\n\t}"
        : "=r"(got), "=&r"(x), "=&r"(y)
        : "r"(smem_u32(answer))
        : "memory");
    return got != 0;
}
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
    float c;         // scale * log2(e)
};

// What a block's warps share beside the tiles.
template <int HD>
struct Aux {
    using C = TCfg<HD>;
    uint64_t q_full, q_empty, out_done, o_done, o_full, drain, s_full[2], p_full[2];
    uint64_t k_full[C::RING], k_empty[C::RING], v_full[C::RING], v_empty[C::RING];
    uint64_t v_in[C::RING];     // a block that is scanned has landed in this buffer
    uint64_t v_ok[SCANS];  // an item's first, second, ... such block is scanned
    uint64_t item_full[ITEMS], item_empty[ITEMS], answer_bar, pad;
    int4 items[ITEMS];
    uint4 answer;
    uint32_t tmem_slot;
    int dead, odd;       // odd: 1 + the last item with a value that is not finite in a scanned block
    uint32_t first[HD];  // there: the first keys whose value in this column is +inf, -inf, NaN
};

// One work item of a block.
struct PromptItem {
    int start, n, blk, head;  // first row and length of the sequence, tile, query head; n = 0: no more items
    __device__ __forceinline__ int q0() const { return blk * BM; }
    __device__ __forceinline__ int blocks() const { return (min(n, q0() + BM) + BN - 1) / BN; }  // of keys
    __device__ __forceinline__ int scan0() const { return q0() / BN; }  // first block with keys behind a query
};

template <typename T, int HD>
__global__ void __launch_bounds__(THREADS, 2)
prompt_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const PromptTcArgs a) {
    using C = TCfg<HD>;
    extern __shared__ __align__(1024) uint8_t base[];  // the tiles, swizzled in units of 1024 bytes, then Aux
    Aux<HD>& aux = *reinterpret_cast<Aux<HD>*>(base + C::TILES);
    auto& q_full = aux.q_full;
    auto& q_empty = aux.q_empty;
    auto& out_done = aux.out_done;
    auto& o_done = aux.o_done;
    auto& o_full = aux.o_full;
    auto& drain = aux.drain;
    auto& s_full = aux.s_full;
    auto& p_full = aux.p_full;
    auto& k_full = aux.k_full;
    auto& k_empty = aux.k_empty;
    auto& v_full = aux.v_full;
    auto& v_empty = aux.v_empty;
    auto& v_in = aux.v_in;
    auto& v_ok = aux.v_ok;
    auto& item_full = aux.item_full;
    auto& item_empty = aux.item_empty;
    auto& answer_bar = aux.answer_bar;
    auto& items = aux.items;
    auto& answer = aux.answer;
    auto& tmem_slot = aux.tmem_slot;
    auto& dead = aux.dead;
    auto& odd = aux.odd;
    auto& first = aux.first;
    const PromptArgs& p = a.p;
    if (block_stopped(p.status)) return;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    uint8_t* ring_k = base + C::QT;
    uint8_t* ring_v = ring_k + C::RING * C::KT;
    for (int i = tid; i < HD; i += THREADS) first[i] = NONE_BAD;
    if (tid == 0) {
        mbar_init(&q_full, 1), mbar_init(&q_empty, 1), mbar_init(&out_done, SOFT * 32);
        mbar_init(&o_done, 1), mbar_init(&o_full, 1), mbar_init(&drain, 1);
        for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_full[i], SOFT * 32);
        for (int i = 0; i < C::RING; ++i)
            mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1), mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], 1), mbar_init(&v_in[i], 1);
        for (int i = 0; i < SCANS; ++i) mbar_init(&v_ok[i], SCAN);
        for (int i = 0; i < ITEMS; ++i) mbar_init(&item_full[i], 1), mbar_init(&item_empty[i], READERS);
        mbar_init(&answer_bar, 1);
        dead = smem_u32(base) % 1024 != 0, odd = 0;
        fence_mbar_init();
    }
    if (warp == SOFT) {
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
    // TMEM is read, and work is issued, by whole warps: their lanes give up together
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    PromptItem it;
    // Item k of this block, which is there.  `leave`: this warp needs it no more.
    auto read_item = [&](int k, PromptItem& to, bool leave) {
        const int at = k % ITEMS;
        const volatile int4& v = items[at];
        const int4 w = make_int4(v.x, v.y, v.z, v.w);
        to.start = w.x, to.n = w.y, to.blk = w.z, to.head = w.w;
        __syncwarp();
        if (leave && lane == 0) mbar_arrive(&item_empty[at]);
    };
    auto item_there = [&](int k) { return wait_warp(&item_full[k % ITEMS], (k / ITEMS) & 1); };

    if (warp == SOFT) {
        // ---- loader: announces the items, loads Q, then K(0), K(1), V(0), K(2), V(1), ... of each
        int x = blockIdx.x, y = blockIdx.y, k = 0, nq = 0, nk = 0, nv = 0, asked = 0;  // n.: loads issued
        uint32_t ins = 0;  // bit i: parity of v_in[i]'s next use
        bool ok = dead == 0, more = true;
        if (lane == 0) tma_prefetch_desc(&tm_q), tma_prefetch_desc(&tm_k), tma_prefetch_desc(&tm_v);
        auto announce = [&](int4 w) {
            const int at = k % ITEMS;
            if (k >= ITEMS) ok = wait_warp(&item_empty[at], (k / ITEMS - 1) & 1);
            if (ok && lane == 0) {
                items[at] = w;
                mbar_arrive(&item_full[at]);
            }
            __syncwarp();
        };
        while (ok && more) {
            if (elect_one()) {
                mbar_arrive_expect_tx(&answer_bar, 16);
                ask_next_block(&answer, &answer_bar);
            }
            const int64_t lin = (int64_t)y * gridDim.x + x;  // heads pass by first
            if (lin == 0) check_rows(p.cu, p.batch, p.rows, p.status);
            int b, blk;
            auto count = [](int, int len) { return (len + BM - 1) / BM; };
            if (find_item(p.cu, p.batch, p.rows, (int)(lin / p.n_heads), count, b, blk)) {
                seq_rows(p.cu, b, p.rows, it.start, it.n);
                it.blk = (it.n + BM - 1) / BM - 1 - blk;  // the longest rows first
                it.head = (int)(lin % p.n_heads);
                announce(make_int4(it.start, it.n, it.blk, it.head));
                const int kvh = it.head / (p.n_heads / p.n_kv), nb = it.blocks(), scan0 = it.scan0();
                if (ok && k >= 1) ok = wait_warp(&q_empty, (k - 1) & 1);
                if (ok && elect_one()) {
                    mbar_arrive_expect_tx(&q_full, C::QT);
                    for (int h = 0; h < HD / 64; ++h)
                        tma_load_2d(base + h * QBOX, &tm_q, &q_full, it.head * HD + 64 * h, it.start + it.q0());
                }
                if (ok) ++nq;
                for (int ik = 0, iv = 0; ok && iv < nb;) {
                    const bool keys = ik < nb && ik - iv < 2;
                    const int kb = keys ? ik : iv, g = keys ? nk : nv, at = g % C::RING;
                    if (g >= C::RING) ok = wait_warp(keys ? &k_empty[at] : &v_empty[at], (g / C::RING - 1) & 1);
                    if (!ok) break;
                    if (elect_one()) {
                        uint64_t* bar = keys ? &k_full[at] : &v_full[at];
                        if (!keys && kb >= scan0) {  // the scan waits for this one alone
                            mbar_arrive(bar);
                            bar = &v_in[at];
                        }
                        mbar_arrive_expect_tx(bar, C::KT);
                        for (int h = 0; h < HD / 64; ++h)
                            tma_load_2d((keys ? ring_k : ring_v) + at * C::KT + h * BN * 128, keys ? &tm_k : &tm_v, bar,
                                        kvh * HD + 64 * h, it.start + kb * BN);
                    }
                    if (keys) ++ik, ++nk;
                    else {
                        if (kb >= scan0) ins ^= 1u << at;
                        ++iv, ++nv;
                    }
                }
                ++k;
            }
            // the answer is waited for in any case: it must not land in a block that has ended
            const bool answered = __all_sync(0xffffffffu, mbar_wait_bounded(&answer_bar, asked & 1, nullptr, landing_limit(p.timeout_ns))) != 0;
            ++asked;
            if (!answered) *reinterpret_cast<volatile int*>(&dead) = 1, ok = false;
            more = answered && next_block(&answer, x, y);
            fence_proxy_async_smem();
            __syncwarp();
        }
        if (ok) announce(make_int4(0, 0, 0, 0));
        // All copies have landed before the block ends, also where a wait ran out.
        if (nq > 0) mbar_wait_bounded(&q_full, (nq - 1) & 1, nullptr, landing_limit(p.timeout_ns));
        for (int g = max(0, nk - C::RING); g < nk; ++g) mbar_wait_bounded(&k_full[g % C::RING], (g / C::RING) & 1, nullptr, landing_limit(p.timeout_ns));
        for (int g = max(0, nv - C::RING); g < nv; ++g) mbar_wait_bounded(&v_full[g % C::RING], (g / C::RING) & 1, nullptr, landing_limit(p.timeout_ns));
        for (int i = 0; i < C::RING; ++i)  // (an unused one passes: the phase before its first counts as done)
            mbar_wait_bounded(&v_in[i], (ins >> i & 1) ^ 1, nullptr, landing_limit(p.timeout_ns));
    } else if (warp == SOFT + 1) {
        // ---- products: the whole warp follows, one lane issues.  The scores run up to two blocks
        // ahead of the products with V, over the ends of items; whichever of the two can go on does (the
        // next item's Q may still be on its way when the last products of this one are due).
        constexpr uint32_t fmt = std::is_same<T, __half>::value ? 0u : 1u;
        constexpr uint32_t idesc_s = idesc_f16(fmt, BM, BN, 0), idesc_o = idesc_f16(fmt, BM, HD, 1);
        auto there = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)) != 0; };
        // the scores: item, its block, block in all; has: the item is read
        PromptItem ahead = it;
        int a_item = 0, a_kb = 0, a_nb = 0, a_x = 0;
        bool end = false, has = false;
        // the products with V: the same
        int k = 0, kb = 0, nb = 0, scan0 = 0, x = 0;
        uint32_t ins = 0, scans = 0;  // parities of the next uses of v_in, v_ok
        uint64_t since = 0;
        for (uint32_t idle = 0;;) {
            bool moved = false;
            if (!end && !has && there(&item_full[a_item % ITEMS], (a_item / ITEMS) & 1)) {
                read_item(a_item, ahead, false);
                end = ahead.n == 0;
                has = !end;
                a_nb = ahead.blocks(), a_kb = 0;
            }
            const int ka = a_x % C::RING;
            // (over the scores of the block two before: its products come first)
            if (has && a_x - x < 2 && (a_kb > 0 || there(&q_full, a_item & 1)) && there(&k_full[ka], (a_x / C::RING) & 1)) {
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t q = smem_u32(base), kk = smem_u32(ring_k + ka * C::KT);
#pragma unroll
                    for (int s = 0; s < HD / 16; ++s)
                        umma_f16(tmem + (a_x & 1) * BN, smem_desc_k128(q + (s >> 2) * QBOX) + 2 * (s & 3),
                                 smem_desc_k128(kk + (s >> 2) * BN * 128) + 2 * (s & 3), idesc_s, s > 0);
                    umma_commit(&s_full[a_x & 1]);
                    umma_commit(&k_empty[ka]);  // K's buffer is free once they are done, and after an item's last ones Q's
                    if (a_kb + 1 == a_nb) umma_commit(&q_empty);
                }
                __syncwarp();
                ++a_x;
                if (++a_kb == a_nb) has = false, ++a_item;
                moved = true;
            }
            if (x < a_x) {  // its scores are under way, so its item was announced
                if (kb == nb) {
                    read_item(k, it, true);
                    nb = it.blocks(), scan0 = it.scan0(), kb = 0, ++k;
                }
                const int at = x % C::RING, j = kb - scan0;
                if (there(&p_full[x & 1], (x >> 1) & 1) && there(&v_full[at], (x / C::RING) & 1) &&
                    (j < 0 || (there(&v_in[at], ins >> at & 1) && there(&v_ok[j], scans >> j & 1)))) {
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t v = smem_u32(ring_v + at * C::KT);
#pragma unroll
                        for (int s = 0; s < BN / 16; ++s)
                            umma_f16_tmem_a(tmem + O_COL, tmem + (x & 1) * BN + s * 8, smem_desc_mn128(v + s * 2048, BN * 128, 1024),
                                            idesc_o, kb > 0 || s > 0);
                        umma_commit(kb + 1 < nb ? &o_done : &o_full);
                        umma_commit(&v_empty[at]);
                    }
                    __syncwarp();
                    if (j >= 0) ins ^= 1u << at, scans ^= 1u << j;
                    ++kb, ++x;
                    moved = true;
                }
            } else if (end) {
                break;
            }
            if (moved) {
                idle = 0;
            } else if ((++idle & 31u) == 0) {
                const uint64_t now = global_ns();
                if (idle == 32) since = now;
                bool over = *reinterpret_cast<volatile int*>(&dead) != 0 || now - since > p.timeout_ns;
                over = __any_sync(0xffffffffu, over);
                if (over) {
                    *reinterpret_cast<volatile int*>(&dead) = 1;
                    break;
                }
            }
        }
        if (elect_one()) umma_commit(&drain);  // all products are done before the block ends
        mbar_wait_bounded(&drain, 0, nullptr, landing_limit(p.timeout_ns));
    } else if (warp > SOFT + 1) {
        // ---- scan of V
        constexpr uint32_t INF = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
        const int me = tid - (SOFT + 2) * 32;
        uint32_t ins = 0;
        bool ok = true;
        for (int k = 0, x = 0;; ++k) {
            // (its warps leave together: they meet at barriers)
            if (!scan_sync<SCAN>(ok && item_there(k))) break;
            read_item(k, it, true);
            if (it.n == 0) break;
            const int nb = it.blocks(), scan0 = it.scan0();
            // what was noted for the item before is read once its outputs are stored
            if (k > 0) ok = wait_warp(&out_done, (k - 1) & 1);
            if (!scan_sync<SCAN>(ok)) break;
            if (*reinterpret_cast<volatile int*>(&odd) == k)
                for (int d = me; d < HD; d += SCAN) first[d] = NONE_BAD;
            scan_sync<SCAN>(true);
            for (int kb = scan0; kb < nb; ++kb) {
                const int at = (x + kb) % C::RING;
                ok = wait_warp(&v_in[at], ins >> at & 1);
                ins ^= 1u << at;
                if (!ok) break;
                uint8_t* v = ring_v + at * C::KT;
                for (int r = me; r < BN; r += SCAN) {
                    const int t = kb * BN + r;
                    uint32_t most = 0;
                    if (t < it.n) {
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
                            note_bad(&first[d], (w & 0x7fffu) > INF ? 2 : w >> 15, t - scan0 * BN);
                            *e = 0;
                        }
                        odd = k + 1;
                    } else {
#pragma unroll
                        for (int ch = 0; ch < HD / 8; ++ch)
                            *reinterpret_cast<uint4*>(v + (ch >> 3) * BN * 128 + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&v_ok[kb - scan0]);
            }
            x += nb;
        }
    } else {
        // ---- softmax, one query per thread
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const uint32_t S0 = tmem + lanes, O = tmem + lanes + O_COL;
        uint32_t scans = 0;
        // g: blocks so far; done: products with V that were not an item's last
        bool ok = true;
        for (int k = 0, g = 0, done = 0;; ++k) {
            // the warps take an item, or leave, together: they meet at a barrier below
            if (!softmax_sync(ok && item_there(k))) break;
            read_item(k, it, true);
            if (it.n == 0) break;
            const int q0 = it.q0(), s = q0 + tid, nb = it.blocks(), scan0 = it.scan0();
            float m = -INFINITY, mc = 0.0f;  // the maximum that the exponentials refer to, and times c less P_UP (0 for -infinity)
            uint64_t sum[4] = {0, 0, 0, 0};  // pairs of partial sums (+0.0)
            for (int kb = 0; kb < nb; ++kb, ++g) {
                const uint32_t S = S0 + (g & 1) * BN;
                ok = wait_warp(&s_full[g & 1], (g >> 1) & 1);
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
                    mc = m == -INFINITY ? 0.0f : m * a.c - P_UP<T>;
                } else if (__any_sync(0xffffffffu, (mx - m) * a.c > GROW)) {
                    // O is at rest once the products of block kb - 1 are done; those of kb - 2 were before S,
                    // those of kb wait for this thread: the phase is the barrier's current or last one
                    ok = wait_warp(&o_done, (done + kb - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    float by = 1.0f;
                    if ((mx - m) * a.c > GROW) {
                        const float now = mx * a.c - P_UP<T>;
                        by = m == -INFINITY ? 0.0f : exp2_fast(mc - now);
                        m = mx, mc = now;
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
                mbar_arrive(&p_full[g & 1]);
            }
            if (ok) ok = wait_warp(&o_full, k & 1);
            // values that are not finite, as noted by the scan
            for (int kb = scan0; ok && kb < nb; ++kb) ok = wait_warp(&v_ok[kb - scan0], scans >> (kb - scan0) & 1);
            for (int kb = scan0; kb < nb; ++kb) scans ^= 1u << (kb - scan0);
            if (ok) {
                tc_fence_after();
                const float2 l2 = one_by_one(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                const float l = l2.x + l2.y, inv = 1.0f / l;
                const bool fix = *reinterpret_cast<volatile int*>(&odd) == k + 1;
                // O / l, rounded, 64 columns at a time through the warp's own shared memory (swizzled like the
                // tiles), so that 8 lanes write 128 bytes of one row
                uint8_t* stage = ring_v + C::RING * C::KT + warp * OUT;
                const int row0 = q0 + warp * 32, rows = min(32, it.n - row0);
                T* to = static_cast<T*>(p.o) + (int64_t)(it.start + row0) * p.ld_o + (int64_t)it.head * HD;
#pragma unroll 1
                for (int h = 0; h < HD / 64; ++h) {
                    uint32_t o[64];
                    tmem_ld_x32(O + 64 * h, o);
                    tmem_ld_x32(O + 64 * h + 32, o + 32);
                    tmem_wait_ld_regs(o);
                    tmem_wait_ld_regs(o + 32);
#pragma unroll
                    for (int e = 0; e < 64; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
                    if (fix) {
                        const int at = s - scan0 * BN;
#pragma unroll
                        for (int e = 0; e < 64; ++e) {
                            const uint32_t w = *reinterpret_cast<const volatile uint32_t*>(&first[64 * h + e]);
                            float f = __uint_as_float(o[e]);
                            if (at >= (int)(w & 511u)) f += INFINITY;
                            if (at >= (int)(w >> 9 & 511u)) f -= INFINITY;
                            if (at >= (int)(w >> 18)) f = NAN;
                            o[e] = __float_as_uint(f);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint4 w;
                        w.x = pack2<T>(__uint_as_float(o[8 * e]), __uint_as_float(o[8 * e + 1]));
                        w.y = pack2<T>(__uint_as_float(o[8 * e + 2]), __uint_as_float(o[8 * e + 3]));
                        w.z = pack2<T>(__uint_as_float(o[8 * e + 4]), __uint_as_float(o[8 * e + 5]));
                        w.w = pack2<T>(__uint_as_float(o[8 * e + 6]), __uint_as_float(o[8 * e + 7]));
                        *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = w;
                    }
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = 4 * e + (lane >> 3), ch = lane & 7;
                        if (r < rows)
                            *reinterpret_cast<uint4*>(to + r * p.ld_o + 64 * h + ch * 8) =
                                *reinterpret_cast<const uint4*>(stage + r * 128 + ((ch ^ (r & 7)) << 4));
                    }
                    __syncwarp();
                }
                tc_fence_before();  // the next item's products write over O
                if (s < it.n && p.lse != nullptr) p.lse[(int64_t)it.head * p.rows + it.start + s] = (mc + log2f(l)) * LN2;
                done += nb - 1;
            }
            mbar_arrive(&out_done);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && dead) status_or(p.status, ENERGON_DEVICE_TIMEOUT);
    if (warp == SOFT) tmem_dealloc(tmem, C::TMEM);
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

template <typename T, int HD>
static cudaError_t prompt_tc(const PromptArgs& p, cudaStream_t st) {
    using C = TCfg<HD>;
    constexpr int SMEM = C::TILES + (int)sizeof(Aux<HD>);
    static_assert(2 * (SMEM + 1024) <= 228 * 1024, "the blocks of an SM share its memory");
    CUtensorMap q, k, v;
    const int64_t wq = (int64_t)p.n_heads * HD, wk = (int64_t)p.n_kv * HD;
    cudaError_t e = rows_map(&q, p.dtype, p.q, wq, p.rows, p.ld_q, BM);
    if (e == cudaSuccess) e = rows_map(&k, p.dtype, p.k, wk, p.rows, p.ld_k, BN);
    if (e == cudaSuccess) e = rows_map(&v, p.dtype, p.v, wk, p.rows, p.ld_v, BN);
    if (e == cudaSuccess) e = prepare_smem((const void*)prompt_tc_kernel<T, HD>, SMEM);
    if (e != cudaSuccess) return e;
    PromptTcArgs a;
    a.p = p;
    a.c = p.scale * LOG2E;
    const int most = p.rows / BM + (p.batch < p.rows ? p.batch : p.rows);
    const dim3 grid(most, p.n_heads);  // (heads pass by first: see the kernel)
    prompt_tc_kernel<T, HD><<<grid, THREADS, SMEM, st>>>(q, k, v, a);
    return cudaGetLastError();
}

cudaError_t launch_prompt_tc(const PromptArgs& p, cudaStream_t st) {
    if (p.dtype == ENERGON_BF16)
        return p.head_dim == 64 ? prompt_tc<__nv_bfloat16, 64>(p, st) : prompt_tc<__nv_bfloat16, 128>(p, st);
    return p.head_dim == 64 ? prompt_tc<__half, 64>(p, st) : prompt_tc<__half, 128>(p, st);
}

}  // namespace energon
