// swa_decode_prefix.cu -- the shared prefix of a batch's decode attention, once for all sequences, on
// Blackwell tensor cores (tcgen05 MMA with TMEM accumulators, pages fetched by TMA): bf16, d = 128.
//
// One query token per sequence makes decode attention a product of a vector with every key, bound by HBM.
// Over a prefix that the batch shares, the queries of all sequences (and of the heads of a group) stand
// against the same keys: a tile of 128 of them turns the work into matrix products, and every key and
// value crosses HBM once for the batch instead of once per sequence.
//
// CTA = (loop, key head, tile of whole sequences) x one split of the blocks of 64 keys that all sequences of
// the tile see (swa_decode_common.cuh; the rest of each sequence's keys is the other kernel's).  So no
// score needs a mask.  Per block j:
//     S  = Q K_j^T          M = 128 queries, N = 64 keys, K = 128
//     P  = exp2(x - m)      x = log2(e) scale S; m raised only when a block exceeds it by more than 8
//     O += P V_j            three times: P as three bf16 numbers, all 24 bits of the weights; A from tensor memory,
//                           the third one's from shared memory
// The tensor core cuts every sum to fp32 instead of rounding it, towards zero each time: over 57 blocks with twelve sums each
// O lost about 2^-15 of itself.  So after every four blocks (a run) O goes to global memory, where it is added
// to the runs before rounded to nearest, and starts from zero.  O, m and the row sums go out as a partial result.
//
// Warps: 0 producer, 1 MMA issuer, 2-5 softmax (a query row per thread).  113 KB of shared memory and 256
// TMEM columns, 168 registers (60 bytes of a thread are in local memory around the rare calls): two CTAs per SM, one's
// softmax under the other's products.  Every wait is bounded; on a
// timeout the CTA records it, drains its copies and MMAs, frees TMEM and exits.
//
// 4 x 64 sequences of 16 heads over 4, 32,768 shared tokens, and up to 1,500 of their own: 287 us in all.  With two parts
// of P (the second rounded) and one run it takes 226, and the outputs are twice as far from those of fp32 arithmetic (their
// bf16 roundings fall the other way 4 times as often); the third part costs 36 us, the runs 25 (their sums added by read and
// write instead of in place: 42; runs of 16 blocks in place of 4: 15).  The softmax's own chain per block is what the
// kernel waits for.  Eight softmax warps spilled their registers and took longer.  Every sequence on its own from
// HBM: 2,595 us in all.
#include <cuda.h>
#include <cuda_runtime.h>

#include "gdr_nvtx.h"
#include "gdr_tc_common.cuh"
#include "gdr_tma_host.h"
#include "sm100_primitives.cuh"
#include "swa_decode_common.cuh"

namespace lt2 {
namespace swap {

using namespace sm100;
using namespace tcc;
using namespace swad;

constexpr int kBM = 128;               // query rows of a tile
constexpr int kBN = 64;                // keys of a block
constexpr int kThreads = 192;
constexpr int kRun = kPrefixRun;       // blocks of a run
constexpr uint64_t kTimeoutNs = kWaitTimeoutNs;

// Shared memory (offsets from a 1024-byte aligned base), 128-byte swizzled panels of 64 bf16 columns.
constexpr uint32_t Q_PANEL = kBM * 128;
constexpr uint32_t KV_PANEL = kBN * 128;
constexpr uint32_t KV_STAGE = 2 * KV_PANEL;
constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_K = OFF_Q + 2 * Q_PANEL;
constexpr uint32_t OFF_V = OFF_K + 2 * KV_STAGE;
constexpr uint32_t OFF_P = OFF_V + 2 * KV_STAGE;       // the third part of P: a panel of 64 columns
constexpr uint32_t PANEL_BYTES = OFF_P + Q_PANEL;
// S, P and O have one place each, so every barrier is at most one phase ahead of its waiter: P_j is written
// after O += P_{j-1} V is done, which the issuer started after it had seen P_{j-1}.
enum Bar : uint32_t {
    B_Q = 0,          // Q written (128 threads)
    B_K_FULL = 1,     // [2] K of a stage landed
    B_K_EMPTY = 3,    // [2] Q K^T is done with a K stage
    B_V_FULL = 5,     // [2]
    B_V_EMPTY = 7,    // [2]
    B_S_FULL = 9,     // S = Q K^T done
    B_S_FREE = 10,    // the softmax warps have read S
    B_P_FULL = 11,    // the first parts of P written, and O rescaled when needed
    B_P_REST = 12,    // the other parts of P written
    B_PV_DONE = 13,   // O += P V done
    B_DRAIN = 14,
    B_COUNT = 15
};
// The barriers and words lie in what the alignment leaves, in front of the panels where they fit there, else behind:
// so two CTAs take all 228 KB of an SM.
constexpr uint32_t OFF_BAR = 0;
constexpr uint32_t OFF_TMEM_SLOT = OFF_BAR + B_COUNT * 8;
constexpr uint32_t OFF_ABORT = OFF_TMEM_SLOT + 16;
constexpr uint32_t WORD_BYTES = OFF_ABORT + 16;
constexpr uint32_t SMEM_BYTES = PANEL_BYTES + 1024;
static_assert(2 * WORD_BYTES + 16 <= 1024, "the words fit in front of the panels or behind them");
static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");

// TMEM columns (lane = query row)
constexpr uint32_t TM_S = 0;           // S, fp32 (64 columns)
constexpr uint32_t TM_P = 64;          // P, bf16 pairs: the first parts in 32 columns, the second in 32
constexpr uint32_t TM_O = 128;         // O, fp32 (128 columns)
constexpr uint32_t TM_COLS = 256;

constexpr int NB_SOFT = 1;
constexpr int kSoftThreads = 128;

// Instruction descriptor, kind::f16 with bf16 A and B, fp32 D.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, int a_mn, int b_mn)
{
    return idesc_f16_f32(M, N, a_mn, b_mn) | (1u << 7) | (1u << 10);
}
constexpr uint32_t ID_QK = idesc_bf16_f32(kBM, kBN, 0, 0);
constexpr uint32_t ID_PV = idesc_bf16_f32(kBM, 128, 0, 1);

// `words`: where the barriers lie
__device__ __forceinline__ uint32_t bar_addr(uint32_t words, uint32_t i) { return words + OFF_BAR + 8u * i; }

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Row r of O times `corr`.
__device__ __noinline__ void rescale_o(uint32_t tm_o, float corr)
{
    #pragma unroll 1
    for (int piece = 0; piece < 4; ++piece) {
        float v[32];
        tmem_load32(tm_o + 32 * piece, v);
        #pragma unroll
        for (int d = 0; d < 32; ++d) v[d] *= corr;
        tmem_st32(tm_o + 32 * piece, v);
    }
    tmem_wait_st();
}
// ---- the sums between two runs --------------------------------------------------------------------
// `sums` is row r's place in the CTA's [column][row], so that a warp's lanes meet neighbouring words.  A place belongs to one
// thread, whose accesses keep their order.
__device__ __forceinline__ float load_sum(const float* p)
{
    float v;
    asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}
// Row r of O on top of the sums times `factor` (the first time: in their place); the result goes to the sums, or BACK to O.
template <bool BACK>
__device__ __noinline__ void add_run(uint32_t tm_o, float* sums, bool first, float factor)
{
    #pragma unroll 1
    for (int piece = 0; piece < 4; ++piece, sums += 32 * kBM) {
        float v[32], a[32];
        tmem_load32(tm_o + 32 * piece, v);
        #pragma unroll
        for (int d = 0; d < 32; ++d) a[d] = first ? 0.f : load_sum(sums + d * kBM);
        #pragma unroll
        for (int d = 0; d < 32; ++d) {
            v[d] = fmaf(a[d], factor, v[d]);
            if (!BACK) sums[d * kBM] = v[d];
        }
        if (BACK) tmem_st32(tm_o + 32 * piece, v);
    }
    if (BACK) tmem_wait_st();
}
// The same where the sums keep their size: added where they lie, without waiting for them.
__device__ __forceinline__ void add_run_in_place(uint32_t tm_o, float* sums)
{
    #pragma unroll 1
    for (int piece = 0; piece < 2; ++piece, sums += 64 * kBM) {
        float v[64];
        tmem_load_2x32(tm_o + 64 * piece, tm_o + 64 * piece + 32, v);
        #pragma unroll
        for (int d = 0; d < 64; ++d)
            asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(sums + d * kBM), "f"(v[d]) : "memory");
    }
}
// Row r of O to global memory (null: nowhere).
__device__ __noinline__ void write_partial(uint32_t tm_o, float* to)
{
    #pragma unroll 1
    for (int piece = 0; piece < 4; ++piece) {
        float v[32];
        tmem_load32(tm_o + 32 * piece, v);
        if (to) {
            #pragma unroll
            for (int d4 = 0; d4 < 32; d4 += 4)
                *reinterpret_cast<float4*>(to + 32 * piece + d4) = make_float4(v[d4], v[d4 + 1], v[d4 + 2], v[d4 + 3]);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 2)
swa_decode_prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ swad::Params p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;
    const uint32_t sw = sb - raw >= WORD_BYTES + 16 ? (raw + 15u) & ~15u : sb + PANEL_BYTES;     // barriers and words
    uint8_t* words = smem_raw + (sw - raw);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(words + OFF_ABORT);
    const DecodeCall& c = p.c;
    unsigned int* err = c.err;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    allow_next_loop_to_start();                            // the other kernel reads none of this one's results

    // blockIdx.x = ((tau * Hkv + h) * tiles + tile) * prefix_splits + split
    unsigned id = blockIdx.x;
    const int split = id % p.plan.prefix_splits;
    id /= p.plan.prefix_splits;
    const int tile = id % p.plan.tiles;
    id /= p.plan.tiles;
    const int64_t h = id % c.Hkv, tau = id / c.Hkv;
    const int G = static_cast<int>(c.Hq / c.Hkv);
    const int64_t b0 = static_cast<int64_t>(tile) * p.plan.seqs_per_tile;
    const int seqs = c.B - b0 < p.plan.seqs_per_tile ? static_cast<int>(c.B - b0) : p.plan.seqs_per_tile;
    const int rows = seqs * G;

    int64_t lo, hi;
    common_range(c, b0, b0 + seqs, lo, hi);
    const int64_t blocks = (hi - lo) / kBN;
    const int64_t share = (blocks + p.plan.prefix_splits - 1) / p.plan.prefix_splits;
    const int64_t j0 = split * share < blocks ? split * share : blocks;
    const int nblk = static_cast<int>(j0 + share < blocks ? share : blocks - j0);
    // row r of the tile: sequence b0 + r / G, query head h G + r % G
    auto row_of = [&](int r) { return (tau * c.B + b0 + r / G) * c.Hq + h * G + r % G; };
    if (nblk <= 0) {
        for (int r = threadIdx.x; r < rows; r += kThreads)
            p.ml[row_of(r) * p.slots + split] = make_float2(-INFINITY, 0.f);
        return;
    }
    const int64_t first = lo + j0 * kBN;
    // the pages of the prefix, from the table row of a sequence of the tile that reaches into it
    int64_t ref = b0;
    {
        bool found = false;
        for (int64_t b = b0; b < b0 + seqs && !found; b += 32) {
            int64_t bl = 0, n = 0;
            if (b + lane < b0 + seqs) key_range(c, b + lane, bl, n);
            const unsigned any = __ballot_sync(0xffffffffu, n > 0);
            if (any) {
                ref = b + __ffs(any) - 1;
                found = true;
            }
        }
    }
    const int32_t* table = c.page_table + ref * c.max_pages;
    const int box_shift = c.page_shift < 6 ? c.page_shift : 6;      // rows of a copy: a page, 64 at most
    const int nbox = kBN >> box_shift;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (uint32_t b = 0; b < B_COUNT; ++b)
            mbar_init(bar_addr(sw, b), b == B_Q || b == B_S_FREE || b == B_P_FULL || b == B_P_REST ? kSoftThreads : 1);
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(sw + OFF_TMEM_SLOT, TM_COLS);
        tmem_relinquish();
        if (lane == 0) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(words + OFF_TMEM_SLOT);

    if (warp == 0) {
        // ================= TMA producer: K_j, then V_{j-1}, as the MMAs free their stages =================
        uint32_t leader = 0;
        int k_issued = 0, v_issued = 0;
        auto load = [&](bool is_v, int j) -> bool {
            const int s = j & 1;
            // the block's pages: lane i has the one of copy i
            const int64_t pos = first + static_cast<int64_t>(j) * kBN + (static_cast<int64_t>(lane) << box_shift);
            int z = 0, y = 1 << c.page_shift;              // past the page: zeros
            if (lane < nbox) {
                const int32_t page = table[pos >> c.page_shift];
                if (page < 0 || page >= c.pages) {
                    atomicOr(err, kDevPages);
                } else {
                    z = static_cast<int>((tau * c.pages + page) * c.Hkv + h);
                    y = static_cast<int>(pos & ((int64_t(1) << c.page_shift) - 1));
                }
            }
            const uint32_t empty = bar_addr(sw, (is_v ? B_V_EMPTY : B_K_EMPTY) + s);
            if (!mbar_wait(empty, ((j >> 1) & 1) ^ 1, abort_flag, err, kTimeoutNs)) return false;
            const uint32_t fb = bar_addr(sw, (is_v ? B_V_FULL : B_K_FULL) + s);
            const uint32_t st = sb + (is_v ? OFF_V : OFF_K) + s * KV_STAGE;
            __syncwarp();
            if (elect_one(leader)) mbar_arrive_expect_tx(fb, KV_STAGE);
            __syncwarp();
            for (int i = 0; i < nbox; ++i) {
                const int zi = __shfl_sync(0xffffffffu, z, i), yi = __shfl_sync(0xffffffffu, y, i);
                const uint32_t at = st + (static_cast<uint32_t>(i) << box_shift) * 128u;
                if (elect_one(leader)) {
                    tma_load_3d(at, is_v ? &tm_v : &tm_k, 0, yi, zi, fb);
                    tma_load_3d(at + KV_PANEL, is_v ? &tm_v : &tm_k, 64, yi, zi, fb);
                }
                __syncwarp();
            }
            return true;
        };
        for (int j = 0; j <= nblk; ++j) {
            if (j < nblk) {
                if (!load(false, j)) break;
                k_issued = j + 1;
            }
            if (j > 0) {
                if (!load(true, j - 1)) break;
                v_issued = j;
            }
        }
        if (lane == 0 && *abort_flag) {
            // the copies in flight land before the CTA's memory goes away
            for (int j = k_issued - 2 < 0 ? 0 : k_issued - 2; j < k_issued; ++j)
                mbar_wait(bar_addr(sw, B_K_FULL + (j & 1)), (j >> 1) & 1, abort_flag, err, kTimeoutNs / 4);
            for (int j = v_issued - 2 < 0 ? 0 : v_issued - 2; j < v_issued; ++j)
                mbar_wait(bar_addr(sw, B_V_FULL + (j & 1)), (j >> 1) & 1, abort_flag, err, kTimeoutNs / 4);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA issuer =================
        uint32_t issuer = 0;
        bool issued_any = false;
        bool ok = mbar_wait(bar_addr(sw, B_Q), 0, abort_flag, err, kTimeoutNs);
        auto issue_pv = [&](int j) -> bool {
            if (!mbar_wait(bar_addr(sw, B_V_FULL + (j & 1)), (j >> 1) & 1, abort_flag, err, kTimeoutNs) ||
                !mbar_wait(bar_addr(sw, B_P_FULL), j & 1, abort_flag, err, kTimeoutNs))
                return false;
            tc_fence_after();
            if (elect_one(issuer)) {
                const uint32_t vt = sb + OFF_V + (j & 1) * KV_STAGE;
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_f16_tmem_a(tmem + TM_O, tmem + TM_P + 8 * k, smem_desc_sw128(vt + k * 2048, KV_PANEL, 1024), ID_PV,
                                    (j % kRun > 0 || k > 0) ? 1u : 0u);
            }
            if (!mbar_wait(bar_addr(sw, B_P_REST), j & 1, abort_flag, err, kTimeoutNs)) return false;
            tc_fence_after();
            if (elect_one(issuer)) {
                const uint32_t vt = sb + OFF_V + (j & 1) * KV_STAGE;
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_f16_tmem_a(tmem + TM_O, tmem + TM_P + 32 + 8 * k, smem_desc_sw128(vt + k * 2048, KV_PANEL, 1024),
                                    ID_PV, 1u);
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_f16(tmem + TM_O, smem_desc_sw128(sb + OFF_P + k * 32, 16, 1024),
                             smem_desc_sw128(vt + k * 2048, KV_PANEL, 1024), ID_PV, 1u);
                umma_commit(bar_addr(sw, B_PV_DONE));
                umma_commit(bar_addr(sw, B_V_EMPTY + (j & 1)));
            }
            return true;
        };
        for (int j = 0; ok && j < nblk; ++j) {
            if (!mbar_wait(bar_addr(sw, B_K_FULL + (j & 1)), (j >> 1) & 1, abort_flag, err, kTimeoutNs) ||
                (j > 0 && !mbar_wait(bar_addr(sw, B_S_FREE), (j - 1) & 1, abort_flag, err, kTimeoutNs))) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (elect_one(issuer)) {
                const uint32_t kt = sb + OFF_K + (j & 1) * KV_STAGE;
                #pragma unroll
                for (int k = 0; k < 8; ++k)
                    umma_f16(tmem + TM_S, smem_desc_sw128(sb + OFF_Q + (k >> 2) * Q_PANEL + (k & 3) * 32, 16, 1024),
                             smem_desc_sw128(kt + (k >> 2) * KV_PANEL + (k & 3) * 32, 16, 1024), ID_QK, k > 0);
                umma_commit(bar_addr(sw, B_S_FULL));
                umma_commit(bar_addr(sw, B_K_EMPTY + (j & 1)));
            }
            issued_any = true;
            if (j > 0 && !issue_pv(j - 1)) ok = false;
        }
        if (ok) ok = issue_pv(nblk - 1);
        if (issued_any && !ok && lane == issuer) {
            // every MMA this thread issued completes before TMEM is released
            umma_commit(bar_addr(sw, B_DRAIN));
            mbar_wait(bar_addr(sw, B_DRAIN), 0, abort_flag, err, kTimeoutNs / 4);
        }
        __syncwarp();
    } else {
        // ================= softmax and output (query row r, TMEM lane r) =================
        const int q4 = warp & 3;
        const int r = 32 * q4 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(32 * q4) << 16;
        const int64_t row = r < rows ? row_of(r) : 0;
        // the row's query to its place in the swizzled panels; rows past the tile are zero
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.q) + row * 128);
        #pragma unroll
        for (int k = 0; k < 16; ++k) {
            const uint4 v = r < rows ? q[k] : make_uint4(0u, 0u, 0u, 0u);
            sts128(sw128(sb + OFF_Q + (k >> 3) * Q_PANEL, r, k & 7), v);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar_addr(sw, B_Q));

        float* const sums = p.between + static_cast<int64_t>(blockIdx.x) * (kBM * 128) + r;
        float m = -INFINITY, l = 0.f, factor = 1.f;
        bool ok = true;
        for (int j = 0; j < nblk; ++j) {
            // keys of a page outside the cache are left out: which of the block's copies have one
            unsigned bad = 0;
            {
                const int64_t pos = first + static_cast<int64_t>(j) * kBN + (static_cast<int64_t>(lane) << box_shift);
                bool wrong = false;
                if (lane < nbox) {
                    const int32_t page = table[pos >> c.page_shift];
                    wrong = page < 0 || page >= c.pages;
                }
                bad = __ballot_sync(0xffffffffu, wrong);
            }
            if (j > 0 && j % kRun == 0) {                  // a run is done: O starts again
                mbar_wait(bar_addr(sw, B_PV_DONE), (j - 1) & 1, abort_flag, err, kTimeoutNs);
                tc_fence_after();
                if (j > kRun && __all_sync(0xffffffffu, factor == 1.f))
                    add_run_in_place(tmem + TM_O + lane_addr, sums);
                else
                    add_run<false>(tmem + TM_O + lane_addr, sums, j == kRun, factor);
            }
            const bool got = mbar_wait(bar_addr(sw, B_S_FULL), j & 1, abort_flag, err, kTimeoutNs);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float x[64];
            tmem_load_2x32(tmem + TM_S + lane_addr, tmem + TM_S + lane_addr + 32, x);
            tc_fence_before();
            mbar_arrive(bar_addr(sw, B_S_FREE));
            if (bad) {
                #pragma unroll
                for (int e = 0; e < kBN; ++e)
                    if ((bad >> (e >> box_shift)) & 1u) x[e] = -INFINITY;
            }
            float mx[4];
            #pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = max3(x[e], x[e + 4], x[e + 8]);
            #pragma unroll
            for (int e = 12; e < 60; e += 8) {
                #pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], x[e + i], x[e + 4 + i]);
            }
            const float bm = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], x[60], x[61]), fmaxf(x[62], x[63])) * p.xscale;
            const bool raise = bm > m + 8.f;
            const float mnew = raise ? bm : m;
            const float corr = raise && m != -INFINITY ? ex2(m - mnew) : 1.f;
            const float msub = mnew == -INFINITY ? 0.f : mnew;
            // (O is rescaled before the weights fill the registers; it is free once O += P_{j-1} V is done.)  The sums of
            // the runs before wait for their factor until the next run is added.
            if (j > 0 && j % kRun == 0) {
                factor = corr;
            } else if (__any_sync(0xffffffffu, corr != 1.f)) {
                if (j >= 1) mbar_wait(bar_addr(sw, B_PV_DONE), (j - 1) & 1, abort_flag, err, kTimeoutNs);
                tc_fence_after();
                rescale_o(tmem + TM_O + lane_addr, corr);
                factor *= corr;
            }
            // the softmax warps' instructions are what the kernel waits for most: pairs where there are paired ones
            const f2 scale2 = pack2(p.xscale, p.xscale), msub2 = pack2(-msub, -msub);
            f2 w[32], ps[2] = {0, 0};
            #pragma unroll
            for (int e = 0; e < 32; ++e) {
                float p0, p1;
                unpack2(fma2(pack2(x[2 * e], x[2 * e + 1]), scale2, msub2), p0, p1);
                w[e] = pack2(ex2(p0), ex2(p1));
                ps[e & 1] = add2(ps[e & 1], w[e]);
            }
            float s0, s1;
            unpack2(add2(ps[0], ps[1]), s0, s1);
            l = l * corr + (s0 + s1);
            m = mnew;
            // P is free once O += P_{j-1} V is done.  split_bf16, pair by pair: the first parts go to the MMA warp while
            // the others are made of what they leave.
            if (j >= 1) mbar_wait(bar_addr(sw, B_PV_DONE), (j - 1) & 1, abort_flag, err, kTimeoutNs);
            tc_fence_after();
            const f2 less2 = pack2(kLess, kLess), minus2 = pack2(-1.f, -1.f);
            const uint32_t tp = tmem + TM_P + lane_addr;
            // the next part of a pair of weights, and the rest in its place
            auto next_part = [&](f2& v) -> uint32_t {
                float h0, h1;
                unpack2(mul2(v, less2), h0, h1);
                v = fma2(pack2(cut_bf16(h0), cut_bf16(h1)), minus2, v);
                return upper_halves(h0, h1);
            };
            #pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t ph[16];
                #pragma unroll
                for (int e = 0; e < 16; ++e) ph[e] = next_part(w[16 * half + e]);
                tmem_st16(tp + 16 * half, ph);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar_addr(sw, B_P_FULL));
            #pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pm[16], pl[16];
                #pragma unroll
                for (int e = 0; e < 16; ++e) {
                    pm[e] = next_part(w[16 * half + e]);
                    float h0, h1;
                    unpack2(w[16 * half + e], h0, h1);
                    pl[e] = upper_halves(h0, h1);
                }
                tmem_st16(tp + 32 + 16 * half, pm);
                #pragma unroll
                for (int i = 0; i < 4; ++i)
                    sts128(sw128(sb + OFF_P, r, 4 * half + i), make_uint4(pl[4 * i], pl[4 * i + 1], pl[4 * i + 2], pl[4 * i + 3]));
            }
            fence_proxy_async_smem();
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar_addr(sw, B_P_REST));
        }
        const bool mine =
            ok && mbar_wait(bar_addr(sw, B_PV_DONE), (nblk - 1) & 1, abort_flag, err, kTimeoutNs);
        uint32_t all;
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                     "bar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(all) : "r"(mine ? 1u : 0u), "r"(NB_SOFT), "r"(kSoftThreads) : "memory");
        // a row whose only scores are NaN has no maximum; it must not count as a row without keys
        if (l != l && m == -INFINITY) m = 0.f;
        if (all) {
            tc_fence_after();
            if (nblk > kRun) add_run<true>(tmem + TM_O + lane_addr, sums, false, factor);
            write_partial(tmem + TM_O + lane_addr, r < rows ? p.acc + (row * p.slots + split) * 128 : nullptr);
        }
        if (r < rows) {
            // an empty sequence (an idle slot of the batch) has no keys here either
            int64_t bl, n;
            key_range(c, b0 + r / G, bl, n);
            p.ml[row * p.slots + split] = all && n > 0 ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, TM_COLS);
}

}  // namespace swap

cudaError_t launch_swa_decode_prefix(const swad::Params& p, cudaStream_t stream)
{
    using namespace swap;
    const DecodeCall& c = p.c;
    CUtensorMap mk, mv;
    const uint32_t box = c.page_shift < 6 ? 1u << c.page_shift : 64u;
    const int64_t units = c.T * c.pages * c.Hkv, size = int64_t(1) << c.page_shift;
    if (!make_bf16_map_3d(&mk, c.k_cache, units, size, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_bf16_map_3d(&mv, c.v_cache, units, size, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(swa_decode_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(SMEM_BYTES));
    if (e != cudaSuccess) return e;
    const int64_t grid = c.T * c.Hkv * p.plan.tiles * p.plan.prefix_splits;
    swa_decode_prefix_kernel<<<static_cast<unsigned>(grid), kThreads, SMEM_BYTES, stream>>>(mk, mv, p);
    return cudaGetLastError();
}

}  // namespace lt2
