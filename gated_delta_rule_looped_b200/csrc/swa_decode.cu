// swa_decode.cu -- decode attention over the paged cache: one query token per (loop, sequence, query
// head), the window of its sequence's last positions, keys and values shared by groups of query heads.
//
//     o = sum_s softmax_s(scale q . k_s) v_s,   s in [max(0, n - window), n)
//
// Every key and value is read once for the heads that share it, so the kernels are bound by HBM; a
// sequence's keys are split between CTAs (each keeps a running maximum and sum), and a second launch
// joins the partial results where there is more than one.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdr_nvtx.h"
#include "swa_decode_common.cuh"

namespace lt2 {
namespace swad {

constexpr int kThreads = 128;          // 4 warps (more where a CTA has an SM to itself), each with its own keys

// A row whose only scores are NaN has no maximum; it must not count as a row without keys.
__device__ __forceinline__ float seen(float m, float l) { return l != l && m == -INFINITY ? 0.f : m; }

// ---- bf16: warp-level products (m16n8k16) ---------------------------------------------------------
// CTA = (loop, sequence, key head, 16 of its query heads) x one split.  A warp of W takes every W-th tile of 16
// keys through a ring of its own (asynchronous copies, no barrier with the other warps): S = Q K^T with
// Q in registers, P = 2^(S - m), O += P V.  With at most 16 query rows the tensor core is far from busy;
// what counts is bytes in flight (8 KB per warp and stage at d = 128; two stages and three CTAs per SM read 5.9 TB/s of
// 4 x 64 x 16 windows of 512, 182 us, three stages and two CTAs 5.0 TB/s, 216 us).  A warp looks 32 tiles' pages up at once (4 x
// 32 x 4 key heads of 64: 140 us, page by page 162).  P enters the
// product as three bf16 numbers, which hold all its bits (swa_decode_common.cuh).  A group of up to 8 heads leaves the
// lower half of the 16 rows empty (R = 1): there the second parts take it, beside the first ones, and O is the sum of
// both halves in the end; so two products do, and half of the exponentials.  The tensor core cuts its fp32 sums
// instead of rounding them (O lost up to 2^-17 of itself over 64 tiles), so each tile's product starts from zero.
template <int DP> struct Ring {
    static constexpr int kHalf = 16 * DP * 2;            // 16 rows of K (or V), bytes
    static constexpr int kStage = 2 * kHalf;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <int DP, int W, int ST, int R>
__global__ void __launch_bounds__(32 * W) swa_decode_kernel(const __grid_constant__ Params p)
{
    constexpr int KS = DP / 16;                          // steps of 16 along d
    constexpr int CPR = DP / 8;                          // 16-byte chunks of a row
    constexpr int NL = 16 * CPR / 32;                    // chunks of K (and of V) that a lane copies per tile
    extern __shared__ __align__(128) uint8_t smem[];
    const DecodeCall& c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = static_cast<int>(c.Hq / c.Hkv);
    allow_next_loop_to_start();                          // the join, which waits for this kernel's end

    // blockIdx.x = ((tau * Hkv + h) * B + b) * group_tiles + row tile; blockIdx.y = split
    unsigned id = blockIdx.x;
    const int rt = id % p.plan.group_tiles;
    id /= p.plan.group_tiles;
    const int64_t b = id % c.B;
    id /= static_cast<unsigned>(c.B);
    const int64_t h = id % c.Hkv, tau = id / c.Hkv;
    const int split = blockIdx.y;
    const int rows = G - 16 * rt < 16 ? G - 16 * rt : 16;
    const int64_t row0 = (tau * c.B + b) * c.Hq + h * G + 16 * rt;
    if (split == 0 && rt == 0 && threadIdx.x == 0) {
        const int64_t n = c.lens[b];
        if (n < 0 || n > (c.max_pages << c.page_shift)) atomicOr(c.err, kDevSeqlens);
    }
    const OwnTiles t = own_tiles(c, p.plan, b);
    int64_t i0, i1;
    split_range(t.total, split, p.plan.own_splits, i0, i1);
    if (i0 >= i1) {
        // no keys in this split: an empty slot, or zeros where it is the only one
        for (int i = threadIdx.x; i < rows * (p.slots ? 1 : static_cast<int>(c.d)); i += 32 * W) {
            if (p.slots)
                p.ml[(row0 + i) * p.slots + p.plan.prefix_splits + split] = make_float2(-INFINITY, 0.f);
            else
                store_out(c.o, row0 * c.d + i, c.out_bf16, 0.f);
        }
        outlast_prefix(p.plan);
        return;
    }

    const uint32_t ring = sm100::smem_addr(smem) + warp * ST * Ring<DP>::kStage;
    const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(c.k_cache);
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(c.v_cache);
    const int32_t* table = c.page_table + b * c.max_pages;
    const int d = static_cast<int>(c.d);

    // The pages of the warp's tiles: lane j holds the one of tile j of 32.
    int64_t next = i0 + warp;                            // the tile to copy next
    int64_t listed = next + lane * W;
    auto list_page = [&]() {
        const int32_t page = listed < i1 ? table[t.pos(listed) >> c.page_shift] : 0;
        listed += 32 * W;
        return page;
    };
    int32_t pages = list_page();
    int at_page = 0;
    uint32_t bad = 0;                                    // one bit per copy, the last one lowest: no such page

    // copies tile `next` into its stage (nothing past the warp's last tile) and closes the group
    auto copy_tile = [&](int stage) {
        bad <<= 1;
        if (next < i1) {
            const int64_t pos = t.pos(next);
            const int64_t at = cache_row(c, tau, h, __shfl_sync(0xffffffffu, pages, at_page), pos);
            if (at < 0) bad |= 1;
            next += W;
            if (++at_page == 32) {
                at_page = 0;
                pages = list_page();
            }
            const uint32_t dst = ring + stage * Ring<DP>::kStage;
            #pragma unroll
            for (int j = 0; j < NL; ++j) {
                const int q = lane + 32 * j;
                const int key = q / CPR, ch = q % CPR;
                // keys outside the range become zeros: a weight of zero must not meet a NaN there
                const bool in = at >= 0 && pos + key >= t.lo && pos + key < t.n && ch * 8 < d;
                const int64_t off = in ? at + static_cast<int64_t>(key) * d + ch * 8 : 0;
                const uint32_t to = dst + key * (DP * 2) + ((ch ^ (key & 7)) << 4);
                cp_async16(to, kc + off, in ? 16u : 0u);
                cp_async16(to + Ring<DP>::kHalf, vc + off, in ? 16u : 0u);
            }
        }
        cp_async_commit();
    };
    #pragma unroll
    for (int s = 0; s < ST - 1; ++s) copy_tile(s);

    // Q: the A operand of S = Q K^T, rows past the group zero
    uint32_t qa[KS][4];
    {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(c.q) + row0 * d);
        const int r = lane >> 2, e = 2 * (lane & 3);
        #pragma unroll
        for (int k = 0; k < KS; ++k) {
            #pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int rr = r + (f & 1) * 8, ee = 16 * k + e + (f >> 1) * 8;
                qa[k][f] = rr < rows && ee < d ? q[(rr * d + ee) >> 1] : 0u;
            }
        }
    }
    float o[2 * KS][4];
    #pragma unroll
    for (int k = 0; k < 2 * KS; ++k)
        #pragma unroll
        for (int f = 0; f < 4; ++f) o[k][f] = 0.f;
    float m[R], l[R];
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
    }

    int stage = 0;
    for (int64_t i = i0 + warp; i < i1; i += W) {
        cp_async_wait<ST - 2>();
        __syncwarp();
        copy_tile(stage == 0 ? ST - 1 : stage - 1);      // the stage of the tile before this one
        const uint32_t kt = ring + stage * Ring<DP>::kStage, vt = kt + Ring<DP>::kHalf;
        stage = stage + 1 == ST ? 0 : stage + 1;

        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        #pragma unroll
        for (int k = 0; k < KS; ++k) {
            const uint32_t key = (lane & 7) + ((lane >> 4) & 1) * 8, ch = 2 * k + ((lane >> 3) & 1);
            uint32_t bf[4];
            sm100::ldsm_x4(kt + key * (DP * 2) + ((ch ^ (key & 7)) << 4), bf);
            mma_bf16(s[0], qa[k], bf[0], bf[1]);
            mma_bf16(s[1], qa[k], bf[2], bf[3]);
        }
        const int64_t pos = t.pos(i);
        const int64_t off = t.lo - pos, end = t.n - pos;
        const int c_lo = off > 0 ? static_cast<int>(off) : 0;
        const int c_hi = bad >> (ST - 1) & 1 ? 0 : end < 16 ? static_cast<int>(end) : 16;
        #pragma unroll
        for (int j = 0; j < 2; ++j)
            #pragma unroll
            for (int f = 0; f < 2 * R; ++f) {
                const int col = 8 * j + 2 * (lane & 3) + (f & 1);
                s[j][f] = col >= c_lo && col < c_hi ? s[j][f] * p.xscale : -INFINITY;
            }
        // the reference maximum of a row is raised only when a tile exceeds it by more than 8 (so
        // weights stay below 2^8); O and the sum then shrink
        float corr[R];
        bool raised = false;
        #pragma unroll
        for (int r = 0; r < R; ++r) {
            float bm = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2));
            corr[r] = 1.f;
            if (bm > m[r] + 8.f) {
                corr[r] = ex2(m[r] - bm);                // 0 for the first keys
                m[r] = bm;
                raised = true;
            }
        }
        if (__any_sync(0xffffffffu, raised)) {
            #pragma unroll
            for (int r = 0; r < R; ++r) l[r] *= corr[r];
            #pragma unroll
            for (int k = 0; k < 2 * KS; ++k) {
                o[k][0] *= corr[0];
                o[k][1] *= corr[0];
                o[k][2] *= corr[R - 1];
                o[k][3] *= corr[R - 1];
            }
        }
        uint32_t ph[4], pm[4], pl[4];
        #pragma unroll
        for (int j = 0; j < 2; ++j)
            #pragma unroll
            for (int r = 0; r < R; ++r) {
                const float ms = m[r] == -INFINITY ? 0.f : m[r];
                const float p0 = ex2(s[j][2 * r] - ms), p1 = ex2(s[j][2 * r + 1] - ms);
                l[r] += p0 + p1;
                if constexpr (R == 1) {
                    split_bf16(p0, p1, ph[2 * j], ph[2 * j + 1], pl[2 * j], 0.5f);
                    pl[2 * j + 1] = pl[2 * j];
                } else {
                    split_bf16(p0, p1, ph[2 * j + r], pm[2 * j + r], pl[2 * j + r], 1.f);
                }
            }
        #pragma unroll
        for (int k = 0; k < KS; ++k) {
            const uint32_t key = (lane & 7) + ((lane >> 3) & 1) * 8, ch = 2 * k + (lane >> 4);
            uint32_t bf[4];
            sm100::ldsm_x4_trans(vt + key * (DP * 2) + ((ch ^ (key & 7)) << 4), bf);
            // the tensor core cuts its sums, so a tile's product starts from zero and is added to O rounded to nearest
            float t[2][4];
            #pragma unroll
            for (int n = 0; n < 2; ++n) {
                mma_bf16_first(t[n], pl, bf[2 * n], bf[2 * n + 1]);
                if constexpr (R == 2) mma_bf16(t[n], pm, bf[2 * n], bf[2 * n + 1]);
                mma_bf16(t[n], ph, bf[2 * n], bf[2 * n + 1]);
                #pragma unroll
                for (int f = 0; f < 4; ++f) o[2 * k + n][f] += t[n][f];
            }
        }
        __syncwarp();                                    // every lane is done with the stage
    }
    cp_async_wait<0>();
    if constexpr (R == 1) {
        #pragma unroll
        for (int k = 0; k < 2 * KS; ++k) {
            o[k][0] += o[k][2];
            o[k][1] += o[k][3];
        }
    }
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        m[r] = seen(m[r], l[r]);
    }
    __syncthreads();                                     // the rings are free

    float* so = reinterpret_cast<float*>(smem);          // [W][16][DP]
    float2* sm = reinterpret_cast<float2*>(smem + W * 16 * DP * 4);
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = (lane >> 2) + 8 * r;
        if ((lane & 3) == 0) sm[warp * 16 + row] = make_float2(m[r], l[r]);
        if (row < rows) {
            #pragma unroll
            for (int k = 0; k < 2 * KS; ++k)
                *reinterpret_cast<float2*>(&so[(warp * 16 + row) * DP + 8 * k + 2 * (lane & 3)]) =
                    make_float2(o[k][2 * r], o[k][2 * r + 1]);
        }
    }
    __syncthreads();
    join_warps<16, DP, W>(p, sm, so, rows, row0, p.plan.prefix_splits + split);
    outlast_prefix(p.plan);
}

// ---- fp32 arithmetic on CUDA cores, any width up to 256 ---------------------------------------------
// CTA = (loop, sequence, key head, R of its query heads) x one split; a warp takes every fourth tile of 16
// keys, four keys and their values at a time, lane j holding E elements of every row, in pieces of V.  fp32
// inputs, and bf16 ones of a width that is no multiple of 8.  With R and E no larger than the call needs, and a
// piece's keys and values on their way together, 4 x 16 x 16 windows of up to 4,096 keys of 128 floats take 457 us
// (6.1 TB/s), one after the other at R = 4 and E = 8 860; with 8 heads a key the arithmetic counts (2 x 16 x 4 such
// key heads: 170 us, HBM 53; R = 8 leaves too few warps, 205).
constexpr int kRowsCc = 4;             // query heads of a CTA at most

template <typename T, int V, int E>
__device__ __forceinline__ void load_row(const T* row, int lane, int d, float (&x)[E])
{
    #pragma unroll
    for (int j = 0; j < E / V; ++j) {
        const int e = (lane + 32 * j) * V;
        if constexpr (V == 4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (e < d) {
                if (sizeof(T) == 4) {
                    v = *reinterpret_cast<const float4*>(row + e);
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(row + e);
                    v = make_float4(sm100::bf16_lo(w.x), sm100::bf16_hi(w.x), sm100::bf16_lo(w.y), sm100::bf16_hi(w.y));
                }
            }
            x[4 * j] = v.x;
            x[4 * j + 1] = v.y;
            x[4 * j + 2] = v.z;
            x[4 * j + 3] = v.w;
        } else {
            x[j] = e < d ? to_f32<T>(row[e]) : 0.f;
        }
    }
}

// Sums each of N values over the warp's lanes, every lane getting all: each exchange halves what a lane still
// carries, so N values take N + N - 1 and a few shuffles more, not 5 N.
template <int N>
__device__ __forceinline__ void warp_sums(float (&x)[N], int lane)
{
    int s = 16;
    #pragma unroll
    for (int n = N / 2; n > 0; n /= 2, s >>= 1) {
        const bool upper = lane & s;
        #pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = upper ? x[i] : x[i + n], keep = upper ? x[i + n] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    }
    float v = x[0];
    #pragma unroll
    for (int r = 32 / N / 2; r > 0; r >>= 1) v += __shfl_xor_sync(0xffffffffu, v, r);
    #pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __shfl_sync(0xffffffffu, v, i * (32 / N));
}

template <typename T, int V, int E, int R>
__global__ void __launch_bounds__(kThreads) swa_decode_cc_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const DecodeCall& c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = static_cast<int>(c.Hq / c.Hkv);
    allow_next_loop_to_start();                          // the join, which waits for this kernel's end
    unsigned id = blockIdx.x;
    const int rt = id % p.plan.group_tiles;
    id /= p.plan.group_tiles;
    const int64_t b = id % c.B;
    id /= static_cast<unsigned>(c.B);
    const int64_t h = id % c.Hkv, tau = id / c.Hkv;
    const int split = blockIdx.y;
    const int rows = G - kRowsCc * rt < kRowsCc ? G - kRowsCc * rt : kRowsCc;
    const int64_t row0 = (tau * c.B + b) * c.Hq + h * G + kRowsCc * rt;
    if (split == 0 && rt == 0 && threadIdx.x == 0) {
        const int64_t n = c.lens[b];
        if (n < 0 || n > (c.max_pages << c.page_shift)) atomicOr(c.err, kDevSeqlens);
    }
    const OwnTiles t = own_tiles(c, p.plan, b);
    int64_t i0, i1;
    split_range(t.total, split, p.plan.own_splits, i0, i1);
    const int d = static_cast<int>(c.d);

    float q[R][E], a[R][E], m[R], l[R];
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        #pragma unroll
        for (int e = 0; e < E; ++e) q[r][e] = a[r][e] = 0.f;
        if (r < rows) load_row<T, V, E>(static_cast<const T*>(c.q) + (row0 + r) * d, lane, d, q[r]);
    }
    const int32_t* table = c.page_table + b * c.max_pages;
    for (int64_t i = i0 + warp; i < i1; i += 4) {
        const int64_t pos = t.pos(i);
        const int64_t at = cache_row(c, tau, h, table[pos >> c.page_shift], pos);
        if (at < 0) continue;
        const T* kr = static_cast<const T*>(c.k_cache) + at;
        const T* vr = static_cast<const T*>(c.v_cache) + at;
        for (int k0 = 0; k0 < 16; k0 += 4) {
            float key[4][E], val[4][E], x[4 * R];
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = pos + k0 + k >= t.lo && pos + k0 + k < t.n;      // the same for the warp
                #pragma unroll
                for (int e = 0; e < E; ++e) key[k][e] = val[k][e] = 0.f;
                if (in) {
                    load_row<T, V, E>(kr + static_cast<int64_t>(k0 + k) * d, lane, d, key[k]);
                    load_row<T, V, E>(vr + static_cast<int64_t>(k0 + k) * d, lane, d, val[k]);
                }
            }
            #pragma unroll
            for (int k = 0; k < 4; ++k)
                #pragma unroll
                for (int r = 0; r < R; ++r) {
                    float s = 0.f;
                    #pragma unroll
                    for (int e = 0; e < E; ++e) s = fmaf(q[r][e], key[k][e], s);
                    x[4 * r + k] = s;
                }
            warp_sums(x, lane);
            #pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r >= rows) break;
                float* xr = x + 4 * r;
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool in = pos + k0 + k >= t.lo && pos + k0 + k < t.n;
                    xr[k] = in ? xr[k] * p.xscale : -INFINITY;
                }
                const float bm = fmaxf(fmaxf(xr[0], xr[1]), fmaxf(xr[2], xr[3]));
                const float mn = fmaxf(m[r], bm);
                const float ms = mn == -INFINITY ? 0.f : mn;
                const float corr = exp2f(m[r] - ms);     // 0 for the first keys
                l[r] *= corr;
                #pragma unroll
                for (int e = 0; e < E; ++e) a[r][e] *= corr;
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float w = exp2f(xr[k] - ms);
                    l[r] += w;
                    #pragma unroll
                    for (int e = 0; e < E; ++e) a[r][e] = fmaf(w, val[k][e], a[r][e]);
                }
                m[r] = mn;
            }
        }
    }
    constexpr int DP = 32 * E;
    float* so = reinterpret_cast<float*>(smem);          // [4][R][DP]
    float2* sm = reinterpret_cast<float2*>(smem + 4 * R * DP * 4);
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        if (lane == 0) sm[warp * R + r] = make_float2(seen(m[r], l[r]), l[r]);
        #pragma unroll
        for (int j = 0; j < E / V; ++j)
            #pragma unroll
            for (int v = 0; v < V; ++v) so[(warp * R + r) * DP + (lane + 32 * j) * V + v] = a[r][j * V + v];
    }
    __syncthreads();
    join_warps<R, DP, 4>(p, sm, so, rows, row0, p.plan.prefix_splits + split);
}

// ---- joining the splits -----------------------------------------------------------------------------
// One CTA per query row: warp w takes slots w, w + 4, ... with eight loads on their way at a time, lane j the elements
// j, j + 32, ...; the four warps' sums are joined in order.  The order is that of the slots, so the result does
// not depend on timing.
constexpr int kMaxSlots = 128;
template <int NE>                                          // elements of a lane: ceil(d / 32)
__global__ void __launch_bounds__(kThreads) swa_decode_join_kernel(const __grid_constant__ Params p)
{
    __shared__ float weight[kMaxSlots];
    __shared__ float part[3][32 * NE];
    __shared__ float total;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const DecodeCall& c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    const float2* ml = p.ml + row * p.slots;
    const float* acc = p.acc + row * p.slots * c.d;
    const int d = static_cast<int>(c.d);
    if (warp == 0) {
        float2 v[kMaxSlots / 32];
        float M = -INFINITY;
        #pragma unroll
        for (int i = 0; i < kMaxSlots / 32; ++i) {
            const int s = lane + 32 * i;
            v[i] = s < p.slots ? ml[s] : make_float2(-INFINITY, 0.f);
            M = fmaxf(M, v[i].x);
        }
        #pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        float l = 0.f;
        #pragma unroll
        for (int i = 0; i < kMaxSlots / 32; ++i) {
            const float f = v[i].x == -INFINITY ? 0.f : ex2(v[i].x - M);
            weight[lane + 32 * i] = f;                   // 0 for an empty slot, whose sums are not written
            l += v[i].y * f;
        }
        #pragma unroll
        for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        if (lane == 0) total = l;
    }
    __syncthreads();
    float a[NE] = {};
    for (int s0 = warp; s0 < p.slots; s0 += 32) {
        float x[8][NE];
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int s = s0 + 4 * i;
            const bool in = s < p.slots && weight[s] > 0.f;
            #pragma unroll
            for (int j = 0; j < NE; ++j) {
                const int e = lane + 32 * j;
                x[i][j] = in && e < d ? acc[static_cast<int64_t>(s) * d + e] : 0.f;
            }
        }
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int s = s0 + 4 * i;
            const float f = s < p.slots ? weight[s] : 0.f;
            #pragma unroll
            for (int j = 0; j < NE; ++j) a[j] = fmaf(x[i][j], f, a[j]);
        }
    }
    if (warp > 0) {
        #pragma unroll
        for (int j = 0; j < NE; ++j) part[warp - 1][lane + 32 * j] = a[j];
    }
    __syncthreads();
    if (warp > 0) return;
    const float inv = total == 0.f ? 0.f : 1.f / total;
    #pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int e = lane + 32 * j;
        const float v = ((a[j] + part[0][e]) + part[1][e]) + part[2][e];
        if (e < d) store_out(c.o, row * d + e, c.out_bf16, v * inv);
    }
}

template <typename K>
cudaError_t launch(K kernel, const Params& p, dim3 grid, size_t smem, bool early, cudaStream_t stream,
                   int threads = kThreads)
{
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int DP, int W, int ST>
cudaError_t launch_tc(const Params& p, dim3 grid, bool early, cudaStream_t stream)
{
    const size_t smem = W * ST * Ring<DP>::kStage;
    return p.c.Hq / p.c.Hkv <= 8 ? launch(swa_decode_kernel<DP, W, ST, 1>, p, grid, smem, early, stream, 32 * W)
                                 : launch(swa_decode_kernel<DP, W, ST, 2>, p, grid, smem, early, stream, 32 * W);
}

// As many rows in a CTA's registers as the group has heads (1, 2 or 4), and no more elements than the width needs.
template <typename T, int V, int E>
cudaError_t launch_cc(const Params& p, dim3 grid, cudaStream_t stream)
{
    const int64_t G = p.c.Hq / p.c.Hkv;
    const size_t row = 4 * (32 * E * 4 + 8);
    return G == 1   ? launch(swa_decode_cc_kernel<T, V, E, 1>, p, grid, row, false, stream)
           : G == 2 ? launch(swa_decode_cc_kernel<T, V, E, 2>, p, grid, 2 * row, false, stream)
                    : launch(swa_decode_cc_kernel<T, V, E, 4>, p, grid, 4 * row, false, stream);
}
template <typename T>
cudaError_t launch_cc(const Params& p, dim3 grid, cudaStream_t stream)
{
    if (p.c.d <= 128) return p.c.d % 4 == 0 ? launch_cc<T, 4, 4>(p, grid, stream) : launch_cc<T, 1, 4>(p, grid, stream);
    return p.c.d % 4 == 0 ? launch_cc<T, 4, 8>(p, grid, stream) : launch_cc<T, 1, 8>(p, grid, stream);
}

}  // namespace swad

bool decode_tc_supports(int bf16, int64_t d) { return bf16 && d % 8 == 0 && d <= 256; }

DecodePlan plan_decode(const DecodeCall& c)
{
    DecodePlan plan = {};
    const int64_t G = c.Hq / c.Hkv;
    const int per = c.tensor_core ? 16 : swad::kRowsCc;
    plan.group_tiles = static_cast<int>((G + per - 1) / per);
    plan.seqs_per_tile = 1;
    // The keys a sequence may have, as far as the host can tell: splits of 512 at least (a split costs a second
    // launch and its partial results; 128 on CUDA cores, which take longer for a key, and 64 gained nothing), and no
    // more CTAs than 16 per SM (4 x 48 ragged sequences of up to 16,384 keys: 8 per SM 648 us, 16 620, 32 627).
    int64_t most = c.max_pages << c.page_shift;
    // A shared prefix: tiles of as many whole sequences as 128 query rows hold, split so that each SM has two CTAs and
    // a CTA four blocks of keys at least.  It pays from the second sequence on: a tile of any size reads the
    // keys once, and its products keep up with HBM.
    if (c.tensor_core && c.d == 128 && c.pages > 0 && c.B > 1 && c.prefix >= 256 && G <= 128 &&
        c.T * c.pages * c.Hkv < (int64_t(1) << 31)) {
        plan.seqs_per_tile = static_cast<int>(128 / G);
        plan.tiles = static_cast<int>((c.B + plan.seqs_per_tile - 1) / plan.seqs_per_tile);
        const int64_t units = c.T * c.Hkv * plan.tiles;
        int64_t n = 2 * 148 / units;
        if (n > c.prefix / 256) n = c.prefix / 256;
        if (n > 64) n = 64;
        plan.prefix_splits = n < 1 ? 1 : static_cast<int>(n);
        most -= c.prefix;
    }
    if (c.window < most) most = c.window;
    const int64_t units = c.T * c.B * c.Hkv * plan.group_tiles;
    const int64_t least = c.tensor_core ? 512 : 128;
    int64_t n = (most + least - 1) / least;
    const int64_t fill = (16 * 148 + units - 1) / units;
    if (n > fill) n = fill;
    if (n > 64) n = 64;
    if (n < 1) n = 1;
    plan.own_splits = static_cast<int>(n);
    return plan;
}

// A shared prefix's sums between two runs, 64 KB for a CTA, where one may have more than a run of blocks.
static size_t between_bytes(const DecodeCall& c, const DecodePlan& plan)
{
    if (plan.prefix_splits == 0) return 0;
    const int64_t blocks = (c.prefix / 64 + plan.prefix_splits - 1) / plan.prefix_splits;
    if (blocks <= swad::kPrefixRun) return 0;
    return static_cast<size_t>(c.T * c.Hkv * plan.tiles) * plan.prefix_splits * (128 * 128 * 4);
}

size_t decode_workspace_bytes(const DecodeCall& c)
{
    const DecodePlan plan = plan_decode(c);
    if (plan.slots() <= 1) return 0;               // (a shared prefix makes two at least)
    const size_t rows = static_cast<size_t>(c.T * c.B * c.Hq) * plan.slots();
    return (rows * 8 + 15) / 16 * 16 + rows * c.d * 4 + between_bytes(c, plan);
}

cudaError_t launch_swa_decode(const DecodeCall& c, cudaStream_t stream)
{
    using namespace swad;
    NvtxRange range("lt2 window decode");
    Params p;
    p.c = c;
    p.plan = plan_decode(c);
    p.xscale = c.scale * kLog2e;
    p.slots = p.plan.slots() > 1 ? p.plan.slots() : 0;
    const size_t rows = static_cast<size_t>(c.T * c.B * c.Hq);
    p.ml = reinterpret_cast<float2*>(c.workspace);
    p.acc = p.slots ? c.workspace + (rows * p.slots * 8 + 15) / 16 * 4 : nullptr;
    p.between = between_bytes(c, p.plan) ? p.acc + rows * p.slots * c.d : nullptr;
    const dim3 grid(static_cast<unsigned>(c.T * c.Hkv * c.B * p.plan.group_tiles), p.plan.own_splits);
    cudaError_t e;
    if (p.plan.prefix_splits > 0) {
        e = launch_swa_decode_prefix(p, stream);
        if (e != cudaSuccess) return e;
    }
    const bool beside = p.plan.prefix_splits > 0;
    if (c.tensor_core) {
        // A warp takes 1.2 us for a tile, however deep its ring.  So where a CTA has an SM to itself, as many warps as
        // shared memory holds share its keys (16 heads of 128, a window of 512: 12 warps 9.1 us, four 11.4; heads of
        // 64: 16 warps 6.7, four 8.9); elsewhere, and beside a prefix, four (three CTAs per SM).
        const bool alone = !beside && static_cast<int64_t>(grid.x) * grid.y <= 148;
        if (c.d <= 64)
            e = alone ? launch_tc<64, 16, 2>(p, grid, false, stream) : launch_tc<64, 4, 4>(p, grid, beside, stream);
        else if (c.d <= 128)
            e = alone ? launch_tc<128, 12, 2>(p, grid, false, stream) : launch_tc<128, 4, 2>(p, grid, beside, stream);
        else
            e = launch_tc<256, 4, 3>(p, grid, beside, stream);
    } else {
        e = c.bf16 ? launch_cc<__nv_bfloat16>(p, grid, stream) : launch_cc<float>(p, grid, stream);
    }
    if (e != cudaSuccess || !p.slots) return e;
    const dim3 jgrid(static_cast<unsigned>(rows));
    return c.d <= 64    ? launch(swa_decode_join_kernel<2>, p, jgrid, 0, true, stream)
           : c.d <= 128 ? launch(swa_decode_join_kernel<4>, p, jgrid, 0, true, stream)
                        : launch(swa_decode_join_kernel<8>, p, jgrid, 0, true, stream);
}

}  // namespace lt2
