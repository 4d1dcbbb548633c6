// swa_decode_common.cuh -- what the kernels of the decode attention share: a sequence's range of keys,
// the part of it that a tile of sequences has in common, and the partial results.
//
// Query of sequence b (its last token): keys [lo_b, n_b), lo_b = max(0, n_b - window).  The first
// `prefix` tokens lie in the same pages for every sequence.  Of those, a tile of sequences takes the
// blocks of 64 keys that all its sequences see, [common_lo, common_hi), in one product for the whole tile;
// each sequence takes the rest, [lo_b, common_lo) and [common_hi, n_b), by itself.  So no product
// of the shared part needs a mask, and a sequence whose window leaves the prefix early costs the others
// their sharing there, not their results.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "cache_launch.h"
#include "f32x2.cuh"
#include "gdr_common.cuh"
#include "lt2_api_common.h"
#include "sm100_primitives.cuh"

namespace lt2 {
namespace swad {

using namespace pairs;

// Blocks of 64 keys whose products the tensor core adds up in a shared prefix before the sum is rounded (a run).
constexpr int kPrefixRun = 4;

struct Params {
    DecodeCall c;
    DecodePlan plan;
    float xscale;          // scale * log2(e)
    int slots;             // partial results per row; 0: o is written directly
    float2* ml;            // [rows][slots]: maximum (log2 units) and sum
    float* acc;            // [rows][slots][d]: sum of 2^(x - max) v
    float* between;        // [CTA][128 columns][128 rows]: the shared prefix's sums between two runs of blocks, or null
};

// Weights p >= 0 as three bf16 numbers whose sum is p exactly, all 24 bits of it: p a little lessened (kLess) and cut to
// 8 bits, the rest treated the same way, and what is left then, which has 8 bits at most.  Lessening by one or two
// units of the last place leaves every part of a weight above 2^-100 above zero, so an infinite value stays infinite
// instead of meeting a zero or a negative part.
constexpr float kLess = 1.f - 0x1p-23f;
__device__ __forceinline__ float cut_bf16(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// The upper halves of two floats: cut to bf16.
__device__ __forceinline__ uint32_t upper_halves(float x0, float x1)
{
    return __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);
}
// (the last one times `share`, a power of two)
__device__ __forceinline__ void split_bf16(float p0, float p1, uint32_t& hi, uint32_t& mid, uint32_t& lo, float share)
{
    const float h0 = cut_bf16(p0 * kLess), h1 = cut_bf16(p1 * kLess);
    hi = upper_halves(h0, h1);
    const float r0 = p0 - h0, r1 = p1 - h1, m0 = cut_bf16(r0 * kLess), m1 = cut_bf16(r1 * kLess);
    mid = upper_halves(m0, m1);
    lo = upper_halves((r0 - m0) * share, (r1 - m1) * share);
}

// Keys of sequence b as [lo, n); an empty sequence, or a length that the table does not hold, is [0, 0).
__device__ __forceinline__ void key_range(const DecodeCall& c, int64_t b, int64_t& lo, int64_t& n)
{
    n = c.lens[b];
    if (n < 0 || n > (c.max_pages << c.page_shift)) n = 0;
    lo = n > c.window ? n - c.window : 0;
}

// The keys that every sequence of [b0, b1) sees in the shared prefix, cut to whole blocks of 64; called by a full
// warp.  Empty sequences do not count.  lo = hi where there are none.
__device__ __forceinline__ void common_range(const DecodeCall& c, int64_t b0, int64_t b1, int64_t& lo, int64_t& hi)
{
    int64_t l = 0, h = c.prefix;
    bool any = false;
    for (int64_t b = b0 + (threadIdx.x & 31); b < b1; b += 32) {
        int64_t bl, n;
        key_range(c, b, bl, n);
        if (n == 0) continue;
        any = true;
        l = bl > l ? bl : l;
        h = n < h ? n : h;
    }
    #pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const int64_t ol = __shfl_xor_sync(0xffffffffu, l, s), oh = __shfl_xor_sync(0xffffffffu, h, s);
        l = ol > l ? ol : l;
        h = oh < h ? oh : h;
    }
    any = __any_sync(0xffffffffu, any);
    lo = (l + 63) & ~int64_t(63);
    hi = h & ~int64_t(63);
    if (!any || hi < lo) lo = hi = 0;
}

// A sequence's own keys as tiles of 16 that never cross a page: `head` tiles from `first` on (in front of
// the common part), the others from `second` on.
struct OwnTiles {
    int64_t lo, n, first, second;
    int64_t head, total;
    __device__ __forceinline__ int64_t pos(int64_t i) const { return i < head ? first + 16 * i : second + 16 * (i - head); }
};
__device__ __forceinline__ OwnTiles own_tiles(const DecodeCall& c, const DecodePlan& plan, int64_t b)
{
    OwnTiles t;
    key_range(c, b, t.lo, t.n);
    t.first = t.lo & ~int64_t(15);
    t.head = 0;
    t.second = t.first;
    if (plan.prefix_splits > 0) {
        const int64_t b0 = b / plan.seqs_per_tile * plan.seqs_per_tile;
        const int64_t b1 = b0 + plan.seqs_per_tile < c.B ? b0 + plan.seqs_per_tile : c.B;
        int64_t clo, chi;
        common_range(c, b0, b1, clo, chi);
        if (chi > clo && t.n > 0) {
            t.head = (clo - t.first) >> 4;
            t.second = chi;
        }
    }
    t.total = t.n > 0 ? t.head + ((t.n - t.second + 15) >> 4) : 0;
    return t;
}

// Tiles [i0, i1) of split s of n splits: equal shares, of 8 tiles at least.
__device__ __forceinline__ void split_range(int64_t total, int s, int n, int64_t& i0, int64_t& i1)
{
    int64_t share = (total + n - 1) / n;
    share = share < 8 ? 8 : (share + 3) & ~int64_t(3);
    i0 = s * share < total ? s * share : total;
    i1 = i0 + share < total ? i0 + share : total;
}

// First element of the cache row of position `pos` (loop tau, key head h), or -1 with the error
// recorded where the table names a page outside the cache.
__device__ __forceinline__ int64_t cache_row(const DecodeCall& c, int64_t tau, int64_t h, int32_t page, int64_t pos)
{
    if (page < 0 || page >= c.pages) {
        atomicOr(c.err, kDevPages);
        return -1;
    }
    return ((((tau * c.pages + page) * c.Hkv + h) << c.page_shift) + (pos & ((int64_t(1) << c.page_shift) - 1))) * c.d;
}

__device__ __forceinline__ void store_out(void* o, int64_t i, int bf16, float v)
{
    if (bf16)
        static_cast<__nv_bfloat16*>(o)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(o)[i] = v;
}

// The kernel of the sequences' own keys may run beside the one of the shared prefix (programmatic launch); the
// join that follows waits for the former alone.  So one CTA of it does not end before the latter has.
__device__ __forceinline__ void outlast_prefix(const DecodePlan& plan)
{
    if (plan.prefix_splits > 0 && blockIdx.x == 0 && blockIdx.y == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Joins the W warps' results of up to `rows` query rows in shared memory and writes them: o where there is
// one slot, else the slot's partial.  sm: [W][ROWS] float2, so: [W][ROWS][DP] floats.
template <int ROWS, int DP, int W>
__device__ __forceinline__ void join_warps(const Params& p, const float2* sm, const float* so, int rows, int64_t row0,
                                           int slot)
{
    const int d = static_cast<int>(p.c.d);
    for (int i = threadIdx.x; i < rows * DP; i += blockDim.x) {
        const int r = i / DP, e = i % DP;
        if (e >= d) continue;
        float M = sm[r].x;
        #pragma unroll
        for (int w = 1; w < W; ++w) M = fmaxf(M, sm[w * ROWS + r].x);
        float l = 0.f, a = 0.f;
        if (M != -INFINITY) {
            #pragma unroll
            for (int w = 0; w < W; ++w) {
                const float2 v = sm[w * ROWS + r];
                if (v.x == -INFINITY) continue;          // this warp saw no key
                const float f = ex2(v.x - M);
                l = fmaf(v.y, f, l);
                a = fmaf(so[(w * ROWS + r) * DP + e], f, a);
            }
        }
        const int64_t row = row0 + r;
        if (p.slots == 0) {
            store_out(p.c.o, row * d + e, p.c.out_bf16, l == 0.f ? 0.f : a / l);
        } else {
            p.acc[(row * p.slots + slot) * d + e] = a;
            if (e == 0) p.ml[row * p.slots + slot] = make_float2(M, l);
        }
    }
}

}  // namespace swad

// The shared prefix's partial results, slots [0, prefix_splits) (swa_decode_prefix.cu).
cudaError_t launch_swa_decode_prefix(const swad::Params& p, cudaStream_t stream);

}  // namespace lt2
