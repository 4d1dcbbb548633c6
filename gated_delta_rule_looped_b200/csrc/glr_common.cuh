// glr_common.cuh -- device helpers of the gated linear recurrence kernels: element loads and
// stores by fours, the gates from their logits, and the carries between the tiles of a scan.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "f32x2.cuh"
#include "gdr_common.cuh"
#include "gdr_tc_common.cuh"

namespace lt2 {
namespace glr {

using namespace pairs;

// ---- two channels at a time ----------------------------------------------------------------------
// With logits the gates take some 40 scalar operations an element, more than HBM leaves time for; paired they fit
// under the loads.
// 2^x of both, rcp of both
__device__ __forceinline__ f2 ex2_2(f2 v)
{
    float a, b;
    unpack2(v, a, b);
    return pack2(ex2(a), ex2(b));
}
__device__ __forceinline__ f2 rcp_2(f2 v)
{
    float a, b;
    unpack2(v, a, b);
    return pack2(sm100::rcp_approx(a), sm100::rcp_approx(b));
}

// alpha = exp(-c softplus(a)) of N pairs, softplus(a) = max(a, 0) + log(1 + exp(-|a|)); nc = -c.
//
// log(1 + e), e in [0, 1], is e times a polynomial fitted at Chebyshev nodes to log(1 + e) / e: full relative
// precision for small e (1.2e-7 at most over the range).
//
// exp(y), y <= 0: a decay near 1 is applied thousands of times, and an error of a few ulps in it (the
// hardware's exp2 has that) would come back multiplied by the memory's length.  So down to y = -1/2 it is
// 1 + y (1 + y q(y)), q fitted at Chebyshev nodes: right to 1.4 units of rounding; below, where at most two or three
// tokens are remembered, the hardware's exp2.
//
// The polynomials go coefficient by coefficient over the N pairs: a coefficient is a pair in two registers,
// and set up once for N products.
template <int N>
__device__ __forceinline__ void decay_of_logits(f2 (&a)[N], f2 nc)
{
    constexpr float kLog[9] = {0.005253458f, -0.029588507f, 0.07836167f, -0.1367477f, 0.1911143f,
                               -0.2484437f, 0.3331927f, -0.49999502f, 1.f};
    constexpr float kExp[7] = {0.0011646036f, 0.008238538f, 0.04165003f, 0.16666564f, 0.5f, 1.f, 1.f};
    f2 e[N], q[N];
    #pragma unroll
    for (int i = 0; i < N; ++i) {
        float a0, a1;
        unpack2(a[i], a0, a1);
        e[i] = pack2(ex2(-fabsf(a0) * kLog2e), ex2(-fabsf(a1) * kLog2e));
        a[i] = pack2(fmaxf(a0, 0.f), fmaxf(a1, 0.f));
        q[i] = both(kLog[0]);
    }
    #pragma unroll
    for (int k = 1; k < 9; ++k) {
        const f2 c = both(kLog[k]);
        #pragma unroll
        for (int i = 0; i < N; ++i) q[i] = fma2(e[i], q[i], c);
    }
    #pragma unroll
    for (int i = 0; i < N; ++i) {
        a[i] = mul2(nc, fma2(e[i], q[i], a[i]));           // y
        q[i] = both(kExp[0]);
    }
    #pragma unroll
    for (int k = 1; k < 7; ++k) {
        const f2 c = both(kExp[k]);
        #pragma unroll
        for (int i = 0; i < N; ++i) q[i] = fma2(a[i], q[i], c);
    }
    #pragma unroll
    for (int i = 0; i < N; ++i) {
        float y0, y1, q0, q1;
        unpack2(a[i], y0, y1);
        unpack2(q[i], q0, q1);
        const float e0 = ex2(y0 * kLog2e), e1 = ex2(y1 * kLog2e);
        a[i] = pack2(y0 >= -0.5f ? q0 : e0, y1 >= -0.5f ? q1 : e1);  // a NaN takes exp2 and stays one
    }
}
// exp(-b), kept finite so that its product with a vanishing sigmoid is 0; a NaN stays one
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 exp_minus(f2 b)
{
    float e0, e1;
    unpack2(ex2_2(mul2(b, both(-kLog2e))), e0, e1);
    return pack2(min_nan(e0, 3e38f), min_nan(e1, 3e38f));
}
__device__ __forceinline__ f2 sigmoid_from(f2 e) { return rcp_2(add2(both(1.f), e)); }
__device__ __forceinline__ f2 sigmoid_of(f2 b) { return sigmoid_from(ex2_2(mul2(b, both(-kLog2e)))); }

// ---- four channels at a time -------------------------------------------------------------------
struct F4 {
    f2 a, b;               // channels 0, 1 and 2, 3
};
__device__ __forceinline__ F4 all4(float v) { return {both(v), both(v)}; }
__device__ __forceinline__ F4 widen(float4 v) { return {pack2(v.x, v.y), pack2(v.z, v.w)}; }
__device__ __forceinline__ F4 widen(uint2 w)
{
    return {pack2(sm100::bf16_lo(w.x), sm100::bf16_hi(w.x)), pack2(sm100::bf16_lo(w.y), sm100::bf16_hi(w.y))};
}
__device__ __forceinline__ float4 floats(F4 v)
{
    float4 r;
    unpack2(v.a, r.x, r.y);
    unpack2(v.b, r.z, r.w);
    return r;
}
__device__ __forceinline__ F4 mul4(F4 x, F4 y) { return {mul2(x.a, y.a), mul2(x.b, y.b)}; }
__device__ __forceinline__ F4 fma4(F4 x, F4 y, F4 z) { return {fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)}; }
// The decays of N fours of logits.
template <int N>
__device__ __forceinline__ void decay4(F4 (&v)[N], f2 nc)
{
    f2 a[2 * N];
    #pragma unroll
    for (int i = 0; i < N; ++i) {
        a[2 * i] = v[i].a;
        a[2 * i + 1] = v[i].b;
    }
    decay_of_logits<2 * N>(a, nc);
    #pragma unroll
    for (int i = 0; i < N; ++i) v[i] = {a[2 * i], a[2 * i + 1]};
}
__device__ __forceinline__ F4 sigmoid4(F4 v) { return {sigmoid_of(v.a), sigmoid_of(v.b)}; }

template <typename T> struct Four;
template <> struct Four<float> { using Raw = float4; };
template <> struct Four<__nv_bfloat16> { using Raw = uint2; };

// Four channels that lie together (shared memory, or a row of a width that is a multiple of 4).
template <typename T>
__device__ __forceinline__ F4 load4(const T* p) { return widen(*reinterpret_cast<const typename Four<T>::Raw*>(p)); }
// The first n of four channels (n = 4 with vec).
template <typename T>
__device__ __forceinline__ F4 load4(const T* p, bool vec, int n)
{
    if (vec) return load4(p);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n > 0) v.x = to_f32<T>(p[0]);
    if (n > 1) v.y = to_f32<T>(p[1]);
    if (n > 2) v.z = to_f32<T>(p[2]);
    if (n > 3) v.w = to_f32<T>(p[3]);
    return widen(v);
}
__device__ __forceinline__ void store4(float* p, F4 x, bool vec, int n)
{
    const float4 v = floats(x);
    if (vec) {
        *reinterpret_cast<float4*>(p) = v;
        return;
    }
    if (n > 0) p[0] = v.x;
    if (n > 1) p[1] = v.y;
    if (n > 2) p[2] = v.z;
    if (n > 3) p[3] = v.w;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, F4 x, bool vec, int n)
{
    const float4 v = floats(x);
    if (vec) {
        *reinterpret_cast<uint2*>(p) = make_uint2(sm100::pack_bf16x2(v.x, v.y), sm100::pack_bf16x2(v.z, v.w));
        return;
    }
    if (n > 0) p[0] = __float2bfloat16_rn(v.x);
    if (n > 1) p[1] = __float2bfloat16_rn(v.y);
    if (n > 2) p[2] = __float2bfloat16_rn(v.z);
    if (n > 3) p[3] = __float2bfloat16_rn(v.w);
}
// From element i of a tensor whose type is known at run time (the same for the whole launch).
__device__ __forceinline__ void store4_as(void* p, int64_t i, int bf16, F4 v, bool vec, int n)
{
    if (bf16)
        store4(static_cast<__nv_bfloat16*>(p) + i, v, vec, n);
    else
        store4(static_cast<float*>(p) + i, v, vec, n);
}

// ---- two channels of a lane (scan) ---------------------------------------------------------------
template <typename T> struct Pair;
template <> struct Pair<float> {
    using Raw = float2;
    __device__ static f2 wide(float2 v) { return pack2(v.x, v.y); }
};
template <> struct Pair<__nv_bfloat16> {
    using Raw = uint32_t;
    __device__ static f2 wide(uint32_t w) { return pack2(sm100::bf16_lo(w), sm100::bf16_hi(w)); }
};
// Two channels that lie together.
template <typename T>
__device__ __forceinline__ f2 load2(const T* p)
{
    return Pair<T>::wide(*reinterpret_cast<const typename Pair<T>::Raw*>(p));
}
__device__ __forceinline__ void put2(float* p, f2 x)
{
    float2 v;
    unpack2(x, v.x, v.y);
    *reinterpret_cast<float2*>(p) = v;
}
__device__ __forceinline__ void put2(__nv_bfloat16* p, f2 x)
{
    float a, b;
    unpack2(x, a, b);
    *reinterpret_cast<uint32_t*>(p) = sm100::pack_bf16x2(a, b);
}
__device__ __forceinline__ void put1(float* p, float x) { *p = x; }
__device__ __forceinline__ void put1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
// To the first n of two channels from element i of a tensor; `pair`: they lie on a pair's boundary.
template <typename T>
__device__ __forceinline__ void store2(T* p, f2 x, bool pair, int n)
{
    if (pair) {
        put2(p, x);
        return;
    }
    float a, b;
    unpack2(x, a, b);
    if (n > 0) put1(p, a);
    if (n > 1) put1(p + 1, b);
}
// The same with a type known at run time (one for the whole launch); `i` counts elements.
__device__ __forceinline__ void store2_as(void* p, int64_t i, int bf16, f2 x, bool pair, int n)
{
    if (bf16)
        store2(static_cast<__nv_bfloat16*>(p) + i, x, pair, n);
    else
        store2(static_cast<float*>(p) + i, x, pair, n);
}

// ---- carries between the tiles of a scan -------------------------------------------------------
// A chain is one unit's block of 64 channels, cut into tiles of tokens.  A tile publishes, per channel,
// its map carry -> A carry + H as one 64-bit word as soon as it has read its tokens, and the carry
// that leaves it as one 32-bit word once it knows the one that enters.  All words start as all ones
// (one memset), which no published value is: a NaN is published as the canonical one.  So a word
// carries its own flag, and no fence is needed.
//
// A tile walks back over its predecessors until one has published its outgoing carry, then applies
// the maps of the tiles between, oldest first.  The carry that a tile publishes is the same
// expression, fmaf(A, carry, H): so every tile's carry is the same left-to-right fold bit for bit,
// however far it had to walk.  A tile waits only for tiles with a lower ticket, which are running
// or done and publish their maps without waiting.
constexpr uint32_t kNotYet = 0xffffffffu;
constexpr uint32_t kNan = 0x7fffffffu;
constexpr int kChannels = 64;          // channels of a tile: two for each lane of a warp

__device__ __forceinline__ uint32_t word_of(float v) { return v != v ? kNan : __float_as_uint(v); }
__device__ __forceinline__ void ld_words(const uint32_t* p, uint32_t (&v)[2])
{
    asm volatile("ld.relaxed.gpu.global.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p) : "memory");
}
__device__ __forceinline__ void ld_words(const uint64_t* p, uint64_t (&v)[2])
{
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "l"(p) : "memory");
}
__device__ __forceinline__ void publish_map(uint64_t* p, f2 A, f2 H)
{
    float a0, a1, h0, h1;
    unpack2(A, a0, a1);
    unpack2(H, h0, h1);
    const uint64_t v0 = static_cast<uint64_t>(word_of(a0)) | (static_cast<uint64_t>(word_of(h0)) << 32);
    const uint64_t v1 = static_cast<uint64_t>(word_of(a1)) | (static_cast<uint64_t>(word_of(h1)) << 32);
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p), "l"(v0), "l"(v1) : "memory");
}
__device__ __forceinline__ void publish_carry(uint32_t* p, f2 v)
{
    float a, b;
    unpack2(v, a, b);
    asm volatile("st.relaxed.gpu.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(word_of(a)), "r"(word_of(b)) : "memory");
}

// The carry that enters tile `tile` (> 0) of a chain, for the two channels of each lane of a full warp; `maps` and
// `carries` point at the lane's words of tile 0.  The warp walks together: a tile counts as ready when all
// its channels are.
__device__ __forceinline__ f2 carry_into(const uint64_t* maps, const uint32_t* carries, int tile, unsigned int* err)
{
    constexpr int W = 4;                                  // predecessors looked at in one go
    constexpr unsigned kAll = 0xffffffffu;
    int j = tile - 1;
    f2 carry = 0;
    uint64_t t0 = 0;
    uint32_t spins = 0;
    while (true) {
        uint32_t c[W][2];
        uint64_t m[W][2];
        #pragma unroll
        for (int i = 0; i < W; ++i) {
            const int64_t k = (j - i < 0 ? 0 : j - i) * static_cast<int64_t>(kChannels);
            ld_words(carries + k, c[i]);
            ld_words(maps + k, m[i]);
        }
        int found = -1, back = 0;
        bool go = true;
        #pragma unroll
        for (int i = 0; i < W; ++i) {
            const bool here = __all_sync(kAll, c[i][0] != kNotYet && c[i][1] != kNotYet);
            const bool map = __all_sync(kAll, m[i][0] != ~uint64_t(0) && m[i][1] != ~uint64_t(0));
            if (go && j - i >= 0) {
                if (here) {
                    found = i;
                    carry = pack2(__uint_as_float(c[i][0]), __uint_as_float(c[i][1]));
                    go = false;
                } else if (map) {
                    ++back;
                } else {
                    go = false;                           // not read yet
                }
            }
        }
        if (found >= 0) {
            // the maps between, oldest first; the nearest are at hand
            #pragma unroll
            for (int i = W - 1; i >= 0; --i)
                if (i < found) carry = fma2(pack2(__uint_as_float(static_cast<uint32_t>(m[i][0])),
                                                  __uint_as_float(static_cast<uint32_t>(m[i][1]))), carry,
                                            pack2(__uint_as_float(static_cast<uint32_t>(m[i][0] >> 32)),
                                                  __uint_as_float(static_cast<uint32_t>(m[i][1] >> 32))));
            j += 1;
            break;
        }
        j -= back;
        if (back == 0 && (++spins & 63u) == 0u) {
            const uint64_t now = sm100::global_timer_ns();
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > tcc::kWaitTimeoutNs) {  // the clock is the same for the warp
                atomicOr(err, kDevTimeout);
                return both(__uint_as_float(kNan));
            }
        }
    }
    // the maps behind those are all published (the walk back saw them)
    for (int k = j; k < tile; ++k) {
        uint64_t m[2];
        ld_words(maps + static_cast<int64_t>(k) * kChannels, m);
        carry = fma2(pack2(__uint_as_float(static_cast<uint32_t>(m[0])), __uint_as_float(static_cast<uint32_t>(m[1]))), carry,
                     pack2(__uint_as_float(static_cast<uint32_t>(m[0] >> 32)),
                           __uint_as_float(static_cast<uint32_t>(m[1] >> 32))));
    }
    return carry;
}

// ---- staging a tile -----------------------------------------------------------------------------
// A warp's ROWS x CB elements of a [.][d] tensor from `g` (the warp's first row, channel 0 of the tile) to
// shared memory; rows from `rows` on and channels from `chans` on become 0.  Rows are packed, in HALVES
// interleaved runs: with two, row i of the first half lies beside row i of the second, so that two half warps that
// read them together meet no bank twice.  `aligned`: every row starts on 16 bytes and d is a multiple of 16 bytes; such
// rows are copied in 16-byte chunks, others that consist of whole 4-byte words (`even`: pairs of bf16) word by word,
// both asynchronously, and bf16 rows of an odd width element by element.
template <int ROWS, int HALVES>
__host__ __device__ constexpr int staged_row(int row)
{
    return HALVES == 1 ? row : (row % (ROWS / 2)) * 2 + row / (ROWS / 2);
}
// Where a lane's first chunk lies: element of the tensor from row 0, channel 0 of the warp's rows.
template <typename T, int CB>
__device__ __forceinline__ int64_t lane_chunk(int64_t d)
{
    constexpr int E = 16 / static_cast<int>(sizeof(T)), CPR = CB / E;
    const int lane = threadIdx.x & 31;
    return lane / CPR * d + lane % CPR * E;
}
template <typename T, int CB, int ROWS, int HALVES>
__device__ __forceinline__ void stage_rows(T* s, const T* g, int64_t chunk, int rows, int chans, int64_t d, bool aligned,
                                           bool even)
{
    const int lane = threadIdx.x & 31;
    if (aligned) {
        constexpr int E = 16 / static_cast<int>(sizeof(T));
        constexpr int CPR = CB / E;                       // chunks of a row
        constexpr int STEP = 32 / CPR;                    // rows between a lane's chunks
        constexpr int SZ = static_cast<int>(sizeof(T));
        static_assert(HALVES == 1 || (ROWS / 2) % STEP == 0, "a lane's chunks step through a half evenly");
        const int row0 = lane / CPR, ch = lane % CPR * E;
        const uint32_t dst = sm100::smem_addr(s) + (row0 * HALVES * CB + ch) * SZ;
        const T* src = g + chunk;
        const int64_t step = STEP * d;
        const bool all = rows >= ROWS && chans == CB;
        #pragma unroll
        for (int i = 0; i < ROWS / STEP; ++i, src += step) {
            const bool in = all || (row0 + i * STEP < rows && ch < chans);
            cp_async16(dst + staged_row<ROWS, HALVES>(i * STEP) * CB * SZ, in ? src : g, in ? 16u : 0u);
        }
    } else if (sizeof(T) == 4 || even) {
        constexpr int E = 4 / static_cast<int>(sizeof(T)), WPR = CB / E;      // words of a row
        const uint32_t dst = sm100::smem_addr(s);
        #pragma unroll 4
        for (int i = 0; i < ROWS * WPR / 32; ++i) {
            const int k = i * 32 + lane;
            const int row = k / WPR, ch = k % WPR * E;
            const bool in = row < rows && ch < chans;
            cp_async4(dst + (staged_row<ROWS, HALVES>(row) * WPR + k % WPR) * 4u, in ? g + row * d + ch : g, in ? 4u : 0u);
        }
    } else {
        #pragma unroll 4
        for (int i = 0; i < ROWS * CB / 32; ++i) {
            const int k = i * 32 + lane;
            const int row = k / CB, ch = k % CB;
            s[staged_row<ROWS, HALVES>(row) * CB + ch] = row < rows && ch < chans ? g[row * d + ch] : from_f32<T>(0.f);
        }
    }
}

}  // namespace glr
}  // namespace lt2
