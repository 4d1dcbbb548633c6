// glr_split.cu -- the gated linear recurrence in three launches, for units too narrow for tiles of 64 channels: every
// sequence is cut into segments of 64 tokens, one thread per segment and two channels.
//
//   1  each segment's map carry -> A carry + H                        (reads alpha, beta, x)
//   2  a warp per channel passes the state over the segments' maps, and keeps the states between them
//   3  each segment runs its tokens from its state                    (reads them again, writes o)
//
// and backward the same from the last segment to the first, the states given.  Nobody waits for another CTA inside a
// launch, and any number of channels per unit fills the lanes.  The inputs are read twice; a launch starts while the one before
// drains.
#include <cuda_runtime.h>

#include "gdr_nvtx.h"
#include "glr_tile.cuh"

namespace lt2 {
namespace glr {

constexpr int kSeg = kGlrChunk;        // tokens of a segment
constexpr int kSplitThreads = 128;
constexpr int kStep = 8;               // tokens whose loads are on their way together

struct SplitParams {
    ScanParams s;
    int64_t segs;          // segments of a sequence
    int64_t slots;         // pairs of channels (single channels for an odd width) of a unit
    int64_t threads;       // units * segs * slots
    int64_t channels;      // units * d
    float2* maps;          // [unit][channel][segment]: A and H (M)
    float* carries;        // [unit][segment][channel]: the state (mu) that enters each segment
    const float* first;    // the state that enters the first segment: S0, dS_L or null
};

// A thread's place: unit, segment, first channel, and the elements of its tokens.
template <bool PAIR>
struct Seg {
    int64_t unit, seg, ch, base;
    int tokens;
    __device__ __forceinline__ Seg(const SplitParams& p, int64_t id)
    {
        const int64_t slot = id % p.slots, rest = id / p.slots;
        ch = slot * (PAIR ? 2 : 1);
        seg = rest % p.segs;
        unit = rest / p.segs;
        const int64_t t0 = seg * kSeg;
        tokens = p.s.L - t0 < kSeg ? static_cast<int>(p.s.L - t0) : kSeg;
        base = (unit * p.s.L + t0) * p.s.d + ch;
    }
    __device__ __forceinline__ int64_t state(const SplitParams& p) const { return (unit * p.segs + seg) * p.s.d + ch; }
};
// One or two channels.
template <bool PAIR, typename T>
__device__ __forceinline__ f2 get(const T* p)
{
    if constexpr (PAIR)
        return load2(p);
    else
        return pack2(to_f32<T>(*p), 0.f);
}
template <bool PAIR, typename T>
__device__ __forceinline__ void put(T* p, f2 v)
{
    if constexpr (PAIR) {
        put2(p, v);
    } else {
        float a, b;
        unpack2(v, a, b);
        put1(p, a);
    }
}
template <bool PAIR>
__device__ __forceinline__ void put_as(void* p, int64_t i, int bf16, f2 v)
{
    if (bf16)
        put<PAIR>(static_cast<__nv_bfloat16*>(p) + i, v);
    else
        put<PAIR>(static_cast<float*>(p) + i, v);
}

// Decays and inputs of tokens [t, t + 8) of a segment; those behind its end are the identity.
template <typename XT, typename GT, bool LOGITS, bool PAIR>
__device__ __forceinline__ void tokens_at(const ScanParams& p, int64_t base, int t, int tokens, Tokens& k)
{
    static_assert(kStep == kTokens, "");
    const int64_t at = base + t * p.d;
    const GT* a = static_cast<const GT*>(p.alpha) + at;
    const XT* x = static_cast<const XT*>(p.x) + at;
    const GT* b = p.beta ? static_cast<const GT*>(p.beta) + at : nullptr;
    f2 bv[kStep];
    #pragma unroll
    for (int i = 0; i < kStep; ++i) {
        const bool in = t + i < tokens;
        k.al[i] = in ? get<PAIR>(a + i * p.d) : both(0.f);
        k.u[i] = in ? get<PAIR>(x + i * p.d) : both(0.f);
        bv[i] = in && b ? get<PAIR>(b + i * p.d) : both(1.f);
    }
    if (LOGITS) {
        #pragma unroll
        for (int i0 = 0; i0 < kStep; i0 += kBlock) {
            f2 v[kBlock];
            #pragma unroll
            for (int i = 0; i < kBlock; ++i) v[i] = k.al[i0 + i];
            decay_of_logits<kBlock>(v, both(-p.scale));
            #pragma unroll
            for (int i = 0; i < kBlock; ++i) k.al[i0 + i] = v[i];
        }
    }
    if (b) {
        #pragma unroll
        for (int i = 0; i < kStep; ++i) k.u[i] = mul2(k.u[i], LOGITS ? sigmoid_of(bv[i]) : bv[i]);
    }
    #pragma unroll
    for (int i = 0; i < kStep; ++i)
        if (t + i >= tokens) {
            k.al[i] = both(1.f);
            k.u[i] = both(0.f);
        }
}

template <bool PAIR>
__device__ __forceinline__ void put_map(const SplitParams& p, const Seg<PAIR>& s, f2 A, f2 H)
{
    float a0, a1, h0, h1;
    unpack2(A, a0, a1);
    unpack2(H, h0, h1);
    float2* m = p.maps + (s.unit * p.s.d + s.ch) * p.segs + s.seg;
    m[0] = make_float2(a0, h0);
    if (PAIR) m[p.segs] = make_float2(a1, h1);
    if (!isfinite(a0) || (PAIR && !isfinite(a1))) atomicOr(p.s.err, kDevRange);
}

template <typename XT, typename GT, bool LOGITS, bool PAIR>
__global__ void __launch_bounds__(kSplitThreads) glr_split_map_kernel(const __grid_constant__ SplitParams p)
{
    allow_next_loop_to_start();
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kSplitThreads + threadIdx.x;
    if (id >= p.threads) return;
    const Seg<PAIR> s(p, id);
    f2 A = both(1.f), H = both(0.f);
    for (int t = 0; t < s.tokens; t += kStep) {
        Tokens k;
        tokens_at<XT, GT, LOGITS, PAIR>(p.s, s.base, t, s.tokens, k);
        #pragma unroll
        for (int i = 0; i < kStep; ++i) {
            A = mul2(A, k.al[i]);
            H = fma2(k.al[i], H, k.u[i]);
        }
    }
    put_map<PAIR>(p, s, A, H);
}

template <typename XT, typename GT, bool LOGITS, bool PAIR>
__global__ void __launch_bounds__(kSplitThreads) glr_split_backward_map_kernel(const __grid_constant__ SplitParams p)
{
    allow_next_loop_to_start();
    asm volatile("griddepcontrol.wait;" ::: "memory");     // the states may be the launch's before
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kSplitThreads + threadIdx.x;
    if (id >= p.threads) return;
    const Seg<PAIR> s(p, id);
    const XT* g = static_cast<const XT*>(p.s.dO) + s.base;
    f2 A = both(1.f), M = both(0.f);
    for (int t = (s.tokens - 1) / kStep * kStep; t >= 0; t -= kStep) {
        Tokens k;
        tokens_at<XT, GT, LOGITS, PAIR>(p.s, s.base, t, s.tokens, k);
        f2 gv[kStep];
        #pragma unroll
        for (int i = 0; i < kStep; ++i) gv[i] = t + i < s.tokens ? get<PAIR>(g + (t + i) * p.s.d) : both(0.f);
        #pragma unroll
        for (int i = kStep - 1; i >= 0; --i) {
            A = mul2(A, k.al[i]);
            M = mul2(k.al[i], add2(gv[i], M));
        }
    }
    put_map<PAIR>(p, s, A, M);
}

// A warp per channel: lane j holds the map of segment j of 32, and the carry passes over them one after another, as it does from
// tile to tile: a product of maps over more than a segment may overflow where the state itself does not.  REVERSE: from
// the last segment to the first.
template <bool REVERSE>
__global__ void __launch_bounds__(kSplitThreads) glr_split_carry_kernel(const __grid_constant__ SplitParams p)
{
    allow_next_loop_to_start();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * (kSplitThreads / 32) + (threadIdx.x >> 5);
    if (c >= p.channels) return;
    const int64_t unit = c / p.s.d, ch = c - unit * p.s.d;
    const float2* m = p.maps + c * p.segs;
    auto at = [&](int64_t i) { return REVERSE ? p.segs - 1 - i : i; };
    auto map_of = [&](int64_t i) { return i < p.segs ? m[at(i)] : make_float2(1.f, 0.f); };
    float carry = p.first ? p.first[c] : 0.f;
    float2 next = map_of(lane);
    for (int64_t i0 = 0; i0 < p.segs; i0 += 32) {
        const float2 v = next;
        next = map_of(i0 + 32 + lane);                     // under the chain of this group's
        float mine = carry;
        #pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (lane == j) mine = carry;
            carry = fmaf(__shfl_sync(0xffffffffu, v.x, j), carry, __shfl_sync(0xffffffffu, v.y, j));
        }
        if (i0 + lane < p.segs) p.carries[(unit * p.segs + at(i0 + lane)) * p.s.d + ch] = mine;
    }
}

template <typename XT, typename GT, bool LOGITS, bool PAIR>
__global__ void __launch_bounds__(kSplitThreads) glr_split_run_kernel(const __grid_constant__ SplitParams p)
{
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kSplitThreads + threadIdx.x;
    if (id >= p.threads) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const Seg<PAIR> s(p, id);
    Tokens k;
    tokens_at<XT, GT, LOGITS, PAIR>(p.s, s.base, 0, s.tokens, k);      // under the launch before
    asm volatile("griddepcontrol.wait;" ::: "memory");
    f2 h = get<PAIR>(p.carries + s.state(p));
    for (int t = 0; t < s.tokens; t += kStep) {
        if (t > 0) tokens_at<XT, GT, LOGITS, PAIR>(p.s, s.base, t, s.tokens, k);
        #pragma unroll
        for (int i = 0; i < kStep; ++i) {
            h = fma2(k.al[i], h, k.u[i]);
            if (t + i < s.tokens) put_as<PAIR>(p.s.o, s.base + (t + i) * p.s.d, p.s.out_bf16, h);
        }
    }
    if (p.s.S_out && s.seg + 1 == p.segs) put<PAIR>(p.s.S_out + s.unit * p.s.d + s.ch, h);
}

template <typename XT, typename GT, bool LOGITS, bool PAIR>
__global__ void __launch_bounds__(kSplitThreads) glr_split_backward_run_kernel(const __grid_constant__ SplitParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kSplitThreads + threadIdx.x;
    if (id >= p.threads) return;
    const Seg<PAIR> s(p, id);
    const ScanParams& q = p.s;
    // the state in front of every eight tokens, then the eights from the last
    f2 at[kSeg / kStep];
    f2 h = get<PAIR>(q.states + s.state(p));
    at[0] = h;                                             // (the last eight are run once)
    #pragma unroll 1
    for (int t = 0; t + kStep < s.tokens; t += kStep) {
        Tokens k;
        tokens_at<XT, GT, LOGITS, PAIR>(q, s.base, t, s.tokens, k);
        #pragma unroll
        for (int i = 0; i < kStep; ++i) h = fma2(k.al[i], h, k.u[i]);
        at[t / kStep + 1] = h;
    }
    f2 m = p.carries ? get<PAIR>(p.carries + s.state(p)) : both(0.f);
    const f2 nc = both(-q.scale);
    #pragma unroll 1
    for (int t = (s.tokens - 1) / kStep * kStep; t >= 0; t -= kStep) {
        Tokens k;
        tokens_at<XT, GT, LOGITS, PAIR>(q, s.base, t, s.tokens, k);
        h = at[t / kStep];
        #pragma unroll
        for (int i = 0; i < kStep; ++i) {
            const f2 next = fma2(k.al[i], h, k.u[i]);
            k.u[i] = h;
            h = next;
        }
        #pragma unroll
        for (int i = kStep - 1; i >= 0; --i) {
            if (t + i >= s.tokens) continue;
            const int64_t e = s.base + (t + i) * q.d;
            const f2 lam = add2(get<PAIR>(static_cast<const XT*>(q.dO) + e), m);
            m = mul2(k.al[i], lam);
            f2 da = mul2(k.u[i], lam);
            if (LOGITS) da = mul2(mul2(da, k.al[i]), mul2(sigmoid_of(get<PAIR>(static_cast<const GT*>(q.alpha) + e)), nc));
            put_as<PAIR>(q.dalpha, e, q.dg_bf16, da);
            f2 dx = lam;
            if (q.beta) {
                f2 bv = get<PAIR>(static_cast<const GT*>(q.beta) + e);
                f2 db = mul2(get<PAIR>(static_cast<const XT*>(q.x) + e), lam);
                if (LOGITS) {
                    const f2 eb = exp_minus(bv);           // beta (1 - beta) = e beta^2
                    bv = sigmoid_from(eb);
                    db = mul2(db, mul2(bv, mul2(bv, eb)));
                }
                put_as<PAIR>(q.dbeta, e, q.dg_bf16, db);
                dx = mul2(lam, bv);
            }
            put_as<PAIR>(q.dx, e, q.dx_bf16, dx);
        }
    }
    if (q.dS0 && s.seg == 0) put<PAIR>(q.dS0 + s.unit * q.d + s.ch, m);
}

SplitParams split_params(const GlrCall& c, const ScanParams& s)
{
    SplitParams p;
    p.s = s;
    p.segs = (c.L + kSeg - 1) / kSeg;
    p.slots = c.d % 2 == 0 ? c.d / 2 : c.d;
    p.threads = c.units * p.segs * p.slots;
    p.channels = c.units * c.d;
    p.maps = static_cast<float2*>(c.workspace);
    p.carries = reinterpret_cast<float*>(p.maps + p.channels * p.segs);
    p.first = nullptr;
    return p;
}

template <typename K>
cudaError_t launch_split(K kernel, const SplitParams& p, int64_t threads, bool early, cudaStream_t stream)
{
    const int64_t grid = (threads + kSplitThreads - 1) / kSplitThreads;
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename XT, typename GT, bool LOGITS, bool PAIR>
cudaError_t split_forward(const GlrCall& c, cudaStream_t stream)
{
    SplitParams p = split_params(c, params_of(c, layout_of(c.units, c.L, c.d, kChannels)));
    p.first = c.S0;
    if (c.states) p.carries = c.states;
    cudaError_t e = launch_split(glr_split_map_kernel<XT, GT, LOGITS, PAIR>, p, p.threads, false, stream);
    if (e == cudaSuccess) e = launch_split(glr_split_carry_kernel<false>, p, p.channels * 32, true, stream);
    if (e == cudaSuccess && c.o) e = launch_split(glr_split_run_kernel<XT, GT, LOGITS, PAIR>, p, p.threads, true, stream);
    return e;
}
template <typename XT, typename GT, bool LOGITS>
cudaError_t split_forward_typed(const GlrCall& c, cudaStream_t stream)
{
    return c.d % 2 == 0 ? split_forward<XT, GT, LOGITS, true>(c, stream) : split_forward<XT, GT, LOGITS, false>(c, stream);
}

template <typename XT, typename GT, bool LOGITS, bool PAIR>
cudaError_t split_backward(const GlrBackwardCall& b, cudaStream_t stream)
{
    const GlrCall& c = b.f;
    SplitParams p = split_params(c, params_of(b, layout_of(c.units, c.L, c.d, kChannels)));
    p.first = b.dS_L;
    if (p.segs == 1) {                                     // nothing to pass on: dS_L enters the one segment
        p.carries = const_cast<float*>(b.dS_L);
        return launch_split(glr_split_backward_run_kernel<XT, GT, LOGITS, PAIR>, p, p.threads, false, stream);
    }
    cudaError_t e = launch_split(glr_split_backward_map_kernel<XT, GT, LOGITS, PAIR>, p, p.threads, false, stream);
    if (e == cudaSuccess) e = launch_split(glr_split_carry_kernel<true>, p, p.channels * 32, true, stream);
    if (e == cudaSuccess) e = launch_split(glr_split_backward_run_kernel<XT, GT, LOGITS, PAIR>, p, p.threads, true, stream);
    return e;
}
template <typename XT, typename GT, bool LOGITS>
cudaError_t split_backward_typed(const GlrBackwardCall& b, cudaStream_t stream)
{
    return b.f.d % 2 == 0 ? split_backward<XT, GT, LOGITS, true>(b, stream) : split_backward<XT, GT, LOGITS, false>(b, stream);
}

}  // namespace glr

size_t glr_split_workspace_bytes(int64_t units, int64_t L, int64_t d)
{
    const size_t n = static_cast<size_t>(units) * d * ((L + glr::kSeg - 1) / glr::kSeg);
    return (n * 12 + 255) / 256 * 256;
}

// Units of up to 16 channels, longer than a segment: 225 units of 18,913
// tokens x 1, training pass, 358 us against 2,540 in tiles; 2 x 16 x 16 units of 4,096 x 8, prefill, 103 against 328.
// At 20 channels the two meet (training 300 against 281 us), and full tiles are faster at any size (16 units of 512 x
// 128: 32 against 7.6 us), since a thread takes its segment's 64 tokens one after another, twice.
bool glr_splits(int64_t, int64_t L, int64_t d) { return d <= 16 && L > glr::kSeg; }

cudaError_t launch_glr_split(const GlrCall& c, cudaStream_t stream)
{
    NvtxRange range("lt2 gated linear recurrence (split)");
    LT2_GLR_DISPATCH(c, glr::split_forward_typed, c, stream);
}

// Up to eight tokens, as the forward pass walks them: a thread runs its tokens in a row from the state in front (8 x 218 x
// 10 units of 158 channels, 2 tokens, forward and backward: 565 us in tiles, 86 so; 4 x 16 x 16 units of 128, 8 tokens 27
// against 20, 16 tokens the same).
bool glr_backward_walks(int64_t units, int64_t L, int64_t d)
{
    return L == 1 || (L <= 8 && units * ((d + 1) / 2) >= 148 * 256);
}

cudaError_t launch_glr_split_backward(const GlrBackwardCall& b, cudaStream_t stream)
{
    NvtxRange range("lt2 gated linear recurrence (split, backward)");
    LT2_GLR_DISPATCH(b.f, glr::split_backward_typed, b, stream);
}

}  // namespace lt2
