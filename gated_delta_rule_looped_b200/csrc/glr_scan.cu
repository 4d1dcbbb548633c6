// glr_scan.cu -- the gated linear recurrence over long sequences where the channels alone do not fill the
// GPU: CTA = one tile of 64 tokens x 64 channels (glr_tile.cuh), and the carry that enters a tile comes from the
// tiles before it, which other CTAs work on (glr_common.cuh).  One pass: each input crosses HBM once and
// each output once; what the tiles exchange is 12 bytes per channel and 64 tokens.
//
// A tile's time is a chain of latencies, in cycles as measured inside the kernel: its ticket 1,100, its rows 2,700, its
// maps 2,800, its carry 2,200, its second half 800.  So three CTAs per SM share it
// (for which a thread keeps up to 48 bytes in local memory), and a small call takes a few such
// chains (16 units of 2,048 x 128 bf16 with logits: 16.4 us, where HBM would take 5).  CTAs that stay and load ahead
// hold tickets that others wait for, and were slower (30 us); where there are channels enough, glr_stream.cu needs
// no such waits.
#include <cuda_runtime.h>

#include "gdr_nvtx.h"
#include "glr_tile.cuh"

namespace lt2 {
namespace glr {

constexpr int CB = kChannels;
using Sh = Shape<CB>;
constexpr int kScanThreads = 32 * kWarps;

// Tickets go tile by tile through all chains, so a tile's predecessors have lower tickets and are at work or done
// (and neighbouring CTAs read neighbouring channels of the same rows).
template <bool REVERSE>
__device__ __forceinline__ Tile take_tile(const ScanParams& p, unsigned* slot)
{
    unsigned id = blockIdx.x;
    if (p.ticket) {
        if (threadIdx.x == 0) *slot = atomicAdd(p.ticket, 1u) + 1u;      // the counter starts at all ones
        __syncthreads();
        id = *slot;
    }
    const int step = static_cast<int>(id / p.nchains);
    return tile_at<CB, REVERSE>(p, id - static_cast<unsigned>(step) * p.nchains, step);
}

// One warp: publishes the tile's map, fetches the carry that enters (`first` where the tile is its chain's first),
// publishes the one that leaves.
__device__ __forceinline__ f2 hand_over(const ScanParams& p, const Tile& t, f2 A, f2 H, f2 first)
{
    float a, b;
    unpack2(A, a, b);
    const int ch = Sh::lane_channel();
    if ((ch < t.chans && !isfinite(a)) || (ch + 1 < t.chans && !isfinite(b))) atomicOr(p.err, kDevRange);
    f2 carry = first;
    if (p.ticket) {
        const int64_t chain = static_cast<int64_t>(t.chain) * p.ntiles * CB + ch;
        const int64_t here = chain + static_cast<int64_t>(t.step) * CB;
        const bool last = t.step + 1 == p.ntiles;
        if (t.step > 0) {
            if (!last) publish_map(p.maps + here, A, H);
            carry = carry_into(p.maps + chain, p.carries + chain, t.step, p.err);
        }
        if (!last) publish_carry(p.carries + here, fma2(A, carry, H));
    }
    return carry;
}

template <typename XT, typename GT, bool LOGITS>
__global__ void __launch_bounds__(kScanThreads, 3) glr_scan_kernel(const __grid_constant__ ScanParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float sA[kWarps][CB], sH[kWarps][CB], sC[CB];
    __shared__ unsigned slot;
    const Tile t = take_tile<false>(p, &slot);
    const Stage<XT, GT, CB, false> st(smem, 0);
    const Place w = place_of<XT, GT, CB>(p);
    st.fill(p, t, w);
    cp_async_commit();
    const int warp = threadIdx.x >> 5, ch = Sh::lane_channel();
    f2 first = 0;
    if (warp == 0 && t.step == 0 && p.S0) first = load_state(p.S0 + t.state, ch, t.chans);
    cp_async_wait<0>();
    __syncwarp();

    Tokens k;
    f2 A, H;
    map_tokens<XT, GT, LOGITS, CB, true>(p, st, t.rows, k, A, H);
    pair_of(sA[warp], ch) = A;
    pair_of(sH[warp], ch) = H;
    __syncthreads();
    if (warp == 0) {
        // the map of the tokens in front of each warp's, in place of its own
        A = both(1.f);
        H = both(0.f);
        #pragma unroll
        for (int v = 0; v < kWarps; ++v) {
            const f2 a = pair_of(sA[v], ch), h = pair_of(sH[v], ch);
            pair_of(sA[v], ch) = A;
            pair_of(sH[v], ch) = H;
            H = fma2(a, H, h);
            A = mul2(A, a);
        }
        pair_of(sC, ch) = hand_over(p, t, A, H, first);
    }
    __syncthreads();
    run_tokens<CB, true>(p, t, w, k, fma2(pair_of(sA[warp], ch), pair_of(sC, ch), pair_of(sH[warp], ch)));
}

template <typename XT, typename GT, bool LOGITS>
__global__ void __launch_bounds__(kScanThreads, 3) glr_scan_backward_kernel(const __grid_constant__ ScanParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float sA[kWarps][CB], sH[kWarps][CB], sM[kWarps][CB], sB[kWarps][CB], sC[CB];
    __shared__ unsigned slot;
    const Tile t = take_tile<true>(p, &slot);              // from the last token to the first
    const Stage<XT, GT, CB, true> st(smem, 0);
    const Place w = place_of<XT, GT, CB>(p);
    st.fill(p, t, w);
    cp_async_commit();
    const int warp = threadIdx.x >> 5, ch = Sh::lane_channel();
    // under the copies: the gradient behind the sequence, and the state in front of the tile
    f2 first = 0;
    if (warp == 0 && t.step == 0 && p.dS_L) first = load_state(p.dS_L + t.state, ch, t.chans);
    f2 h = load_state(p.states + t.kept, ch, t.chans);
    cp_async_wait<0>();
    __syncwarp();

    Tokens k;
    f2 A, H;
    map_tokens<XT, GT, LOGITS, CB, true>(p, st, t.rows, k, A, H);
    pair_of(sA[warp], ch) = A;
    pair_of(sH[warp], ch) = H;
    pair_of(sM[warp], ch) = map_gradients<CB>(st, t.rows, k);
    __syncthreads();
    // the state that enters this warp's tokens
    for (int v = 0; v < warp; ++v) h = fma2(pair_of(sA[v], ch), h, pair_of(sH[v], ch));
    if (warp == 0) {
        // the map of the tokens behind each warp's
        A = both(1.f);
        f2 M = both(0.f);
        #pragma unroll
        for (int v = kWarps - 1; v >= 0; --v) {
            const f2 a = pair_of(sA[v], ch), m = pair_of(sM[v], ch);
            pair_of(sB[v], ch) = A;
            pair_of(sM[v], ch) = M;
            M = fma2(a, M, m);
            A = mul2(A, a);
        }
        pair_of(sC, ch) = hand_over(p, t, A, M, first);
    }
    __syncthreads();
    run_gradients<XT, GT, LOGITS, CB>(p, t, w, st, k, h, fma2(pair_of(sB[warp], ch), pair_of(sC, ch), pair_of(sM[warp], ch)));
}

template <typename K>
cudaError_t run_scan(K kernel, ScanParams p, const Layout& l, void* workspace, size_t ws_bytes, size_t smem,
                     cudaStream_t stream)
{
    if (l.ntiles > 1) {
        uint8_t* w = static_cast<uint8_t*>(workspace);
        p.ticket = reinterpret_cast<unsigned int*>(w);
        p.maps = reinterpret_cast<uint64_t*>(w + 256);
        p.carries = reinterpret_cast<uint32_t*>(w + 256 + static_cast<int64_t>(l.tiles) * CB * 8);
        const cudaError_t e = cudaMemsetAsync(workspace, 0xff, ws_bytes, stream);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    kernel<<<p.total, kScanThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <typename XT, typename GT, bool LOGITS>
cudaError_t forward_typed(const GlrCall& c, cudaStream_t stream)
{
    const Layout l = layout_of(c.units, c.L, c.d, CB);
    return run_scan(glr_scan_kernel<XT, GT, LOGITS>, params_of(c, l), l, c.workspace,
                    glr_scan_workspace_bytes(c.units, c.L, c.d), Stage<XT, GT, CB, false>::kBytes, stream);
}
template <typename XT, typename GT, bool LOGITS>
cudaError_t backward_typed(const GlrBackwardCall& b, cudaStream_t stream)
{
    const GlrCall& c = b.f;
    const Layout l = layout_of(c.units, c.L, c.d, CB);
    return run_scan(glr_scan_backward_kernel<XT, GT, LOGITS>, params_of(b, l), l, c.workspace,
                    glr_scan_workspace_bytes(c.units, c.L, c.d), Stage<XT, GT, CB, true>::kBytes, stream);
}

}  // namespace glr

__int128 glr_scan_tiles(int64_t units, int64_t L, int64_t d) { return glr::layout_of(units, L, d, glr::CB).tiles; }

size_t glr_scan_workspace_bytes(int64_t units, int64_t L, int64_t d)
{
    const glr::Layout l = glr::layout_of(units, L, d, glr::CB);
    if (l.ntiles <= 1) return 0;
    return (256 + static_cast<size_t>(l.tiles) * glr::CB * 12 + 255) / 256 * 256;
}

cudaError_t launch_glr_scan(const GlrCall& c, cudaStream_t stream)
{
    NvtxRange range("lt2 gated linear recurrence (scan)");
    LT2_GLR_DISPATCH(c, glr::forward_typed, c, stream);
}

cudaError_t launch_glr_scan_backward(const GlrBackwardCall& b, cudaStream_t stream)
{
    NvtxRange range("lt2 gated linear recurrence (scan, backward)");
    LT2_GLR_DISPATCH(b.f, glr::backward_typed, b, stream);
}

}  // namespace lt2
