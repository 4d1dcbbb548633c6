// glr_stream.cu -- the gated linear recurrence over long sequences where there are channels enough to fill the
// GPU: CTAs that stay, an equal share of all chains' tiles each, the state passed on inside the CTA.
//
// A chain is one unit's block of 64 (or 32) channels.  The tiles of all chains, chain by chain, are dealt out
// evenly; with at least as many chains as CTAs, a share is the end of one chain, some whole chains and
// the start of another.  The CTA takes the start first and publishes the state that leaves it, then the whole
// chains, and last the end, whose entering state the CTA before it published long ago.  So nobody waits, and
// each input crosses HBM once and each output once.
//
// Eight warps work on the tokens; a ninth passes the state over the groups' maps (glr_tile.cuh) and describes the
// tiles to come.  The eight do the first half of the next tile before the second half of the present one,
// and each copies its own rows two tiles ahead: loads and hand-overs run under the arithmetic, whose latency at 18 warps per
// SM (two CTAs, up to 44 bytes of a thread in local memory) bounds the kernel with logits (35 instructions an element on 54 % of the issue slots; 4 x 4 x 16 units of 8,192 x 128
// bf16: 470 us with logits, 372 us with decays as values, where HBM's copy rate would take 327).
#include <cuda_runtime.h>

#include "gdr_nvtx.h"
#include "glr_tile.cuh"
#include "per_device.h"

namespace lt2 {
namespace glr {

constexpr int kStreamThreads = 32 * (kWarps + 1);

// What the warps of a CTA share.  Tile n uses the places n % 2 of the maps and n % 8 of the descriptions.
// The hand-overs are named barriers, one each for even and for odd tiles:
//   kMaps:   the eight warps have written their maps of tile n    -> the ninth passes the state over them
//   kCarry:  the ninth warp is done with tile n, and has described tile n + 3
// A warp writes its maps of tile n + 2 behind its own second half of tile n, and the ninth writes places of tile
// n + 2 behind kMaps of it, when all eight have left tile n.  So no place is written before it has been read.
template <int CB>
struct Shared {
    float A[2][Shape<CB>::kGroups][CB];    // maps of the forward recurrence
    float H[2][Shape<CB>::kGroups][CB];    // then the states that enter the groups
    Tile tile[8];
    unsigned index;
};
template <int CB>
struct SharedBackward : Shared<CB> {
    float M[2][Shape<CB>::kGroups][CB];    // maps of the reverse recurrence, with A; then the mu that enter
};
enum : int { kMaps = 1, kCarry = 3 };

__device__ __forceinline__ void bar_arrive(int id)
{
    __syncwarp();
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kStreamThreads) : "memory");
}
__device__ __forceinline__ void bar_wait(int id)
{
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kStreamThreads) : "memory");
}

// A CTA's share, in the order of its work: `start` tiles of the chain that it begins, `whole` tiles of whole
// chains, `end` tiles of the chain that the CTA before it began.  Tiles are numbered chain by chain.
struct Share {
    unsigned start, whole, end;
    unsigned at_start, at_whole, at_end;
    __device__ __forceinline__ Share(const ScanParams& p, unsigned index)
    {
        const unsigned n = p.ntiles;
        const unsigned lo = static_cast<unsigned>(static_cast<uint64_t>(p.total) * index / gridDim.x);
        const unsigned hi = static_cast<unsigned>(static_cast<uint64_t>(p.total) * (index + 1) / gridDim.x);
        at_end = lo;
        at_whole = (lo + n - 1) / n * n;
        at_start = hi / n * n;
        end = at_whole - lo;
        whole = at_start - at_whole;
        start = hi - at_start;
    }
    __device__ __forceinline__ unsigned count() const { return start + whole + end; }
    template <int CB, bool REVERSE>
    __device__ __forceinline__ Tile tile(const ScanParams& p, unsigned n) const
    {
        Tile t;
        t.valid = 0;
        if (n >= count()) return t;
        const unsigned id = n < start ? at_start + n : n < start + whole ? at_whole + (n - start) : at_end + (n - start - whole);
        const unsigned chain = id / static_cast<unsigned>(p.ntiles);
        return tile_at<CB, REVERSE>(p, chain, static_cast<int>(id - chain * static_cast<unsigned>(p.ntiles)));
    }
};

// The CTA's share goes by the order in which CTAs start, so the CTA before it, whose state it needs at the end, has
// started; that one publishes the state without waiting.
template <int CB, bool REVERSE, typename SH>
__device__ __forceinline__ Share open_share(const ScanParams& p, SH& sh)
{
    if (threadIdx.x == 0) sh.index = p.ticket ? atomicAdd(p.ticket, 1u) + 1u : blockIdx.x;    // from all ones
    __syncthreads();
    const Share share(p, sh.index);
    if (threadIdx.x < 3) sh.tile[threadIdx.x] = share.template tile<CB, REVERSE>(p, threadIdx.x);
    __syncthreads();
    return share;
}

// The state that the CTA before published for a channel; bounded as every wait.
__device__ __forceinline__ float published_state(const uint32_t* p, unsigned int* err)
{
    uint64_t t0 = 0;
    for (uint32_t spins = 1;; ++spins) {
        uint32_t v;
        asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
        if (v != kNotYet) return __uint_as_float(v);
        if ((spins & 63u) == 0u) {
            const uint64_t now = sm100::global_timer_ns();
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > tcc::kWaitTimeoutNs) {
                atomicOr(err, kDevTimeout);
                return __uint_as_float(kNan);
            }
        }
    }
}

// The ninth warp: lane j owns channels j (and j + 32) of the tiles.  fetch(tile, channel): what the
// tile needs from global memory; pass(tile, parity, channel, carry, fetched) -> the state behind the tile.
template <int CB, bool REVERSE, typename SH, typename FETCH, typename PASS>
__device__ __forceinline__ void carry_warp(const ScanParams& p, SH& sh, const Share& share, const float* first, FETCH fetch,
                                           PASS pass)
{
    constexpr int N = CB / 32;
    const int lane = threadIdx.x & 31;
    float carry[N] = {}, fetched[N];
    for (unsigned n = 0; n < share.count(); ++n) {
        const int par = n & 1;
        const Tile t = sh.tile[n & 7];
        #pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = lane + 32 * j;
            fetched[j] = fetch(t, c);
            if (t.step == 0)
                carry[j] = first && c < t.chans ? first[t.state + c] : 0.f;
            else if (n == share.start + share.whole)
                carry[j] = published_state(p.carries + static_cast<int64_t>(t.chain) * CB + c, p.err);
        }
        bar_wait(kMaps + par);
        #pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = lane + 32 * j;
            carry[j] = pass(t, par, c, carry[j], fetched[j]);
            if (n + 1 == share.start) {
                const uint32_t w = word_of(carry[j]);
                asm volatile("st.relaxed.gpu.global.u32 [%0], %1;"
                             ::"l"(p.carries + static_cast<int64_t>(t.chain) * CB + c), "r"(w) : "memory");
            }
        }
        if (lane == 0) sh.tile[(n + 3) & 7] = share.template tile<CB, REVERSE>(p, n + 3);
        bar_arrive(kCarry + par);
    }
}

// Passes a state over the groups' maps of one channel in the order first, first + dir, ...: each group's H becomes
// the state that enters it.  A map that is not finite is reported.
template <int CB>
__device__ __forceinline__ float pass_state(float (*A)[CB], float (*H)[CB], int c, float s, bool report, unsigned int* err,
                                            bool reverse)
{
    constexpr int G = Shape<CB>::kGroups;
    float a[G], h[G];
    #pragma unroll
    for (int g = 0; g < G; ++g) {
        a[g] = A[g][c];
        h[g] = H[g][c];
    }
    bool fine = true;
    #pragma unroll
    for (int i = 0; i < G; ++i) {
        const int g = reverse ? G - 1 - i : i;
        fine = fine && isfinite(a[g]);
        H[g][c] = s;
        s = fmaf(a[g], s, h[g]);
    }
    if (report && !fine) atomicOr(err, kDevRange);
    return s;
}

template <typename XT, typename GT, bool LOGITS, int CB>
__global__ void __launch_bounds__(kStreamThreads, 2) glr_stream_kernel(const __grid_constant__ ScanParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) Shared<CB> sh;
    using Table = typename std::conditional<LOGITS && sizeof(GT) == 2, DecayTable, NoTable>::type;
    __shared__ __align__(16) Table table;
    const int warp = threadIdx.x >> 5;
    table.build(p.scale, threadIdx.x, kStreamThreads);     // open_share's barriers follow
    const Share share = open_share<CB, false>(p, sh);
    if (warp == kWarps) {
        carry_warp<CB, false>(p, sh, share, p.S0, [](const Tile&, int) { return 0.f; },
                              [&](const Tile& t, int par, int c, float s, float) {
            return pass_state<CB>(sh.A[par], sh.H[par], c, s, c < t.chans, p.err, false);
        });
        return;
    }
    using St = Stage<XT, GT, CB, false>;
    const int ch = Shape<CB>::lane_channel(), g = Shape<CB>::group();
    const Place w = place_of<XT, GT, CB>(p);
    auto first_half = [&](unsigned n, Tokens& k) {
        f2 A, H;
        map_tokens<XT, GT, LOGITS, CB, false>(p, St(smem, n & 1), sh.tile[n & 7].rows, k, A, H, &table);
        pair_of(sh.A[n & 1][g], ch) = A;
        pair_of(sh.H[n & 1][g], ch) = H;
        bar_arrive(kMaps + (n & 1));
    };
    auto fill = [&](unsigned n) {
        if (sh.tile[n & 7].valid) St(smem, n & 1).fill(p, sh.tile[n & 7], w);
        cp_async_commit();
    };
    if (!sh.tile[0].valid) return;
    fill(0);
    fill(1);
    Tokens even, odd;
    cp_async_wait<1>();
    __syncwarp();
    first_half(0, even);
    fill(2);
    // first half of tile n + 1, then the second half of tile n; false behind the last tile
    auto step = [&](unsigned n, Tokens& cur, Tokens& next) -> bool {
        const bool more = sh.tile[(n + 1) & 7].valid;
        if (more) {
            cp_async_wait<1>();
            __syncwarp();
            first_half(n + 1, next);
        }
        bar_wait(kCarry + (n & 1));
        if (more) fill(n + 3);                             // over tile n + 1's rows, which the warp has read
        run_tokens<CB, false>(p, sh.tile[n & 7], w, cur, pair_of(sh.H[n & 1][g], ch));
        return more;
    };
    for (unsigned n = 0;; n += 2) {
        if (!step(n, even, odd)) break;
        if (!step(n + 1, odd, even)) break;
    }
}

// The backward pass takes its tiles in one of two ways.  With a table of decays (bf16 logits) one tile after the other,
// two stages: two sets of tokens and a third stage would leave no room for the table, which is worth more (forward and
// backward pass of 4 x 4 x 16 units of 8,192 x 128: 1,518 -> 1,464 us).  Without one the first half of the next tile
// precedes the second half of the present, three stages (2 x 4 x 32 units of 4,096 x 128 with fp32 decays: 810 us
// against 870).  Neither is unrolled: the code would outgrow the instruction cache (1,570 us against 1,530).
template <typename GT, bool LOGITS>
constexpr bool kBackwardTable = LOGITS && sizeof(GT) == 2;
template <typename GT, bool LOGITS>
constexpr int kBackwardStages = kBackwardTable<GT, LOGITS> ? 2 : 3;

template <typename XT, typename GT, bool LOGITS, int CB>
__global__ void __launch_bounds__(kStreamThreads, sizeof(GT) == 2 ? 2 : 1)
glr_stream_backward_kernel(const __grid_constant__ ScanParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) SharedBackward<CB> sh;
    using Table = typename std::conditional<kBackwardTable<GT, LOGITS>, DecayTable, NoTable>::type;
    __shared__ __align__(16) Table table;
    const int warp = threadIdx.x >> 5;
    table.build(p.scale, threadIdx.x, kStreamThreads);     // open_share's barriers follow
    const Share share = open_share<CB, true>(p, sh);
    if (warp == kWarps) {
        // the states that enter the groups, from the kept one in front of the tile; then the gradients
        carry_warp<CB, true>(p, sh, share, p.dS_L,
                             [&](const Tile& t, int c) { return c < t.chans ? p.states[t.kept + c] : 0.f; },
                             [&](const Tile& t, int par, int c, float mu, float h) {
            pass_state<CB>(sh.A[par], sh.H[par], c, h, false, p.err, false);
            return pass_state<CB>(sh.A[par], sh.M[par], c, mu, c < t.chans, p.err, true);
        });
        return;
    }
    using St = Stage<XT, GT, CB, true>;
    constexpr int STAGES = kBackwardStages<GT, LOGITS>;
    const int ch = Shape<CB>::lane_channel(), g = Shape<CB>::group();
    const Place w = place_of<XT, GT, CB>(p);
    auto first_half = [&](unsigned n, Tokens& k) {
        f2 A, H;
        const St st(smem, n % STAGES);
        map_tokens<XT, GT, LOGITS, CB, false>(p, st, sh.tile[n & 7].rows, k, A, H, &table);
        pair_of(sh.A[n & 1][g], ch) = A;
        pair_of(sh.H[n & 1][g], ch) = H;
        pair_of(sh.M[n & 1][g], ch) = map_gradients<CB>(st, sh.tile[n & 7].rows, k);
        bar_arrive(kMaps + (n & 1));
    };
    auto fill = [&](unsigned n) {
        if (sh.tile[n & 7].valid) St(smem, n % STAGES).fill(p, sh.tile[n & 7], w);
        cp_async_commit();
    };
    if (!sh.tile[0].valid) return;
    fill(0);
    fill(1);
    auto second_half = [&](unsigned n, Tokens& k) {
        bar_wait(kCarry + (n & 1));
        run_gradients<XT, GT, LOGITS, CB>(p, sh.tile[n & 7], w, St(smem, n % STAGES), k, pair_of(sh.H[n & 1][g], ch),
                                          pair_of(sh.M[n & 1][g], ch));
        __syncwarp();                                      // tile n's rows are free
    };
    Tokens cur;
    if constexpr (STAGES == 2) {
        #pragma unroll 1
        for (unsigned n = 0; sh.tile[n & 7].valid; ++n) {
            cp_async_wait<1>();
            __syncwarp();
            first_half(n, cur);
            second_half(n, cur);
            fill(n + 2);
        }
    } else {
        fill(2);
        Tokens next;
        cp_async_wait<2>();
        __syncwarp();
        first_half(0, cur);
        #pragma unroll 1
        for (unsigned n = 0;; ++n) {
            const bool more = sh.tile[(n + 1) & 7].valid;
            if (more) {
                cp_async_wait<1>();
                __syncwarp();
                first_half(n + 1, next);
            }
            second_half(n, cur);
            if (!more) break;
            fill(n + 3);
            cur = next;
        }
    }
}

// Scratch: the index counter, and the states that CTAs hand on.
inline size_t stream_bytes(__int128 chains, int channels)
{
    return (256 + static_cast<size_t>(chains) * channels * 4 + 255) / 256 * 256;
}

// CTAs of a kernel that the current GPU holds at once.
template <typename K>
cudaError_t resident_ctas(K kernel, size_t smem, PerDevice& kept, int* out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    *out = kept.get(dev, [&]() {
        int sms = 0, per = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
            (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kStreamThreads, smem)) != cudaSuccess)
            return 0;
        return sms * (per > 0 ? per : 1);
    });
    return e;
}

template <typename XT, typename GT, bool LOGITS, int CB, bool BACKWARD>
cudaError_t run_stream(ScanParams p, const Layout& l, void* workspace, cudaStream_t stream)
{
    void (*kernel)(const ScanParams);
    if constexpr (BACKWARD)
        kernel = glr_stream_backward_kernel<XT, GT, LOGITS, CB>;
    else
        kernel = glr_stream_kernel<XT, GT, LOGITS, CB>;
    const size_t smem = (BACKWARD ? kBackwardStages<GT, LOGITS> : 2) * Stage<XT, GT, CB, BACKWARD>::kBytes;
    static PerDevice kept;
    int ctas = 0;
    cudaError_t e = resident_ctas(kernel, smem, kept, &ctas);
    if (e != cudaSuccess) return e;
    const unsigned grid = l.chains < ctas ? static_cast<unsigned>(l.chains) : static_cast<unsigned>(ctas);
    if (l.chains % grid != 0) {                            // some chain is shared
        uint8_t* w = static_cast<uint8_t*>(workspace);
        p.ticket = reinterpret_cast<unsigned int*>(w);
        p.carries = reinterpret_cast<uint32_t*>(w + 256);
        e = cudaMemsetAsync(workspace, 0xff, stream_bytes(l.chains, CB), stream);
        if (e != cudaSuccess) return e;
    }
    kernel<<<grid, kStreamThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <typename XT, typename GT, bool LOGITS>
cudaError_t forward_typed(const GlrCall& c, cudaStream_t stream)
{
    const int cb = glr_stream_channels(c.units, c.L, c.d);
    const Layout l = layout_of(c.units, c.L, c.d, cb);
    return cb == 64 ? run_stream<XT, GT, LOGITS, 64, false>(params_of(c, l), l, c.workspace, stream)
                    : run_stream<XT, GT, LOGITS, 32, false>(params_of(c, l), l, c.workspace, stream);
}
template <typename XT, typename GT, bool LOGITS>
cudaError_t backward_typed(const GlrBackwardCall& b, cudaStream_t stream)
{
    const GlrCall& c = b.f;
    const int cb = glr_stream_channels(c.units, c.L, c.d);
    const Layout l = layout_of(c.units, c.L, c.d, cb);
    return cb == 64 ? run_stream<XT, GT, LOGITS, 64, true>(params_of(b, l), l, c.workspace, stream)
                    : run_stream<XT, GT, LOGITS, 32, true>(params_of(b, l), l, c.workspace, stream);
}

}  // namespace glr

size_t glr_stream_workspace_bytes(int64_t units, int64_t L, int64_t d)
{
    const int cb = glr_stream_channels(units, L, d);
    return glr::stream_bytes(glr::layout_of(units, L, d, cb).chains, cb);
}
// Chains of 64 channels where they give every resident CTA (two per SM) one at least, else chains of 32 where these
// keep most CTAs busy.  Below that a scan is faster, although its tiles wait for one another: 160 chains of 32 channels
// (2 x 4,099 tokens x 2,560, training pass) 182 us streamed, 150 scanned; 256 chains (2 x 32 units of 65,536 x 128)
// 1,177 against 1,385; 8,192 chains of 64 (4 x 64 x 16 units of 128 tokens) 123 against 168.  Narrow units count by their
// channels, as a CTA takes a mostly empty chain no faster than a full one (225 units of 18,913 tokens x 1: 2,300 us).
// A single tile has nothing to pass on.
int glr_stream_channels(int64_t units, int64_t L, int64_t d)
{
    if (L <= kGlrChunk || d < 32) return 0;
    if (glr::layout_of(units, L, d, 64).chains >= 296 && d > 32) return 64;
    if (L > 8 * kGlrChunk && glr::layout_of(units, L, d, 32).chains >= 222) return 32;
    return 0;
}

cudaError_t launch_glr_stream(const GlrCall& c, cudaStream_t stream)
{
    NvtxRange range("lt2 gated linear recurrence (stream)");
    LT2_GLR_DISPATCH(c, glr::forward_typed, c, stream);
}

cudaError_t launch_glr_stream_backward(const GlrBackwardCall& b, cudaStream_t stream)
{
    NvtxRange range("lt2 gated linear recurrence (stream, backward)");
    LT2_GLR_DISPATCH(b.f, glr::backward_typed, b, stream);
}

}  // namespace lt2
