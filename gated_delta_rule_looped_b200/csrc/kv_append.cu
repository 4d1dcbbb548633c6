// kv_append.cu -- new tokens' keys and values into a paged cache, with the position rotation of q and
// k applied on the way: one launch, every element read once and written once.
//
//     (u, w) -> (u cos - w sin, w cos + u sin),   angle = position * frequency of the pair
//
// An angle at position 10^6 loses its fraction in fp32 (a step of fp32 is 0.06 rad there), so positions are
// turned into fractions of a turn in 64-bit fixed point: frequency / 2 pi is an integer number of
// 2^-64 turns, its product with the position wraps modulo whole turns exactly, and the remainder's
// cosine and sine are taken in fp64, once for all loops and heads, and rounded once.
//
// CTA = up to 8 tokens and a share of their (loop, head) rows.  The tokens' cos and sin go to shared
// memory once and serve every loop and head; a thread then moves two 16-byte vectors of a row, the two halves of
// rotated pairs together, of two rows at a time.  The work is a copy: bound by HBM for prompts
// (4 x 9 ragged prompts of up to 4,001 tokens, 16 + 2 x 4 heads of 128: 151 us, 5.9 TB/s), by the launch for a
// decode step (4 x 64 sequences of 16 heads: 3.9 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache_launch.h"
#include "gdr_common.cuh"
#include "gdr_nvtx.h"
#include "lt2_api_common.h"
#include "sm100_primitives.cuh"

namespace lt2 {
namespace kva {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;

struct Params {
    AppendCall c;
    int64_t rows;          // T * (Hq + 2 Hkv) rows of a token
    int rows_per_cta;
    int tokens;            // tokens of a CTA: 1, 2, 4 or 8
    int lanes;             // threads of a row, a power of two
};

template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    static constexpr int E = 8;
    uint4 w;
    __device__ float get(int i) const
    {
        const uint32_t x = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
        return i & 1 ? sm100::bf16_hi(x) : sm100::bf16_lo(x);
    }
    __device__ static Vec of(const float (&f)[8])
    {
        Vec v;
        v.w = make_uint4(sm100::pack_bf16x2(f[0], f[1]), sm100::pack_bf16x2(f[2], f[3]), sm100::pack_bf16x2(f[4], f[5]),
                         sm100::pack_bf16x2(f[6], f[7]));
        return v;
    }
};
template <> struct Vec<float> {
    static constexpr int E = 4;
    float4 w;
    __device__ float get(int i) const { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
    __device__ static Vec of(const float (&f)[4])
    {
        Vec v;
        v.w = make_float4(f[0], f[1], f[2], f[3]);
        return v;
    }
};

// Vector i of a row whose first `rotated` vectors hold neighbouring pairs.
template <typename T>
__device__ __forceinline__ Vec<T> turn_pairs(const Vec<T>& a, const float2* t, int i, int rotated)
{
    constexpr int E = Vec<T>::E;
    if (i < 0 || i >= rotated) return a;
    float x[E];
    #pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float2 w = t[(i * E + e) >> 1];
        x[e] = a.get(e) * w.x - a.get(e + 1) * w.y;
        x[e + 1] = a.get(e + 1) * w.x + a.get(e) * w.y;
    }
    return Vec<T>::of(x);
}

// The sequence that packed token n of N belongs to, and its place there; -1 where it belongs to none (before the first or
// behind the last one) or to one with a bad offset: below 0, past N, or out of order with a neighbour.
__device__ __forceinline__ int64_t sequence_of(const int64_t* cu, int64_t B, int64_t N, int64_t n, int64_t& i)
{
    int64_t lo = 0, hi = B;                        // the last b in [0, B] with cu[b] <= n, if any
    if (cu[0] > n) return -1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= n) lo = mid; else hi = mid - 1;
    }
    if (lo == B) return -1;
    const int64_t first = cu[lo], end = cu[lo + 1];
    if (first < 0 || first > n || end <= n || end > N) return -1;
    if ((lo > 0 && cu[lo - 1] > first) || (lo + 2 <= B && cu[lo + 2] < end)) return -1;
    i = n - first;
    return lo;
}

// A row's two or three places: source, destination, and a second destination (k_out beside the cache row).
template <typename T>
struct Row {
    const T* src;
    T* dst;
    T* dst2;
    int pairs;             // rotated pairs
    int token;             // its token's cos and sin; -1: no row
};
// Row i of a CTA (token i % tokens, row i / tokens of the token).
template <typename T>
__device__ __forceinline__ Row<T> row_at(const Params& p, const int64_t* place, int64_t n0, int64_t r0, int i, int count)
{
    const AppendCall& c = p.c;
    Row<T> row;
    const int tk = i & (p.tokens - 1);
    row.token = i < count && place[tk] >= 0 ? tk : -1;
    if (row.token < 0) return row;
    const unsigned per_loop = static_cast<unsigned>(c.Hq + 2 * c.Hkv);
    const unsigned r = static_cast<unsigned>(r0) + (i >> (__ffs(p.tokens) - 1));
    const unsigned tau = r / per_loop;
    unsigned h = r - tau * per_loop;
    const bool is_q = h < c.Hq;
    if (!is_q) h -= static_cast<unsigned>(c.Hq);
    const bool is_v = !is_q && h >= c.Hkv;
    if (is_v) h -= static_cast<unsigned>(c.Hkv);
    const int64_t H = is_q ? c.Hq : c.Hkv, n = n0 + tk;
    const int64_t at = (c.token_major ? (tau * c.N + n) * H + h : (tau * H + h) * c.N + n) * c.d;
    row.src = static_cast<const T*>(is_q ? c.q : is_v ? c.v : c.k) + at;
    row.pairs = is_v ? 0 : c.rot_pairs;
    row.dst2 = nullptr;
    if (is_q) {
        row.dst = static_cast<T*>(c.q_out) + at;
    } else {
        const int64_t slot = (((static_cast<int64_t>(tau) * c.pages * c.Hkv) << c.page_shift) + place[tk] +
                              (static_cast<int64_t>(h) << c.page_shift)) * c.d;
        row.dst = static_cast<T*>(is_v ? c.v_cache : c.k_cache) + slot;
        if (!is_v && c.k_out) row.dst2 = static_cast<T*>(c.k_out) + at;
    }
    return row;
}
// The two vectors of a row that a lane moves (-1: none).  Rotated halves: the two partners; elsewhere any two.
__device__ __forceinline__ void lane_vectors(int lane, int lanes, int nv, int half_vectors, int& i0, int& i1)
{
    if (lane < half_vectors) {
        i0 = lane;
        i1 = lane + half_vectors;
        return;
    }
    const int rest = nv - 2 * half_vectors, r = lane - half_vectors, step = half_vectors ? (rest + 1) / 2 : lanes;
    i0 = r < rest && r < step ? 2 * half_vectors + r : -1;
    i1 = r < step && r + step < rest ? 2 * half_vectors + r + step : -1;
}

// How rows are moved: kElements one by one (a width that is no whole number of 16-byte vectors); kVectors, the
// rotated halves being whole vectors too; kShared, where they are not: a row passes through shared memory, from which
// each lane takes the partners of its elements.
enum Mode : int { kElements, kVectors, kShared };
template <typename T, Mode MODE>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ Params p)
{
    const AppendCall& c = p.c;
    __shared__ float2 cs[kMaxTokens][kMaxRotPairs];
    __shared__ int64_t place[kMaxTokens];          // row of the cache (page, offset) without loop and head; -1: none
    __shared__ int64_t posn[kMaxTokens];
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * p.tokens;

    // one thread of the grid looks at the order of the offsets
    if (blockIdx.x == 0 && blockIdx.y == 0 && c.cu) {
        bool bad = false;
        for (int64_t b = threadIdx.x; b < c.B; b += kThreads)
            bad |= c.cu[b] < 0 || c.cu[b] > c.cu[b + 1] || c.cu[b + 1] > c.N;
        if (bad) atomicOr(c.err, kDevSeqlens);
    }
    if (threadIdx.x < p.tokens) {
        const int64_t n = n0 + threadIdx.x;
        int64_t at = -1, pos = 0;
        if (n < c.N) {
            int64_t i = 0;
            const int64_t b = c.cu ? sequence_of(c.cu, c.B, c.N, n, i) : n;
            if (b >= 0) {
                const int64_t first = c.start[b], cap = c.max_pages << c.page_shift;
                if (first < 0 || first >= cap || i >= cap - first) {
                    atomicOr(c.err, kDevSeqlens);
                } else {
                    pos = first + i;
                    const int64_t page = c.page_table[b * c.max_pages + (pos >> c.page_shift)];
                    if (page < 0 || page >= c.pages)
                        atomicOr(c.err, kDevPages);
                    else
                        at = (page * c.Hkv << c.page_shift) + (pos & ((int64_t(1) << c.page_shift) - 1));
                }
            }
        }
        place[threadIdx.x] = at;
        posn[threadIdx.x] = pos;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.tokens * c.rot_pairs; i += kThreads) {
        const int tk = i / c.rot_pairs, j = i - tk * c.rot_pairs;
        const uint64_t turn = c.turns[j] * static_cast<uint64_t>(posn[tk]);
        double s, co;
        sincospi(static_cast<double>(static_cast<int64_t>(turn)) * 0x1p-63, &s, &co);      // in half turns
        cs[tk][j] = make_float2(static_cast<float>(co), static_cast<float>(s));
    }
    __syncthreads();

    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * p.rows_per_cta;
    const int nrows = static_cast<int>(p.rows - r0 < p.rows_per_cta ? p.rows - r0 : p.rows_per_cta);
    const int count = nrows * p.tokens;
    const int lane = threadIdx.x & (p.lanes - 1);
    const int stride = kThreads / p.lanes;
    if constexpr (MODE == kVectors) {
        constexpr int E = Vec<T>::E;
        constexpr int U = 2;                               // rows of a thread on their way at a time
        const int nv = static_cast<int>(c.d) / E;
        for (int i = threadIdx.x / p.lanes; i < count; i += U * stride) {
            Row<T> row[U];
            Vec<T> a[U], b[U];
            int i0[U], i1[U];
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                row[u] = row_at<T>(p, place, n0, r0, i + u * stride, count);
                i0[u] = i1[u] = -1;
                if (row[u].token < 0) continue;
                lane_vectors(lane, p.lanes, nv, c.interleaved ? 0 : row[u].pairs / E, i0[u], i1[u]);
                const Vec<T>* src = reinterpret_cast<const Vec<T>*>(row[u].src);
                if (i0[u] >= 0) a[u] = src[i0[u]];
                if (i1[u] >= 0) b[u] = src[i1[u]];
            }
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                if (row[u].token < 0) continue;
                const float2* t = cs[row[u].token];
                if (!c.interleaved && lane < row[u].pairs / E) {
                    float x[E], y[E];
                    #pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float2 w = t[lane * E + e];
                        x[e] = a[u].get(e) * w.x - b[u].get(e) * w.y;
                        y[e] = b[u].get(e) * w.x + a[u].get(e) * w.y;
                    }
                    a[u] = Vec<T>::of(x);
                    b[u] = Vec<T>::of(y);
                } else if (c.interleaved) {
                    a[u] = turn_pairs(a[u], t, i0[u], 2 * row[u].pairs / E);
                    b[u] = turn_pairs(b[u], t, i1[u], 2 * row[u].pairs / E);
                }
                Vec<T>* dst = reinterpret_cast<Vec<T>*>(row[u].dst);
                Vec<T>* dst2 = reinterpret_cast<Vec<T>*>(row[u].dst2);
                if (i0[u] >= 0) dst[i0[u]] = a[u];
                if (i1[u] >= 0) dst[i1[u]] = b[u];
                if (dst2) {
                    if (i0[u] >= 0) dst2[i0[u]] = a[u];
                    if (i1[u] >= 0) dst2[i1[u]] = b[u];
                }
            }
        }
    } else if constexpr (MODE == kShared) {
        constexpr int E = Vec<T>::E;
        __shared__ Vec<T> rows[2 * kThreads];
        const int nv = static_cast<int>(c.d) / E;
        Vec<T>* mine = rows + threadIdx.x / p.lanes * nv;  // (a row has at most two vectors for each of its lanes)
        const T* elements = reinterpret_cast<const T*>(mine);
        for (int i0 = 0; i0 < count; i0 += stride) {
            const Row<T> row = row_at<T>(p, place, n0, r0, i0 + static_cast<int>(threadIdx.x) / p.lanes, count);
            if (row.token >= 0) {
                const Vec<T>* src = reinterpret_cast<const Vec<T>*>(row.src);
                for (int v = lane; v < nv; v += p.lanes) mine[v] = src[v];
            }
            __syncwarp();                                  // a row's lanes are in one warp
            if (row.token >= 0) {
                const float2* t = cs[row.token];
                const int half = row.pairs;
                for (int v = lane; v < nv; v += p.lanes) {
                    float x[E];
                    #pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int at = v * E + e;
                        x[e] = to_f32<T>(elements[at]);
                        if (at >= 2 * half) continue;
                        const bool first = c.interleaved ? !(at & 1) : at < half;
                        const int pair = c.interleaved ? at >> 1 : first ? at : at - half;
                        const int partner = c.interleaved ? at ^ 1 : first ? at + half : at - half;
                        const float b = to_f32<T>(elements[partner]);
                        const float2 w = t[pair];
                        x[e] = first ? x[e] * w.x - b * w.y : x[e] * w.x + b * w.y;
                    }
                    const Vec<T> out = Vec<T>::of(x);
                    reinterpret_cast<Vec<T>*>(row.dst)[v] = out;
                    if (row.dst2) reinterpret_cast<Vec<T>*>(row.dst2)[v] = out;
                }
            }
            __syncwarp();                                  // the place is free for the next row
        }
    } else {
        for (int i = threadIdx.x / p.lanes; i < count; i += stride) {
            const Row<T> row = row_at<T>(p, place, n0, r0, i, count);
            if (row.token < 0) continue;
            const float2* t = cs[row.token];
            const int half = row.pairs;
            for (int u = lane; u < half; u += p.lanes) {
                const int i0 = c.interleaved ? 2 * u : u, i1 = c.interleaved ? 2 * u + 1 : u + half;
                const float a = to_f32<T>(row.src[i0]), b = to_f32<T>(row.src[i1]);
                const float2 w = t[u];
                const T x = from_f32<T>(a * w.x - b * w.y), y = from_f32<T>(b * w.x + a * w.y);
                row.dst[i0] = x;
                row.dst[i1] = y;
                if (row.dst2) {
                    row.dst2[i0] = x;
                    row.dst2[i1] = y;
                }
            }
            for (int u = 2 * half + lane; u < c.d; u += p.lanes) {
                const T a = row.src[u];
                row.dst[u] = a;
                if (row.dst2) row.dst2[u] = a;
            }
        }
    }
}

template <typename T>
cudaError_t launch_typed(const AppendCall& c, cudaStream_t stream)
{
    constexpr int E = Vec<T>::E;
    Params p;
    p.c = c;
    p.rows = c.T * (c.Hq + 2 * c.Hkv);
    const Mode mode = c.d % E != 0 ? kElements : (c.interleaved ? 2 * c.rot_pairs : c.rot_pairs) % E == 0 ? kVectors : kShared;
    const int units = mode != kElements ? static_cast<int>((c.d / E + 1) / 2) : static_cast<int>((c.d + 1) / 2);
    p.lanes = 1;
    while (p.lanes < units && p.lanes < 32) p.lanes *= 2;
    // tokens share nothing but neighbouring rows in memory: as many to a CTA as leave every SM two
    p.tokens = kMaxTokens;
    while (p.tokens > 1 && (c.N + p.tokens - 1) / p.tokens < 2 * 148) p.tokens /= 2;
    const int64_t gx = (c.N + p.tokens - 1) / p.tokens;
    // the rows of a token are shared out while there are fewer than eight CTAs per SM and a CTA
    // keeps a row for each of its groups of threads
    const int64_t least = kThreads / p.lanes / p.tokens > 1 ? kThreads / p.lanes / p.tokens : 1;
    int64_t gy = (8 * 148 + gx - 1) / gx;
    if (gy > (p.rows + least - 1) / least) gy = (p.rows + least - 1) / least;
    if (gy > 65535) gy = 65535;
    p.rows_per_cta = static_cast<int>((p.rows + gy - 1) / gy);
    gy = (p.rows + p.rows_per_cta - 1) / p.rows_per_cta;
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
    if (mode == kVectors)
        kv_append_kernel<T, kVectors><<<grid, kThreads, 0, stream>>>(p);
    else if (mode == kShared)
        kv_append_kernel<T, kShared><<<grid, kThreads, 0, stream>>>(p);
    else
        kv_append_kernel<T, kElements><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kva

cudaError_t launch_kv_append(const AppendCall& c, cudaStream_t stream)
{
    NvtxRange range("lt2 kv append");
    return c.bf16 ? kva::launch_typed<__nv_bfloat16>(c, stream) : kva::launch_typed<float>(c, stream);
}

}  // namespace lt2
