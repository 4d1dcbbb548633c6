// lt2_cache_api.cu -- the entry points of the paged key/value cache declared in include/lt2_gdr.h
// (appending rotated tokens, decode attention): argument checks and the calls' descriptions.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "cache_launch.h"
#include "gdr_nvtx.h"
#include "lt2_api_common.h"

namespace {

using namespace lt2::api;
using lt2::NvtxRange;

// Elements up to which a product of sizes is taken (each factor < 2^31).
bool product_ok(std::initializer_list<int64_t> f, int64_t* out)
{
    __int128 v = 1;
    for (int64_t x : f) {
        v *= x;
        if (v > (static_cast<__int128>(1) << 59)) return false;
    }
    *out = static_cast<int64_t>(v);
    return true;
}

// Pages of 16 to 256 tokens, a power of two; the shift, or -1.
int page_shift(int64_t size)
{
    for (int s = 4; s <= 8; ++s)
        if (size == (int64_t(1) << s)) return s;
    return -1;
}

lt2_status sizes_ok(std::initializer_list<int64_t> v)
{
    for (int64_t x : v)
        if (x < 0 || x >= kMaxDim) return LT2_ERR_INVALID_ARGUMENT;
    return LT2_OK;
}

// Angles of one position in 2^-64 turns.
lt2_status fill_turns(const lt2_rope* r, int64_t d, lt2::AppendCall* c)
{
    c->rot_pairs = 0;
    c->interleaved = 0;
    if (!r || r->rot_dim == 0) return LT2_OK;
    if (r->rot_dim < 0 || r->rot_dim % 2 != 0 || r->rot_dim > d) return LT2_ERR_INVALID_ARGUMENT;
    if (r->rot_dim / 2 > lt2::kMaxRotPairs) return LT2_ERR_UNSUPPORTED;    // more than the tables below hold
    if (r->interleaved != 0 && r->interleaved != 1) return LT2_ERR_INVALID_ARGUMENT;
    if (!r->inv_freq && !(r->base > 0.0 && std::isfinite(r->base))) return LT2_ERR_INVALID_ARGUMENT;
    c->rot_pairs = r->rot_dim / 2;
    c->interleaved = r->interleaved;
    // A program rotates by the same frequencies call after call, and the powers take longer than the rest of the
    // call: the last frequencies' angles are kept, by their values.
    struct Kept {
        int pairs = 0;
        double f[lt2::kMaxRotPairs];
        uint64_t turns[lt2::kMaxRotPairs];
        double base = 0.0;                                     // of f, where it was computed from one
        int rot_dim = 0;
    };
    static thread_local Kept kept;
    const size_t n = static_cast<size_t>(c->rot_pairs);
    const bool same = r->inv_freq ? kept.pairs == c->rot_pairs && std::memcmp(kept.f, r->inv_freq, n * sizeof(double)) == 0
                                  : kept.rot_dim == r->rot_dim && kept.base == r->base;
    if (!same) {
        kept.pairs = kept.rot_dim = 0;
        const long double two_pi = 6.283185307179586476925286766559005768L;
        for (size_t i = 0; i < n; ++i) {
            const double f = r->inv_freq ? r->inv_freq[i] : std::pow(r->base, -2.0 * static_cast<double>(i) / r->rot_dim);
            if (!std::isfinite(f)) return LT2_ERR_INVALID_ARGUMENT;
            long double t = static_cast<long double>(f) / two_pi;
            t -= std::floor(t);                                // whole turns do nothing
            const long double scaled = std::ldexp(t, 64);
            kept.f[i] = f;
            kept.turns[i] = scaled >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(scaled);
        }
        kept.pairs = c->rot_pairs;
        kept.rot_dim = r->inv_freq ? 0 : r->rot_dim;
        kept.base = r->base;
    }
    std::memcpy(c->turns, kept.turns, n * sizeof(uint64_t));
    return LT2_OK;
}

struct DecodeSizes {
    int64_t q, cache;
    int esz, osz;
};

lt2_status decode_call(const lt2_swa_decode_dims* d, DecodeSizes* sz, lt2::DecodeCall* c)
{
    if (!d) return LT2_ERR_INVALID_ARGUMENT;
    lt2_status st = sizes_ok({d->T, d->B, d->Hq, d->Hkv, d->pages, d->max_pages});
    if (st != LT2_OK) return st;
    if (d->d < 1 || d->d >= kMaxDim || d->window < 1 || d->prefix_len < 0) return LT2_ERR_INVALID_ARGUMENT;
    if (d->dtype != LT2_DTYPE_F32 && d->dtype != LT2_DTYPE_BF16) return LT2_ERR_INVALID_ARGUMENT;
    if (d->algo < LT2_ALGO_AUTO || d->algo > LT2_ALGO_CUDA_CORE) return LT2_ERR_INVALID_ARGUMENT;
    if (d->out_dtype < LT2_OUT_SAME || d->out_dtype > LT2_OUT_BF16) return LT2_ERR_INVALID_ARGUMENT;
    if (!(d->scale >= 0.f && d->scale <= 3.4e38f)) return LT2_ERR_INVALID_ARGUMENT;
    if (d->Hkv == 0 ? d->Hq != 0 : d->Hq % d->Hkv != 0) return LT2_ERR_INVALID_ARGUMENT;
    const int shift = page_shift(d->page_size);
    if (shift < 0 || d->d > 256) return LT2_ERR_UNSUPPORTED;
    if (!product_ok({d->T, d->B, d->Hq, d->d}, &sz->q) || !product_ok({d->T, d->pages, d->Hkv, d->page_size, d->d}, &sz->cache))
        return LT2_ERR_INVALID_ARGUMENT;
    int64_t rows, table;
    if (!product_ok({d->T, d->B, d->Hq}, &rows) || rows >= kMaxDim || !product_ok({d->B, d->max_pages}, &table))
        return LT2_ERR_UNSUPPORTED;
    const int bf16 = d->dtype == LT2_DTYPE_BF16;
    sz->esz = bf16 ? 2 : 4;
    sz->osz = d->out_dtype == LT2_OUT_F32 ? 4 : d->out_dtype == LT2_OUT_BF16 ? 2 : sz->esz;
    const bool tc = lt2::decode_tc_supports(bf16, d->d);
    if (d->algo == LT2_ALGO_TENSOR_CORE && !tc) return LT2_ERR_UNSUPPORTED;
    *c = {};
    c->T = d->T;
    c->B = d->B;
    c->Hq = d->Hq;
    c->Hkv = d->Hkv;
    c->d = d->d;
    c->pages = d->pages;
    c->max_pages = d->max_pages;
    c->page_shift = shift;
    c->window = d->window;
    const int64_t cap = d->max_pages << shift;
    c->prefix = (d->prefix_len < cap ? d->prefix_len : cap) >> shift << shift;
    c->scale = d->scale > 0.f ? d->scale : 1.f / std::sqrt(static_cast<float>(d->d));
    c->bf16 = bf16;
    c->out_bf16 = sz->osz == 2;
    c->tensor_core = tc && d->algo != LT2_ALGO_CUDA_CORE;
    return LT2_OK;
}

}  // namespace

extern "C" {

lt2_status lt2_kv_append(const lt2_kv_dims* d, const lt2_rope* rope, const void* q, const void* k, const void* v,
                         const int64_t* start, const int64_t* cu_seqlens, const int32_t* page_table, void* k_cache,
                         void* v_cache, void* q_out, void* k_out, void* stream)
{
    if (!d) return LT2_ERR_INVALID_ARGUMENT;
    lt2_status st = sizes_ok({d->T, d->B, d->Hq, d->Hkv, d->N, d->pages, d->max_pages});
    if (st != LT2_OK) return st;
    if (d->d < 1 || d->d >= kMaxDim || d->reserved != 0) return LT2_ERR_INVALID_ARGUMENT;
    if (d->dtype != LT2_DTYPE_F32 && d->dtype != LT2_DTYPE_BF16) return LT2_ERR_INVALID_ARGUMENT;
    if (!cu_seqlens && d->N != d->B) return LT2_ERR_INVALID_ARGUMENT;
    const int shift = page_shift(d->page_size);
    if (shift < 0 || d->d > 256) return LT2_ERR_UNSUPPORTED;
    lt2::AppendCall c = {};
    st = fill_turns(rope, d->d, &c);
    if (st != LT2_OK) return st;
    int64_t nq, nk, ncache, ntable, rows;
    if (!product_ok({d->T, d->N, d->Hq, d->d}, &nq) || !product_ok({d->T, d->N, d->Hkv, d->d}, &nk) ||
        !product_ok({d->T, d->pages, d->Hkv, d->page_size, d->d}, &ncache) || !product_ok({d->B, d->max_pages}, &ntable))
        return LT2_ERR_INVALID_ARGUMENT;
    // rows of a token are numbered in 28 bits (times the 8 tokens of a block)
    if (!product_ok({d->T, d->Hq + 2 * d->Hkv}, &rows) || rows >= (int64_t(1) << 28)) return LT2_ERR_UNSUPPORTED;
    if (!tensor_ok(q, nq) || !tensor_ok(k, nk) || !tensor_ok(v, nk) || !tensor_ok(q_out, nq) || (k_out && !aligned16(k_out)))
        return LT2_ERR_INVALID_ARGUMENT;
    if (nk > 0 && (!tensor_ok(k_cache, ncache) || !tensor_ok(v_cache, ncache))) return LT2_ERR_INVALID_ARGUMENT;
    if (rows > 0 && d->N > 0) {
        if (d->B > 0 && (!start || reinterpret_cast<uintptr_t>(start) % 8)) return LT2_ERR_INVALID_ARGUMENT;
        if (reinterpret_cast<uintptr_t>(cu_seqlens) % 8) return LT2_ERR_INVALID_ARGUMENT;
        if (ntable > 0 && (!page_table || reinterpret_cast<uintptr_t>(page_table) % 4)) return LT2_ERR_INVALID_ARGUMENT;
    }
    const int64_t e = d->dtype == LT2_DTYPE_BF16 ? 2 : 4;
    const Range in[6] = {range_of(q, nq * e), range_of(k, nk * e), range_of(v, nk * e), range_of(start, start ? d->B * 8 : 0),
                         range_of(cu_seqlens, cu_seqlens ? (d->B + 1) * 8 : 0), range_of(page_table, ntable * 4)};
    const Range out[4] = {range_of(q_out, nq * e), range_of(k_out, k_out ? nk * e : 0), range_of(k_cache, ncache * e),
                          range_of(v_cache, ncache * e)};
    for (int a = 0; a < 4; ++a) {
        for (int i = 0; i < 6; ++i) {
            if ((a == 0 && i == 0 && q_out == q) || (a == 1 && i == 1 && k_out == k)) continue;     // in place
            if (overlap(out[a], in[i])) return LT2_ERR_INVALID_ARGUMENT;
        }
        for (int b = a + 1; b < 4; ++b)
            if (overlap(out[a], out[b])) return LT2_ERR_INVALID_ARGUMENT;
    }
    if (d->N == 0 || rows == 0 || d->B == 0) return LT2_OK;
    st = on_current_device({nq ? q : nullptr, nk ? k : nullptr, nk ? v : nullptr, nq ? q_out : nullptr,
                            nk ? k_out : nullptr, ncache ? k_cache : nullptr, ncache ? v_cache : nullptr, start,
                            cu_seqlens, ntable ? page_table : nullptr});
    if (st != LT2_OK) return st;

    NvtxRange range("lt2_kv_append");
    st = status_word(&c.err);
    if (st != LT2_OK) return st;
    c.q = q;
    c.k = k;
    c.v = v;
    c.q_out = q_out;
    c.k_out = k_out;
    c.k_cache = k_cache;
    c.v_cache = v_cache;
    c.page_table = page_table;
    c.start = start;
    c.cu = cu_seqlens;
    c.T = d->T;
    c.B = d->B;
    c.Hq = d->Hq;
    c.Hkv = d->Hkv;
    c.N = d->N;
    c.d = d->d;
    c.pages = d->pages;
    c.max_pages = d->max_pages;
    c.page_shift = shift;
    c.token_major = cu_seqlens == nullptr;
    c.bf16 = e == 2;
    const cudaError_t ce = lt2::launch_kv_append(c, static_cast<cudaStream_t>(stream));
    if (ce != cudaSuccess) return cuda_fail(ce, "lt2_kv_append");
    return LT2_OK;
}

size_t lt2_swa_decode_workspace_bytes(const lt2_swa_decode_dims* dims)
{
    DecodeSizes sz;
    lt2::DecodeCall c;
    if (decode_call(dims, &sz, &c) != LT2_OK || sz.q == 0) return 0;
    return lt2::decode_workspace_bytes(c);
}

lt2_status lt2_swa_decode(const lt2_swa_decode_dims* dims, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* page_table, const int64_t* seq_lens, void* o, void* workspace,
                          size_t workspace_bytes, void* stream)
{
    DecodeSizes sz;
    lt2::DecodeCall c;
    lt2_status st = decode_call(dims, &sz, &c);
    if (st != LT2_OK) return st;
    if (!tensor_ok(q, sz.q) || !tensor_ok(o, sz.q)) return LT2_ERR_INVALID_ARGUMENT;
    if (sz.q == 0) return LT2_OK;
    if (!tensor_ok(k_cache, sz.cache) || !tensor_ok(v_cache, sz.cache)) return LT2_ERR_INVALID_ARGUMENT;
    const int64_t ntable = c.B * c.max_pages;
    if (!seq_lens || reinterpret_cast<uintptr_t>(seq_lens) % 8) return LT2_ERR_INVALID_ARGUMENT;
    if (ntable > 0 && (!page_table || reinterpret_cast<uintptr_t>(page_table) % 4)) return LT2_ERR_INVALID_ARGUMENT;
    const size_t need = lt2::decode_workspace_bytes(c);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return LT2_ERR_WORKSPACE;
    if (need == 0) workspace = nullptr;
    const Range in[5] = {range_of(q, sz.q * sz.esz), range_of(k_cache, sz.cache * sz.esz),
                         range_of(v_cache, sz.cache * sz.esz), range_of(page_table, ntable * 4), range_of(seq_lens, c.B * 8)};
    const Range ro = range_of(o, sz.q * sz.osz), rw = range_of(workspace, static_cast<int64_t>(need));
    for (const Range& r : in)
        if (overlap(ro, r) || overlap(rw, r)) return LT2_ERR_INVALID_ARGUMENT;
    if (overlap(ro, rw)) return LT2_ERR_INVALID_ARGUMENT;
    const lt2::DecodePlan plan = lt2::plan_decode(c);
    if (static_cast<__int128>(c.T) * c.B * c.Hkv * plan.group_tiles >= kMaxDim) return LT2_ERR_UNSUPPORTED;
    st = on_current_device({q, sz.cache ? k_cache : nullptr, sz.cache ? v_cache : nullptr, ntable ? page_table : nullptr,
                            seq_lens, o, workspace});
    if (st != LT2_OK) return st;

    NvtxRange range("lt2_swa_decode");
    st = status_word(&c.err);
    if (st != LT2_OK) return st;
    c.q = q;
    c.k_cache = k_cache;
    c.v_cache = v_cache;
    c.page_table = page_table;
    c.lens = seq_lens;
    c.o = o;
    c.workspace = static_cast<float*>(workspace);
    const cudaError_t e = lt2::launch_swa_decode(c, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "lt2_swa_decode");
    return LT2_OK;
}

}  // extern "C"
