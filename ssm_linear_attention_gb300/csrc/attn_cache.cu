// attn_cache.cu -- the paged key-value cache of a hybrid model's attention layers: new
// tokens written (rounded to bf16, or to e4m3 with a scale per token and head), tokens
// read back, lengths advanced.
//
// All three move bytes and compute next to nothing: a vector of D values is read once and
// written once, so HBM bounds the large calls and launch latency the small ones. A CTA
// takes a few consecutive tokens: its first threads look up each token's row, position
// and page (one dependent chain per token instead of one per vector), then all threads
// move the tokens' vectors, D / 8 lanes to a vector, 8 values to a lane (one 16-byte load
// of bf16).
#include <cuda_fp8.h>

#include "attn.cuh"

namespace rssm {
namespace attn {

constexpr int kThreads = 256;
constexpr int kTokMax = 16;  // tokens per CTA of a large call

struct MoveArgs {
    const void* src[2];   // append: k, v; read: the caches
    void* dst[2];         // append: the caches; read: k_out, v_out
    float* scale[2];      // k_scale, v_scale
    long stride[2];       // append: token strides of k, v (elements)
    const int32_t* cu;    // nullable
    const int32_t* first; // read only, nullable
    const int32_t* ci;
    const int32_t* page_table;
    const int32_t* slot_len;
    int32_t* dev_err;
    int n_tokens, batch, T, heads, ps_log2, num_pages, max_pages, num_slots;
    int tok_per_cta;
};

// Row of token t: t / T, or the row whose [cu[b], cu[b+1]) holds t (the first row b with
// cu[b+1] > t). -1 when the list does not cover t.
__device__ __forceinline__ int row_of(const int32_t* cu, int batch, int T, int t, int* in_row) {
    if (!cu) {
        *in_row = t % T;
        return t / T;
    }
    int lo = 0, hi = batch;  // first b in [lo, hi) with cu[b + 1] > t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    if (lo >= batch) return -1;
    *in_row = t - cu[lo];
    return *in_row < 0 ? -1 : lo;
}

// Cache vector index of token t's head 0 ((page * heads) * ps + offset), or -1 (padding
// row, or a flagged token).
template <bool READ>
__device__ __forceinline__ long locate(const MoveArgs& a, int t) {
    int in_row = 0;
    const int b = row_of(a.cu, a.batch, a.T, t, &in_row);
    if (b < 0) {
        set_dev_err(a.dev_err, RSSM_DEVERR_CURSOR);
        return -1;
    }
    const int s = a.ci[b];
    if (s < 0) return -1;
    if (s >= a.num_slots) {
        set_dev_err(a.dev_err, RSSM_DEVERR_SLOT);
        return -1;
    }
    const long cap = (long)a.max_pages << a.ps_log2;
    const int len = a.slot_len[s];
    const long pos = (READ ? (a.first ? (long)a.first[b] : 0) : (long)len) + in_row;
    if (len < 0 || len > cap || pos < 0 || pos >= (READ ? (long)len : cap)) {
        set_dev_err(a.dev_err, RSSM_DEVERR_CURSOR);
        return -1;
    }
    const int page = a.page_table[(long)s * a.max_pages + (pos >> a.ps_log2)];
    if (page < 0 || page >= a.num_pages) {
        set_dev_err(a.dev_err, RSSM_DEVERR_PAGE);
        return -1;
    }
    return (((long)page * a.heads) << a.ps_log2) + (pos & ((1 << a.ps_log2) - 1));
}

// The 8-bit form of 8 values x (already multiplied by 448 / amax).
__device__ __forceinline__ uint2 pack8_e4m3(const float* x) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]),
                                                     __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void unpack8_e4m3(uint2 v, float* f) {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 p = __half22float2(__half2(h));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

// D / 8 lanes share a vector; E4M3: the cache is 8-bit; ABF: bf16 activations.
template <int D, bool E4M3, bool ABF>
__global__ void __launch_bounds__(kThreads) append_kernel(const MoveArgs a) {
    __shared__ long where[kTokMax];
    constexpr int LPV = D / 8;
    const int t0 = blockIdx.x * a.tok_per_cta;
    const int nt = min(a.tok_per_cta, a.n_tokens - t0);
    if (threadIdx.x < nt) where[threadIdx.x] = locate<false>(a, t0 + threadIdx.x);
    __syncthreads();
    const int lane = threadIdx.x % LPV;
    const int nvec = nt * 2 * a.heads;
    for (int i = threadIdx.x / LPV; i < nvec; i += kThreads / LPV) {
        const int h = i % a.heads, r = i / a.heads, w = r & 1, t = r >> 1;
        const long base = where[t];
        // the group of lanes that shares a vector takes the same branch
        if (base < 0) continue;
        float x[8];
        load8(static_cast<const char*>(a.src[w]) +
                  ((long)(t0 + t) * a.stride[w] + h * D + lane * 8) * (ABF ? 2 : 4),
              ABF, x);
        const long vec = base + ((long)h << a.ps_log2);
        if (!E4M3) {
            store8(static_cast<char*>(a.dst[w]) + (vec * D + lane * 8) * 2, true, x);
            continue;
        }
        // the largest |x| by its bit pattern: an infinity or a NaN stays on top
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
        const unsigned mask = LPV == 32 ? 0xffffffffu
                                        : ((1u << LPV) - 1u) << ((threadIdx.x & 31) / LPV * LPV);
#pragma unroll
        for (int o = LPV / 2; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
        const bool finite = m < 0x7f800000u;
        const float amax = fmaxf(__uint_as_float(m), kAmaxFloor);
        // a vector that is not finite is marked by its scale; its values are stored as zeros
        const float inv = __fdiv_rn(kE4M3Max, amax);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = finite ? x[j] * inv : 0.f;
        *reinterpret_cast<uint2*>(static_cast<char*>(a.dst[w]) + vec * D + lane * 8) = pack8_e4m3(x);
        if (lane == 0)
            a.scale[w][vec] = finite ? __fdiv_rn(amax, kE4M3Max) : __uint_as_float(0x7fc00000u);
    }
}

template <int D, bool E4M3, bool OBF>
__global__ void __launch_bounds__(kThreads) read_kernel(const MoveArgs a) {
    __shared__ long where[kTokMax];
    constexpr int LPV = D / 8;
    const int t0 = blockIdx.x * a.tok_per_cta;
    const int nt = min(a.tok_per_cta, a.n_tokens - t0);
    if (threadIdx.x < nt) where[threadIdx.x] = locate<true>(a, t0 + threadIdx.x);
    __syncthreads();
    const int lane = threadIdx.x % LPV;
    const int nvec = nt * 2 * a.heads;
    for (int i = threadIdx.x / LPV; i < nvec; i += kThreads / LPV) {
        const int h = i % a.heads, r = i / a.heads, w = r & 1, t = r >> 1;
        const long base = where[t];
        if (base < 0) continue;
        const long vec = base + ((long)h << a.ps_log2);
        float x[8];
        if (E4M3) {
            unpack8_e4m3(*reinterpret_cast<const uint2*>(static_cast<const char*>(a.src[w]) +
                                                         vec * D + lane * 8),
                         x);
            const float sc = a.scale[w][vec];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= sc;
        } else {
            load8(static_cast<const char*>(a.src[w]) + (vec * D + lane * 8) * 2, true, x);
        }
        store8(static_cast<char*>(a.dst[w]) +
                   (((long)(t0 + t) * a.heads + h) * D + lane * 8) * (OBF ? 2 : 4),
               OBF, x);
    }
}

__global__ void advance_kernel(const int32_t* cu, const int32_t* acc, const int32_t* ci,
                               int32_t* slot_len, int batch, int T, long cap, int num_slots,
                               int32_t* dev_err) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= batch) return;
    const int s = ci[b];
    if (s < 0) return;
    if (s >= num_slots) {
        set_dev_err(dev_err, RSSM_DEVERR_SLOT);
        return;
    }
    const int n = cu ? cu[b + 1] - cu[b] : T;
    const int add = acc ? acc[b] : n;
    const int len = slot_len[s];
    if (add < 0 || add > n || len < 0 || (long)len + add > cap) {
        set_dev_err(dev_err, RSSM_DEVERR_CURSOR);
        return;
    }
    slot_len[s] = len + add;
}

// Tokens per CTA: few when the call is small, so that its vectors spread over the SMs;
// kTokMax when there are enough CTAs all the same (one look-up per token either way).
static int tokens_per_cta(const rssm_attn_dims* d, int n_tokens, int sm_count) {
    const int per_pass = kThreads / (d->head_dim / 8);  // vectors a CTA moves at once
    int tok = kTokMax;
    while (tok > 1 && (n_tokens + tok - 1) / tok < 4 * sm_count &&
           tok * 2 * d->num_kv_heads > per_pass)
        tok >>= 1;
    return tok;
}

static int check_move(const rssm_attn_dims* d, const rssm_attn_cache* c, int n_tokens,
                      const int32_t* cu, const int32_t* ci) {
    const int st = check_dims(d);
    if (st != RSSM_OK) return st;
    if (n_tokens < 0 || (!cu && (int64_t)d->batch * d->q_tokens != n_tokens)) return RSSM_ERR_INVALID_ARG;
    if (n_tokens == 0) return RSSM_OK;
    if (d->batch == 0 || !ok_cache(d, c) || !ok_ptr(ci) || !ok_opt_ptr(cu)) return RSSM_ERR_INVALID_ARG;
    return RSSM_OK;
}

static MoveArgs move_args(const rssm_attn_dims* d, const rssm_attn_cache* c, int n_tokens,
                          const int32_t* cu, const int32_t* ci, int32_t* dev_err, int sm_count) {
    MoveArgs a{};
    a.scale[0] = c->k_scale;
    a.scale[1] = c->v_scale;
    a.cu = cu;
    a.ci = ci;
    a.page_table = c->page_table;
    a.slot_len = c->slot_len;
    a.dev_err = dev_err;
    a.n_tokens = n_tokens;
    a.batch = d->batch;
    a.T = d->q_tokens;
    a.heads = d->num_kv_heads;
    a.ps_log2 = log2_of(d->page_size);
    a.num_pages = d->num_pages;
    a.max_pages = d->max_pages;
    a.num_slots = d->num_slots;
    a.tok_per_cta = tokens_per_cta(d, n_tokens, sm_count);
    return a;
}

template <bool READ, int D, bool E4M3>
static void launch_move(const MoveArgs& a, bool dense_bf16, cudaStream_t st) {
    const int grid = (a.n_tokens + a.tok_per_cta - 1) / a.tok_per_cta;
    if (READ) {
        if (dense_bf16) read_kernel<D, E4M3, true><<<grid, kThreads, 0, st>>>(a);
        else read_kernel<D, E4M3, false><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (dense_bf16) append_kernel<D, E4M3, true><<<grid, kThreads, 0, st>>>(a);
        else append_kernel<D, E4M3, false><<<grid, kThreads, 0, st>>>(a);
    }
}

template <bool READ>
static int run_move(const rssm_attn_dims* d, const MoveArgs& a, int dense_dtype, cudaStream_t st) {
    const bool bf = dense_dtype == RSSM_BF16, q = d->cache_dtype == RSSM_E4M3;
    if (d->head_dim == 64) {
        if (q) launch_move<READ, 64, true>(a, bf, st);
        else launch_move<READ, 64, false>(a, bf, st);
    } else {
        if (q) launch_move<READ, 128, true>(a, bf, st);
        else launch_move<READ, 128, false>(a, bf, st);
    }
    return launch_status();
}

}  // namespace attn
}  // namespace rssm

using namespace rssm;

extern "C" int rssm_attn_append(const rssm_attn_dims* d, const rssm_attn_cache* c, int32_t n_tokens,
                                const int32_t* cu_tokens, const void* k, int64_t k_stride,
                                const void* v, int64_t v_stride, const int32_t* cache_indices,
                                int32_t* dev_err, rssm_stream_t stream) {
    const int st = attn::check_move(d, c, n_tokens, cu_tokens, cache_indices);
    if (st != RSSM_OK || n_tokens == 0) return st;
    if (!ok_ptr(k) || !ok_ptr(v) || !attn::ok_stride(d, k_stride, d->num_kv_heads) ||
        !attn::ok_stride(d, v_stride, d->num_kv_heads))
        return RSSM_ERR_INVALID_ARG;
    DeviceInfo di;
    if (!device_info(&di)) return RSSM_ERR_CUDA;
    attn::MoveArgs a = attn::move_args(d, c, n_tokens, cu_tokens, cache_indices, dev_err, di.sm_count);
    a.src[0] = k;
    a.src[1] = v;
    a.dst[0] = c->k;
    a.dst[1] = c->v;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    return attn::run_move<false>(d, a, d->act_dtype, (cudaStream_t)stream);
}

extern "C" int rssm_attn_read(const rssm_attn_dims* d, const rssm_attn_cache* c, int32_t n_tokens,
                              const int32_t* cu_tokens, const int32_t* first,
                              const int32_t* cache_indices, void* k_out, void* v_out,
                              int32_t* dev_err, rssm_stream_t stream) {
    const int st = attn::check_move(d, c, n_tokens, cu_tokens, cache_indices);
    if (st != RSSM_OK || n_tokens == 0) return st;
    if (!ok_ptr(k_out) || !ok_ptr(v_out) || !ok_opt_ptr(first)) return RSSM_ERR_INVALID_ARG;
    DeviceInfo di;
    if (!device_info(&di)) return RSSM_ERR_CUDA;
    attn::MoveArgs a = attn::move_args(d, c, n_tokens, cu_tokens, cache_indices, dev_err, di.sm_count);
    a.src[0] = c->k;
    a.src[1] = c->v;
    a.dst[0] = k_out;
    a.dst[1] = v_out;
    a.first = first;
    return attn::run_move<true>(d, a, d->out_dtype, (cudaStream_t)stream);
}

extern "C" int rssm_attn_advance(const rssm_attn_dims* d, const rssm_attn_cache* c,
                                 const int32_t* cu_tokens, const int32_t* num_accepted,
                                 const int32_t* cache_indices, int32_t* dev_err,
                                 rssm_stream_t stream) {
    const int st = attn::check_dims(d);
    if (st != RSSM_OK) return st;
    if (d->batch == 0) return RSSM_OK;
    if (!c || !ok_ptr(c->slot_len) || !ok_ptr(cache_indices) || !ok_opt_ptr(cu_tokens) ||
        !ok_opt_ptr(num_accepted))
        return RSSM_ERR_INVALID_ARG;
    attn::advance_kernel<<<(d->batch + 255) / 256, 256, 0, (cudaStream_t)stream>>>(
        cu_tokens, num_accepted, cache_indices, c->slot_len, d->batch, d->q_tokens,
        (long)d->max_pages * d->page_size, d->num_slots, dev_err);
    return launch_status();
}
