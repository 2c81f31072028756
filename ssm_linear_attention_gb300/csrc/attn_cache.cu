// attn_cache.cu -- the paged key-value cache of a hybrid model's attention layers: new
// tokens written (rounded to bf16, or to e4m3 with a scale per token and head), tokens
// read back, lengths advanced.
//
// All three move bytes: a vector of D values is read once and written once, so HBM bounds
// the large calls (the 8-bit append comes near the issue rate too: an absolute maximum, a
// division and a conversion per 8 values) and launch latency the small ones. CTAs loop over
// blocks of consecutive tokens. One warp looks up row, position and page of the next block's
// tokens, a chain of dependent loads, while the others move this block's vectors, D / 8
// lanes to a vector, 8 values to a lane (one 16-byte load of bf16), a vector of each of
// several tokens at once.
//
// Measured (one GB300, GPU time of a call; "of" the measured copy bandwidth; 8 heads, D 128,
// bf16 against an 8-bit cache): append of 61k tokens 72.3 us, 5.2 TB/s, 77 % of it; read-back
// of 156k tokens 159 us, 6.1 TB/s, 90 %; append of one token of 512 rows 3.4 us. Loading the
// next vectors while these are rounded costs more in CTAs (registers) than it hides: append
// 83 us with 3 CTAs an SM, 88 with 4 and spills.
#include <cuda_fp8.h>

#include "attn.cuh"

namespace rssm {
namespace attn {

constexpr int kMovers = 256;          // threads that move vectors
constexpr int kThreads = kMovers + 32;  // and the warp that looks tokens up
constexpr int kTokMax = 32;            // tokens of a block: one per lane of that warp
constexpr int kCtas = 4;               // of an SM: 3 or 5 cost 8 to 27 % on the large cases
constexpr int kAhead = 4;              // vectors whose loads a thread has in flight

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
    int block;  // tokens of a block
};

// Row of token t, one token per lane of a warp: t / T, or the row whose [cu[b], cu[b+1])
// holds t (the first row b with cu[b+1] > t), found among 32 evenly spaced entries held by
// the lanes and then between two of them. -1 when the list does not cover t.
__device__ __forceinline__ int row_of(const MoveArgs& a, int t, int* in_row) {
    if (!a.cu) {
        *in_row = t % a.T;
        return t / a.T;
    }
    const int lane = threadIdx.x & 31, step = (a.batch + 31) / 32;
    const int mine = a.cu[min((lane + 1) * step, a.batch)];
    int piece = 0;  // entries that are <= t
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) {
        const int v = __shfl_sync(0xffffffffu, mine, piece + w - 1);
        if (v <= t) piece += w;
    }
    if (__shfl_sync(0xffffffffu, mine, piece) <= t || piece * step >= a.batch) return -1;
    int lo = piece * step, hi = min(lo + step, a.batch) - 1;  // first b in [lo, hi] with cu[b + 1] > t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    *in_row = t - a.cu[lo];
    return *in_row < 0 ? -1 : lo;
}

// Cache vector index of token t's head 0 ((page * heads) * ps + offset), or -1 (padding
// row, or a flagged token).
template <bool READ>
__device__ __forceinline__ long locate(const MoveArgs& a, int t) {
    int in_row = 0;
    const int b = row_of(a, min(t, a.n_tokens - 1), &in_row);  // the whole warp
    if (t >= a.n_tokens) return -1;
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

// Runs over the CTA's blocks of tokens: body(first token, count, where) with where[i] the
// place of token i.
template <bool READ, bool SMALL, class Body>
__device__ __forceinline__ void for_blocks(const MoveArgs& a, Body body) {
    __shared__ long where[2][kTokMax];
    if (SMALL) let_next_in();  // (a large call's CTAs want the room)
    wait_for_stream();
    const int nblk = (a.n_tokens + a.block - 1) / a.block;
    const bool looks = threadIdx.x >= kMovers;
    const int lane = threadIdx.x & 31;
    auto look = [&](int blk, int half) {
        const int t = blk * a.block + lane;
        const long w = locate<READ>(a, lane < a.block ? t : a.n_tokens);
        where[half][lane] = w;
    };
    if (looks) look(blockIdx.x, 0);
    __syncthreads();
    int half = 0;
    for (int blk = blockIdx.x; blk < nblk; blk += gridDim.x, half ^= 1) {
        if (looks) {
            if (blk + (int)gridDim.x < nblk) look(blk + gridDim.x, half ^ 1);
        } else {
            body(blk * a.block, min(a.block, a.n_tokens - blk * a.block), where[half]);
        }
        __syncthreads();
    }
}

// The vectors of a block: body(w, h, t, dt) for the vectors of k (w 0) or v (w 1), head h, of
// tokens t, t + dt, ... Groups of D / 8 lanes take one vector of the 2 heads each, and
// share the tokens where there are more groups than vectors. Every group makes the same
// calls (t beyond any block: nothing to do), so that a warp stays together.
template <int LPV, class Body>
__device__ __forceinline__ void for_vectors(int heads, Body body) {
    constexpr int GROUPS = kMovers / LPV, NONE = 1 << 20;
    const int g = threadIdx.x / LPV, n = 2 * heads;
    const int dt = n <= GROUPS ? GROUPS / n : 1;
    for (int j0 = 0; j0 < n; j0 += GROUPS) {
        const int t = n <= GROUPS ? g / n : 0, j = n <= GROUPS ? g - t * n : j0 + g;
        const bool have = t < dt && j < n;
        body(have && j >= heads, have ? (j >= heads ? j - heads : j) : 0, have ? t : NONE, dt);
    }
}

// Largest |x| of 8 loaded values, as the bits of a float32: an infinity or a NaN stays on top.
__device__ __forceinline__ uint32_t abs_max8(uint4 v) {  // bf16
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
}

// D / 8 lanes share a vector; E4M3: the cache is 8-bit; ABF: bf16 activations; AHEAD: vectors
// of a thread at once.
template <int D, bool E4M3, bool ABF, int AHEAD>
__global__ void __launch_bounds__(kThreads, kCtas) append_kernel(const MoveArgs a) {
    constexpr int LPV = D / 8;
    const int lane = threadIdx.x % LPV;
    for_blocks<false, AHEAD == 1>(a, [&](int t0, int nt, const long* where) {
        for_vectors<LPV>(a.heads, [&](bool w, int h, int t1, int dt) {
            constexpr int SA = ABF ? 2 : 4;
            const char* src = static_cast<const char*>(w ? a.src[1] : a.src[0]);
            const long stride = (w ? a.stride[1] : a.stride[0]) * SA;
            src += t0 * stride + (h * D + lane * 8) * SA;
            char* dst = static_cast<char*>(w ? a.dst[1] : a.dst[0]) + lane * 8 * (E4M3 ? 1 : 2);
            float* scales = w ? a.scale[1] : a.scale[0];
            const long head = (long)h << a.ps_log2;
#pragma unroll 1
            for (int done = 0; done < nt; done += AHEAD * dt) {
                uint4 x[AHEAD][ABF ? 1 : 2];
                long vec[AHEAD];
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const int t = done + t1 + u * dt, at = min(t, nt - 1);  // (a token of this block)
                    vec[u] = t < nt ? where[at] : -1;
                    const uint4* p = reinterpret_cast<const uint4*>(src + at * stride);
#pragma unroll
                    for (int e = 0; e < (ABF ? 1 : 2); ++e) x[u][e] = p[e];
                }
                float scale = 0.f, inv = 0.f;
                if (E4M3) {
                    // Each lane of a vector's group takes one of the AHEAD maxima, so that the
                    // two divisions are made once for all of them.
                    uint32_t mine = 0;
#pragma unroll
                    for (int u = 0; u < AHEAD; ++u) {
                        uint32_t m = 0;
                        if (ABF) {
                            m = abs_max8(x[u][0]);
                        } else {
                            const uint32_t* f = reinterpret_cast<const uint32_t*>(x[u]);
#pragma unroll
                            for (int e = 0; e < 8; ++e) m = max(m, f[e] & 0x7fffffffu);
                        }
#pragma unroll
                        for (int o = LPV / 2; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                        if ((lane & (AHEAD - 1)) == u) mine = m;
                    }
                    // a vector that is not finite is marked by its scale; its values are stored
                    // as zeros
                    const bool finite = mine < 0x7f800000u;
                    const float amax = fmaxf(__uint_as_float(mine), kAmaxFloor);
                    scale = finite ? __fdiv_rn(amax, kE4M3Max) : __uint_as_float(0x7fc00000u);
                    inv = finite ? __fdiv_rn(kE4M3Max, amax) : 0.f;
                }
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    float f[8];
                    load8(x[u], ABF, f);
                    const long to = vec[u] + head;
                    if (E4M3) {
                        const float by = __shfl_sync(0xffffffffu, inv, u, LPV);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] *= by;
                        uint2 q = pack8_e4m3(f);
                        if (__builtin_expect(by == 0.f, 0)) q = make_uint2(0, 0);
                        if (vec[u] >= 0) {
                            *reinterpret_cast<uint2*>(dst + to * D) = q;
                            if (lane == u) scales[to] = scale;
                        }
                    } else if (vec[u] >= 0) {
                        store8(dst + to * D * 2, true, f);
                    }
                }
            }
        });
    });
}

template <int D, bool E4M3, bool OBF, int AHEAD>
__global__ void __launch_bounds__(kThreads, kCtas) read_kernel(const MoveArgs a) {
    constexpr int LPV = D / 8;
    const int lane = threadIdx.x % LPV;
    for_blocks<true, AHEAD == 1>(a, [&](int t0, int nt, const long* where) {
        for_vectors<LPV>(a.heads, [&](bool w, int h, int t1, int dt) {
            const char* src = static_cast<const char*>(w ? a.src[1] : a.src[0]) + lane * 8 * (E4M3 ? 1 : 2);
            char* dst = static_cast<char*>(w ? a.dst[1] : a.dst[0]) +
                        (((long)t0 * a.heads + h) * D + lane * 8) * (OBF ? 2 : 4);
            const float* scales = w ? a.scale[1] : a.scale[0];
            const long head = (long)h << a.ps_log2;
#pragma unroll 1
            for (int t = t1; t < nt; t += AHEAD * dt) {
                uint4 raw[AHEAD];  // 8 values: 8 bytes (in x, y) or 16
                float sc[AHEAD];
                bool have[AHEAD];
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const long vec = t + u * dt < nt ? where[t + u * dt] : -1;
                    have[u] = vec >= 0;
                    if (!have[u]) continue;
                    const char* p = src + (vec + head) * (D * (E4M3 ? 1 : 2));
                    if (E4M3) {
                        const uint2 q = *reinterpret_cast<const uint2*>(p);
                        raw[u] = make_uint4(q.x, q.y, 0, 0);
                        sc[u] = scales[vec + head];
                    } else {
                        raw[u] = *reinterpret_cast<const uint4*>(p);
                    }
                }
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    if (!have[u]) continue;
                    float x[8];
                    if (E4M3) {
                        unpack8_e4m3(make_uint2(raw[u].x, raw[u].y), x);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] *= sc[u];
                    } else {
                        load8(&raw[u], true, x);
                    }
                    store8(dst + (long)(t + u * dt) * a.heads * (D * (OBF ? 2 : 4)), OBF, x);
                }
            }
        });
    });
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

// Tokens of a block: few when the call is small, so that its vectors spread over the SMs,
// but a vector for every group of lanes; else kTokMax.
static int block_tokens(const rssm_attn_dims* d, int n_tokens, int sm_count) {
    const int groups = kMovers / (d->head_dim / 8);
    int tok = kTokMax;
    while (tok > 1 && (n_tokens + tok - 1) / tok < 4 * sm_count && tok * 2 * d->num_kv_heads > groups)
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
    a.block = block_tokens(d, n_tokens, sm_count);
    return a;
}

template <bool READ, int D, bool E4M3, bool DBF>
static void launch_move(const MoveArgs& a, int sm_count, cudaStream_t st) {
    const int grid = min((a.n_tokens + a.block - 1) / a.block, kCtas * sm_count);
    // a block with no more vectors than groups of lanes: one each (4.8 -> 3.6 us for one token of
    // 512 rows)
    const bool one = a.block * 2 * a.heads <= kMovers / (D / 8);
    if (READ && one) launch_early(read_kernel<D, E4M3, DBF, 1>, grid, kThreads, 0, st, a);
    if (READ && !one) launch_early(read_kernel<D, E4M3, DBF, kAhead>, grid, kThreads, 0, st, a);
    if (!READ && one) launch_early(append_kernel<D, E4M3, DBF, 1>, grid, kThreads, 0, st, a);
    if (!READ && !one) launch_early(append_kernel<D, E4M3, DBF, kAhead>, grid, kThreads, 0, st, a);
}

template <bool READ>
static int run_move(const rssm_attn_dims* d, const MoveArgs& a, int dense_dtype, int sms, cudaStream_t st) {
    const bool bf = dense_dtype == RSSM_BF16, q = d->cache_dtype == RSSM_E4M3;
#define RSSM_MOVE(D_, Q_) (bf ? launch_move<READ, D_, Q_, true>(a, sms, st) : launch_move<READ, D_, Q_, false>(a, sms, st))
    if (d->head_dim == 64) q ? RSSM_MOVE(64, true) : RSSM_MOVE(64, false);
    else q ? RSSM_MOVE(128, true) : RSSM_MOVE(128, false);
#undef RSSM_MOVE
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
    return attn::run_move<false>(d, a, d->act_dtype, di.sm_count, (cudaStream_t)stream);
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
    return attn::run_move<true>(d, a, d->out_dtype, di.sm_count, (cudaStream_t)stream);
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
