// attn_decode.cu -- attention of a few new tokens per row over the paged cache.
#include <cuda_fp8.h>

#include "attn.cuh"

namespace rssm {
namespace attn {

struct DecArgs {
    const void* q;
    long q_stride;
    const void* k;
    const void* v;
    const float* k_scale;
    const float* v_scale;
    const int32_t* page_table;
    const int32_t* slot_len;
    const int32_t* ci;
    void* o;
    float* lse;
    int32_t* dev_err;
    float scale;
    int batch, T, hq, hkv, ps_log2, num_pages, max_pages, num_slots, window, appended;
    bool abf, obf, e4m3;
};

// One warp per (row, query token, query head), tokens one after the other with the
// running maximum and sum of the softmax.
template <int D>
__global__ void __launch_bounds__(128) decode_simple(const DecArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long item = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (item >= (long)a.batch * a.T * a.hq) return;
    const int h = (int)(item % a.hq);
    const int j = (int)(item / a.hq % a.T);
    const int b = (int)(item / a.hq / a.T);
    const int s = a.ci[b];
    if (s < 0) return;
    if (s >= a.num_slots) {
        set_dev_err(a.dev_err, RSSM_DEVERR_SLOT);
        return;
    }
    const int len = a.slot_len[s];
    const long cap = (long)a.max_pages << a.ps_log2;
    if (len < 0 || (long)len + (a.appended ? a.T : 0) > cap) {
        set_dev_err(a.dev_err, RSSM_DEVERR_CURSOR);
        return;
    }
    const int end = len + (a.appended ? j + 1 : 0);
    const int begin = a.window && end > a.window ? end - a.window : 0;
    float q[E], o[E];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = load1(a.q, ((long)b * a.T + j) * a.q_stride + h * D + lane * E + e, a.abf) * a.scale;
        o[e] = 0.f;
    }
    const int hk = h / (a.hq / a.hkv);
    for (int p = begin; p < end; ++p) {
        const int page = a.page_table[(long)s * a.max_pages + (p >> a.ps_log2)];
        if (page < 0 || page >= a.num_pages) {
            set_dev_err(a.dev_err, RSSM_DEVERR_PAGE);
            continue;
        }
        const long vec = (((long)page * a.hkv + hk) << a.ps_log2) + (p & ((1 << a.ps_log2) - 1));
        float k[E], v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const long i = vec * D + lane * E + e;
            if (a.e4m3) {
                k[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(
                    static_cast<const uint8_t*>(a.k)[i], __NV_E4M3)));
                v[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(
                           static_cast<const uint8_t*>(a.v)[i], __NV_E4M3))) * a.v_scale[vec];
            } else {
                k[e] = load1(a.k, i, true);
                v[e] = load1(a.v, i, true);
            }
        }
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x += q[e] * k[e];
#pragma unroll
        for (int w = 16; w >= 1; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        if (a.e4m3) x *= a.k_scale[vec];
        const float mn = fmaxf(m, x), base = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - base), p1 = expf(x - base);
        m = x != x ? x : mn;
        l = l * f + p1;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + p1 * v[e];
    }
    const long out = (((long)b * a.T + j) * a.hq + h);
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e)
        store1(a.o, out * D + lane * E + e, a.obf, l == 0.f ? 0.f : o[e] * inv);
    if (a.lse && lane == 0) a.lse[out] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace attn
}  // namespace rssm

using namespace rssm;

extern "C" size_t rssm_attn_workspace_size(const rssm_attn_dims* d) {
    if (attn::check_dims(d) != RSSM_OK) return 0;
    return 256;
}

extern "C" int rssm_attn_decode(const rssm_attn_dims* d, const rssm_attn_cache* c, int appended,
                                float scale, int32_t window, const void* q, int64_t q_stride,
                                const int32_t* cache_indices, void* workspace,
                                size_t workspace_bytes, void* o, float* lse, int32_t* dev_err,
                                rssm_stream_t stream) {
    const int st = attn::check_dims(d);
    if (st != RSSM_OK) return st;
    if (window < 0) return RSSM_ERR_INVALID_ARG;
    if (d->q_tokens * (d->num_q_heads / d->num_kv_heads) > 64) return RSSM_ERR_UNSUPPORTED;
    if (d->batch == 0) return RSSM_OK;
    if (!attn::ok_cache(d, c) || !ok_ptr(q) || !attn::ok_stride(d, q_stride, d->num_q_heads) ||
        !ok_ptr(cache_indices) || !ok_ptr(workspace) ||
        workspace_bytes < rssm_attn_workspace_size(d) || !ok_ptr(o) || !ok_opt_ptr(lse))
        return RSSM_ERR_INVALID_ARG;
    attn::DecArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.k = c->k;
    a.v = c->v;
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    a.page_table = c->page_table;
    a.slot_len = c->slot_len;
    a.ci = cache_indices;
    a.o = o;
    a.lse = lse;
    a.dev_err = dev_err;
    a.scale = scale;
    a.batch = d->batch;
    a.T = d->q_tokens;
    a.hq = d->num_q_heads;
    a.hkv = d->num_kv_heads;
    a.ps_log2 = attn::log2_of(d->page_size);
    a.num_pages = d->num_pages;
    a.max_pages = d->max_pages;
    a.num_slots = d->num_slots;
    a.window = window;
    a.appended = appended != 0;
    a.abf = d->act_dtype == RSSM_BF16;
    a.obf = d->out_dtype == RSSM_BF16;
    a.e4m3 = d->cache_dtype == RSSM_E4M3;
    const long items = (long)a.batch * a.T * a.hq;
    if (d->head_dim == 64)
        attn::decode_simple<64><<<(int)((items + 3) / 4), 128, 0, (cudaStream_t)stream>>>(a);
    else
        attn::decode_simple<128><<<(int)((items + 3) / 4), 128, 0, (cudaStream_t)stream>>>(a);
    return launch_status();
}
