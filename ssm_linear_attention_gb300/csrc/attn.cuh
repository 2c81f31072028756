// attn.cuh -- what the paged-attention translation units share: the dims checks and the
// row and page look-ups of the paged cache.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace rssm {
namespace attn {

constexpr float kE4M3Max = 448.f;              // largest e4m3 value
constexpr float kAmaxFloor = 7.888609052e-31f;  // 2^-100: 448 / a stays finite for every a >= it

// Status of a call's dims (the batch may be 0).
inline int check_dims(const rssm_attn_dims* d) {
    if (!d || d->batch < 0 || d->q_tokens < 1 || d->num_q_heads < 1 || d->num_kv_heads < 1 ||
        d->num_pages < 1 || d->max_pages < 1 || d->num_slots < 1)
        return RSSM_ERR_INVALID_ARG;
    if (!ok_dtype(d->act_dtype) || !ok_dtype(d->out_dtype) ||
        (d->cache_dtype != RSSM_BF16 && d->cache_dtype != RSSM_E4M3))
        return RSSM_ERR_INVALID_ARG;
    if (d->num_q_heads % d->num_kv_heads) return RSSM_ERR_CONFIG;
    if (d->head_dim != 64 && d->head_dim != 128) return RSSM_ERR_UNSUPPORTED;
    const int ps = d->page_size;
    if (ps < 16 || ps > 256 || (ps & (ps - 1))) return RSSM_ERR_UNSUPPORTED;
    if ((int64_t)d->max_pages * ps > (1 << 30)) return RSSM_ERR_UNSUPPORTED;
    if ((int64_t)d->num_pages * d->num_kv_heads * ps >= (int64_t)1 << 31) return RSSM_ERR_UNSUPPORTED;
    return RSSM_OK;
}

inline bool ok_cache(const rssm_attn_dims* d, const rssm_attn_cache* c) {
    if (!c || !ok_ptr(c->k) || !ok_ptr(c->v) || !ok_ptr(c->page_table) || !ok_ptr(c->slot_len))
        return false;
    return d->cache_dtype != RSSM_E4M3 || (ok_ptr(c->k_scale) && ok_ptr(c->v_scale));
}

// Element strides between tokens of dense [heads][D] blocks.
inline bool ok_stride(const rssm_attn_dims* d, int64_t stride, int heads) {
    return stride >= (int64_t)heads * d->head_dim && stride % 8 == 0;
}

// A kernel launched with launch_early may start while the one before it in the stream still ends
// (its launch, first instructions and barriers then cost nothing): every thread waits here for
// that one's completion before it touches memory. Of a stream of calls: 1 row of 300 tokens 10.9
// -> 8.8 us, norm of 509 x 8192 8.2 -> 6.9, append of 61k tokens 75.0 -> 72.4.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel's CTAs in before this one's are gone: where it helps (attention 9.0 -> 8.7 us on 1
// row; level or worse for the norm and large moves, whose own CTAs want the room).
__device__ __forceinline__ void let_next_in() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <class... P, class... A>
inline void launch_early(void (*kernel)(P...), int grid, int block, size_t smem, cudaStream_t st, const A&... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = at;
    c.numAttrs = 1;
    cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

inline int log2_of(int v) {
    int l = 0;
    while ((1 << l) < v) ++l;
    return l;
}

}  // namespace attn
}  // namespace rssm
