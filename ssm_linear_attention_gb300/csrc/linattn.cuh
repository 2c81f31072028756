// linattn.cuh -- what the linear-attention translation units share: argument checks, kernel
// arguments, and a row's part of the token list.
#pragma once

#include "attn.cuh"

namespace rssm {
namespace linattn {

struct Args {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* w;
    long q_stride, k_stride, v_stride, g_stride, w_stride;
    float scale;
    const int32_t* cu;       // null: `each` tokens a row
    const uint8_t* resume;
    const int32_t* slots;
    void* state;
    void* o;
    int32_t* dev_err;
    int batch, tokens, each;
    int H, G, num_slots;
    bool sbf, obf;           // bf16 state, bf16 output
};

inline int check_dims(const rssm_linattn_dims* d) {
    if (!d || d->batch < 0 || d->num_heads < 1 || d->num_k_heads < 1 || d->num_slots < 1)
        return RSSM_ERR_INVALID_ARG;
    if (!ok_dtype(d->state_dtype) || !ok_dtype(d->act_dtype) || !ok_dtype(d->out_dtype))
        return RSSM_ERR_INVALID_ARG;
    if (d->num_heads % d->num_k_heads) return RSSM_ERR_CONFIG;
    if ((d->key_dim != 64 && d->key_dim != 128) || (d->value_dim != 64 && d->value_dim != 128))
        return RSSM_ERR_UNSUPPORTED;
    // (launch sizes and tensor-map widths)
    if (d->num_heads > 8192 || (int64_t)d->batch * d->num_heads >= (1 << 27)) return RSSM_ERR_UNSUPPORTED;
    return RSSM_OK;
}

inline bool ok_stride(int64_t s, int64_t least, int64_t unit) { return s >= least && s % unit == 0 && s < ((int64_t)1 << 36); }

inline bool ok_inputs(const rssm_linattn_dims* d, const rssm_linattn_inputs* in) {
    if (!in || !ok_ptr(in->q) || !ok_ptr(in->k) || !ok_ptr(in->v) || !ok_ptr(in->g) || !ok_opt_ptr(in->w)) return false;
    const int64_t kw = (int64_t)d->num_k_heads * d->key_dim, vw = (int64_t)d->num_heads * d->value_dim;
    return ok_stride(in->q_stride, kw, 8) && ok_stride(in->k_stride, kw, 8) && ok_stride(in->v_stride, vw, 8) &&
           (in->g_stride == 0 || ok_stride(in->g_stride, d->num_heads, 1)) &&
           (!in->w || ok_stride(in->w_stride, d->num_heads, 1));
}

inline Args make_args(const rssm_linattn_dims* d, const rssm_linattn_inputs* in, void* state, const int32_t* slots,
                      void* o, int32_t* dev_err) {
    Args a{};
    a.q = in->q; a.k = in->k; a.v = in->v; a.g = in->g; a.w = in->w;
    a.q_stride = in->q_stride; a.k_stride = in->k_stride; a.v_stride = in->v_stride;
    a.g_stride = in->g_stride; a.w_stride = in->w_stride;
    a.scale = in->scale;
    a.slots = slots; a.state = state; a.o = o; a.dev_err = dev_err;
    a.batch = d->batch; a.H = d->num_heads; a.G = d->num_k_heads; a.num_slots = d->num_slots;
    a.sbf = d->state_dtype == RSSM_BF16; a.obf = d->out_dtype == RSSM_BF16;
    return a;
}

// Row b's tokens [begin, end) and slot; false when the row is left alone (errors flagged by
// whoever passes report).
__device__ __forceinline__ bool row_of(const Args& a, int b, bool report, int& begin, int& end, int& slot) {
    slot = a.slots[b];
    begin = a.cu ? a.cu[b] : b * a.each;
    end = a.cu ? a.cu[b + 1] : begin + a.each;
    if (slot < 0) return false;
    const bool bad_slot = slot >= a.num_slots, bad_part = begin < 0 || end < begin || end > a.tokens;
    if (bad_slot || bad_part) {
        if (report) set_dev_err(a.dev_err, bad_slot ? RSSM_DEVERR_SLOT : RSSM_DEVERR_CURSOR);
        return false;
    }
    return end > begin;
}

// bf16 activations (linattn_chunk.cu).
size_t chunk_workspace(const rssm_linattn_dims* d, int n_tokens);
int prompt_chunks(const rssm_linattn_dims* d, const Args& a, void* workspace, uint64_t wait_ns, cudaStream_t st);

}  // namespace linattn
}  // namespace rssm
