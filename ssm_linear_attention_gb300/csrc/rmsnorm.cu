// rmsnorm.cu -- residual add and RMS norm of the stream between a model's layers, with an
// output in float32, bf16, or e4m3 with float32 scales.
//
// r = x + residual, y = r * rsqrt(mean(r^2) + eps) * weight. Every element is read once
// and written once, so HBM bounds a large call and the launch a small one. One CTA takes a
// row and keeps it in registers between the sum of squares and the output.
#include <cuda_fp8.h>

#include "attn.cuh"

namespace rssm {
namespace norm {

struct Args {
    const void* x;
    const void* res;
    const float* w;
    void* res_out;
    void* y;
    float* y_scale;
    float eps;
    int rows, cols, group;
    bool abf;
    int out_dtype;
};

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) t += red[i];
    return t;
}

__device__ __forceinline__ void store_out(const Args& a, long i, float v) {
    if (a.out_dtype == RSSM_E4M3)
        static_cast<uint8_t*>(a.y)[i] = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
    else
        store1(a.y, i, a.out_dtype == RSSM_BF16, v);
}

// One CTA per row, the row in dynamic shared memory.
__global__ void __launch_bounds__(256) simple_kernel(const Args a) {
    extern __shared__ float row[];
    __shared__ float red[8];
    __shared__ unsigned amax[256];
    const long base = (long)blockIdx.x * a.cols;
    float ss = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float r = load1(a.x, base + c, a.abf);
        if (a.res) r += load1(a.res, base + c, a.abf);
        if (a.res_out) store1(a.res_out, base + c, a.abf, r);
        row[c] = r;
        ss += r * r;
    }
    const float rstd = rsqrtf(block_sum(ss, red) / (float)a.cols + a.eps);
    const int groups = a.group ? a.cols / a.group : 1, gs = a.group ? a.group : a.cols;
    for (int i = threadIdx.x; i < groups; i += blockDim.x) amax[i] = 0;
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        const float y = row[c] * rstd * a.w[c];
        row[c] = y;
        if (a.out_dtype == RSSM_E4M3) atomicMax(&amax[c / gs], __float_as_uint(y) & 0x7fffffffu);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float y = row[c];
        if (a.out_dtype == RSSM_E4M3) {
            const unsigned m = amax[c / gs];
            const float am = fmaxf(__uint_as_float(m), attn::kAmaxFloor);
            y *= __fdiv_rn(attn::kE4M3Max, am);
            if (c % gs == 0)
                a.y_scale[(long)blockIdx.x * groups + c / gs] =
                    m < 0x7f800000u ? __fdiv_rn(am, attn::kE4M3Max) : __uint_as_float(0x7fc00000u);
        }
        store_out(a, base + c, y);
    }
}

}  // namespace norm
}  // namespace rssm

using namespace rssm;

extern "C" int rssm_add_rmsnorm(const rssm_norm_dims* d, const void* x, const void* residual,
                                const float* weight, float eps, void* residual_out, void* y,
                                float* y_scale, rssm_stream_t stream) {
    if (!d || d->rows < 0 || d->cols < 1 || !ok_dtype(d->act_dtype) ||
        (!ok_dtype(d->out_dtype) && d->out_dtype != RSSM_E4M3))
        return RSSM_ERR_INVALID_ARG;
    const bool q = d->out_dtype == RSSM_E4M3;
    if (d->cols > 32768 || (q && d->scale_group != 0 && d->scale_group != 128))
        return RSSM_ERR_UNSUPPORTED;
    if (q && d->scale_group && d->cols % d->scale_group) return RSSM_ERR_CONFIG;
    if (d->rows == 0) return RSSM_OK;
    if (!ok_ptr(x) || !ok_opt_ptr(residual) || !ok_ptr(weight) || !ok_opt_ptr(residual_out) ||
        !ok_ptr(y) || (q && !ok_ptr(y_scale)))
        return RSSM_ERR_INVALID_ARG;
    norm::Args a{x, residual, weight, residual_out, y, y_scale, eps, d->rows, d->cols,
                 q ? d->scale_group : 0, d->act_dtype == RSSM_BF16, d->out_dtype};
    const int smem = d->cols * 4;
    if (!ensure_smem_limit((const void*)norm::simple_kernel, smem)) return RSSM_ERR_CUDA;
    norm::simple_kernel<<<d->rows, 256, smem, (cudaStream_t)stream>>>(a);
    return launch_status();
}
