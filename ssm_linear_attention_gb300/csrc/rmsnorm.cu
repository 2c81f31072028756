// rmsnorm.cu -- residual add and RMS norm of the stream between a model's layers, with an
// output in float32, bf16, or e4m3 with float32 scales.
//
// r = x + residual, y = r * rsqrt(mean(r^2) + eps) * weight. Every element is read once
// and written once, so HBM bounds a large call and the launch a small one. A CTA takes a
// row, keeps it in registers between the sum of squares and the output, and loops over
// rows with the next row's loads issued before this row's sums, its weights in registers
// throughout.
//
// Measured (one GB300, GPU time of a call; "of" the measured copy bandwidth): 32768 x 4096 bf16
// to e4m3 in groups of 128: 146.5 us, 6.4 TB/s, 95 % of it. 509 x 8192 bf16: 6.8 us, 4.9 TB/s,
// of which a launch that does nothing much (one row of 4096: 2.1 us) is a third.
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

// 8 values times f as e4m3.
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float* v, float f) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * f, v[4 * i + 1] * f), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * f, v[4 * i + 3] * f), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// Sum, or the largest, over the CTA. Consecutive calls use different arrays: `red` may be
// written again once a later call's barrier has passed.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (blockDim.x == 32) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int n = blockDim.x >> 5;
    v = (threadIdx.x & 31) < n ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (blockDim.x == 32) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int n = blockDim.x >> 5;
    return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < n ? red[threadIdx.x & 31] : 0u);
}

// The 8-bit scale rule: amax's bits m -> (448 / amax, amax / 448), NaN for what is not finite.
__device__ __forceinline__ float2 scale_of(uint32_t m) {
    if (m >= 0x7f800000u) return make_float2(__uint_as_float(0x7fc00000u), __uint_as_float(0x7fc00000u));
    const float a = fmaxf(__uint_as_float(m), attn::kAmaxFloor);
    return make_float2(__fdiv_rn(attn::kE4M3Max, a), __fdiv_rn(a, attn::kE4M3Max));
}

// 8 values as loaded.
template <bool BF>
struct Raw;
template <>
struct Raw<true> {
    uint4 v;
    __device__ __forceinline__ void load(const void* p, long i) {
        v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
        f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
    }
};
template <>
struct Raw<false> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p, long i) {
        a = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)[0];
        b = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)[1];
    }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

// Rows of a multiple of 8 columns: thread t has the 8-column pieces t, t + threads, ... (V of
// them at most).
constexpr int max_threads(int v) { return v == 1 ? 1024 : 512; }

template <bool ABF, int OUT, int V>
__global__ void __launch_bounds__(max_threads(V), V == 2 ? 2 : 1) vector_kernel(const Args a) {
    __shared__ float red_s[2][32];
    __shared__ uint32_t red_m[2][32];
    constexpr bool AHEAD = V <= 4;               // the next row's loads before this row's sums
    constexpr bool WREG = V == 1 || (V == 2 && ABF);  // weights in registers before they are used
    attn::wait_for_stream();
    const int np = a.cols >> 3;
    Raw<ABF> x[V], r[V];
    long row = blockIdx.x;
    auto load_row = [&](long at) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int p = threadIdx.x + k * blockDim.x;
            if (p < np) {
                x[k].load(a.x, at * a.cols + p * 8);
                if (a.res) r[k].load(a.res, at * a.cols + p * 8);
            }
        }
    };
    if (AHEAD) load_row(row);
    for (int turn = 0; row < a.rows; row += gridDim.x, turn ^= 1) {
        float y[V][8], ss = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int p = threadIdx.x + k * blockDim.x;
            if (p < np) {
                if (!AHEAD) {
                    x[k].load(a.x, row * a.cols + p * 8);
                    if (a.res) r[k].load(a.res, row * a.cols + p * 8);
                }
                x[k].get(y[k]);
                if (a.res) {
                    float f[8];
                    r[k].get(f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[k][e] += f[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[k][e] = 0.f;
            }
        }
        // the next row, while this one is summed
        if (AHEAD && row + gridDim.x < a.rows) load_row(row + gridDim.x);
        float w[WREG ? V : 1][8];
        if (WREG) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (threadIdx.x + k * blockDim.x < np) load8(a.w + (threadIdx.x + k * blockDim.x) * 8, false, w[WREG ? k : 0]);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int p = threadIdx.x + k * blockDim.x;
            if (a.res_out && p < np)
                store8(static_cast<char*>(a.res_out) + (row * a.cols + p * 8) * (ABF ? 2 : 4), ABF, y[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += y[k][e] * y[k][e];
        }
        const float rstd = rsqrtf(block_sum(ss, red_s[turn]) / (float)a.cols + a.eps);
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int p = threadIdx.x + k * blockDim.x;
            float* wk = w[WREG ? k : 0];
            if (!WREG && p < np) load8(a.w + p * 8, false, wk);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (p < np) y[k][e] = y[k][e] * rstd * wk[e];
                if (OUT == RSSM_E4M3) top = max(top, __float_as_uint(y[k][e]) & 0x7fffffffu);
            }
            const long at = row * a.cols + p * 8;
            if (OUT != RSSM_E4M3) {
                if (p < np) store8(static_cast<char*>(a.y) + at * (OUT == RSSM_BF16 ? 2 : 4), OUT == RSSM_BF16, y[k]);
            } else if (a.group) {  // 128 columns: 16 lanes
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float2 sc = scale_of(top);
                if (p < np) {
                    store8_e4m3(static_cast<uint8_t*>(a.y) + at, y[k], sc.x);
                    if ((threadIdx.x & 15) == 0) a.y_scale[at >> 7] = sc.y;
                }
                top = 0;
            }
        }
        if (OUT == RSSM_E4M3 && !a.group) {
            const float2 sc = scale_of(block_max(top, red_m[turn]));
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int p = threadIdx.x + k * blockDim.x;
                if (p < np) store8_e4m3(static_cast<uint8_t*>(a.y) + row * a.cols + p * 8, y[k], sc.x);
            }
            if (threadIdx.x == 0) a.y_scale[row] = sc.y;
        }
    }
}

// Rows of other lengths (their starts are not 16-byte aligned): element by element, the row
// in dynamic shared memory. A 128-column scale group never comes here.
__global__ void __launch_bounds__(256) element_kernel(const Args a) {
    extern __shared__ float row[];
    __shared__ float red_s[32];
    __shared__ uint32_t red_m[32];
    const long base = (long)blockIdx.x * a.cols;
    float ss = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float r = load1(a.x, base + c, a.abf);
        if (a.res) r += load1(a.res, base + c, a.abf);
        if (a.res_out) store1(a.res_out, base + c, a.abf, r);
        row[c] = r;
        ss += r * r;
    }
    const float rstd = rsqrtf(block_sum(ss, red_s) / (float)a.cols + a.eps);
    uint32_t top = 0;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        const float y = row[c] * rstd * a.w[c];
        row[c] = y;
        if (a.out_dtype != RSSM_E4M3) store1(a.y, base + c, a.out_dtype == RSSM_BF16, y);
        top = max(top, __float_as_uint(y) & 0x7fffffffu);
    }
    if (a.out_dtype != RSSM_E4M3) return;
    const float2 sc = scale_of(block_max(top, red_m));
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x)
        static_cast<uint8_t*>(a.y)[base + c] = __nv_cvt_float_to_fp8(row[c] * sc.x, __NV_SATFINITE, __NV_E4M3);
    if (threadIdx.x == 0) a.y_scale[blockIdx.x] = sc.y;
}

template <bool ABF, int OUT, int V>
static int launch(const Args& a, const DeviceInfo& di, cudaStream_t st) {
    const int threads = ((a.cols / 8 + V - 1) / V + 31) / 32 * 32;
    // as many CTAs as fit the SMs by threads, and 32 of one warp
    const int per_sm = min(max(1, (V <= 2 ? 1024 : 512) / threads), 32);
    const long grid = min((long)a.rows, (long)di.sm_count * per_sm);
    attn::launch_early(vector_kernel<ABF, OUT, V>, (int)grid, threads, 0, st, a);
    return launch_status();
}

// Pieces per thread: one where rows are few and the latency of one counts, two to have more
// bytes in flight, as many as the row wants beyond.
template <bool ABF, int OUT>
static int launch_v(const Args& a, const DeviceInfo& di, cudaStream_t st) {
    const int np = a.cols / 8;
    if (a.rows <= 2 * di.sm_count && np <= max_threads(1)) return launch<ABF, OUT, 1>(a, di, st);
    if (np <= 2 * max_threads(2)) return launch<ABF, OUT, 2>(a, di, st);
    if (np <= 4 * max_threads(4)) return launch<ABF, OUT, 4>(a, di, st);
    return launch<ABF, OUT, 8>(a, di, st);
}

template <bool ABF>
static int launch_out(const Args& a, const DeviceInfo& di, cudaStream_t st) {
    return a.out_dtype == RSSM_E4M3   ? launch_v<ABF, RSSM_E4M3>(a, di, st)
           : a.out_dtype == RSSM_BF16 ? launch_v<ABF, RSSM_BF16>(a, di, st)
                                      : launch_v<ABF, RSSM_F32>(a, di, st);
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
    DeviceInfo di;
    if (!device_info(&di)) return RSSM_ERR_CUDA;
    const norm::Args a{x, residual, weight, residual_out, y, y_scale, eps, d->rows, d->cols,
                       q ? d->scale_group : 0, d->act_dtype == RSSM_BF16, d->out_dtype};
    const cudaStream_t st = (cudaStream_t)stream;
    if (d->cols % 8 == 0)
        return a.abf ? norm::launch_out<true>(a, di, st) : norm::launch_out<false>(a, di, st);
    const int smem = d->cols * 4;
    if (!ensure_smem_limit((const void*)norm::element_kernel, smem)) return RSSM_ERR_CUDA;
    norm::element_kernel<<<d->rows, 256, smem, st>>>(a);
    return launch_status();
}
