// linattn.cu -- linear attention with a decay for each head: the entry points, the recurrence over a
// prompt, and the step of one token.
//
//   S_t = exp(g_t) S_{t-1} + w_t v_t k_t^T,   o_t = scale S_t q_t      (S [P][N] per head)
//
// The step reads and writes every state once and is bound by that; a lane has pieces of 16 bytes
// of one value row, eight lanes a row, so that a sum over N takes three shuffles.
//
// The recurrence over a prompt keeps 16 value rows of a head in the registers of a CTA and takes one token
// after another.
#include "linattn.cuh"

namespace rssm {
namespace linattn {

// ------------------------------------------------------------------ one token ----

// VEC elements of 16 bytes: 4 float32 or 8 bf16.
template <bool BF>
__device__ __forceinline__ void unpack16(const uint4& x, float* f) {
    if (BF) {
        f[0] = bf16_lo(x.x); f[1] = bf16_hi(x.x); f[2] = bf16_lo(x.y); f[3] = bf16_hi(x.y);
        f[4] = bf16_lo(x.z); f[5] = bf16_hi(x.z); f[6] = bf16_lo(x.w); f[7] = bf16_hi(x.w);
    } else {
        f[0] = __uint_as_float(x.x); f[1] = __uint_as_float(x.y);
        f[2] = __uint_as_float(x.z); f[3] = __uint_as_float(x.w);
    }
}
template <bool BF>
__device__ __forceinline__ uint4 pack16(const float* f) {
    if (BF) return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// SBF: bf16 state. R value rows a lane group of eight, V pieces of each.
template <bool ABF, bool SBF, int N>
struct Step {
    static constexpr int E = SBF ? 8 : 4;            // elements of a piece
    static constexpr int V = N / (8 * E);            // pieces of a row in a lane
    static constexpr int R = 8 / V < 4 ? 8 / V : 4;  // rows of a lane
    static constexpr int WARPS = 4;
    static constexpr int ROWS = WARPS * 4 * R;       // value rows of a CTA
};

template <bool ABF, bool SBF, int N>
__global__ void __launch_bounds__(128) step_kernel(const Args a, int P) {
    using C = Step<ABF, SBF, N>;
    constexpr int E = C::E, V = C::V, R = C::R;
    attn::wait_for_stream();
    const int parts = P / C::ROWS;
    const int part = blockIdx.x % parts, bh = blockIdx.x / parts, b = bh / a.H, h = bh - b * a.H;
    const int slot = a.slots[b];
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        if (threadIdx.x == 0) set_dev_err(a.dev_err, RSSM_DEVERR_SLOT);
        return;
    }
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int p0 = part * C::ROWS + (threadIdx.x >> 5) * 4 * R + (lane >> 3);  // rows p0, p0 + 4, ...
    uint4* const s = reinterpret_cast<uint4*>(static_cast<char*>(a.state) +
                                              (((long)slot * a.H + h) * P + p0) * N * (SBF ? 2 : 4)) + l;
    constexpr int ROW = N / E;  // pieces of a row
    uint4 x[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < V; ++j) x[r][j] = __ldcs(s + r * 4 * ROW + j * 8);
    const int kh = h / (a.H / a.G);
    const long q0 = b * a.q_stride + kh * N, k0 = b * a.k_stride + kh * N;
    const long v0 = b * a.v_stride + (long)h * P + p0;
    float q[V][E], k[V][E], v[R];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int at = (j * 8 + l) * E;
        if constexpr (E == 8) {
            load8(static_cast<const char*>(a.q) + (q0 + at) * (ABF ? 2 : 4), ABF, q[j]);
            load8(static_cast<const char*>(a.k) + (k0 + at) * (ABF ? 2 : 4), ABF, k[j]);
        } else {
            load4(static_cast<const char*>(a.q) + (q0 + at) * (ABF ? 2 : 4), 0, ABF, q[j]);
            load4(static_cast<const char*>(a.k) + (k0 + at) * (ABF ? 2 : 4), 0, ABF, k[j]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = load1(a.v, v0 + r * 4, ABF);
    const float f = expf(a.g[b * a.g_stride + h]);
    const float w = a.w ? a.w[b * a.w_stride + h] : 1.f;
    float o[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float u = w * v[r];
        o[r] = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float y[E];
            unpack16<SBF>(x[r][j], y);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                y[e] = f * y[e] + u * k[j][e];
                o[r] += y[e] * q[j][e];
            }
            __stcs(s + r * 4 * ROW + j * 8, pack16<SBF>(y));
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int m = 4; m >= 1; m >>= 1) o[r] += __shfl_xor_sync(0xffffffffu, o[r], m);
        if (l == 0) store1(a.o, ((long)b * a.H + h) * P + p0 + r * 4, a.obf, a.scale * o[r]);
    }
}

template <bool ABF, bool SBF>
static int launch_step(const Args& a, int N, int P, cudaStream_t st) {
    const long rows = (long)a.batch * a.H;
    if (N == 64) attn::launch_early(step_kernel<ABF, SBF, 64>, (int)(rows * (P / Step<ABF, SBF, 64>::ROWS)), 128, 0, st, a, P);
    else attn::launch_early(step_kernel<ABF, SBF, 128>, (int)(rows * (P / Step<ABF, SBF, 128>::ROWS)), 128, 0, st, a, P);
    return launch_status();
}

// ------------------------------------------------ a prompt, token by token ----

constexpr int kRows = 16;  // value rows of a CTA
constexpr int kTile = 16;  // tokens staged at a time

// Thread t: value row t / 8, keys 4 (t % 8) + 32 j + 0..3.
template <bool ABF, int N>
__global__ void __launch_bounds__(128) recurrence_kernel(const Args a, int P) {
    constexpr int J = N / 32;
    __shared__ __align__(16) float sq[kTile][N], sk[kTile][N];
    __shared__ float sv[kTile][kRows], so[kTile][kRows], sf[kTile], sw[kTile];
    attn::wait_for_stream();
    const int parts = P / kRows, part = blockIdx.x % parts, bh = blockIdx.x / parts, b = bh / a.H, h = bh - b * a.H;
    int begin, end, slot;
    if (!row_of(a, b, threadIdx.x == 0 && part == 0, begin, end, slot)) return;
    const int t = threadIdx.x, p = t >> 3, l = t & 7;
    const int kh = h / (a.H / a.G);
    const long at = (((long)slot * a.H + h) * P + part * kRows + p) * N;
    float s[J][4];
    if (a.resume && a.resume[b]) {
#pragma unroll
        for (int j = 0; j < J; ++j) load4(static_cast<const char*>(a.state) + (at + 4 * l + 32 * j) * (a.sbf ? 2 : 4), 0, a.sbf, s[j]);
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
    }
    for (int i0 = begin; i0 < end; i0 += kTile) {
        const int n = min(kTile, end - i0);
        for (int e = t; e < n * (N / 4); e += 128) {
            const int i = e / (N / 4), c = e % (N / 4) * 4;
            const long row = i0 + i;
            load4(static_cast<const char*>(a.q) + (row * a.q_stride + kh * N + c) * (ABF ? 2 : 4), 0, ABF, &sq[i][c]);
            load4(static_cast<const char*>(a.k) + (row * a.k_stride + kh * N + c) * (ABF ? 2 : 4), 0, ABF, &sk[i][c]);
        }
        for (int e = t; e < n * kRows; e += 128) {
            const int i = e / kRows, c = e % kRows;
            sv[i][c] = load1(a.v, (i0 + i) * a.v_stride + (long)h * P + part * kRows + c, ABF);
        }
        if (t < n) {
            sf[t] = expf(a.g[(i0 + t) * a.g_stride + h]);
            sw[t] = a.w ? a.w[(i0 + t) * a.w_stride + h] : 1.f;
        }
        __syncthreads();
        for (int i = 0; i < n; ++i) {
            const float f = sf[i], u = sw[i] * sv[i][p];
            float o = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float4 k = *reinterpret_cast<const float4*>(&sk[i][4 * l + 32 * j]);
                const float4 q = *reinterpret_cast<const float4*>(&sq[i][4 * l + 32 * j]);
                s[j][0] = f * s[j][0] + u * k.x;
                s[j][1] = f * s[j][1] + u * k.y;
                s[j][2] = f * s[j][2] + u * k.z;
                s[j][3] = f * s[j][3] + u * k.w;
                o += s[j][0] * q.x + s[j][1] * q.y + (s[j][2] * q.z + s[j][3] * q.w);
            }
#pragma unroll
            for (int m = 4; m >= 1; m >>= 1) o += __shfl_xor_sync(0xffffffffu, o, m);
            if (l == 0) so[i][p] = o;
        }
        __syncthreads();
        for (int e = t; e < n * kRows; e += 128) {
            const int i = e / kRows, c = e % kRows;
            store1(a.o, ((long)(i0 + i) * a.H + h) * P + part * kRows + c, a.obf, a.scale * so[i][c]);
        }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        char* const to = static_cast<char*>(a.state) + (at + 4 * l + 32 * j) * (a.sbf ? 2 : 4);
        if (a.sbf) *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(s[j][0], s[j][1]), pack_bf16x2(s[j][2], s[j][3]));
        else *reinterpret_cast<float4*>(to) = make_float4(s[j][0], s[j][1], s[j][2], s[j][3]);
    }
}

template <bool ABF>
static int launch_recurrence(const Args& a, int N, int P, cudaStream_t st) {
    const int grid = a.batch * a.H * (P / kRows);
    if (N == 64) attn::launch_early(recurrence_kernel<ABF, 64>, grid, 128, 0, st, a, P);
    else attn::launch_early(recurrence_kernel<ABF, 128>, grid, 128, 0, st, a, P);
    return launch_status();
}

}  // namespace linattn
}  // namespace rssm

using namespace rssm;

extern "C" size_t rssm_linattn_workspace_size(const rssm_linattn_dims* d, int32_t n_tokens) {
    if (linattn::check_dims(d) != RSSM_OK || n_tokens < 0 || d->act_dtype != RSSM_BF16) return 0;
    return linattn::chunk_workspace(d, n_tokens);
}

extern "C" int rssm_linattn_prompt(const rssm_linattn_dims* d, const rssm_linattn_inputs* in, int32_t n_tokens,
                                   const int32_t* cu_tokens, const uint8_t* resume, void* state,
                                   const int32_t* cache_indices, void* workspace, size_t workspace_bytes, void* o,
                                   int32_t* dev_err, rssm_stream_t stream) {
    if (const int rc = linattn::check_dims(d)) return rc;
    if (n_tokens < 0) return RSSM_ERR_INVALID_ARG;
    if (!cu_tokens && d->batch && n_tokens % d->batch) return RSSM_ERR_CONFIG;
    if (d->batch == 0 || n_tokens == 0) return RSSM_OK;
    if (!linattn::ok_inputs(d, in) || !ok_opt_ptr(cu_tokens) || !ok_opt_ptr(resume) || !ok_ptr(state) ||
        !ok_ptr(cache_indices) || !ok_ptr(o))
        return RSSM_ERR_INVALID_ARG;
    linattn::Args a = linattn::make_args(d, in, state, cache_indices, o, dev_err);
    a.cu = cu_tokens;
    a.resume = resume;
    a.tokens = n_tokens;
    a.each = n_tokens / d->batch;
    const cudaStream_t st = (cudaStream_t)stream;
    if (d->act_dtype == RSSM_BF16) {
        const size_t need = linattn::chunk_workspace(d, n_tokens);
        if (need && (!ok_ptr(workspace) || workspace_bytes < need)) return RSSM_ERR_INVALID_ARG;
        return linattn::prompt_chunks(d, a, workspace, RSSM_WAIT_NS, st);
    }
    return linattn::launch_recurrence<false>(a, d->key_dim, d->value_dim, st);
}

extern "C" int rssm_linattn_step(const rssm_linattn_dims* d, const rssm_linattn_inputs* in, void* state,
                                 const int32_t* cache_indices, void* o, int32_t* dev_err, rssm_stream_t stream) {
    if (const int rc = linattn::check_dims(d)) return rc;
    if (d->batch == 0) return RSSM_OK;
    if (!linattn::ok_inputs(d, in) || !ok_ptr(state) || !ok_ptr(cache_indices) || !ok_ptr(o)) return RSSM_ERR_INVALID_ARG;
    const linattn::Args a = linattn::make_args(d, in, state, cache_indices, o, dev_err);
    const cudaStream_t st = (cudaStream_t)stream;
    const int N = d->key_dim, P = d->value_dim;
    if (d->act_dtype == RSSM_BF16)
        return a.sbf ? linattn::launch_step<true, true>(a, N, P, st) : linattn::launch_step<true, false>(a, N, P, st);
    return a.sbf ? linattn::launch_step<false, true>(a, N, P, st) : linattn::launch_step<false, false>(a, N, P, st);
}
