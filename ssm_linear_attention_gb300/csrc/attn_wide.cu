// attn_wide.cu -- paged attention where 9 to 64 queries (8-bit cache: 17 to 64) share a key head,
// bf16 activations.
//
// The mathematics and the tile list are attn_decode.cu's. With so many queries the products and
// the softmax of a warp-level kernel cost more than the bytes (every warp of 8 queries reads
// each tile from shared memory again and turns four scores a lane into weights), so here they
// go to the tensor memory: a chunk is up to 128 consecutive tokens (8 tiles) of a (row, key
// head), and for its N queries (M rounded up to 16, 32 or 64)
//     S [128 tokens][N]     = K Q^T     A = K, its rows as the cache has them
//     O^T [D][2 N]         += V^T P     A = V transposed by its descriptor, P = [hi | lo]
// with a token a lane of S: a thread makes its token's weights for N / 2 (N / 4) queries without
// looking at another lane, and writes them as rows of P. The weights are two bf16 parts,
// side by side in P, so that V is read once for both; their sums meet when a (row, head) ends.
// As there, the weights' base is 8 (log2 units) above the largest score, and O is rescaled only when a
// score passes it.
//
// One CTA per SM, a range of the tile list each. Warps 0 to 7 (or 15): softmax, a quarter of the
// tensor memory's lanes and half (a quarter) of the queries each. Then a warp for loads
// (TMA), one for the products, two for the queries of the next (row, head), and with an 8-bit
// cache eight that turn the loaded tiles into operands (four K in f16, four V in bf16). They meet at
// mbarriers; S has two buffers, so that the products of a chunk run beside the softmax of the
// one before. The descriptors are made by the whole warp and only stepped by the elected lane:
// built inside its branch they cost more than the products (1100 against 480 cycles for eight).
//
// The list's unit is a chunk here, and a (row, head) counts for one more (its first maxima, its
// output): a cut never leaves two CTAs a part of one chunk each.
//
// Measured (one GB300, GPU time of a call; in brackets the warp-level kernel that took these
// calls before): 128 rows of 500 to 2000 tokens, 4 drafts, 4 key heads of 8 queries, D 128, bf16
// cache: 65 us, 5.0 TB/s, 73 % of the measured copy bandwidth [88]; 26 rows of 2.8k to 11k
// tokens, M 32, 8-bit cache: 136 us, 43 % [203], where the conversions' and the softmax's shared-
// memory accesses wait on one another; 147 rows of 500 to 2090 tokens, M 32, D 64, bf16: 104 us
// [130]; 34 rows of 120 to 470, M 32, bf16: 12.6 us [17.4]; 24 rows of 28 to 113, M 64, bf16: 19 us
// [22.6]; 64 rows of 1000 to 4000 tokens, M 64, D 128, bf16: 80 us [147], 8-bit: 125 [159].
// Short (row, head)s over an 8-bit cache, several to a CTA, are level: 55 rows of 100 to 384, M 32,
// D 64: 28 us [25.6]. Tried, when values were f16, too: 16 softmax warps for 32 queries (level), integer
// conversions of e4m3 (148 us against 136), conversions by four warps for K and V in turn (140
// against 137).
#include <cstring>

#include "attn_decode.cuh"
#include "umma.cuh"

namespace rssm {
namespace attn {

constexpr int kChunk = 128;            // tokens of a product
constexpr int kChunkTiles = kChunk / kTok;
constexpr int kBlk = kChunk * 128;     // bytes of 64 operand columns of a chunk
constexpr int kWideRows = 512;         // rows of a launch
constexpr int kWideRowBytes = 7168;    // their facts in shared memory
constexpr int kInfo = 8;               // chunks whose look-ups are kept
// (row, head)s whose queries' factors are kept. Those of (row, head) s are written once the products of s - 2
// are done; these waited for every softmax warp to take the scores of two chunks before, but a warp
// reads the factors after that: where each (row, head) is one chunk, those of s - 4 may still be read.
constexpr int kFactors = 8;
// What a (row, head) costs beside its chunks, in chunks, where the list is cut: 147 rows, D 64, 116 us with
// 0, 104 with 1, 100 with 2; 55 rows of 384, 8-bit, 34, 27 and 29; 128 rows of 4 drafts, D 128, level.
constexpr int kHeadCost = 1;

template <int D, bool E4M3, int N>
struct Wide {
    static constexpr int PARTS = N == 64 ? 4 : 2;  // softmax threads of a token
    static constexpr int NH = N / PARTS;           // queries of one
    static constexpr int SOFT = kChunk * PARTS;    // softmax threads
    static constexpr int W0 = SOFT / 32;           // the warp after them
    static constexpr int THREADS = SOFT + (E4M3 ? 384 : 128);
    static constexpr int OPER = D / 64 * kBlk;   // K or V operand of a chunk
    // operand buffers of K and V, loaded chunks of 8-bit values
    static constexpr int SK = D == 64 ? (E4M3 ? 2 : 4) : E4M3 ? 1 : 2;
    static constexpr int SV = D == 64 ? (E4M3 ? 2 : 4) : E4M3 ? 2 : 3;
    static constexpr int RS = E4M3 ? (D == 64 ? 4 : 2) : 0;
    static constexpr int RAW = 2 * kChunk * D;   // K then V
    static constexpr int QBYTES = N * D * 2;
    static constexpr int QB = N == 64 && D == 128 ? 1 : 2;
    static constexpr int PK = 2 * N / 8 * 128;   // P: bytes of 8 tokens
    static constexpr int PBYTES = kChunk / 8 * PK;
    static constexpr int SC = RS + SV;           // chunks whose scales are kept
    static constexpr int SCBYTES = E4M3 ? SC * kChunk * 2 * 4 : 0;
    static constexpr int SMEM = PBYTES + QB * QBYTES + SK * OPER + SV * OPER + RS * RAW + SCBYTES + kWideRowBytes;
    // Tensor memory: two buffers of S in SA sums each, then O's hi and lo parts. (The tensor core
    // cuts what it adds to a sum: each of D / 16 additions can cost a large score its last bit; two
    // sums instead of one: at most 2 % of a call.)
    static constexpr int SA = 2;
    static constexpr uint32_t OCOL = 2 * SA * N;
    static constexpr uint32_t COLS = 8 * N;
};

// The whole warp's bounded wait.
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, volatile int* abort, const DecArgs& a) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_long(bar, parity, abort, a.wait_ns, a.dev_err);
}
// Barrier of the THREADS softmax threads; true where x is on any of them.
template <int THREADS>
__device__ __forceinline__ bool any_soft(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(THREADS)
        : "memory");
    return r != 0;
}
// Combine v[q] over the warp's lanes; a lane ends with that of query lane / (32 / NH) in v[0].
template <int NH, bool MAX>
__device__ __forceinline__ void combine(float (&v)[NH], int lane) {
    int cnt = NH;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        if (cnt > 1) {
            cnt >>= 1;
#pragma unroll
            for (int k = 0; k < NH / 2; ++k) {
                if (k >= cnt) break;
                const bool up = lane & o;
                const float send = up ? v[k] : v[k + cnt], keep = up ? v[k + cnt] : v[k];
                const float got = __shfl_xor_sync(0xffffffffu, send, o);
                v[k] = MAX ? fmaxf(keep, got) : keep + got;
            }
        } else {
            const float got = __shfl_xor_sync(0xffffffffu, v[0], o);
            v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
        }
    }
}
// Two float32 as an operand pair.
template <bool F16>
__device__ __forceinline__ uint32_t pair16(float lo, float hi) {
    uint32_t r;
    if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// One (row, head) of a range: its chunks are units t .. end of the list, x.at the first one's number;
// all of its chunks. (Its first kHeadCost units stand for no chunk.)
struct Seg {
    Tile x;
    uint32_t t, end, chunks;
    uint32_t after;  // the unit where the next (row, head) begins
};
// The (row, head) that begins at unit s0, cut to the range; false when it has no chunk there.
__device__ __forceinline__ bool clip_seg(const uint32_t* cum, uint32_t s0, uint32_t c0, uint32_t c1, Seg& s) {
    const uint32_t units = cum[s.x.b + 1] - cum[s.x.b], first = s0 + kHeadCost;
    s.after = s0 + units;
    s.chunks = units - kHeadCost;
    s.t = max(c0, first);
    s.end = min(c1, s.after);
    s.x.at = (int)(s.t - first);
    return s.t < s.end;
}
// The one after s; t = c1 when there is none.
__device__ __forceinline__ void next_seg(const DecArgs& a, const uint32_t* cum, uint32_t c1, Seg& s) {
    const uint32_t s0 = s.after;
    s.t = c1;
    if (s0 >= c1) return;
    if (++s.x.h == a.hkv) {
        s.x.h = 0;
        do ++s.x.b;
        while (cum[s.x.b + 1] == cum[s.x.b]);
    }
    if (!clip_seg(cum, s0, s0, c1, s)) s.t = c1;
}
__device__ __forceinline__ Seg first_seg(const DecArgs& a, const uint32_t* cum, uint32_t c0, uint32_t c1,
                                         bool single) {
    Seg s;
    s.x = find_tile(a, cum, c0, single);
    if (!clip_seg(cum, c0 - s.x.at, c0, c1, s)) next_seg(a, cum, c1, s);
    return s;
}
template <int D, bool E4M3, int N>
__global__ void __launch_bounds__((Wide<D, E4M3, N>::THREADS), 1)
    wide_kernel(const __grid_constant__ DecArgs a, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
    using C = Wide<D, E4M3, N>;
    constexpr int NH = C::NH;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    unsigned char* const sp = smem;                  // P
    unsigned char* const sq = sp + C::PBYTES;        // queries
    unsigned char* const sk = sq + C::QB * C::QBYTES;
    unsigned char* const sv = sk + C::SK * C::OPER;
    unsigned char* const raw = sv + C::SV * C::OPER;
    float* const scales = reinterpret_cast<float*>(raw + C::RS * C::RAW);
    Rows rows;
    rows.cum = reinterpret_cast<uint32_t*>(raw + C::RS * C::RAW + C::SCBYTES);
    rows.len = reinterpret_cast<int*>(rows.cum) + kWideRows + 4;
    rows.slot = rows.len + kWideRows;
    uint32_t* const cum = rows.cum;

    __shared__ uint64_t kfull[4], kfree[4], vfull[4], vfree[4], rfull[4], rfree[4];
    __shared__ uint64_t sfull[2], sfree[2], qfull[2], qfree[2], pfull, pfree, drain;
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    __shared__ int q_row[64], q_tok[64];
    __shared__ uint2 scan[C::THREADS / 32];
    __shared__ int info_y[kInfo][kChunkTiles];  // the tiles' rows in the cache, -1: no page
    __shared__ uint32_t info_ok[kInfo];         // and which have one
    __shared__ uint32_t odd[2][4][C::PARTS];  // cleared tokens to add below, of a warp's 32
    __shared__ __align__(16) float rs[kFactors][N];           // score factors of the queries (8-bit cache)
    __shared__ __align__(16) float ms[N], mb[N], fs[N];  // running maxima, finite; the last rescaling
    __shared__ __align__(16) float red[4][N], sums[4][N];
    __shared__ Run runs[2];
    __shared__ int nruns, last_flag[2];

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&kfull[i], E4M3 ? 4 : 1);
            mbar_init(&vfull[i], E4M3 ? 4 : 1);
            mbar_init(&kfree[i], 1);
            mbar_init(&vfree[i], 1);
            mbar_init(&rfull[i], 1);
            mbar_init(&rfree[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 2);
            mbar_init(&sfree[i], C::W0);
            mbar_init(&qfull[i], 2);
            mbar_init(&qfree[i], 1);
        }
        mbar_init(&pfull, C::W0);
        mbar_init(&pfree, 1);
        mbar_init(&drain, 1);
        fence_barrier_init();
        abort_flag = 0;
        nruns = 0;
        last_flag[0] = last_flag[1] = 0;
    }
    if (tid < a.M) {
        const int j = tid / a.G;
        q_tok[tid] = j;
        q_row[tid] = j * a.hq + tid - j * a.G;
    }
    const uint32_t longest = list_tiles<C::THREADS, kWideRows, kChunkTiles, kHeadCost>(a, rows, scan);
    write_empty_rows<D, C::THREADS>(a, rows);
    Cuts rg;
    uint32_t c0, c1;  // this CTA's range
    bool single;
    if (!cut_tiles(a, cum, longest, 2 + kHeadCost, kWholeTiles / kChunkTiles + kHeadCost, rg, c0, c1, single)) return;

    if (warp == C::W0 + 1) umma::tmem_alloc(&tmem_at, C::COLS);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = tmem_at;
    volatile int* const stop = &abort_flag;

    if (warp < C::W0) {
        // ------------------------------------------------------------- softmax
        const int half = warp >> 2;              // which of the queries
        const int tok = (warp & 3) * 32 + lane;  // of the chunk; lane of the tensor memory
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        const uint32_t ocol = lanes + C::OCOL + half * NH;
        const int q0 = half * NH;
        Ring sb, vb, pb;  // (pb: the parity of P's present use)
        int scb = 0;      // scales
        uint32_t i = 0, seg_no = 0;
        bool dead = false;
        for (Seg g = first_seg(a, cum, c0, c1, single); g.t < c1 && !dead; next_seg(a, cum, c1, g), ++seg_no) {
            const uint32_t t = g.t;
            const int len = rows.len[g.x.b];
            const RowSpan span = row_span(a, len);
            const int pos_t = (span.first + g.x.at * kChunkTiles) * kTok, left = span.tiles - g.x.at * kChunkTiles;
            const int app = a.appended ? 1 : 0;
            const int n_min = len + app, n_max = len + (app ? a.T : 0);
            const int b_min = a.window && n_min > a.window ? n_min - a.window : 0;
            const int b_max = a.window && n_max > a.window ? n_max - a.window : 0;
            float l[NH];
#pragma unroll
            for (int q = 0; q < NH; ++q) l[q] = 0.f;

            for (uint32_t u = t; u < g.end; ++u, ++i) {
                const bool first = u == t;
                const int n = min(left - (int)(u - t) * kChunkTiles, kChunkTiles);
                dead |= !await(&vfull[vb.slot], vb.parity, stop, a);
                const int pos0 = pos_t + (int)(u - t) * kChunk, pos = pos0 + tok;
                const uint32_t oks = info_ok[i % kInfo];
                const bool edge = oks != (1u << kChunkTiles) - 1 || pos0 + kChunk > n_min || pos0 < b_max;
                float ks = 1.f, vs = 1.f;
                if (E4M3) {
                    // (the value scale multiplies the weight where that meets the value: the maxima
                    // and l are the scores' alone)
                    const float* ts = scales + scb * 2 * kChunk + tok;
                    ks = ts[0];
                    vs = ts[kChunk];
                }
                dead |= !await(&sfull[sb.slot], sb.parity, stop, a);
                umma::fence_after_sync();
                float p[NH];
                umma::ld_cols<NH>(lanes + sb.slot * C::SA * N + q0, p);
                {
                    float p1[NH];
                    umma::ld_cols<NH>(lanes + (sb.slot * C::SA + 1) * N + q0, p1);
#pragma unroll
                    for (int q = 0; q < NH; ++q) p[q] += p1[q];
                }
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_plain(&sfree[sb.slot]);
                if (E4M3) {
                    const float* f = rs[seg_no % kFactors] + q0;
#pragma unroll
                    for (int q = 0; q < NH; q += 4) {
                        const float4 r = *reinterpret_cast<const float4*>(f + q);
                        p[q] *= r.x * ks;
                        p[q + 1] *= r.y * ks;
                        p[q + 2] *= r.z * ks;
                        p[q + 3] *= r.w * ks;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < NH; ++q) p[q] *= a.qscale;
                }
                int from = 0, to = NH;  // the queries that see this position
                if (__builtin_expect(edge, 0)) {  // hide what a query does not see, whatever it holds
                    // queries r of tokens jlo .. jhi see this position: r in [from, to)
                    const bool ok = oks >> (tok / kTok) & 1;
                    const int past = pos - n_min;
                    const int jlo = app ? max(0, past + 1) : past < 0 ? 0 : a.T;
                    const int in = past + a.window;
                    const int jhi = !a.window ? a.T - 1 : app ? min(a.T - 1, in) : in >= 0 ? a.T - 1 : -1;
                    from = ok ? jlo * a.G - q0 : NH, to = (jhi + 1) * a.G - q0;
#pragma unroll
                    for (int q = 0; q < NH; ++q)
                        if (q < from || q >= to) p[q] = -INFINITY;
                    // A weight of zero does not silence an infinity or a NaN in a value. Tokens that no
                    // query sees are cleared; one that only some see and that is not finite is
                    // cleared too, and added below for those that see it.
                    // (16 bytes a lane; the warps of the same tokens share them)
                    constexpr int PIECES = D / 8;
                    constexpr uint32_t share = C::PARTS == 2 ? 0x55555555u : 0x11111111u;
                    const bool mine = tok < n * kTok, hidden = !ok || pos >= n_max || pos < b_min;
                    unsigned char* const at = sv + vb.slot * C::OPER + (warp & 3) * 32 * 128 +
                                              ((lane % PIECES) >> 3) * kBlk + (lane & 7) * 16;
                    uint32_t is_odd = 0;
                    if (!E4M3 && a.T > 1) {
                        uint32_t some = __ballot_sync(0xffffffffu, mine && !hidden && (pos >= n_min || pos < b_max)) &
                                        (share << half);
                        for (; some; some &= some - 1) {
                            const int k = __ffs(some) - 1;
                            const uint4 v = *reinterpret_cast<const uint4*>(at + k * 128);
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                            bool bad = false;
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                bad |= (w[x] & 0x7f80u) == 0x7f80u || (w[x] & 0x7f800000u) == 0x7f800000u;
                            if (__any_sync(0xffffffffu, bad)) is_odd |= 1u << k;
                        }
                        if (lane == 0) odd[i & 1][warp & 3][half] = is_odd;
                    }
                    uint32_t clear = (__ballot_sync(0xffffffffu, mine && hidden) & (share << half)) | is_odd;
                    for (; clear; clear &= clear - 1)
                        if (lane < PIECES)
                            *reinterpret_cast<uint4*>(at + (__ffs(clear) - 1) * 128) = make_uint4(0, 0, 0, 0);
                }
                bool grow = first;
                float e[NH];  // exponents
                if (!first)
#pragma unroll
                    for (int q = 0; q < NH; q += 4) {
                        const float4 b = *reinterpret_cast<const float4*>(mb + q0 + q);
                        e[q] = p[q] - b.x;
                        e[q + 1] = p[q + 1] - b.y;
                        e[q + 2] = p[q + 2] - b.z;
                        e[q + 3] = p[q + 3] - b.w;
                        grow |= e[q] > 0.f;
                        grow |= e[q + 1] > 0.f;
                        grow |= e[q + 2] > 0.f;
                        grow |= e[q + 3] > 0.f;
                    }
                if (first || any_soft<C::SOFT>(grow || dead)) {
                    // the maxima move: theirs over the chunk, then l and O follow
                    float top[NH];
#pragma unroll
                    for (int q = 0; q < NH; ++q) top[q] = p[q];
                    combine<NH, true>(top, lane);
                    if (lane % (32 / NH) == 0) red[warp & 3][q0 + lane / (32 / NH)] = top[0];
                    dead = any_soft<C::SOFT>(dead);
                    if (dead) break;
                    if (tid < N) {
                        const float old = first ? -INFINITY : ms[tid];
                        const float top = fmaxf(fmaxf(red[0][tid], red[1][tid]), fmaxf(red[2][tid], red[3][tid]));
                        const float m = top > old ? top + kSlack : old;
                        ms[tid] = m;
                        // (seen only -infinity: weights of zero, and any score passes it)
                        mb[tid] = m == -INFINITY ? -1e30f : m;
                        fs[tid] = m == old ? 1.f : exp2_fast(old - m);
                    }
                    any_soft<C::SOFT>(false);
                    if (!first) {
                        dead |= !await(&pfree, pb.parity ^ 1, stop, a);  // O has the chunk before
                        umma::fence_after_sync();
                        float o[NH];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            umma::ld_cols<NH>(ocol + x * N, o);
#pragma unroll
                            for (int q = 0; q < NH; ++q) o[q] *= fs[q0 + q];
                            umma::st_cols<NH>(ocol + x * N, o);
                        }
                        umma::wait_st();
#pragma unroll
                        for (int q = 0; q < NH; ++q) l[q] *= fs[q0 + q];
                    }
#pragma unroll
                    for (int q = 0; q < NH; q += 4) {
                        const float4 b = *reinterpret_cast<const float4*>(mb + q0 + q);
                        e[q] = p[q] - b.x;
                        e[q + 1] = p[q + 1] - b.y;
                        e[q + 2] = p[q + 2] - b.z;
                        e[q + 3] = p[q + 3] - b.w;
                    }
                }
                bool careful = false;
                if (!E4M3 && edge && a.T > 1)
#pragma unroll
                    for (int k = 0; k < 4 * C::PARTS; ++k) careful |= odd[i & 1][k / C::PARTS][k % C::PARTS] != 0;
#pragma unroll
                for (int q = 0; q < NH; ++q) p[q] = exp2_fast(e[q]);
#pragma unroll
                for (int q = 0; q < NH; ++q) l[q] += p[q];
                if (E4M3 && __builtin_expect(edge, 0)) {  // a hidden token's scale may be anything
#pragma unroll
                    for (int q = 0; q < NH; ++q) p[q] = q < from || q >= to ? 0.f : p[q] * vs;
                } else if (E4M3) {
#pragma unroll
                    for (int q = 0; q < NH; ++q) p[q] *= vs;
                }
                if (i > 0) dead |= !await(&pfree, pb.parity ^ 1, stop, a);  // P is free
                unsigned char* const row = sp + (tok >> 3) * C::PK + (tok & 7) * 16 + q0 / 8 * 128;
#pragma unroll
                for (int q = 0; q < NH; q += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        hi[x] = pair16<false>(p[q + 2 * x], p[q + 2 * x + 1]);
                        lo[x] = pair16<false>(p[q + 2 * x] - bf16_lo(hi[x]), p[q + 2 * x + 1] - bf16_hi(hi[x]));
                    }
                    *reinterpret_cast<uint4*>(row + q * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(row + (N + q) * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_async_smem();
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_plain(&pfull);
                if (__builtin_expect(careful, 0)) {
                    dead |= !await(&pfree, pb.parity, stop, a);
                    umma::fence_after_sync();
                    float o[NH];
                    umma::ld_cols<NH>(ocol, o);
#pragma unroll 1
                    for (int k = 0; k < kChunk; ++k) {
                        if (!(odd[i & 1][k >> 5][k % C::PARTS] >> (k & 31) & 1)) continue;
                        const long y = info_y[i % kInfo][k / kTok] + k % kTok;
                        const float v = bf16_to_f(reinterpret_cast<const uint16_t*>(a.v)[y * D + tok % D]);
#pragma unroll
                        for (int q = 0; q < NH; ++q) {
                            const int r = q0 + q, end = n_min + (r < a.M ? q_tok[r] : 0) * app;
                            const int beg = a.window && end > a.window ? end - a.window : 0;
                            const unsigned char* w = sp + (k >> 3) * C::PK + (k & 7) * 16 + r / 8 * 128 + r % 8 * 2;
                            if (r < a.M && pos0 + k < end && pos0 + k >= beg)
                                o[q] += (bf16_to_f(*reinterpret_cast<const uint16_t*>(w)) +
                                         bf16_to_f(*reinterpret_cast<const uint16_t*>(w + N * 16))) * v;
                        }
                    }
                    umma::st_cols<NH>(ocol, o);
                    umma::wait_st();
                }
                sb.next(2);
                vb.next(C::SV);
                pb.next(1);
                if (++scb == C::SC) scb = 0;
            }
            // ------------------------------------------------ the (row, head) ends
            combine<NH, false>(l, lane);
            if (lane % (32 / NH) == 0) sums[warp & 3][q0 + lane / (32 / NH)] = l[0];
            dead = any_soft<C::SOFT>(dead);
            if (dead) break;
            const uint32_t nt = g.chunks, s0 = t - g.x.at;
            const bool whole = s0 >= c0 && s0 + nt <= c1;
            const int cta0 = s0 < c0 ? cta_of(rg, s0) : (int)blockIdx.x;
            const long slot = 2L * blockIdx.x + (cta0 < (int)blockIdx.x ? 0 : 1);
            const long out0 = (long)g.x.b * a.T * a.hq + g.x.h * a.G;
            float f[NH];
#pragma unroll
            for (int q = 0; q < NH; q += 4) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 y = *reinterpret_cast<const float4*>(&sums[k][q0 + q]);
                    x.x += y.x;
                    x.y += y.y;
                    x.z += y.z;
                    x.w += y.w;
                }
                f[q] = x.x;
                f[q + 1] = x.y;
                f[q + 2] = x.z;
                f[q + 3] = x.w;
            }
            dead |= !await(&pfree, pb.parity ^ 1, stop, a);  // O has the last chunk
            umma::fence_after_sync();
            // through P's buffer, which is free: rows of D values
            const bool as16 = whole && a.obf;
            {
                float o[NH], o2[NH], inv[NH];
#pragma unroll
                for (int q = 0; q < NH; ++q) inv[q] = whole ? reciprocal(f[q]) : 1.f;
                umma::ld_cols<NH>(ocol, o);
                umma::ld_cols<NH>(ocol + N, o2);
                umma::fence_before_sync();
#pragma unroll
                for (int q = 0; q < NH; ++q) {
                    o[q] = (o[q] + o2[q]) * inv[q];
                    if (whole && f[q] == 0.f) o[q] = 0.f;  // nothing was seen, whatever O holds
                }
                if (tok < D) {
                    if (as16) {
                        uint16_t* const dst = reinterpret_cast<uint16_t*>(sp) + q0 * D + tok;
#pragma unroll
                        for (int q = 0; q < NH; q += 2) {
                            const uint32_t y = pair16<false>(o[q], o[q + 1]);
                            dst[q * D] = (uint16_t)y;
                            dst[(q + 1) * D] = (uint16_t)(y >> 16);
                        }
                    } else {
                        float* const dst = reinterpret_cast<float*>(sp) + q0 * D + tok;
#pragma unroll
                        for (int q = 0; q < NH; ++q) dst[q * D] = o[q];
                    }
                }
            }
            dead = any_soft<C::SOFT>(dead);
            if (dead) break;
            const int pieces = D * (as16 ? 2 : 4) / 16;  // of a row, 16 bytes each
            for (int e = tid; e < a.M * pieces; e += C::SOFT) {
                const int r = e / pieces;
                const uint4 v = *reinterpret_cast<const uint4*>(sp + e * 16);
                if (whole)
                    reinterpret_cast<uint4*>(a.o)[(out0 + q_row[r]) * pieces + e - r * pieces] = v;
                else
                    reinterpret_cast<uint4*>(a.part)[slot * a.M * pieces + e] = v;
            }
            if (tid < a.M) {
                const float sum = sums[0][tid] + sums[1][tid] + sums[2][tid] + sums[3][tid];
                if (!whole)
                    reinterpret_cast<float2*>(a.part_ml)[slot * a.M + tid] = make_float2(ms[tid], sum);
                else if (a.lse)
                    a.lse[out0 + q_row[tid]] = sum == 0.f ? -INFINITY : (ms[tid] + log2_fast(sum)) * kLn2;
            }
            if (tid == 0 && !whole) {
                Run r;
                r.b = g.x.b;
                r.h = g.x.h;
                r.rec0 = r.rec1 = 0;
                r.cta0 = cta0;
                r.cta1 = s0 + nt > c1 ? cta_of(rg, s0 + nt - 1) : (int)blockIdx.x;
                runs[nruns++] = r;
            }
        }
    } else if (warp == C::W0) {
        // --------------------------------------------------------------- loads
        const uint64_t pol = policy_evict_first();
        Ring kb, vb, rb;
        int scb = 0;
        uint32_t i = 0;
        bool ok = true;
        for (Seg g = first_seg(a, cum, c0, c1, single); g.t < c1 && ok; next_seg(a, cum, c1, g)) {
            const uint32_t t = g.t;
            const RowSpan span = row_span(a, rows.len[g.x.b]);
            const int pos_t = (span.first + g.x.at * kChunkTiles) * kTok, left = span.tiles - g.x.at * kChunkTiles;
            const int32_t* pages = a.page_table + (long)rows.slot[g.x.b] * a.max_pages;
            int look = -1;  // rows of the next 32 tiles, one a lane
            for (uint32_t u = t; u < g.end; ++u, ++i) {
                const int tile = (int)(u - t) * kChunkTiles;
                if ((tile & 31) == 0) {
                    look = -1;
                    if (tile + lane < left) {  // (tiles past this range are looked up in vain)
                        const int pos = pos_t + (tile + lane) * kTok;
                        const int page = pages[pos >> a.ps_log2];
                        if (page < 0 || page >= a.num_pages) set_dev_err(a.dev_err, RSSM_DEVERR_PAGE);
                        else look = ((page * a.hkv + g.x.h) << a.ps_log2) + (pos & ((1 << a.ps_log2) - 1));
                    }
                }
                const int y = __shfl_sync(0xffffffffu, look, (tile & 31) + (lane & (kChunkTiles - 1)));
                const bool have = lane < kChunkTiles && y >= 0;
                const uint32_t oks = __ballot_sync(0xffffffffu, have);
                const uint32_t count = __popc(oks);
                if (lane < kChunkTiles) info_y[i % kInfo][lane] = y;
                if (lane == 0) info_ok[i % kInfo] = oks;
                __syncwarp();
                if (!E4M3) {
                    ok = await(&kfree[kb.slot], kb.parity ^ 1, stop, a);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&kfull[kb.slot], count * kTok * D * 2 + ((int)u == a.stall ? 16 : 0));
                    __syncwarp();
                    if (have)
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_2d(sk + kb.slot * C::OPER + c * kBlk + lane * kTok * 128, &kmap, 64 * c, y,
                                        &kfull[kb.slot], pol);
                    __syncwarp();
                    ok = await(&vfree[vb.slot], vb.parity ^ 1, stop, a);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&vfull[vb.slot], count * kTok * D * 2);
                    __syncwarp();
                    if (have)
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_2d(sv + vb.slot * C::OPER + c * kBlk + lane * kTok * 128, &vmap, 64 * c, y,
                                        &vfull[vb.slot], pol);
                    __syncwarp();
                    kb.next(C::SK);
                    vb.next(C::SV);
                } else {
                    ok = await(&rfree[rb.slot], rb.parity ^ 1, stop, a);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&rfull[rb.slot], count * kTok * (2 * D + 8) + ((int)u == a.stall ? 16 : 0));
                    __syncwarp();
                    if (have) {
                        unsigned char* dst = raw + rb.slot * C::RAW + lane * kTok * D;
                        float* sc = scales + scb * 2 * kChunk + lane * kTok;
                        bulk_g2s_hint(dst, a.k + (long)y * D, kTok * D, &rfull[rb.slot], pol);
                        bulk_g2s_hint(dst + kChunk * D, a.v + (long)y * D, kTok * D, &rfull[rb.slot], pol);
                        bulk_g2s_hint(sc, a.k_scale + y, kTok * 4, &rfull[rb.slot], pol);
                        bulk_g2s_hint(sc + kChunk, a.v_scale + y, kTok * 4, &rfull[rb.slot], pol);
                    }
                    __syncwarp();
                    rb.next(C::RS);
                    if (++scb == C::SC) scb = 0;
                }
            }
        }
    } else if (warp == C::W0 + 1) {
        // ------------------------------------------------------------ products
        constexpr uint32_t is = umma::idesc_16bit(128, N, !E4M3, false);
        constexpr uint32_t io = umma::idesc_16bit(128, 2 * N, true, true);
        const uint32_t sk_at = smem_addr(sk), sv_at = smem_addr(sv);
        const uint64_t pd = umma::smem_desc_mnmajor(smem_addr(sp), C::PK, 128);
        Ring kb, sb, qb, vb, pb;
        int before = 0;  // tiles of the chunk before, whose values are still to be added
        bool before_first = false, ok = true;
        // O^T (+)= V^T P of the chunk before
        auto add_values = [&]() {
            if (!await(&vfull[vb.slot], vb.parity, stop, a) || !await(&pfull, pb.parity, stop, a))
                return false;
            umma::fence_after_sync();
            // (D = 64: the second half of the accumulator's rows is not read)
            const uint64_t vd = umma::smem_desc_swizzle128(sv_at + vb.slot * C::OPER, D == 128 ? kBlk : 1024, 1024);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kChunkTiles; ++k)
                    if (k < before)
                        umma::mma_bf16(tmem + C::OCOL, vd + k * (2048 >> 4), pd + k * (2 * C::PK >> 4), io,
                                       k > 0 || !before_first);
                umma::commit_to(&pfree);
                umma::commit_to(&vfree[vb.slot]);
            }
            __syncwarp();
            vb.next(C::SV);
            pb.next(1);
            return true;
        };
        for (Seg g = first_seg(a, cum, c0, c1, single); g.t < c1 && ok; next_seg(a, cum, c1, g)) {
            const uint32_t t = g.t;
            ok = await(&qfull[qb.slot], qb.parity, stop, a);
            const int left = row_span(a, rows.len[g.x.b]).tiles - g.x.at * kChunkTiles;
            for (uint32_t u = t; u < g.end && ok; ++u) {
                ok = await(&kfull[kb.slot], kb.parity, stop, a) &&
                     await(&sfree[sb.slot], sb.parity ^ 1, stop, a);
                if (!ok) break;
                umma::fence_after_sync();
                const uint64_t kd = umma::smem_desc_swizzle128(sk_at + kb.slot * C::OPER, 16, 1024);
                const uint64_t qd = umma::smem_desc_kmajor(sq + qb.slot * C::QBYTES, 128, D / 8 * 128);
                const bool last = u + 1 == g.end;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma::mma_bf16(tmem + (sb.slot * C::SA + kk % C::SA) * N, kd + ((kk / 4 * kBlk + kk % 4 * 32) >> 4),
                                       qd + (kk * 256 >> 4), is, kk >= C::SA);
                    umma::commit_to(&kfree[kb.slot]);
                    if (last) umma::commit_to(&qfree[qb.slot]);
                    umma::commit_to(&sfull[sb.slot]);
                    mbar_arrive_plain(&sfull[sb.slot]);
                }
                __syncwarp();
                kb.next(C::SK);
                sb.next(2);
                if (before) ok = add_values();
                before = min(left - (int)(u - t) * kChunkTiles, kChunkTiles);
                before_first = u == t;
            }
            qb.next(C::QB);
        }
        if (ok) add_values();
    } else if (warp < C::W0 + 4) {
        // ------------------------------------------------------------- queries
        const int ql = tid - C::SOFT - 64;  // 64 threads, 8 values of a query each
        constexpr int LPQ = D / 8;     // lanes of a query
        Ring qb;
        uint32_t seg_no = 0;
        for (Seg g = first_seg(a, cum, c0, c1, single); g.t < c1; next_seg(a, cum, c1, g), ++seg_no) {
            const long row0 = (long)g.x.b * a.T;
            constexpr int PER = N * LPQ / 64, AT = PER < 4 ? PER : 4;
            bool ok = true;
#pragma unroll 1
            for (int k0 = 0; k0 < PER; k0 += AT) {
                uint4 x[AT];
#pragma unroll
                for (int k = 0; k < AT; ++k) {
                    const int r = (k0 + k) * (64 / LPQ) + ql / LPQ;
                    x[k] = make_uint4(0, 0, 0, 0);
                    if (r < a.M) {
                        const int j = q_tok[r];
                        x[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (row0 + j) * a.q_stride +
                                                               (long)(g.x.h * a.G + r - j * a.G) * D + ql % LPQ * 8);
                    }
                }
                if (k0 == 0) ok = await(&qfree[qb.slot], qb.parity ^ 1, stop, a);
                if (!ok) break;
#pragma unroll
                for (int k = 0; k < AT; ++k) {
                    const int r = (k0 + k) * (64 / LPQ) + ql / LPQ;
                    if (E4M3) {  // into f16's range: divide by the power of two at the largest
                        float v[8], top = 0.f;
                        load8(&x[k], true, v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
                        for (int o = LPQ / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        float p2 = __uint_as_float(__float_as_uint(top) & 0x7f800000u);
                        if (p2 == 0.f || p2 == INFINITY) p2 = 1.f;
                        const float inv = 1.f / p2;
                        x[k] = make_uint4(pair16<true>(v[0] * inv, v[1] * inv), pair16<true>(v[2] * inv, v[3] * inv),
                                          pair16<true>(v[4] * inv, v[5] * inv), pair16<true>(v[6] * inv, v[7] * inv));
                        if (ql % LPQ == 0) rs[seg_no % kFactors][r] = a.qscale * p2;
                    }
                    *reinterpret_cast<uint4*>(sq + qb.slot * C::QBYTES + (r >> 3) * (D / 8 * 128) + ql % LPQ * 128 +
                                              (r & 7) * 16) = x[k];
                }
            }
            if (!ok) break;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_plain(&qfull[qb.slot]);
            qb.next(C::QB);
        }
    } else if (E4M3) {
        // ------------------------------------- operands of 8-bit tiles: K in f16, V in bf16
        const bool w = warp >= C::W0 + 8;  // four warps for K, four for V
        const int ct = (tid - C::SOFT) & 127;
        // 16-byte pieces of the loaded rows: a thread's are tokens tk, tk + 32, ..., of D = 128 the
        // halves of each in turn. Eight lanes take pieces that neither meet at a bank when read
        // nor, as two chunks of a swizzled row, when written.
        const int hi = ct >> 2 & 1, tk = D == 128 ? (ct >> 3) * 2 + hi : ct >> 2;
        const int from = tk * D + (ct & 3) * 16 + (D == 128 ? hi * 64 : 0);
        const int into = tk * 128 + (((ct & 3) * 2 ^ (tk & 7)) << 4) + (D == 128 ? hi * kBlk : 0);
        const int flip = D == 128 ? (hi ? -kBlk : kBlk) : 0;  // to the other half's block
        const int sn = w ? C::SV : C::SK;
        uint64_t* const full = w ? vfull : kfull;
        uint64_t* const free = w ? vfree : kfree;
        unsigned char* const oper = w ? sv : sk;
        Ring rb, ob;
        uint32_t i = 0;
        bool ok = true;
        for (Seg g = first_seg(a, cum, c0, c1, single); g.t < c1 && ok; next_seg(a, cum, c1, g)) {
            for (uint32_t u = g.t; u < g.end; ++u, ++i) {
                ok = await(&rfull[rb.slot], rb.parity, stop, a) &&
                     await(&free[ob.slot], ob.parity ^ 1, stop, a);
                if (!ok) break;
                const uint32_t oks = info_ok[i % kInfo];
                const unsigned char* src = raw + rb.slot * C::RAW + (w ? kChunk * D : 0);
                unsigned char* dst = oper + ob.slot * C::OPER;
#pragma unroll
                for (int x0 = 0; x0 < D / 16; x0 += 4) {
                    uint4 v[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int k = D == 128 ? (x0 + x) / 2 : x;  // token tk + 32 k
                        v[x] = *reinterpret_cast<const uint4*>(src + k * 32 * D + (D == 128 && x % 2 ? from ^ 64 : from));
                    }
                    if (__builtin_expect(oks != (1u << kChunkTiles) - 1, 0))  // no page: zeros, whatever the stage holds
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int k = D == 128 ? (x0 + x) / 2 : x;
                            if (!(oks >> ((tk + 32 * k) / kTok) & 1)) v[x] = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int k = D == 128 ? (x0 + x) / 2 : x;
                        uint4 y, z;
                        e4m3x4_to_f16(v[x].x, y.x, y.y);
                        e4m3x4_to_f16(v[x].y, y.z, y.w);
                        e4m3x4_to_f16(v[x].z, z.x, z.y);
                        e4m3x4_to_f16(v[x].w, z.z, z.w);
                        if (w) {  // values: on to bf16, exact as well
                            uint32_t* const pairs[8] = {&y.x, &y.y, &y.z, &y.w, &z.x, &z.y, &z.z, &z.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 f = f16x2_to_f(*pairs[e]);
                                *pairs[e] = pair16<false>(f.x, f.y);
                            }
                        }
                        unsigned char* const at = dst + k * 32 * 128 + (x % 2 ? flip : 0);
                        *reinterpret_cast<uint4*>(at + into) = y;
                        *reinterpret_cast<uint4*>(at + (into ^ 16)) = z;
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_plain(&full[ob.slot]);
                    mbar_arrive_plain(&rfree[rb.slot]);
                }
                rb.next(C::RS);
                ob.next(sn);
            }
        }
    }
    __syncthreads();
    if (abort_flag) {
        // A wait ran out: no copy and no product may still be in flight when the CTA ends.
        if (warp == C::W0 + 1) {
            if (elect_one()) umma::commit_to(&drain);
            __syncwarp();
            mbar_wait_bounded(&drain, 0, RSSM_WAIT_NS / 100);
        } else if (tid < 4) {
            uint64_t* full[3] = {E4M3 ? &rfull[tid] : &kfull[tid], E4M3 ? &rfull[tid] : &vfull[tid], nullptr};
            for (int x = 0; x < 2; ++x) {
                mbar_wait_bounded(full[x], 0, RSSM_WAIT_NS / 100);
                mbar_wait_bounded(full[x], 1, RSSM_WAIT_NS / 100);
            }
        }
        __syncthreads();
    }
    if (warp == C::W0 + 1) umma::tmem_dealloc(tmem, C::COLS);
    if (abort_flag) return;
    join_ctas<D, C::THREADS>(a, runs, nruns, q_row, last_flag, sk);
}

template <int D, bool E4M3, int N>
static int launch_n(const rssm_attn_dims* d, const DecArgs& a, const DeviceInfo& di, cudaStream_t st) {
    using C = Wide<D, E4M3, N>;
    static_assert((kWideRows + 4 + 2 * kWideRows) * 4 <= kWideRowBytes, "rows");
    const int smem = C::SMEM + 1024;
    if (smem > di.max_smem_optin) return RSSM_ERR_UNSUPPORTED;
    CUtensorMap km, vm;
    memset(&km, 0, sizeof km);
    memset(&vm, 0, sizeof vm);
    if (!E4M3) {
        const uint64_t nr = (uint64_t)d->num_pages * d->num_kv_heads * d->page_size;
        if (!make_tmap_rows128(&km, a.k, 2, nr, D, kTok) || !make_tmap_rows128(&vm, a.v, 2, nr, D, kTok))
            return RSSM_ERR_CUDA;
    }
    if (!ensure_smem_limit((const void*)wide_kernel<D, E4M3, N>, smem)) return RSSM_ERR_CUDA;
    const int grid = di.sm_count < kMaxCtas ? di.sm_count : kMaxCtas;
    return launch_rows(d, a, kWideRows, [&](const DecArgs& x) {
        launch_early(wide_kernel<D, E4M3, N>, grid, C::THREADS, smem, st, x, km, vm);
    });
}

template <int D, bool E4M3>
static int launch_wide(const rssm_attn_dims* d, const DecArgs& a, const DeviceInfo& di, cudaStream_t st) {
    if constexpr (!E4M3)
        if (a.M <= 16) return launch_n<D, E4M3, 16>(d, a, di, st);
    return a.M <= 32 ? launch_n<D, E4M3, 32>(d, a, di, st) : launch_n<D, E4M3, 64>(d, a, di, st);
}

int decode_wide(const rssm_attn_dims* d, const DecArgs& a, const DeviceInfo& di, cudaStream_t st) {
    const bool q8 = d->cache_dtype == RSSM_E4M3;
    if (d->head_dim == 64) return q8 ? launch_wide<64, true>(d, a, di, st) : launch_wide<64, false>(d, a, di, st);
    return q8 ? launch_wide<128, true>(d, a, di, st) : launch_wide<128, false>(d, a, di, st);
}

}  // namespace attn
}  // namespace rssm
