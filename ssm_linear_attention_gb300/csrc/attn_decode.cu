// attn_decode.cu -- attention of a few new tokens per row over the paged cache: up to 8 queries a
// key head, up to 16 over an 8-bit cache, any number with float32 activations (attn_wide.cu has
// the others).
//
// For a row's T query tokens and the G = HQ / HKV query heads of one key / value head, the
// M = T G queries read the same cached tokens, so every cached vector is read once for all
// of them:
//     S^T = K Q^T (tokens x M),  P = exp2(S - m),  O^T += V^T P^T,
// with the softmax's base m (the largest score and 8) and sum l kept per query while the tokens
// stream by and O, l rescaled when a score passes m (float32 sums and bf16 operands lose nothing by
// the 8, and most tiles then need no maximum across lanes). Two
// partial results (m, l, O) over different tokens join as O = O_1 2^(m_1 - m) +
// O_2 2^(m_2 - m), l likewise, m = max(m_1, m_2); that makes the token axis free to split.
//
// Bound: the cached bytes, M flops per byte at most -- HBM. The contractions are far too
// small for a tcgen05 tile of 128 rows (M is 1 to 64, mostly 4 to 8). A warp-level mma.sync
// m16n8k16 takes 16 cached tokens (then 16 value columns) as its rows and 8 queries as its
// columns, and keeps S, P and O in one warp's registers; with the queries as rows (16 of
// them) half of every product and of the softmax was padding at M <= 8.
//
// Work: 16 cached tokens of one (row, key head) are a tile, all tiles of the call form one
// list (row, head, tokens in order), and the list is cut into equal contiguous ranges,
// one per group of warps (a group: 1, 2, 4 or 8 warps that take 8 queries each over the same
// tiles). Lengths are read on the device: no length reaches the host, ragged batches balance
// to a tile, a single long row fills the machine. A group streams its tiles into a ring of
// stages of its own, 16-byte chunks swizzled within 128 bytes (conflict-free ldmatrix), and
// never meets another group before its range ends. A (row, head) that lies inside one range
// is written out by its group. One that is cut leaves partial results; the groups of a CTA
// join theirs through shared memory, and the last CTA of a (row, head) to arrive at a counter
// joins the CTAs' results, in an order that the lengths and the machine alone fix.
//
// Measured (one GB300, GPU time of a call; "of" the measured copy bandwidth): 256 rows of 2k
// to 8k tokens, 8 key heads of 4 queries, D 128, 8-bit cache: 444 us, 6.4 TB/s, 94 % of it;
// 2 rows of 131k and 64k tokens, bf16 cache: 129 us, 6.2 TB/s, 91 %. 64 rows of 1000 to 4000 tokens, 4 key
// heads, D 128, in float32: 67 us with 8 queries (74 %), 137 with 32, 266 with 64, where the products of
// three parts and a pass over the tile for every 8 queries bind. 16 rows in float32 under a window of
// 1000 tokens: 11.8 us, 64 (row, head)s on as many of the SMs. One row of 300 tokens: 8.7 us, latency
// throughout (three dependent look-ups, one round trip of loads, two joins, and instructions fetched
// for the first time).
#include <cstring>

#include "attn_decode.cuh"

namespace rssm {
namespace attn {

// ---------------------------------------------------------------- mma pieces

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// cp.async with an L2 policy, a 4-byte one, and the wait for all but the last N commits.
__device__ __forceinline__ void cp_async16_hint(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// (or some fewer: 0, 1, 2, 4 and 6 are told apart)
__device__ __forceinline__ void cp_async_wait_but(int n) {
    if (n >= 4) {
        if (n >= 6) asm volatile("cp.async.wait_group 6;" ::: "memory");
        else asm volatile("cp.async.wait_group 4;" ::: "memory");
    } else if (n >= 2) {
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    } else if (n == 1) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
}
template <bool F16>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit values, a row's pair per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// Byte offset of 16-byte chunk c of token t in a [16 tokens][ROWB bytes] tile in shared
// memory: 128-byte row segments, chunk j of row r at j ^ (r % 8).
template <int ROWB>
__device__ __forceinline__ uint32_t tile_off(int t, int c) {
    if (ROWB >= 128) {
        return (uint32_t)((c >> 3) * (kTok * 128) + t * 128 + (((c & 7) ^ (t & 7)) << 4));
    } else {  // 64-byte vectors: two tokens to a 128-byte row
        const int r = t >> 1;
        return (uint32_t)(r * 128 + (((((t & 1) << 2) | c) ^ (r & 7)) << 4));
    }
}

// Warps of a CTA: 16 of 128 registers hide more than 8 (569 -> 481 us on 256 rows over an 8-bit
// cache when that was measured); float32 operands need more registers, and 16 rings of wide tiles
// do not fit.
constexpr int warps_of(int D, bool e4m3, bool af32, bool share) {
    return af32 || (!e4m3 && D == 128 && !share) ? 8 : 16;
}

// D: head dim, E4M3: 8-bit cache, AF32: float32 activations. The products' operands:
//   bf16 cache: bf16, the cached values as they are. A weight in one bf16 part would add
//     an error as large as the output's own rounding (1.41 times it together), so it takes
//     two; float32 activations take three parts of each, all 24 bits.
//   8-bit cache: keys and queries f16, which holds every e4m3 value; a query row is divided by
//     the power of two at its largest element and takes one part, two of float32. Values and
//     weights (times the value scales) are bf16, in as many parts as with a bf16 cache: f16
//     has no room below 2^-25 for the weights of a hundred thousand tokens that stand far behind
//     one, which may add up to all of an output. (f16 took 443 us of the 256-row case, too; with
//     float32 activations, 64 rows of 4000 tokens, 72 us against 80 with three parts.)
template <int D, bool E4M3, bool AF32, bool SHARE>
struct Cfg {
    static constexpr bool WIDE = !E4M3 && D == 128;
    // Tiles of a step: two give a warp independent work between the dependent pieces of one; a
    // ring of three wide tiles wants them one by one.
    static constexpr int TP = WIDE && !SHARE ? 1 : 2;
    static constexpr int WARPS = warps_of(D, E4M3, AF32, SHARE);
    // Wide tiles come by TMA (cp.async keeps fewer bytes in flight: 128 against 154 us on the
    // 2 x 128k case when both were built); for narrow ones the two were level (437 and 431 us on
    // the 256-row 8-bit case), and where warps share a tile each copies its part.
    static constexpr bool TMA = WIDE && !SHARE;
    static constexpr int ROWB = D * (E4M3 ? 1 : 2);  // bytes of a cached vector
    static constexpr int KB = kTok * ROWB;           // K (or V) bytes of a tile
    static constexpr int QP = AF32 ? (E4M3 ? 2 : 3) : 1;
    static constexpr int PP = AF32 ? 3 : 2;
    static constexpr int DB = D / 16;                // 16-column blocks of O^T
    static constexpr int TD = D + 4;                 // row pitch of tails: stores hit all banks
    static constexpr int AUX = E4M3 ? 2 * kTok * 4 : 0;  // scales of a tile
    static constexpr int STAGE = 2 * KB;
    // O^T column of block c that lane row n holds in its first (half 0) or second register
    // pair: 8-bit values come as even and odd columns, bf16 ones as the block's two halves.
    __device__ static __forceinline__ int col(int c, int n, int half) {
        return 16 * c + (E4M3 ? 2 * n + half : 8 * half + n);
    }
};

// Two float32 as a bf16 pair, one conversion.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Split v0, v1 into bf16 (f16) pairs: part i is the rounding of what the parts before it
// leave.
template <int N, bool F16>
__device__ __forceinline__ void split2(float v0, float v1, uint32_t* out) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (F16) {
            const __half2 h = __floats2half2_rn(v0, v1);
            out[i] = *reinterpret_cast<const uint32_t*>(&h);
            if (i + 1 < N) {
                v0 -= __low2float(h);
                v1 -= __high2float(h);
            }
        } else {
            const uint32_t p = pack2(v0, v1);
            out[i] = p;
            if (i + 1 < N) {
                v0 -= bf16_lo(p);
                v1 -= bf16_hi(p);
            }
        }
    }
}

template <int D, bool E4M3, bool AF32, bool SHARE>
__global__ void __launch_bounds__((Cfg<D, E4M3, AF32, SHARE>::WARPS * 32), 1)
    decode_kernel(const __grid_constant__ DecArgs a, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<D, E4M3, AF32, SHARE>;
    constexpr int kWarps = C::WARPS, kDecThreads = kWarps * 32;
    extern __shared__ unsigned char smem_raw[];
    // 128-byte swizzled boxes want their base on 1024 bytes
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int MT = SHARE ? a.MT : 1;
    const int ngroups = a.ngroups;
    const int group = warp / MT, mt = warp - group * MT;
    const int stages = a.stages;
    const int nst = stages * ngroups;

    // shared memory: the rows, stages (at the end the tails lie over them and what follows),
    // scales
    Rows rows;
    rows.cum = reinterpret_cast<uint32_t*>(smem);
    rows.len = reinterpret_cast<int*>(smem) + kMaxRows + 4;
    rows.slot = rows.len + kMaxRows;
    uint32_t* const cum = rows.cum;
    unsigned char* st_kv = smem + kRowBytes;
    float* st_scale = reinterpret_cast<float*>(st_kv + (size_t)nst * C::STAGE);
    uint64_t* full = reinterpret_cast<uint64_t*>(st_kv + (size_t)nst * (C::STAGE + C::AUX));
    __shared__ int abort_flag;
    __shared__ int q_row[64];  // query r of a key head among its row's T HQ: token * HQ + r % G
    __shared__ int q_tok[64];  // its token
    __shared__ uint2 scan[kWarps];  // tiles and longest row of the warps' rows
    __shared__ int rec_b[2 * kWarps], rec_h[2 * kWarps];  // records; b < 0: none
    __shared__ Run runs[2 * kWarps];
    __shared__ int nruns, last_flag[2];
    __shared__ float2 rec_ml[2 * kWarps * 8];  // [record][M] m and l

    if (C::TMA) {
        if (tid < nst) {
            mbar_init(&full[tid], 1);
            fence_barrier_init();
        }
        if (tid == 0) {
            abort_flag = 0;
            asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
        }
    }
    if (tid < 2 * kWarps) rec_b[tid] = -1;
    if (tid < a.M) {
        const int j = tid / a.G;
        q_tok[tid] = j;
        q_row[tid] = j * a.hq + tid - j * a.G;
    }

    // ------------------------------------------------------- the call's tile list
    const uint32_t longest = list_tiles<kDecThreads, kMaxRows, 1, 0>(a, rows, scan);
    write_empty_rows<D, kDecThreads>(a, rows);
    Cuts rg;
    uint32_t c0, c1;  // this CTA's range
    bool single;
    if (!cut_tiles(a, cum, longest, (uint32_t)kMinTiles * ngroups, kWholeTiles, rg, c0, c1, single)) return;
    const uint32_t gbase = (c1 - c0) / (uint32_t)ngroups, grem = (c1 - c0) - gbase * (uint32_t)ngroups;

    // ------------------------------------------------------- stream the range
    // Lane layout of the products: n = lane / 4 numbers S^T's tokens (n and n + 8) and O^T's
    // columns, qd = lane % 4 its queries 2 qd and 2 qd + 1 of each block of 8.
    float o[C::DB][4];
    float m[2], l[2];
    const int n8 = lane >> 2, qd = lane & 3;
    const int q0 = mt * 8;  // this warp's first query

    const uint32_t t0 = c0 + group * gbase + min((uint32_t)group, grem);
    const int ntile = group < ngroups ? (int)(gbase + (group < (int)grem ? 1 : 0)) : 0;
    if (ntile > 0) {
        const bool leader = mt == 0;
        unsigned char* kv = st_kv + (size_t)group * stages * C::STAGE;
        float* sc = st_scale + group * stages * (C::AUX / 4);
        const uint64_t pol = policy_evict_first();
        // ldmatrix: lane 8 i + r points at row r of matrix i. Of K, matrices are tokens 0-7 and
        // 8-15 of one chunk, then of the next; of V as well, chunk and tokens swapped for bf16.
        const uint32_t kbase = smem_addr(kv);
        const uint32_t ko = tile_off<C::ROWB>((lane >> 3 & 1) * 8 + (lane & 7), lane >> 4);
        const uint32_t vo = E4M3 ? ko : tile_off<C::ROWB>((lane >> 4) * 8 + (lane & 7), lane >> 3 & 1);

        // The next 32 tiles of the range are looked up at once, one per lane. Tile `sent` goes
        // into stage sent % stages, each warp of the group copying its share; a commit follows
        // whether or not there is a tile, so that the waits can count commits.
        int look = -1;
        int sent = 0, sent_s = 0;
        uint32_t bad = 0;  // stages whose tile has no page
        uint64_t* fb = full + group * stages;
        uint32_t parity = 0;  // of the stages' barriers, a bit each
        constexpr int LPR = C::ROWB / 16, TPI = 32 / LPR;  // cp.async: lanes of a token, tokens at once
        constexpr int INSTR = kTok / TPI;                  // instructions of a tile's k (or v)
        constexpr int ROWS = C::ROWB >= 128 ? TPI : TPI / 2;  // 128-byte rows of one
        const int share = !SHARE ? INSTR : INSTR / MT > 0 ? INSTR / MT : mt < INSTR ? 1 : 0;
        const int tok0 = (mt < INSTR ? mt * share : 0) * TPI + lane / LPR;
        const char* k_lane = a.k + (long)tok0 * C::ROWB + lane % LPR * 16;
        const long v_minus_k = a.v - a.k;
        const uint32_t st_base = smem_addr(kv) + tile_off<C::ROWB>(tok0, lane % LPR);
        auto issue = [&]() {
            if (sent < ntile) {
                if ((sent & 31) == 0 && sent + lane < ntile)
                    look = locate_tile(a, rows, t0 + sent + lane, single);
                const int y = __shfl_sync(0xffffffffu, look, sent & 31);
                bad = (bad & ~(1u << sent_s)) | (y < 0 ? 1u << sent_s : 0u);
                if (C::TMA) {  // (one warp a group)
                    if (y >= 0) {
                        unsigned char* dst = kv + (size_t)sent_s * C::STAGE;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&fb[sent_s], C::STAGE + ((int)t0 + sent == a.stall ? 16 : 0));
#pragma unroll
                            for (int x = 0; x < C::ROWB / 128; ++x) {
                                tma_load_2d(dst + x * kTok * 128, &kmap, 64 * x, y, &fb[sent_s], pol);
                                tma_load_2d(dst + C::KB + x * kTok * 128, &vmap, 64 * x, y, &fb[sent_s], pol);
                            }
                        }
                        __syncwarp();
                    }
                } else if (__all_sync(0xffffffffu, y >= 0)) {
                    // instruction j copies tokens TPI j .. of k and of v; the swizzle makes a step of j
                    // an exclusive or of the chunk bits
                    const uint32_t dst = st_base + sent_s * C::STAGE;
                    const char* src = k_lane + (long)y * C::ROWB;
#pragma unroll
                    for (int j = 0; j < (SHARE ? (INSTR + 1) / 2 : INSTR); ++j) {
                        if (SHARE && j >= share) break;
                        const uint32_t to = (dst ^ (uint32_t)(j * ROWS % 8 * 16)) + j * ROWS * 128;
                        cp_async16_hint(to, src + j * TPI * C::ROWB, pol);
                        cp_async16_hint(to + C::KB, src + v_minus_k + j * TPI * C::ROWB, pol);
                    }
                    if (E4M3 && leader)
                        cp_async4(smem_addr(sc + sent_s * 2 * kTok + lane),
                                  (lane < kTok ? a.k_scale : a.v_scale) + y + (lane & (kTok - 1)));
                }
                ++sent;
                if (++sent_s == stages) sent_s = 0;
            }
            if (!C::TMA) cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < stages; ++i) issue();

        uint32_t qf[D / 16][C::QP][2];  // [k step][part][k half]
        float rs[2];                    // score factor of the queries
        int end[2], beg[2];         // the positions they see
        int n_min = 0, n_max = 0, b_min = 0, b_max = 0;
        const bool works = q0 < a.M;
        int cb = 0, ch = 0;      // current (row, head)
        bool begun = false;      // its tiles began before this range
        int next = 0;            // tile of the range at which it ends
        int s = 0;               // stage of tile i
        int pos0 = 0;            // position of tile 0 of the range, were all of them this head's
        int used = 0;            // tiles of the step before

#pragma unroll 1
        for (int i = 0;;) {
            if (i == next || i == ntile) {
                if (i > 0) {
                    // The result of the current (row, head): out when all of its tiles lie in this
                    // range, else a record. The last one stays in registers until the stages are
                    // free.
                    const bool whole = i == next && !begun, tail = i == ntile;
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1)
                                l[x] += __shfl_xor_sync(0xffffffffu, l[x], w);
                    if (!whole && leader && lane == 0) {
                        rec_b[2 * group + (tail ? 1 : 0)] = cb;
                        rec_h[2 * group + (tail ? 1 : 0)] = ch;
                    }
                    if (whole) {
                        const long out0 = (long)cb * a.T * a.hq + ch * a.G;
                        const float i0 = l[0] == 0.f ? 0.f : reciprocal(l[0]);
                        const float i1 = l[1] == 0.f ? 0.f : reciprocal(l[1]);
                        if (a.obf) {
                            // transposed, a lane has two columns of query n8
                            const int r = q0 + n8;
                            const long row = r < a.M ? out0 + q_row[r] : 0;
                            uint16_t* dst = static_cast<uint16_t*>(a.o) + row * D;
#pragma unroll
                            for (int c = 0; c < C::DB; ++c) {
                                float v[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const bool none = l[x & 1] == 0.f;
                                    v[x] = none ? 0.f : o[c][x] * (x & 1 ? i1 : i0);
                                }
                                uint32_t lo = transpose8(pack2(v[0], v[1]));
                                uint32_t hi = transpose8(pack2(v[2], v[3]));
                                if (r >= a.M) continue;
                                if (E4M3) {  // even and odd columns 4 qd .. 4 qd + 3
                                    *reinterpret_cast<uint2*>(dst + 16 * c + 4 * qd) = make_uint2(
                                        __byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
                                } else {
                                    *reinterpret_cast<uint32_t*>(dst + 16 * c + 2 * qd) = lo;
                                    *reinterpret_cast<uint32_t*>(dst + 16 * c + 8 + 2 * qd) = hi;
                                }
                            }
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int r = q0 + 2 * qd + x;
                            if (r >= a.M) continue;
                            const long row = out0 + q_row[r];
                            const bool none = l[x] == 0.f;
                            if (!a.obf) {
                                float* dst = static_cast<float*>(a.o) + row * D;
#pragma unroll
                                for (int c = 0; c < C::DB; ++c) {
                                    dst[C::col(c, n8, 0)] = none ? 0.f : o[c][x] * (x ? i1 : i0);
                                    dst[C::col(c, n8, 1)] = none ? 0.f : o[c][2 + x] * (x ? i1 : i0);
                                }
                            }
                            if (a.lse && n8 == 0)
                                a.lse[row] = none ? -INFINITY : (m[x] + log2_fast(l[x])) * kLn2;
                        }
                    } else if (!tail) {
                        const long slot = 2L * gridDim.x + (int)blockIdx.x * ngroups + group;
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int r = q0 + 2 * qd + x;
                                if (r >= a.M) continue;
                                float* dst = a.part + (slot * a.M + r) * D;
#pragma unroll
                                for (int c = 0; c < C::DB; ++c) {
                                    dst[C::col(c, n8, 0)] = o[c][x];
                                    dst[C::col(c, n8, 1)] = o[c][2 + x];
                                }
                                if (n8 == 0) rec_ml[2 * group * a.M + r] = make_float2(m[x], l[x]);
                            }
                    }
                }
                if (i == ntile) break;

                // Start a (row, head): its queries as mma operands, the positions they see.
                const Tile x = find_tile(a, cum, t0 + i, single);
                cb = x.b;
                ch = x.h;
                begun = x.at > 0;
                next = i + (int)(cum[cb + 1] - cum[cb]) - x.at;
                const int len = rows.len[cb];
                pos0 = (row_span(a, len).first + x.at - i) * kTok;
                const int app = a.appended ? 1 : 0;
                n_min = len + app;
                n_max = len + (app ? a.T : 0);
                b_min = a.window && n_min > a.window ? n_min - a.window : 0;
                b_max = a.window && n_max > a.window ? n_max - a.window : 0;
#pragma unroll
                for (int c = 0; c < C::DB; ++c)
                    o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = q0 + 2 * qd + x;
                    const int e = len + (app ? (r < a.M ? q_tok[r] : 0) + 1 : 0);
                    end[x] = e;
                    beg[x] = a.window && e > a.window ? e - a.window : 0;
                    m[x] = -INFINITY;
                    l[x] = 0.f;
                    rs[x] = a.qscale;
                }
                const int r = q0 + n8;  // the query whose operand values this lane has
                const int j = r < a.M ? q_tok[r] : 0;
                const long base = ((long)cb * a.T + j) * a.q_stride + (ch * a.G + (r - j * a.G)) * D;
                float v[D / 16][4];
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    // columns of a k16 step: pairs at 2 qd and 2 qd + 8; for 8-bit keys, of
                    // which a lane gets 4 bytes, 4 qd and 4 qd + 2
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const int col = 16 * kk + (E4M3 ? 4 * qd + e : 2 * qd + 4 * e);
                        v[kk][e] = v[kk][e + 1] = 0.f;
                        if (r < a.M) {
                            if (AF32) {
                                const float2 f = *reinterpret_cast<const float2*>(
                                    static_cast<const float*>(a.q) + base + col);
                                v[kk][e] = f.x;
                                v[kk][e + 1] = f.y;
                            } else {
                                const uint32_t f = *reinterpret_cast<const uint32_t*>(
                                    static_cast<const uint16_t*>(a.q) + base + col);
                                v[kk][e] = bf16_lo(f);
                                v[kk][e + 1] = bf16_hi(f);
                            }
                        }
                    }
                }
                if (E4M3) {  // into f16's range: divide by the power of two at the largest
                    float top = 0.f;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                        for (int x = 0; x < 4; ++x) top = fmaxf(top, fabsf(v[kk][x]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    float p2 = __uint_as_float(__float_as_uint(top) & 0x7f800000u);
                    if (p2 == 0.f || p2 == INFINITY) p2 = 1.f;
                    const float inv = 1.f / p2;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                        for (int x = 0; x < 4; ++x) v[kk][x] *= inv;
                    rs[0] = a.qscale * __shfl_sync(0xffffffffu, p2, 8 * qd);
                    rs[1] = a.qscale * __shfl_sync(0xffffffffu, p2, 8 * qd + 4);
                }
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t lo[C::QP], hi[C::QP];
                    split2<C::QP, E4M3>(v[kk][0], v[kk][1], lo);
                    split2<C::QP, E4M3>(v[kk][2], v[kk][3], hi);
#pragma unroll
                    for (int p = 0; p < C::QP; ++p) {
                        qf[kk][p][0] = lo[p];
                        qf[kk][p][1] = hi[p];
                    }
                }
            }

            // the step's tiles: TP, or what the (row, head) or the range has left
            const int steps = min(C::TP, min(next, ntile) - i);
            int2 t[C::TP];  // position, -1 for a tile that is not there or has no page
            int st[C::TP];
            bool ok = true;
            if (C::TMA) {  // (one tile a step)
                if (!(bad >> s & 1)) {
                    if (!__all_sync(0xffffffffu, mbar_try_wait(&fb[s], parity >> s & 1)))
                        ok = wait_long(&fb[s], parity >> s & 1, &abort_flag, a.wait_ns, a.dev_err);
                    parity ^= 1u << s;
                }
            } else {
                cp_async_wait_but(stages - (SHARE ? 2 : 1) * C::TP);
            }
            if (!SHARE) {
                __syncwarp();
            } else {
                // the group's copies of this step are here; the stages of the step before are free
                asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(MT * 32) : "memory");
#pragma unroll 1
                for (; used > 0; --used) issue();
            }
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < C::TP; ++u) {
                st[u] = s;
                t[u] = make_int2(pos0 + (i + u) * kTok, -1);
                if (u < steps) {
                    t[u].y = bad >> s & 1 ? -1 : 0;
                    if (++s == stages) s = 0;
                }
            }
            bool some = t[0].y >= 0;
            if (C::TP > 1) some = some || t[C::TP - 1].y >= 0;
            if (some && works) {
                // ------------------------------------------------ S^T = K Q^T
                // One tile: two chains of sums. Float32 queries: one of the first parts and one of the
                // rest, which an infinite key (or query) turns into NaN where the first has the sign.
                constexpr int SA = C::TP == 1 || AF32 ? 2 : 1;
                float sa[C::TP][SA][4];
#pragma unroll
                for (int u = 0; u < C::TP; ++u)
#pragma unroll
                        for (int x = 0; x < 4; ++x) sa[u][0][x] = sa[u][SA - 1][x] = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; kk += E4M3 ? 2 : 1)
#pragma unroll
                    for (int u = 0; u < C::TP; ++u) {
                        // chunk 2 kk (8-bit: kk) of the lane's token and half: the swizzle makes a
                        // step of it an exclusive or
                        const uint32_t at = (kbase + st[u] * C::STAGE + ko) ^ (uint32_t)((E4M3 ? kk : 2 * kk) % 8 * 16);
                        uint32_t r[4];
                        if (E4M3) {
                            uint32_t f[2][4];
                            ldsm4(at, r);
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                e4m3x4_to_f16(r[x], f[x >> 1][x & 1], f[x >> 1][2 + (x & 1)]);
#pragma unroll
                            for (int p = 0; p < C::QP; ++p) {
                                    mma16816<true>(sa[u][AF32 && p > 0 ? 1 : 0], f[0], qf[kk][p][0], qf[kk][p][1]);
                                    mma16816<true>(sa[u][AF32 ? p > 0 : SA - 1], f[1], qf[kk + 1][p][0], qf[kk + 1][p][1]);
                            }
                        } else {
                            ldsm4(at + kk / 4 * (kTok * 128), r);
#pragma unroll
                            for (int p = 0; p < C::QP; ++p)
                                    mma16816<false>(sa[u][AF32 ? p > 0 : SA == 2 ? kk & 1 : 0], r, qf[kk][p][0], qf[kk][p][1]);
                        }
                    }
                // ------------------------------------------------ softmax
                // Scores in log2 units. With an 8-bit cache a token's value scale multiplies its
                // weight where that meets the value: m and l are the scores' alone.
                float p[C::TP][4], vs[C::TP][2];
                bool edge[C::TP], edges = false, grow = false;
#pragma unroll
                for (int u = 0; u < C::TP; ++u) {
                    float ks[2] = {1.f, 1.f};
                    if (E4M3) {
                        const float* ts = sc + st[u] * 2 * kTok + n8;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            ks[x] = ts[8 * x];
                            vs[u][x] = ts[kTok + 8 * x];
                        }
                    }
                    // a tile that is not there (or has no page) is all hidden
                    edge[u] = t[u].y < 0 || t[u].x + kTok > n_min || t[u].x < b_max;
                    edges = edges || edge[u];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            float f = sa[u][0][x];
                            if (SA == 2 && !(AF32 && isinf(f))) f += sa[u][SA - 1][x];
                            f *= rs[x & 1];
                            if (E4M3) f *= ks[x >> 1];
                            p[u][x] = f;
                        }
                }
                if (__builtin_expect(edges, 0)) {  // hide what a query does not see, whatever it holds
#pragma unroll
                    for (int u = 0; u < C::TP; ++u)
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const int tok = t[u].x + n8 + 8 * (x >> 1);
                                if (tok >= end[x & 1] || tok < beg[x & 1] || t[u].y < 0)
                                    p[u][x] = -INFINITY;
                            }
                }
#pragma unroll
                for (int u = 0; u < C::TP; ++u)
#pragma unroll
                        for (int x = 0; x < 4; ++x) grow |= p[u][x] > m[x & 1];
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float top = fmaxf(p[0][x], p[0][2 + x]);
                            if (C::TP > 1) top = fmaxf(top, fmaxf(p[C::TP - 1][x], p[C::TP - 1][2 + x]));
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1)
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                            // (a query whose base holds keeps it)
                            top = top > m[x] ? top + kSlack : m[x];
                            const float f = top == m[x] ? 1.f : exp2_fast(m[x] - top);
                            m[x] = top;
                            l[x] *= f;
#pragma unroll
                            for (int c = 0; c < C::DB; ++c) {
                                o[c][x] *= f;
                                o[c][2 + x] *= f;
                            }
                        }
                }
                uint32_t pf[C::TP][C::PP][2];
#pragma unroll
                for (int u = 0; u < C::TP; ++u) {
                        // a query that has seen only -infinity keeps weights of zero
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float c = m[x & 1] == -INFINITY ? 0.f : m[x & 1];
                            p[u][x] = exp2_fast(p[u][x] - c);
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x) l[x & 1] += p[u][x];
                        if (E4M3 && __builtin_expect(edges, 0)) {  // a hidden token's scale may be anything
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const int tok = t[u].x + n8 + 8 * (x >> 1);
                                const bool hidden = tok >= end[x & 1] || tok < beg[x & 1] || t[u].y < 0;
                                p[u][x] = hidden ? 0.f : p[u][x] * vs[u][x >> 1];
                            }
                        } else if (E4M3) {
#pragma unroll
                            for (int x = 0; x < 4; ++x) p[u][x] *= vs[u][x >> 1];
                        }
                        uint32_t lo[C::PP], hi[C::PP];
                        split2<C::PP, false>(p[u][0], p[u][1], lo);
                        split2<C::PP, false>(p[u][2], p[u][3], hi);
#pragma unroll
                        for (int x = 0; x < C::PP; ++x) {
                            pf[u][x][0] = transpose8(lo[x]);
                            pf[u][x][1] = transpose8(hi[x]);
                        }
                }
                // ------------------------------------------------ O^T += V^T P^T
                bool careful[C::TP];
#pragma unroll
                for (int u = 0; u < C::TP; ++u) {
                    careful[u] = false;
                    if (__builtin_expect(!edge[u], 1)) continue;
                    // A weight of zero does not silence an infinity or a NaN in a value. Tokens
                    // that no query sees are cleared (a tile that is not there as a whole); if
                    // one that only some see is not finite, the tile's products run value by
                    // value below (8-bit values are finite: what is not is marked in the scale,
                    // which a hidden score leaves out).
                    const int pos = t[u].x;
                    unsigned char* vt = kv + (size_t)st[u] * C::STAGE + C::KB;
                    if (t[u].y < 0) {
                        careful[u] = true;  // nothing to add
                        continue;
                    }
                    if (pos + kTok > n_max || pos < b_min) {
#pragma unroll 1
                        for (int e = lane; e < kTok * (C::ROWB / 16); e += 32) {
                            const int tok = e / (C::ROWB / 16), c = e % (C::ROWB / 16);
                            if (pos + tok >= n_max || pos + tok < b_min)
                                *reinterpret_cast<uint4*>(vt + tile_off<C::ROWB>(tok, c)) = make_uint4(0, 0, 0, 0);
                        }
                        if (C::TMA) fence_async_smem();  // the stage's next load comes after these stores
                        __syncwarp();
                    }
                    if (!E4M3 && a.T > 1) {
                        bool odd = false;
#pragma unroll 1
                        for (int e = lane; e < kTok * (C::ROWB / 16); e += 32) {
                            const int tok = e / (C::ROWB / 16), c = e % (C::ROWB / 16), at = pos + tok;
                            if ((at >= n_min && at < n_max) || (at >= b_min && at < b_max)) {
                                const uint4 v = *reinterpret_cast<const uint4*>(vt + tile_off<C::ROWB>(tok, c));
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    odd |= (w[x] & 0x7f80u) == 0x7f80u || (w[x] & 0x7f800000u) == 0x7f800000u;
                            }
                        }
                        careful[u] = __any_sync(0xffffffffu, odd);
                    }
                }
#pragma unroll
                for (int u = 0; u < C::TP; ++u) {
                    const unsigned char* vt = kv + (size_t)st[u] * C::STAGE + C::KB;
                    const uint32_t vbase = kbase + st[u] * C::STAGE + C::KB + vo;
                    if (!careful[u]) {
#pragma unroll
                        for (int c = 0; c < C::DB; ++c) {
                            uint32_t f[4];
                            if (E4M3) {
                                // a register holds two tokens' codes of columns 2 n, 2 n + 1; paired
                                // by token they are one k pair of the even and of the odd columns
                                if (c & 1) continue;
                                uint32_t r[4], g[4];
                                ldsm4_t(vbase ^ (uint32_t)(c % 8 * 16), r);
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    uint32_t lo, hi;
                                    e4m3x4_to_f16(r[x], lo, hi);
                                    const float2 t0 = f16x2_to_f(lo), t1 = f16x2_to_f(hi);
                                    uint32_t* d = x < 2 ? f : g;
                                    d[2 * (x & 1)] = pack2(t0.x, t1.x);
                                    d[2 * (x & 1) + 1] = pack2(t0.y, t1.y);
                                }
#pragma unroll
                                for (int x = 0; x < C::PP; ++x) {
                                        mma16816<false>(o[c], f, pf[u][x][0], pf[u][x][1]);
                                        mma16816<false>(o[c + 1], g, pf[u][x][0], pf[u][x][1]);
                                }
                            } else {
                                ldsm4_t((vbase ^ (uint32_t)(2 * c % 8 * 16)) + c / 4 * (kTok * 128), f);
#pragma unroll
                                for (int x = 0; x < C::PP; ++x)
                                        mma16816<false>(o[c], f, pf[u][x][0], pf[u][x][1]);
                            }
                        }
                    } else if (!E4M3 && t[u].y >= 0) {
                        const int pos = t[u].x;
#pragma unroll 1
                        for (int tok = 0; tok < kTok; ++tok) {
                            const int src = (tok & 7) * 4 + qd;
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const float w = __shfl_sync(0xffffffffu, tok < 8 ? p[u][x] : p[u][2 + x], src);
                                    if (pos + tok >= end[x] || pos + tok < beg[x]) continue;
#pragma unroll
                                    for (int c = 0; c < C::DB; ++c) {
                                        const uint16_t* v = reinterpret_cast<const uint16_t*>(
                                            vt + tile_off<C::ROWB>(tok, 2 * c) + 2 * n8);
                                        const uint16_t* w2 = reinterpret_cast<const uint16_t*>(
                                            vt + tile_off<C::ROWB>(tok, 2 * c + 1) + 2 * n8);
                                        o[c][x] += w * bf16_to_f(*v);
                                        o[c][2 + x] += w * bf16_to_f(*w2);
                                    }
                                }
                        }
                    }
                }
            }
            // ---------------------------------------------------- hand the stages back
            __syncwarp();
            i += steps;
            used = steps;
            if (!SHARE)
#pragma unroll 1
                for (; used > 0; --used) issue();
        }
        cp_async_wait_but(0);
    }
    __syncthreads();
    if (C::TMA && abort_flag) {
        // A wait ran out: no copy may still be in flight when the CTA ends. Every stage's
        // barrier is watched for a while, whatever its phase. The group that gave up left no
        // record of its tiles: nothing is joined, what the CTA had not written stays unwritten.
        if (tid < nst) {
            mbar_wait_bounded(&full[tid], 0, RSSM_WAIT_NS / 100);
            mbar_wait_bounded(&full[tid], 1, RSSM_WAIT_NS / 100);
        }
        return;
    }

    // ------------------------------------------------------- join the CTA's records
    // Tails into shared memory (the stages are free now).
    float* tail = reinterpret_cast<float*>(st_kv);  // [group][M][TD]
    if (ntile > 0 && rec_b[2 * group + 1] >= 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = q0 + 2 * qd + x;
                if (r >= a.M) continue;
                float* dst = tail + (group * a.M + r) * C::TD;
#pragma unroll
                for (int c = 0; c < C::DB; ++c) {
                    dst[C::col(c, n8, 0)] = o[c][x];
                    dst[C::col(c, n8, 1)] = o[c][2 + x];
                }
                if (n8 == 0) rec_ml[(2 * group + 1) * a.M + r] = make_float2(m[x], l[x]);
            }
    }
    // Runs of records: a record whose (row, head) differs from that of the record before it
    // starts one.
    if (warp == 0) {
        const int i = lane;
        const bool is = i < 2 * ngroups && rec_b[i] >= 0;
        const unsigned have = __ballot_sync(0xffffffffu, is);
        const unsigned before = have & ((1u << i) - 1u);
        const int prev = before ? 31 - __clz(before) : -1;
        const bool starts = is && (prev < 0 || rec_b[prev] != rec_b[i] || rec_h[prev] != rec_h[i]);
        const unsigned start = __ballot_sync(0xffffffffu, starts);
        if (starts) {
            Run r;
            r.b = rec_b[i];
            r.h = rec_h[i];
            r.rec0 = i;
            const unsigned later = start & ~((2u << i) - 1u);  // the runs after this one
            const unsigned mine = have & ~((1u << i) - 1u) & ((later & (0u - later)) - 1u);
            r.rec1 = 32 - __clz(mine);
            const uint32_t nt = cum[r.b + 1] - cum[r.b];
            const uint32_t s0 = cum[r.b] * (uint32_t)a.hkv + (uint32_t)r.h * nt;
            r.cta0 = r.cta1 = blockIdx.x;
            if (s0 < c0) r.cta0 = cta_of(rg, s0);
            if (s0 + nt > c1) r.cta1 = cta_of(rg, s0 + nt - 1);
            runs[__popc(start & ((1u << i) - 1u))] = r;
        }
        if (lane == 0) {
            nruns = __popc(start);
            last_flag[0] = last_flag[1] = 0;
        }
    }
    __syncthreads();

    // Join each run, 4 columns to a thread. A run is tails (in shared memory) and at most one
    // head, its last record, in global memory.
    const int nv = a.M * (D / 4);
#pragma unroll 1
    for (int i = 0; i < nruns; ++i) {
        const Run r = runs[i];
        const int last = r.rec1 - 1;
        const float* head = a.part + (2L * gridDim.x + (int)blockIdx.x * ngroups + (last >> 1)) * a.M * D;
        const long slot = 2L * blockIdx.x + (r.cta0 < (int)blockIdx.x ? 0 : 1);
#pragma unroll 1
        for (int v0 = tid; v0 < nv; v0 += kItems * kDecThreads) {
            float4 x[kItems];  // the heads, whose loads start together
#pragma unroll
            for (int u = 0; u < kItems; ++u) {
                const int v = v0 + u * kDecThreads;
                if (v < nv && !(last & 1)) x[u] = *reinterpret_cast<const float4*>(head + v * 4);
            }
#pragma unroll
            for (int u = 0; u < kItems; ++u) {
                const int v = v0 + u * kDecThreads;
                if (v >= nv) break;
                const int row = v / (D / 4), d = (v % (D / 4)) * 4;
                Partial acc;
#pragma unroll 1
                for (int k = r.rec0 | 1; k < r.rec1; k += 2)
                    if (rec_b[k] >= 0)
                        acc.add(rec_ml[k * a.M + row],
                                *reinterpret_cast<const float4*>(tail + ((k >> 1) * a.M + row) * C::TD + d));
                if (!(last & 1)) acc.add(rec_ml[last * a.M + row], x[u]);
                if (r.cta0 == r.cta1) {
                    store_partial(a, acc, (long)r.b * a.T * a.hq + r.h * a.G + q_row[row], D, d);
                } else {
                    *reinterpret_cast<float4*>(a.part + slot * a.M * D + v * 4) = acc.v;
                    if (d == 0) reinterpret_cast<float2*>(a.part_ml)[slot * a.M + row] = acc.ml;
                }
            }
        }
    }

    join_ctas<D, kDecThreads>(a, runs, nruns, q_row, last_flag, st_kv);
}

// ---------------------------------------------------------------- host side

// The kernel that a call's dims take, and its groups' layout.
struct Form {
    int M, MT;    // queries per key head, warps per group (each 8 queries)
    bool wide;    // attn_wide.cu's
    int groups;   // of a CTA at most, else
};
static Form form_of(const rssm_attn_dims* d) {
    const bool e4m3 = d->cache_dtype == RSSM_E4M3, af32 = d->act_dtype == RSSM_F32;
    Form f;
    f.M = d->q_tokens * (d->num_q_heads / d->num_kv_heads);
    f.MT = f.M <= 8 ? 1 : f.M <= 16 ? 2 : f.M <= 32 ? 4 : 8;
    // The tensor-memory kernel takes more than 8 queries, but for float32 activations, whose operands
    // would be three parts each, and an 8-bit cache under up to 16 queries, whose conversions cost it
    // more than it saves (64 rows of 1000 to 4000 tokens, 4 key heads of 16 queries: D 64 65 us
    // against 45 here, D 128 70 and 63; of 32 queries 64 against 70, 73 against 104).
    f.wide = f.MT > 1 && !af32 && !(e4m3 && f.M <= 16);
    f.groups = warps_of(d->head_dim, e4m3, af32, f.MT > 1) / f.MT;
    return f;
}
static bool too_many_queries(const rssm_attn_dims* d) {
    return (int64_t)d->q_tokens * (d->num_q_heads / d->num_kv_heads) > 64;
}

// Workspace: counters (one per CTA), then (m, l) of the CTAs' partial results (two each), then the
// values of these and, of the kernel of few queries, of the groups' heads.
struct Workspace {
    size_t ml, part, bytes;
};
static Workspace workspace_of(const rssm_attn_dims* d, const Form& f) {
    DeviceInfo di;
    const size_t ctas = device_info(&di) && di.sm_count < kMaxCtas ? di.sm_count : kMaxCtas;
    Workspace w;
    w.ml = kMaxCtas * sizeof(int32_t);
    w.part = (w.ml + ctas * 2 * f.M * 2 * sizeof(float) + 255) / 256 * 256;
    w.bytes = w.part + ctas * (2 + (f.wide ? 0 : f.groups)) * f.M * d->head_dim * sizeof(float);
    return w;
}

template <int D, bool E4M3, bool AF32, bool SHARE>
static int launch_kernel(const rssm_attn_dims* d, DecArgs a, const DeviceInfo& di, cudaStream_t st) {
    using C = Cfg<D, E4M3, AF32, SHARE>;
    const int fixed = kRowBytes + 1024;
    const int per = C::STAGE + C::AUX + 8;
    // what the kernel's static arrays take: (m, l) of the records, and the lists
    const int statics = C::WARPS * (128 + 2 * (int)sizeof(Run) + 24) + 768;
    const int budget = di.max_smem_optin - statics - fixed;
    // a ring holds a step's tiles at least, and those of the step before where warps share them
    const int least = (SHARE ? 2 : 1) * C::TP;
    a.ngroups = C::WARPS / a.MT;
    if (budget / (per * a.ngroups) < least) a.ngroups = budget / (per * least);
    if (a.ngroups < 1) return RSSM_ERR_UNSUPPORTED;
    a.stages = budget / (per * a.ngroups);
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    int smem = fixed + a.stages * a.ngroups * per;
    const int tails = fixed + C::WARPS * 8 * C::TD * 4;
    if (smem < tails) smem = tails;
    CUtensorMap km, vm;
    memset(&km, 0, sizeof km);
    memset(&vm, 0, sizeof vm);
    if (C::TMA) {
        const uint64_t nr = (uint64_t)d->num_pages * d->num_kv_heads * d->page_size;
        if (!make_tmap_rows128(&km, a.k, 2, nr, D, kTok) || !make_tmap_rows128(&vm, a.v, 2, nr, D, kTok))
            return RSSM_ERR_CUDA;
    }
    const void* kern = (const void*)decode_kernel<D, E4M3, AF32, SHARE>;
    if (!ensure_smem_limit(kern, smem)) return RSSM_ERR_CUDA;
    const int grid = di.sm_count < kMaxCtas ? di.sm_count : kMaxCtas;
    return launch_rows(d, a, kMaxRows, [&](const DecArgs& x) {
        launch_early(decode_kernel<D, E4M3, AF32, SHARE>, grid, C::WARPS * 32, smem, st, x, km, vm);
    });
}

template <int D, bool E4M3, bool AF32>
static int launch(const rssm_attn_dims* d, const DecArgs& a, bool wide, const DeviceInfo& di, cudaStream_t st) {
    if (a.MT == 1) return launch_kernel<D, E4M3, AF32, false>(d, a, di, st);
    if constexpr (AF32 || E4M3)
        if (!wide) return launch_kernel<D, E4M3, AF32, true>(d, a, di, st);
    if constexpr (!AF32) return decode_wide(d, a, di, st);
}

}  // namespace attn
}  // namespace rssm

using namespace rssm;

extern "C" size_t rssm_attn_workspace_size(const rssm_attn_dims* d) {
    if (attn::check_dims(d) != RSSM_OK || attn::too_many_queries(d)) return 0;
    return attn::workspace_of(d, attn::form_of(d)).bytes;
}

static int decode_call(const rssm_attn_dims* d, const rssm_attn_cache* c, int appended, float scale,
                       int32_t window, const void* q, int64_t q_stride, const int32_t* cache_indices,
                       void* workspace, size_t workspace_bytes, void* o, float* lse, int stall,
                       uint64_t wait_ns, int32_t* dev_err, rssm_stream_t stream) {
    const int st = attn::check_dims(d);
    if (st != RSSM_OK) return st;
    if (window < 0) return RSSM_ERR_INVALID_ARG;
    if (attn::too_many_queries(d)) return RSSM_ERR_UNSUPPORTED;
    if (d->batch == 0) return RSSM_OK;
    const attn::Form form = attn::form_of(d);
    const attn::Workspace ws = attn::workspace_of(d, form);
    if (!attn::ok_cache(d, c) || !ok_ptr(q) || !attn::ok_stride(d, q_stride, d->num_q_heads) ||
        !ok_ptr(cache_indices) || !ok_ptr(workspace) || workspace_bytes < ws.bytes || !ok_ptr(o) ||
        !ok_opt_ptr(lse))
        return RSSM_ERR_INVALID_ARG;
    DeviceInfo di;
    if (!device_info(&di)) return RSSM_ERR_CUDA;
    attn::DecArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.k = static_cast<const char*>(c->k);
    a.v = static_cast<const char*>(c->v);
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    a.page_table = c->page_table;
    a.slot_len = c->slot_len;
    a.ci = cache_indices;
    a.o = o;
    a.lse = lse;
    a.dev_err = dev_err;
    a.counters = static_cast<int32_t*>(workspace);
    a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.ml);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.part);
    a.qscale = scale * attn::kLog2e;
    a.T = d->q_tokens;
    a.G = d->num_q_heads / d->num_kv_heads;
    a.hq = d->num_q_heads;
    a.hkv = d->num_kv_heads;
    a.ps_log2 = attn::log2_of(d->page_size);
    a.num_pages = d->num_pages;
    a.max_pages = d->max_pages;
    a.num_slots = d->num_slots;
    a.window = window < (1 << 30) ? window : 1 << 30;  // (no row is longer: sums with it stay in 32 bits)
    a.appended = appended != 0;
    a.M = form.M;
    a.MT = form.MT;
    a.obf = d->out_dtype == RSSM_BF16;
    a.wait_ns = wait_ns;
    a.stall = stall;
    const bool q8 = d->cache_dtype == RSSM_E4M3, f32 = d->act_dtype == RSSM_F32;
    const cudaStream_t s = (cudaStream_t)stream;
#define RSSM_ATTN_D(D_)                                                            \
    (q8 ? (f32 ? attn::launch<D_, true, true>(d, a, form.wide, di, s)                      \
               : attn::launch<D_, true, false>(d, a, form.wide, di, s))                    \
        : (f32 ? attn::launch<D_, false, true>(d, a, form.wide, di, s)                     \
               : attn::launch<D_, false, false>(d, a, form.wide, di, s)))
    return d->head_dim == 64 ? RSSM_ATTN_D(64) : RSSM_ATTN_D(128);
#undef RSSM_ATTN_D
}

extern "C" int rssm_attn_decode(const rssm_attn_dims* d, const rssm_attn_cache* c, int appended,
                                float scale, int32_t window, const void* q, int64_t q_stride,
                                const int32_t* cache_indices, void* workspace,
                                size_t workspace_bytes, void* o, float* lse, int32_t* dev_err,
                                rssm_stream_t stream) {
    return decode_call(d, c, appended, scale, window, q, q_stride, cache_indices, workspace,
                       workspace_bytes, o, lse, -1, RSSM_WAIT_NS, dev_err, stream);
}

extern "C" int rssm_debug_attn_decode(const rssm_attn_dims* d, const rssm_attn_cache* c,
                                      int appended, float scale, int32_t window, const void* q,
                                      int64_t q_stride, const int32_t* cache_indices,
                                      void* workspace, size_t workspace_bytes, void* o, float* lse,
                                      int stall_tile, int wait_us, int32_t* dev_err,
                                      rssm_stream_t stream) {
    if (wait_us < 1 || wait_us > 2000000) return RSSM_ERR_INVALID_ARG;
    return decode_call(d, c, appended, scale, window, q, q_stride, cache_indices, workspace,
                       workspace_bytes, o, lse, stall_tile < 0 ? -1 : stall_tile,
                       (uint64_t)wait_us * 1000ull, dev_err, stream);
}
