// attn_decode.cu -- attention of a few new tokens per row over the paged cache.
//
// For a row's T query tokens and the G = HQ / HKV query heads of one key / value head, the
// T G queries read the same cached tokens, so they form one operand of M = T G rows and
// every cached vector is read once:
//     S = Q K^T (M x tokens),  P = exp2(S - running row maximum),  O += P V,
// with the softmax's maximum m and sum l kept per row while the tokens stream by and O, l
// rescaled when m grows. Two such partial results (m, l, O) over different tokens join as
// O = O_1 2^(m_1 - m) + O_2 2^(m_2 - m), l likewise, m = max(m_1, m_2); that makes the
// token axis free to split.
//
// Bound: the cached bytes, M flops per byte and two bytes per value at most -- HBM. The
// contractions are far too small for a tcgen05 tile of 128 rows (M is 1 to 64, mostly 4
// to 8), and a warp-level mma.sync m16n8k16 whose rows are the queries keeps S, P and O in
// the registers of one warp, with no tensor-memory round trips between the two products.
//
// Work: 16 cached tokens of one (row, key head) are a tile, all tiles of the call form one
// list (row, head, tokens in order), and the list is cut into equal contiguous ranges,
// one per group of warps (a group: ceil(M / 16) warps that take 16 queries each over the
// same tiles). Lengths are read on the device: no length reaches the host, ragged batches
// balance to a tile, a single long row fills the machine. A group streams its tiles with
// TMA boxes of 128-byte swizzled row segments into a ring of stages of its own (conflict-
// free ldmatrix), and never meets another group before its range ends. A (row, head) that
// lies inside one range is written out by its group. One that is cut leaves partial
// results; the groups of a CTA join theirs through shared memory, and the last CTA of a
// (row, head) to arrive at a counter joins the CTAs' results, in an order that the
// lengths alone fix.
#include "attn.cuh"

namespace rssm {
namespace attn {

constexpr int kTok = 16;       // tokens per tile: the smallest page
constexpr int kWarps = 8;
constexpr int kDecThreads = kWarps * 32;
constexpr int kMaxRows = 1024;  // rows per launch (prefix sums in shared memory)
constexpr int kMaxStages = 8;   // per group
// A range shorter than this is not cut further: the partial results of a cut cost about as
// much as these tiles.
constexpr int kMinTiles = 4;
constexpr float kLog2e = 1.4426950408889634f;

struct DecArgs {
    const void* q;
    long q_stride;
    const float* k_scale;
    const float* v_scale;
    const int32_t* page_table;
    const int32_t* slot_len;
    const int32_t* ci;
    void* o;
    float* lse;
    int32_t* dev_err;
    float* part;       // [2 x CTAs][M][D] partial results of CTAs, then of groups
    float* part_ml;    // [2 x CTAs + groups][M][2]
    int32_t* counters; // [CTAs]
    float qscale;      // scale * log2 e
    int batch, T, G, hq, hkv, ps_log2, num_pages, max_pages, num_slots, window, appended;
    int M, MT;         // queries per key head, warps per group
    int stages;        // per group
    int obf;
};

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
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four e4m3 codes w as bf16 pairs: lo = codes 0 and 2, hi = codes 1 and 3, each its value
// times 2^-120. An e4m3 code has its exponent and significand in the bits below its sign;
// moved under a bf16 sign, four bits further down, they read as the same number with the
// bf16 bias (127 against 7), subnormal codes included. Exact, and three instructions a
// pair. The factor is undone in the score scale and the output (kUnscale).
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    hi = (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u);
    lo = ((w << 8) & 0x80008000u) | ((w << 4) & 0x07f007f0u);
}
// Queries and weights are raised by 2^64 against the codes' 2^-120, so that neither the
// products nor their sums come near float32's subnormal range; 2^56 remains.
constexpr float kRaise = 18446744073709551616.f;  // 2^64
constexpr float kUnscale = 72057594037927936.f;   // 2^56

// Byte offset of 16-byte chunk c of token t in a [16 tokens][ROWB bytes] tile as the TMA
// boxes leave it: 128-byte row segments, chunk j of row r at j ^ (r % 8).
template <int ROWB>
__device__ __forceinline__ uint32_t tile_off(int t, int c) {
    if (ROWB >= 128) {
        return (uint32_t)((c >> 3) * (kTok * 128) + t * 128 + (((c & 7) ^ (t & 7)) << 4));
    } else {  // 64-byte vectors: two tokens to a 128-byte row
        const int r = t >> 1;
        return (uint32_t)(r * 128 + (((((t & 1) << 2) | c) ^ (r & 7)) << 4));
    }
}

// Tiles of a row: tokens from the first one any query sees to the last, in whole tiles.
struct RowSpan {
    int first;  // first tile
    int tiles;
};
__device__ __forceinline__ RowSpan row_span(const DecArgs& a, int len) {
    const int end = len + (a.appended ? a.T : 0);
    const int e0 = len + (a.appended ? 1 : 0);
    const int begin = a.window && e0 > a.window ? e0 - a.window : 0;
    RowSpan s;
    s.first = begin / kTok;
    s.tiles = end > begin ? (end + kTok - 1) / kTok - s.first : 0;
    return s;
}

// Length of row b's slot, or -1 for a row that is skipped. `flag`: this thread reports.
__device__ __forceinline__ int row_len(const DecArgs& a, int b, bool flag) {
    const int s = a.ci[b];
    if (s < 0) return -1;
    if (s >= a.num_slots) {
        if (flag) set_dev_err(a.dev_err, RSSM_DEVERR_SLOT);
        return -1;
    }
    const int len = a.slot_len[s];
    const long cap = (long)a.max_pages << a.ps_log2;
    if (len < 0 || (long)len + (a.appended ? a.T : 0) > cap) {
        if (flag) set_dev_err(a.dev_err, RSSM_DEVERR_CURSOR);
        return -1;
    }
    return len;
}

// Where one tile lies: row, head, first position, row of its first token in the cache
// matrix (-1: its page is out of range).
struct Tile {
    int b, h, pos, y;
};

struct Ranges {
    long total;
    int per_cta;  // groups of a CTA that have a range
    int workers;
};
// First tile of worker w's range: the remainder of total / workers goes to the first ones.
__device__ __forceinline__ long range_start(const Ranges& r, long w) {
    const long base = r.total / r.workers, rem = r.total - base * r.workers;
    return w * base + (w < rem ? w : rem);
}
// The worker whose range holds tile t.
__device__ __forceinline__ int worker_of(const Ranges& r, long t) {
    const long base = r.total / r.workers, rem = r.total - base * r.workers;
    const long cut = rem * (base + 1);
    return (int)(t < cut ? t / (base + 1) : rem + (t - cut) / base);
}

// The whole warp's bounded wait for phase `parity` of `bar`; false, with the CTA's abort
// flag set, when it ran out on any lane or another warp had given up.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         int32_t* dev_err) {
    const int w = mbar_wait_abortable(bar, parity, RSSM_WAIT_NS, abort);
    if (__all_sync(0xffffffffu, w > 0)) return true;
    if (w == 0) {
        set_dev_err(dev_err, RSSM_DEVERR_TIMEOUT);
        *abort = 1;
    }
    __syncwarp();
    return false;
}

// Last row b with cum[b] <= i (rows without tiles are passed over).
__device__ __forceinline__ int find_row(const long* cum, int batch, long i) {
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ Tile locate_tile(const DecArgs& a, const long* cum, long t) {
    const int b = find_row(cum, a.batch, t / a.hkv);
    const long nt = cum[b + 1] - cum[b];
    const long in_row = t - cum[b] * a.hkv;
    const int s = a.ci[b];
    const RowSpan sp = row_span(a, a.slot_len[s]);
    Tile x;
    x.b = b;
    x.h = (int)(in_row / nt);
    x.pos = (sp.first + (int)(in_row - x.h * nt)) * kTok;
    const int page = a.page_table[(long)s * a.max_pages + (x.pos >> a.ps_log2)];
    if (page < 0 || page >= a.num_pages) {
        set_dev_err(a.dev_err, RSSM_DEVERR_PAGE);
        x.y = -1;
    } else {
        x.y = ((page * a.hkv + x.h) << a.ps_log2) + (x.pos & ((1 << a.ps_log2) - 1));
    }
    return x;
}

// o and lse of query row r of (b, h): elements d, d + 1.
__device__ __forceinline__ long out_row(const DecArgs& a, int b, int h, int r) {
    const int j = r / a.G;
    return ((long)b * a.T + j) * a.hq + h * a.G + (r - j * a.G);
}

// A run: the consecutive records (partial results of groups) of one (row, head) in a CTA.
struct Run {
    int b, h;
    int rec0, rec1;  // records [rec0, rec1): 2 g: group g's head, 2 g + 1: its tail
    int whole;       // the CTA has all of its tiles
    int slot;        // else: 2 CTA + (0: began in an earlier CTA, 1: begins here)
    int cta0, cta1;  // first and last CTA
};

// D: head dim, E4M3: 8-bit cache, PARTS: bf16 parts of a query and of a weight (1 and 2
// for bf16 activations, 3 and 3 for float32 ones, which keeps all 24 bits).
template <int D, bool E4M3, bool AF32>
struct Cfg {
    static constexpr int ROWB = D * (E4M3 ? 1 : 2);  // bytes of a cached vector
    static constexpr int KB = kTok * ROWB;           // K (or V) bytes of a tile
    static constexpr int QP = AF32 ? 3 : 1;
    static constexpr int PP = AF32 ? 3 : 2;
    static constexpr int NB = D / 8;                 // n blocks of O
    static constexpr int AUX = E4M3 ? 2 * kTok * 4 : 0;  // scales of a tile
    static constexpr int STAGE = 2 * KB;
};

// Split v into bf16 parts: part i the rounding of what the parts before it leave.
template <int N>
__device__ __forceinline__ void split2(float v0, float v1, uint32_t (*out)[4], int reg) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t p = pack_bf16x2(v0, v1);
        out[i][reg] = p;
        if (i + 1 < N) {
            v0 -= bf16_lo(p);
            v1 -= bf16_hi(p);
        }
    }
}

template <int D, bool E4M3, bool AF32>
__global__ void __launch_bounds__(kDecThreads, 1)
    decode_kernel(const DecArgs a, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<D, E4M3, AF32>;
    extern __shared__ unsigned char smem_raw[];
    // 128-byte swizzled boxes want their base on 1024 bytes
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ngroups = kWarps / a.MT;
    const int group = warp / a.MT, mt = warp - group * a.MT;
    const bool in_group = group < ngroups;

    // shared memory: stages, then scales, tiles, barriers, prefix sums
    unsigned char* st_kv = smem;
    const int nst = a.stages * ngroups;
    float* st_scale = reinterpret_cast<float*>(smem + (size_t)nst * C::STAGE);
    Tile* st_tile = reinterpret_cast<Tile*>(smem + (size_t)nst * (C::STAGE + C::AUX));
    uint64_t* full = reinterpret_cast<uint64_t*>(st_tile + nst);
    uint64_t* empty = full + nst;
    long* cum = reinterpret_cast<long*>(empty + nst);
    __shared__ long scan[kWarps];
    __shared__ int abort_flag;
    __shared__ int rec_b[2 * kWarps], rec_h[2 * kWarps];  // records; b < 0: none
    __shared__ Run runs[2 * kWarps + 1];
    __shared__ int nruns, last_flag[2];
    __shared__ float tail_ml[kWarps * 16][2];

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < nst; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], a.MT);
        }
        fence_barrier_init();
    }
    if (tid < 2 * kWarps) rec_b[tid] = -1;

    // ------------------------------------------------------- the call's tile list
    {
        constexpr int R = kMaxRows / kDecThreads;
        long n[R], sum = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int b = tid * R + i;
            n[i] = 0;
            if (b < a.batch) {
                const int len = row_len(a, b, blockIdx.x == 0);
                n[i] = len < 0 ? 0 : row_span(a, len).tiles;
                // a row that sees nothing has no tiles: its outputs are written here
                if (len >= 0 && n[i] == 0 && b % gridDim.x == blockIdx.x) {
                    const long o0 = (long)b * a.T * a.hq, no = (long)a.T * a.hq;
                    for (long e = 0; e < no * D; ++e) store1(a.o, o0 * D + e, a.obf, 0.f);
                    if (a.lse)
                        for (long e = 0; e < no; ++e) a.lse[o0 + e] = -INFINITY;
                }
            }
            sum += n[i];
        }
        long inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        long before = inc - sum;
        for (int w = 0; w < warp; ++w) before += scan[w];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int b = tid * R + i;
            if (b <= a.batch) cum[b] = before;
            before += n[i];
        }
        if (tid == kDecThreads - 1 && a.batch == kMaxRows) cum[kMaxRows] = before;
        __syncthreads();
    }
    Ranges rg;
    rg.total = cum[a.batch] * a.hkv;
    if (rg.total == 0) return;
    {
        long want = (rg.total + kMinTiles - 1) / kMinTiles;
        const long ctas = gridDim.x;
        long k = (want + ctas - 1) / ctas;
        rg.per_cta = (int)(k < ngroups ? k : ngroups);
        const long w = ctas * rg.per_cta;
        rg.workers = (int)(w < want ? w : want);
    }
    const int w0 = blockIdx.x * rg.per_cta;  // this CTA's first worker
    const int nw = min(rg.per_cta, rg.workers - w0);
    if (nw <= 0) return;

    // ------------------------------------------------------- stream the range
    float o[C::NB][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    int cb = -1, ch = -1;   // current (row, head)
    int rec_begin = 0;      // its tiles began before the range
    const int r0 = mt * 16 + (lane >> 2), r1 = r0 + 8;
    const int qd = lane & 3;

    if (in_group && group < nw) {
        const long t0 = range_start(rg, w0 + group), t1 = range_start(rg, w0 + group + 1);
        const int ntile = (int)(t1 - t0);
        const bool leader = mt == 0;
        const uint64_t pol = policy_evict_first();
        unsigned char* kv = st_kv + (size_t)group * a.stages * C::STAGE;
        float* sc = st_scale + group * a.stages * (C::AUX / 4);
        Tile* tl = st_tile + group * a.stages;
        uint64_t* fb = full + group * a.stages;
        uint64_t* eb = empty + group * a.stages;

        // tiles 32 w .. 32 w + 31 of the range sit one per lane; the next 32 are looked up
        // while these are issued
        Tile cur{}, nxt{};
        int win = 0;
        if (leader) {
            if (lane < ntile) cur = locate_tile(a, cum, t0 + lane);
            if (32 + lane < ntile) nxt = locate_tile(a, cum, t0 + 32 + lane);
        }
        // issue tile i of the range into its stage (leader warp only)
        auto issue = [&](int i) {
            if (i >= ntile) return;
            if ((i >> 5) != win) {
                win = i >> 5;
                cur = nxt;
                if (32 * (win + 1) + lane < ntile) nxt = locate_tile(a, cum, t0 + 32 * (win + 1) + lane);
            }
            if (lane == (i & 31)) {
                const int s = i % a.stages;
                unsigned char* dst = kv + (size_t)s * C::STAGE;
                tl[s] = cur;
                if (cur.y < 0) {
                    mbar_arrive_plain(&fb[s]);
                } else {
                    mbar_arrive_expect_tx(&fb[s], C::STAGE + C::AUX);
                    constexpr int EB = E4M3 ? 1 : 2;
                    const int y = C::ROWB >= 128 ? cur.y : cur.y >> 1;
#pragma unroll
                    for (int x = 0; x < (C::ROWB + 127) / 128; ++x) {
                        tma_load_2d(dst + x * kTok * 128, &kmap, x * 128 / EB, y, &fb[s], pol);
                        tma_load_2d(dst + C::KB + x * kTok * 128, &vmap, x * 128 / EB, y, &fb[s], pol);
                    }
                    if (E4M3) {
                        bulk_g2s(sc + s * 2 * kTok, a.k_scale + cur.y, kTok * 4, &fb[s]);
                        bulk_g2s(sc + s * 2 * kTok + kTok, a.v_scale + cur.y, kTok * 4, &fb[s]);
                    }
                }
            }
            __syncwarp();
        };
        // A stage is refilled one tile late when several warps read it, so that the
        // leader seldom waits for them.
        const int lag = a.MT > 1 ? 1 : 0;
        if (leader)
            for (int i = 0; i < a.stages; ++i) issue(i);

        uint32_t qf[D / 16][C::QP][4];
        int end0 = 0, end1 = 0, beg0 = 0, beg1 = 0;  // visible positions of rows r0 and r1
        int n_min = 0, n_max = 0, b_min = 0, b_max = 0;
        const bool works = mt * 16 < a.M;

        // Write the current (row, head)'s result: out when its tiles all lie in this range,
        // else as a record. `tail`: the range ends with it.
        auto finish = [&](bool ends, bool tail) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            const float un = E4M3 ? kUnscale : 1.f;
            if (ends && !rec_begin) {
                const float i0 = l0 == 0.f ? 0.f : un / l0, i1 = l1 == 0.f ? 0.f : un / l1;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int r = half ? r1 : r0;
                    if (r >= a.M) continue;
                    const long row = out_row(a, cb, ch, r);
                    const float inv = half ? i1 : i0, l = half ? l1 : l0, m = half ? m1 : m0;
#pragma unroll
                    for (int n = 0; n < C::NB; n += 2) {
                        // bf16: block n has columns 8 n + 2 qd, + 1; e4m3: blocks n, n + 1
                        // have the even and odd columns of 8 n + 4 qd .. + 3
                        float v[4] = {o[n][2 * half], E4M3 ? o[n + 1][2 * half] : o[n][2 * half + 1],
                                      E4M3 ? o[n][2 * half + 1] : o[n + 1][2 * half], o[n + 1][2 * half + 1]};
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = l == 0.f ? 0.f : v[i] * inv;
                        const long e0 = row * D + 8 * n + (E4M3 ? 4 * qd : 2 * qd);
                        const long e1 = E4M3 ? e0 + 2 : e0 + 8;
                        if (a.obf) {
                            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + e0) = pack_bf16x2(v[0], v[1]);
                            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + e1) = pack_bf16x2(v[2], v[3]);
                        } else {
                            *reinterpret_cast<float2*>(static_cast<float*>(a.o) + e0) = make_float2(v[0], v[1]);
                            *reinterpret_cast<float2*>(static_cast<float*>(a.o) + e1) = make_float2(v[2], v[3]);
                        }
                    }
                    if (a.lse && qd == 0)
                        a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                }
                return;
            }
            if (leader && lane == 0) {
                rec_b[2 * group + (tail ? 1 : 0)] = cb;
                rec_h[2 * group + (tail ? 1 : 0)] = ch;
            }
            if (tail) return;  // stays in registers until the stages are free
            const long slot = 2L * gridDim.x + w0 + group;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = half ? r1 : r0;
                if (r >= a.M) continue;
                float* dst = a.part + (slot * a.M + r) * D;
#pragma unroll
                for (int n = 0; n < C::NB; ++n) {
                    const int d = E4M3 ? 16 * (n >> 1) + 4 * qd + (n & 1) : 8 * n + 2 * qd;
                    dst[d] = o[n][2 * half] * un;
                    dst[d + (E4M3 ? 2 : 1)] = o[n][2 * half + 1] * un;
                }
                if (qd == 0) {
                    a.part_ml[(slot * a.M + r) * 2] = half ? m1 : m0;
                    a.part_ml[(slot * a.M + r) * 2 + 1] = half ? l1 : l0;
                }
            }
        };

        for (int i = 0; i < ntile; ++i) {
            const int s = i % a.stages;
            if (!wait_all(&fb[s], (i / a.stages) & 1, &abort_flag, a.dev_err)) break;
            const Tile t = tl[s];
            if (t.b != cb || t.h != ch) {
                if (cb >= 0) finish(true, false);
                // the new (row, head): its queries as mma operands
                rec_begin = 0;
                if (i == 0) {
                    const long nt = cum[t.b + 1] - cum[t.b];
                    rec_begin = t0 > cum[t.b] * a.hkv + t.h * nt;
                }
                cb = t.b;
                ch = t.h;
                m0 = m1 = -INFINITY;
                l0 = l1 = 0.f;
#pragma unroll
                for (int n = 0; n < C::NB; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
                const int len = a.slot_len[a.ci[cb]];
                const int app = a.appended ? 1 : 0;
                n_min = len + app;
                n_max = len + (app ? a.T : 0);
                b_min = a.window && n_min > a.window ? n_min - a.window : 0;
                b_max = a.window && n_max > a.window ? n_max - a.window : 0;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int r = half ? r1 : r0;
                    const int j = r < a.M ? r / a.G : 0;
                    const int e = len + (app ? j + 1 : 0);
                    const int bg = a.window && e > a.window ? e - a.window : 0;
                    if (half) end1 = e, beg1 = bg;
                    else end0 = e, beg0 = bg;
                    const long base = ((long)cb * a.T + j) * a.q_stride + (ch * a.G + (r - j * a.G)) * D;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        // columns of the k16 step that this lane's registers 0/1 and 2/3 hold
                        float v[4];
#pragma unroll
                        for (int e2 = 0; e2 < 4; ++e2) {
                            const int col = E4M3 ? 4 * qd + (e2 & 1) * 2 + (e2 >> 1)
                                                 : 2 * qd + (e2 & 1) + (e2 >> 1) * 8;
                            v[e2] = r < a.M ? load1(a.q, base + 16 * kk + col, !AF32) : 0.f;
                            if (E4M3) v[e2] *= kRaise;
                        }
                        split2<C::QP>(v[0], v[1], qf[kk], half);
                        split2<C::QP>(v[2], v[3], qf[kk], 2 + half);
                    }
                }
            }
            if (t.y >= 0 && works) {
                const uint32_t kbase = smem_addr(kv + (size_t)s * C::STAGE), vbase = kbase + C::KB;
                // ------------------------------------------------ S = Q K^T
                float sa[2][2][4];
#pragma unroll
                for (int x = 0; x < 16; ++x) sa[x >> 3][(x >> 2) & 1][x & 3] = 0.f;
                const int lr = lane & 7, lm = lane >> 3;
                if (E4M3) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; kk += 2) {
                        uint32_t r[4], lo, hi;
                        ldsm4(kbase + tile_off<C::ROWB>((lm & 1) * 8 + lr, kk + (lm >> 1)), r);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            e4m3x4_to_bf16(r[x], lo, hi);
#pragma unroll
                            for (int p = 0; p < C::QP; ++p)
                                mma16816(sa[x >> 1][x & 1], qf[kk + (x >> 1)][p], lo, hi);
                        }
                    }
                } else {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        uint32_t r[4];
                        ldsm4(kbase + tile_off<C::ROWB>((lm >> 1) * 8 + lr, 2 * kk + (lm & 1)), r);
#pragma unroll
                        for (int p = 0; p < C::QP; ++p) {
                            mma16816(sa[kk & 1][0], qf[kk][p], r[0], r[1]);
                            mma16816(sa[kk & 1][1], qf[kk][p], r[2], r[3]);
                        }
                    }
                }
                // ------------------------------------------------ softmax
                float p[2][4];
                const float* ks = sc + s * 2 * kTok;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float f0 = a.qscale, f1 = a.qscale;
                    if (E4M3) {
                        const float2 k2 = *reinterpret_cast<const float2*>(ks + n * 8 + 2 * qd);
                        f0 *= k2.x * kUnscale;
                        f1 *= k2.y * kUnscale;
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        p[n][x] = (sa[0][n][x] + sa[1][n][x]) * (x & 1 ? f1 : f0);
                }
                const bool edge = t.pos + kTok > n_min || t.pos < b_max;
                if (edge) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int tok = t.pos + n * 8 + 2 * qd + (x & 1);
                            const bool vis = x < 2 ? tok < end0 && tok >= beg0 : tok < end1 && tok >= beg1;
                            if (!vis) p[n][x] = -INFINITY;
                        }
                }
                float x0 = fmaxf(fmaxf(p[0][0], p[0][1]), fmaxf(p[1][0], p[1][1]));
                float x1 = fmaxf(fmaxf(p[0][2], p[0][3]), fmaxf(p[1][2], p[1][3]));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
                const float nm0 = fmaxf(m0, x0), nm1 = fmaxf(m1, x1);
                if (__any_sync(0xffffffffu, nm0 != m0 || nm1 != m1)) {
                    const float f0 = m0 == nm0 ? 1.f : exp2_fast(m0 - nm0);
                    const float f1 = m1 == nm1 ? 1.f : exp2_fast(m1 - nm1);
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int n = 0; n < C::NB; ++n) {
                        o[n][0] *= f0;
                        o[n][1] *= f0;
                        o[n][2] *= f1;
                        o[n][3] *= f1;
                    }
                    m0 = nm0;
                    m1 = nm1;
                }
                // a row that has seen only -infinity keeps weights of zero
                const float c0 = m0 == -INFINITY ? 0.f : m0, c1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) p[n][x] = exp2_fast(p[n][x] - (x < 2 ? c0 : c1));
                    l0 += p[n][0] + p[n][1];
                    l1 += p[n][2] + p[n][3];
                }
                if (E4M3) {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float2 v2 = *reinterpret_cast<const float2*>(ks + kTok + n * 8 + 2 * qd);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            float w = p[n][x] * ((x & 1 ? v2.y : v2.x) * kRaise);
                            if (edge) {
                                const int tok = t.pos + n * 8 + 2 * qd + (x & 1);
                                const bool vis = x < 2 ? tok < end0 && tok >= beg0 : tok < end1 && tok >= beg1;
                                if (!vis) w = 0.f;  // whatever the scale there holds
                            }
                            p[n][x] = w;
                        }
                    }
                }
                // ------------------------------------------------ O += P V
                bool careful = false;
                if (!E4M3 && edge) {
                    // A weight of zero does not silence an infinity or a NaN in a value. Tokens
                    // that no query sees are cleared; if one that only some see is not finite,
                    // the tile's products run value by value below.
                    unsigned char* vt = kv + (size_t)s * C::STAGE + C::KB;
                    const bool outside = t.pos + kTok > n_max || t.pos < b_min;
                    if (outside) {
                        for (int e = lane; e < kTok * (C::ROWB / 16); e += 32) {
                            const int tok = e / (C::ROWB / 16), c = e % (C::ROWB / 16);
                            if (t.pos + tok >= n_max || t.pos + tok < b_min)
                                *reinterpret_cast<uint4*>(vt + tile_off<C::ROWB>(tok, c)) = make_uint4(0, 0, 0, 0);
                        }
                        fence_async_smem();  // the stage's next TMA load comes after these stores
                        __syncwarp();
                    }
                    if (a.T > 1) {
                        bool odd = false;
                        for (int e = lane; e < kTok * (C::ROWB / 16); e += 32) {
                            const int tok = e / (C::ROWB / 16), c = e % (C::ROWB / 16), pos = t.pos + tok;
                            if ((pos >= n_min && pos < n_max) || (pos >= b_min && pos < b_max)) {
                                const uint4 v = *reinterpret_cast<const uint4*>(vt + tile_off<C::ROWB>(tok, c));
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    odd |= (w[x] & 0x7f80u) == 0x7f80u || (w[x] & 0x7f800000u) == 0x7f800000u;
                            }
                        }
                        careful = __any_sync(0xffffffffu, odd);
                    }
                }
                if (!careful) {
                    uint32_t pf[C::PP][4];
                    split2<C::PP>(p[0][0], p[0][1], pf, 0);
                    split2<C::PP>(p[0][2], p[0][3], pf, 1);
                    split2<C::PP>(p[1][0], p[1][1], pf, 2);
                    split2<C::PP>(p[1][2], p[1][3], pf, 3);
                    constexpr int CH = C::ROWB / 16;  // 16-byte chunks of a vector
#pragma unroll
                    for (int c = 0; c < CH; c += 2) {
                        uint32_t r[4];
                        ldsm4_t(vbase + tile_off<C::ROWB>((lm & 1) * 8 + lr, c + (lm >> 1)), r);
                        if (E4M3) {
                            uint32_t lo0, hi0, lo1, hi1, lo2, hi2, lo3, hi3;
                            e4m3x4_to_bf16(r[0], lo0, hi0);
                            e4m3x4_to_bf16(r[1], lo1, hi1);
                            e4m3x4_to_bf16(r[2], lo2, hi2);
                            e4m3x4_to_bf16(r[3], lo3, hi3);
#pragma unroll
                            for (int x = 0; x < C::PP; ++x) {
                                mma16816(o[2 * c], pf[x], lo0, lo1);
                                mma16816(o[2 * c + 1], pf[x], hi0, hi1);
                                mma16816(o[2 * c + 2], pf[x], lo2, lo3);
                                mma16816(o[2 * c + 3], pf[x], hi2, hi3);
                            }
                        } else {
#pragma unroll
                            for (int x = 0; x < C::PP; ++x) {
                                mma16816(o[c], pf[x], r[0], r[1]);
                                mma16816(o[c + 1], pf[x], r[2], r[3]);
                            }
                        }
                    }
                } else {
                    const unsigned char* vt = kv + (size_t)s * C::STAGE + C::KB;
                    for (int tok = 0; tok < kTok; ++tok) {
                        const int src = (lane & ~3) | ((tok & 7) >> 1);
                        const int n = tok >> 3, x = tok & 1;
                        const float w0f = n ? (x ? p[1][1] : p[1][0]) : (x ? p[0][1] : p[0][0]);
                        const float w1f = n ? (x ? p[1][3] : p[1][2]) : (x ? p[0][3] : p[0][2]);
                        const float w0v = __shfl_sync(0xffffffffu, w0f, src);
                        const float w1v = __shfl_sync(0xffffffffu, w1f, src);
                        const int pos = t.pos + tok;
                        const bool see0 = pos < end0 && pos >= beg0, see1 = pos < end1 && pos >= beg1;
#pragma unroll
                        for (int nb = 0; nb < C::NB; ++nb) {
                            const uint32_t v = *reinterpret_cast<const uint32_t*>(
                                vt + tile_off<C::ROWB>(tok, nb) + 4 * qd);
                            if (see0) {
                                o[nb][0] += w0v * bf16_lo(v);
                                o[nb][1] += w0v * bf16_hi(v);
                            }
                            if (see1) {
                                o[nb][2] += w1v * bf16_lo(v);
                                o[nb][3] += w1v * bf16_hi(v);
                            }
                        }
                    }
                }
            }
            // ---------------------------------------------------- hand the stage back
            __syncwarp();
            if (a.MT > 1 && lane == 0) mbar_arrive_plain(&eb[s]);
            if (leader && i >= lag) {
                const int done = i - lag;
                if (a.MT > 1 && done + a.stages < ntile &&
                    !wait_all(&eb[done % a.stages], (done / a.stages) & 1, &abort_flag, a.dev_err))
                    break;
                issue(done + a.stages);
            }
        }
        if (cb >= 0) {
            const long nt = cum[cb + 1] - cum[cb];
            finish(t1 == cum[cb] * a.hkv + (ch + 1) * nt, true);
        }
    }
    __syncthreads();
    if (abort_flag) {
        // A wait ran out: no copy may still be in flight when the CTA ends. Every stage's
        // barrier is watched for a while, whatever its phase.
        if (tid < nst) {
            mbar_wait_bounded(&full[tid], 0, RSSM_WAIT_NS / 100);
            mbar_wait_bounded(&full[tid], 1, RSSM_WAIT_NS / 100);
        }
        __syncthreads();
    }

    // ------------------------------------------------------- join the CTA's records
    // Tails into shared memory (the stages are free now).
    float* tail = reinterpret_cast<float*>(smem);  // [group][M][D]
    if (in_group && group < nw && rec_b[2 * group + 1] >= 0) {
        const float un = E4M3 ? kUnscale : 1.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = half ? r1 : r0;
            if (r >= a.M) continue;
            float* dst = tail + ((long)group * a.M + r) * D;
#pragma unroll
            for (int n = 0; n < C::NB; ++n) {
                const int d = E4M3 ? 16 * (n >> 1) + 4 * qd + (n & 1) : 8 * n + 2 * qd;
                dst[d] = o[n][2 * half] * un;
                dst[d + (E4M3 ? 2 : 1)] = o[n][2 * half + 1] * un;
            }
            if (qd == 0) {
                tail_ml[group * a.M + r][0] = half ? m1 : m0;
                tail_ml[group * a.M + r][1] = half ? l1 : l0;
            }
        }
    }
    if (tid == 0) {
        int n = 0;
        last_flag[0] = last_flag[1] = 0;
        for (int i = 0; i < 2 * nw; ++i) {
            if (rec_b[i] < 0) continue;
            if (n && runs[n - 1].b == rec_b[i] && runs[n - 1].h == rec_h[i]) {
                runs[n - 1].rec1 = i + 1;
                continue;
            }
            Run r;
            r.b = rec_b[i];
            r.h = rec_h[i];
            r.rec0 = i;
            r.rec1 = i + 1;
            const long nt = cum[r.b + 1] - cum[r.b];
            const long s0 = cum[r.b] * a.hkv + r.h * nt;
            r.cta0 = worker_of(rg, s0) / rg.per_cta;
            r.cta1 = worker_of(rg, s0 + nt - 1) / rg.per_cta;
            r.whole = r.cta0 == r.cta1;
            r.slot = 2 * (int)blockIdx.x + (r.cta0 < (int)blockIdx.x ? 0 : 1);
            runs[n++] = r;
        }
        nruns = n;
    }
    __threadfence_block();
    __syncthreads();

    // (run, part of its values) pairs over the warps; a lane takes 4 values at a time
    const int parts = nruns >= kWarps ? 1 : kWarps / max(nruns, 1);
    for (int item = warp; item < nruns * parts; item += kWarps) {
        const Run r = runs[item / parts];
        const int nv = a.M * D / 4, part = item % parts;
        for (int v = part * 32 + lane; v < nv; v += 32 * parts) {
            const int row = v / (D / 4), d = (v % (D / 4)) * 4;
            float m = -INFINITY, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            // the rows' maxima first, then the weighted sums, in record order
            for (int i = r.rec0; i < r.rec1; ++i) {
                if (rec_b[i] < 0) continue;
                const float* ml = i & 1 ? tail_ml[(i >> 1) * a.M + row]
                                        : a.part_ml + ((2L * gridDim.x + w0 + (i >> 1)) * a.M + row) * 2;
                m = fmaxf(m, ml[0]);
            }
            const float base = m == -INFINITY ? 0.f : m;
            for (int i = r.rec0; i < r.rec1; ++i) {
                if (rec_b[i] < 0) continue;
                const float* ml;
                const float* src;
                if (i & 1) {
                    ml = tail_ml[(i >> 1) * a.M + row];
                    src = tail + ((long)(i >> 1) * a.M + row) * D + d;
                } else {
                    const long slot = 2L * gridDim.x + w0 + (i >> 1);
                    ml = a.part_ml + (slot * a.M + row) * 2;
                    src = a.part + (slot * a.M + row) * D + d;
                }
                const float f = exp2_fast(ml[0] - base);
                const float4 x = *reinterpret_cast<const float4*>(src);
                l += ml[1] * f;
                acc.x += x.x * f;
                acc.y += x.y * f;
                acc.z += x.z * f;
                acc.w += x.w * f;
            }
            if (r.whole) {
                const long out = out_row(a, r.b, r.h, row);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                float y[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store1(a.o, out * D + d + i, a.obf, l == 0.f ? 0.f : y[i] * inv);
                if (a.lse && d == 0)
                    a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            } else {
                *reinterpret_cast<float4*>(a.part + ((long)r.slot * a.M + row) * D + d) = acc;
                if (d == 0) {
                    a.part_ml[((long)r.slot * a.M + row) * 2] = m;
                    a.part_ml[((long)r.slot * a.M + row) * 2 + 1] = l;
                }
            }
        }
    }

    // ------------------------------------------------------- join the CTAs
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        // at most the first run (begun earlier) and the last (goes on) are shared; the
        // counter is the first CTA's
        for (int i = 0; i < nruns; ++i) {
            if (runs[i].whole) continue;
            const int n = runs[i].cta1 - runs[i].cta0 + 1;
            if (atomicAdd(&a.counters[runs[i].cta0], 1) == n - 1) {
                a.counters[runs[i].cta0] = 0;
                last_flag[i == 0 ? 0 : 1] = i + 1;
            }
        }
        __threadfence();
    }
    __syncthreads();
#pragma unroll 1
    for (int f = 0; f < 2; ++f) {
        if (!last_flag[f]) continue;
        const Run r = runs[last_flag[f] - 1];
        const int n = r.cta1 - r.cta0 + 1;
        const int nv = a.M * D / 4;
        for (int v = tid; v < nv; v += kDecThreads) {
            const int row = v / (D / 4), d = (v % (D / 4)) * 4;
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < n; ++i) {
                const long slot = 2L * (r.cta0 + i) + (i == 0 ? 1 : 0);
                m = fmaxf(m, __ldcg(a.part_ml + (slot * a.M + row) * 2));
            }
            const float base = m == -INFINITY ? 0.f : m;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const long slot = 2L * (r.cta0 + i) + (i == 0 ? 1 : 0);
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot * a.M + row);
                const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part + (slot * a.M + row) * D + d));
                const float w = exp2_fast(ml.x - base);
                l += ml.y * w;
                acc.x += x.x * w;
                acc.y += x.y * w;
                acc.z += x.z * w;
                acc.w += x.w * w;
            }
            const long out = out_row(a, r.b, r.h, row);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            float y[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                store1(a.o, out * D + d + i, a.obf, l == 0.f ? 0.f : y[i] * inv);
            if (a.lse && d == 0)
                a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
    }
}

// ---------------------------------------------------------------- host side

// Workspace: counters (one per CTA), then [2 CTAs + groups] partial results (m, l), then
// their values. The CTA count is that of the largest machine the library runs on.
constexpr int kMaxCtas = 256;

struct Workspace {
    size_t ml, part, bytes;
};
static Workspace workspace_of(const rssm_attn_dims* d) {
    const size_t M = (size_t)d->q_tokens * (d->num_q_heads / d->num_kv_heads);
    const size_t slots = kMaxCtas * (2 + kWarps);
    Workspace w;
    w.ml = kMaxCtas * sizeof(int32_t);
    w.part = (w.ml + slots * M * 2 * sizeof(float) + 255) / 256 * 256;
    w.bytes = w.part + slots * M * d->head_dim * sizeof(float);
    return w;
}

template <int D, bool E4M3, bool AF32>
static int launch(const rssm_attn_dims* d, const rssm_attn_cache* c, DecArgs a, const DeviceInfo& di,
                  cudaStream_t st) {
    using C = Cfg<D, E4M3, AF32>;
    const int ngroups = kWarps / a.MT;
    const int fixed = (kMaxRows + 1) * 8 + 1024;
    const int per = C::STAGE + C::AUX + (int)sizeof(Tile) + 16;
    int stages = (di.max_smem_optin - 2560 - fixed) / (per * ngroups);
    if (stages > kMaxStages) stages = kMaxStages;
    if (stages < 2) return RSSM_ERR_UNSUPPORTED;
    a.stages = stages;
    int smem = stages * ngroups * per + fixed;
    const int tails = kWarps * 16 * D * 4 + 1024;
    if (smem < tails) smem = tails;
    const void* kern = (const void*)decode_kernel<D, E4M3, AF32>;
    if (!ensure_smem_limit(kern, smem)) return RSSM_ERR_CUDA;
    // rows of 128 bytes at least: 64-byte vectors go in pairs
    const uint64_t rows = (uint64_t)d->num_pages * d->num_kv_heads * d->page_size;
    const bool pair = C::ROWB < 128;
    CUtensorMap km, vm;
    if (!make_tmap_rows128(&km, c->k, E4M3 ? 1 : 2, pair ? rows / 2 : rows, pair ? 2 * D : D, pair ? kTok / 2 : kTok) ||
        !make_tmap_rows128(&vm, c->v, E4M3 ? 1 : 2, pair ? rows / 2 : rows, pair ? 2 * D : D, pair ? kTok / 2 : kTok))
        return RSSM_ERR_CUDA;
    const int grid = di.sm_count < kMaxCtas ? di.sm_count : kMaxCtas;
    for (int b = 0; b < d->batch; b += kMaxRows) {
        DecArgs x = a;
        x.batch = d->batch - b < kMaxRows ? d->batch - b : kMaxRows;
        x.ci = a.ci + b;
        x.q = static_cast<const char*>(a.q) + (long)b * a.T * a.q_stride * (AF32 ? 4 : 2);
        x.o = static_cast<char*>(a.o) + (long)b * a.T * a.hq * D * (a.obf ? 2 : 4);
        if (a.lse) x.lse = a.lse + (long)b * a.T * a.hq;
        decode_kernel<D, E4M3, AF32><<<grid, kDecThreads, smem, st>>>(x, km, vm);
    }
    return launch_status();
}

}  // namespace attn
}  // namespace rssm

using namespace rssm;

extern "C" size_t rssm_attn_workspace_size(const rssm_attn_dims* d) {
    if (attn::check_dims(d) != RSSM_OK) return 0;
    return attn::workspace_of(d).bytes;
}

extern "C" int rssm_attn_decode(const rssm_attn_dims* d, const rssm_attn_cache* c, int appended,
                                float scale, int32_t window, const void* q, int64_t q_stride,
                                const int32_t* cache_indices, void* workspace,
                                size_t workspace_bytes, void* o, float* lse, int32_t* dev_err,
                                rssm_stream_t stream) {
    const int st = attn::check_dims(d);
    if (st != RSSM_OK) return st;
    if (window < 0) return RSSM_ERR_INVALID_ARG;
    const int G = d->num_q_heads / d->num_kv_heads;
    if ((int64_t)d->q_tokens * G > 64) return RSSM_ERR_UNSUPPORTED;
    if (d->batch == 0) return RSSM_OK;
    const attn::Workspace ws = attn::workspace_of(d);
    if (!attn::ok_cache(d, c) || !ok_ptr(q) || !attn::ok_stride(d, q_stride, d->num_q_heads) ||
        !ok_ptr(cache_indices) || !ok_ptr(workspace) || workspace_bytes < ws.bytes || !ok_ptr(o) ||
        !ok_opt_ptr(lse))
        return RSSM_ERR_INVALID_ARG;
    DeviceInfo di;
    if (!device_info(&di)) return RSSM_ERR_CUDA;
    attn::DecArgs a{};
    a.q = q;
    a.q_stride = q_stride;
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
    a.G = G;
    a.hq = d->num_q_heads;
    a.hkv = d->num_kv_heads;
    a.ps_log2 = attn::log2_of(d->page_size);
    a.num_pages = d->num_pages;
    a.max_pages = d->max_pages;
    a.num_slots = d->num_slots;
    a.window = window;
    a.appended = appended != 0;
    a.M = a.T * G;
    a.MT = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
    a.obf = d->out_dtype == RSSM_BF16;
    const bool q8 = d->cache_dtype == RSSM_E4M3, f32 = d->act_dtype == RSSM_F32;
    const cudaStream_t s = (cudaStream_t)stream;
#define RSSM_ATTN_D(D_)                                                            \
    (q8 ? (f32 ? attn::launch<D_, true, true>(d, c, a, di, s)                      \
               : attn::launch<D_, true, false>(d, c, a, di, s))                    \
        : (f32 ? attn::launch<D_, false, true>(d, c, a, di, s)                     \
               : attn::launch<D_, false, false>(d, c, a, di, s)))
    return d->head_dim == 64 ? RSSM_ATTN_D(64) : RSSM_ATTN_D(128);
#undef RSSM_ATTN_D
}
