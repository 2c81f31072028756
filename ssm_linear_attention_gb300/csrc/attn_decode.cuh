// attn_decode.cuh -- what the attention kernels share: the call's tile list and its cuts,
// partial results and how the CTAs' are joined.
#pragma once

#include <cuda_fp16.h>

#include "attn.cuh"
#include "warps.cuh"

namespace rssm {
namespace attn {

constexpr int kTok = 16;       // tokens per tile: the smallest page
constexpr int kMaxStages = 8;  // per group
constexpr int kMaxWarps = 16;  // per CTA
constexpr int kMaxCtas = 256;  // more than the SMs of any machine the library runs on
constexpr int kMaxRows = 1024;  // rows per launch (prefix sums in shared memory)
constexpr int kRowBytes = 13312;  // prefix sums, lengths and slots of kMaxRows rows, up to the
                                  // stages' alignment
// Tiles that each group of a CTA gets at least before another CTA joins in.
constexpr int kMinTiles = 2;
// Longest (row, head), in tiles, up to which no CTA shares one. Meeting in global memory
// costs a call some 3 to 6 us; an uneven cut costs at most this many tiles over a CTA's groups
// (16 rows of 1500 tokens: 24 us with 48 here, 21 with 96 or 160; 64 of 1200: 37, 38, 39).
constexpr int kWholeTiles = 96;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The base m of the weights 2^(s - m) is the largest score and this much (log2 units): it moves when a
// score passes it, so most tiles need no maximum across lanes, and no weight is above 1 (a sum of
// weighted values overflows only where one of plain softmax weights would).
constexpr float kSlack = 8.f;

struct DecArgs {
    const void* q;
    long q_stride;
    const char* k;
    const char* v;
    const float* k_scale;
    const float* v_scale;
    const int32_t* page_table;
    const int32_t* slot_len;
    const int32_t* ci;
    void* o;
    float* lse;
    int32_t* dev_err;
    float* part;       // [2 x CTAs][M][D] partial results of CTAs, then [CTAs][groups][M][D] of
                       // the groups' heads (few queries)
    float* part_ml;    // [2 x CTAs][M][2]
    int32_t* counters; // [CTAs]
    float qscale;      // scale * log2 e
    int batch, T, G, hq, hkv, ps_log2, num_pages, max_pages, num_slots, window, appended;
    int M, MT;         // queries per key head, warps per group (each 8 queries)
    int ngroups;       // of a CTA
    int stages;        // per group
    int obf;
    uint64_t wait_ns;  // limit of a wait on a copy or a product
    int stall;         // test: the tile (many queries: chunk) of the list whose wait runs out; -1: none
};

__device__ __forceinline__ float log2_fast(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x to 1 ulp of float32
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The four e4m3 codes of w as f16 pairs (exact): lo = codes 0, 1, hi = codes 2, 3.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ float2 f16x2_to_f(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
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

// The call's rows in shared memory.
struct Rows {
    uint32_t* cum;  // [batch + 1] tiles of the rows before
    int* len;       // committed tokens; -1: the row is skipped
    int* slot;
};

// Where one tile lies: row, head, number among the (row, head)'s tiles.
struct Tile {
    int b, h, at;
};

// The tile list (fewer than 2^31 tiles) cut into the CTAs' ranges. Even cuts share (row,
// head)s between CTAs, whose results then meet in global memory; where every (row, head)
// is short, the cuts move up to the next (row, head) instead.
struct Cuts {
    uint32_t total, base, rem;  // an even range has base tiles, the first rem of them one more
    int ctas;                   // that have a range
};
__device__ __forceinline__ uint32_t even_cut(const Cuts& r, uint32_t c) {
    return c * r.base + min(c, r.rem);
}
// The CTA whose even range holds tile t.
__device__ __forceinline__ int cta_of(const Cuts& r, uint32_t t) {
    const uint32_t cut = r.rem * (r.base + 1);
    return (int)(t < cut ? t / (r.base + 1) : r.rem + (t - cut) / r.base);
}

// Last row b with cum[b] <= i (rows without tiles are passed over).
__device__ __forceinline__ int find_row(const uint32_t* cum, int batch, uint32_t i) {
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Row and head of tile t, and its number among the (row, head)'s tiles; `single` says that
// CTA i has (row, head) i.
static __device__ __noinline__ Tile find_tile(const DecArgs& a, const uint32_t* cum, uint32_t t, bool single) {
    Tile x;
    if (single)
        x.b = (int)blockIdx.x / a.hkv;
    else
        x.b = a.batch == 1 ? 0 : find_row(cum, a.batch, t / (uint32_t)a.hkv);
    const uint32_t nt = cum[x.b + 1] - cum[x.b];
    const uint32_t in_row = t - cum[x.b] * (uint32_t)a.hkv;
    x.h = single ? (int)blockIdx.x - x.b * a.hkv : (int)(in_row / nt);
    x.at = (int)(in_row - (uint32_t)x.h * nt);
    return x;
}

// The first tile from t (the same on all lanes) on that begins a (row, head). The lanes look for
// the row together, 32 places at a time.
static __device__ __noinline__ uint32_t next_head(const DecArgs& a, const uint32_t* cum, uint32_t t) {
    if (t >= cum[a.batch] * (uint32_t)a.hkv) return t;
    const uint32_t i = t / (uint32_t)a.hkv;
    const int lane = threadIdx.x & 31;
    int b = 0, n = a.batch;  // the row is one of the n from b on
    while (n > 1) {
        const int step = (n + 31) / 32, at = lane * step;
        const int k = __popc(__ballot_sync(0xffffffffu, at < n && cum[b + min(at, n - 1)] <= i)) - 1;
        b += k * step;
        n = min(step, n - k * step);
    }
    const uint32_t nt = cum[b + 1] - cum[b], rest = (t - cum[b] * (uint32_t)a.hkv) % nt;
    return rest == 0 ? t : t - rest + nt;
}

// Row of tile t's first token in the cache matrix; -1, with the flag set, when its page is
// out of range.
static __device__ __noinline__ int locate_tile(const DecArgs& a, const Rows& rows, uint32_t t, bool single) {
    const Tile x = find_tile(a, rows.cum, t, single);
    const int pos = (row_span(a, rows.len[x.b]).first + x.at) * kTok;
    // (a plain load: a kernel that starts early may not take a table for constant that one before
    // it still writes)
    const int page = a.page_table[(long)rows.slot[x.b] * a.max_pages + (pos >> a.ps_log2)];
    if (page < 0 || page >= a.num_pages) {
        set_dev_err(a.dev_err, RSSM_DEVERR_PAGE);
        return -1;
    }
    return ((page * a.hkv + x.h) << a.ps_log2) + (pos & ((1 << a.ps_log2) - 1));
}

// A partial result of one query over four columns: (m, l) and O. Adding one rescales to
// the larger m; a sum's order is that of the adds.
struct Partial {
    float2 ml = make_float2(-INFINITY, 0.f);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float2 bl, float4 x) {
        const float top = fmaxf(ml.x, bl.x), base = top == -INFINITY ? 0.f : top;
        const float f = exp2_fast(ml.x - base), g = exp2_fast(bl.x - base);
        ml = make_float2(top, ml.y * f + bl.y * g);
        v.x = v.x * f + x.x * g;
        v.y = v.y * f + x.y * g;
        v.z = v.z * f + x.z * g;
        v.w = v.w * f + x.w * g;
    }
};
// Columns d .. d + 3 of output row r: O / l, zeros where nothing was seen; its lse.
static __device__ __noinline__ void store_partial(const DecArgs& a, const Partial p, long r, int D, int d) {
    const bool none = p.ml.y == 0.f;
    const float inv = none ? 0.f : reciprocal(p.ml.y);
    const float y[4] = {none ? 0.f : p.v.x * inv, none ? 0.f : p.v.y * inv, none ? 0.f : p.v.z * inv,
                        none ? 0.f : p.v.w * inv};
    if (a.obf)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + r * D + d) =
            make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(a.o) + r * D + d) = make_float4(y[0], y[1], y[2], y[3]);
    if (d == 0 && a.lse) a.lse[r] = none ? -INFINITY : (p.ml.x + log2_fast(p.ml.y)) * kLn2;
}
constexpr int kItems = 2;  // pieces of a CTA's join that a thread has in flight
constexpr int kJoin = 4;   // partial results of CTAs whose loads a thread has in flight

// A run: the consecutive records (partial results of groups) of one (row, head) in a CTA.
struct Run {
    int b, h;
    int rec0, rec1;  // its first record and one past its last (2 g: group g's head, 2 g + 1: its tail)
    int cta0, cta1;  // first and last CTA that has tiles of it
};

// Tiles of the call's rows into `rows`, bad slots and lengths flagged; returns the tiles of the
// longest row, all in units of UNIT tiles, EXTRA more to a row that has any. All THREADS threads of the CTA, ROWS rows at most;
// scan: a value of shared memory per warp.
template <int THREADS, int ROWS, int UNIT, int EXTRA>
__device__ __forceinline__ uint32_t list_tiles(const DecArgs& a, const Rows& rows, uint2* scan) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t* const cum = rows.cum;
    uint32_t longest = 0;  // tiles of the longest (row, head)
    {
        constexpr int R = (ROWS + THREADS - 1) / THREADS;
        uint32_t n[R], sum = 0;
        int slot[R], len[R];
        let_next_in();
        wait_for_stream();
#pragma unroll
        for (int i = 0; i < R; ++i) slot[i] = tid * R + i < a.batch ? a.ci[tid * R + i] : -1;
#pragma unroll
        for (int i = 0; i < R; ++i)
            len[i] = slot[i] >= 0 && slot[i] < a.num_slots ? a.slot_len[slot[i]] : -1;
        const long cap = ((long)a.max_pages << a.ps_log2) - (a.appended ? a.T : 0);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (slot[i] >= a.num_slots) {
                if (blockIdx.x == 0) set_dev_err(a.dev_err, RSSM_DEVERR_SLOT);
            } else if (slot[i] >= 0 && (len[i] < 0 || len[i] > cap)) {
                if (blockIdx.x == 0) set_dev_err(a.dev_err, RSSM_DEVERR_CURSOR);
                len[i] = -1;
            }
            n[i] = len[i] < 0 ? 0 : (row_span(a, len[i]).tiles + UNIT - 1) / UNIT;
            if (EXTRA && n[i]) n[i] += EXTRA;
            if (tid * R + i < a.batch) {
                rows.len[tid * R + i] = len[i];
                rows.slot[tid * R + i] = slot[i];
            }
            sum += n[i];
        }
        uint32_t inc = sum, top = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) top = max(top, n[i]);
        top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) scan[warp] = make_uint2(inc, top);
        __syncthreads();
        uint32_t before = inc - sum;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += scan[w].x;
            longest = max(longest, scan[w].y);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int b = tid * R + i;
            if (b <= a.batch) cum[b] = before;
            before += n[i];
        }
        if (tid == THREADS - 1 && a.batch == R * THREADS) cum[a.batch] = before;
        __syncthreads();
    }
    return longest;
}

// Rows that see nothing have no tiles: their outputs are written here.
template <int D, int THREADS>
__device__ __forceinline__ void write_empty_rows(const DecArgs& a, const Rows& rows) {
    const uint32_t* const cum = rows.cum;
    const int tid = threadIdx.x;
#pragma unroll 1
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
        if (cum[b + 1] != cum[b] || rows.len[b] < 0) continue;
        const long o0 = (long)b * a.T * a.hq;
        const int no = a.T * a.hq;
#pragma unroll 1
        for (int e = tid; e < no * D; e += THREADS) store1(a.o, o0 * D + e, a.obf, 0.f);
        if (a.lse)
#pragma unroll 1
            for (int e = tid; e < no; e += THREADS) a.lse[o0 + e] = -INFINITY;
    }
}

// This CTA's range [c0, c1) of the tile list; false when it has none. least_tiles: a CTA gets at least
// so many before another joins in. whole: the longest (row, head) that no CTAs share. single: every CTA has a (row, head) of its own.
__device__ __forceinline__ bool cut_tiles(const DecArgs& a, const uint32_t* cum, uint32_t longest,
                                          uint32_t least_tiles, uint32_t whole, Cuts& rg, uint32_t& c0, uint32_t& c1,
                                          bool& single) {
    rg.total = cum[a.batch] * (uint32_t)a.hkv;
    if (rg.total == 0) return false;
    // Short (row, head)s, and a CTA for each: no cuts at all, and no search for them.
    single = longest <= whole && a.batch * a.hkv <= (int)gridDim.x;
    if (single) {
        const int b = (int)blockIdx.x / a.hkv, h = (int)blockIdx.x - b * a.hkv;
        if (b >= a.batch) return false;
        const uint32_t nt = cum[b + 1] - cum[b];
        if (nt == 0) return false;
        c0 = cum[b] * (uint32_t)a.hkv + h * nt;
        c1 = c0 + nt;
    } else {
        // short (row, head)s: as many CTAs as there may be (row, head)s
        const uint32_t least = longest <= whole ? min(least_tiles, longest) : least_tiles;
        rg.ctas = (int)min(gridDim.x, (rg.total + least - 1) / least);
        rg.base = rg.total / (uint32_t)rg.ctas;
        rg.rem = rg.total - rg.base * (uint32_t)rg.ctas;
        if ((int)blockIdx.x >= rg.ctas) return false;
        c0 = even_cut(rg, blockIdx.x);
        c1 = even_cut(rg, blockIdx.x + 1);
        if (longest <= whole) {
            c0 = next_head(a, cum, c0);
            c1 = next_head(a, cum, c1);
            if (c0 >= c1) return false;
        }
    }
    return true;
}

// Join the CTAs of this CTA's shared (row, head)s, whose partial results are in global memory.
// All THREADS threads; last_flag: two values of shared memory, 0; scratch: a Partial per thread.
template <int D, int THREADS>
__device__ __forceinline__ void join_ctas(const DecArgs& a, const Run* runs, int nruns, const int* q_row,
                                          int* last_flag, void* scratch) {
    const int tid = threadIdx.x, nv = a.M * (D / 4);
    // Only the first run (begun in an earlier CTA) and the last (which goes on) can be
    // shared. The counter of a shared (row, head) is its first CTA's.
    if (nruns == 0 || (runs[0].cta0 == runs[0].cta1 && runs[nruns - 1].cta0 == runs[nruns - 1].cta1)) return;
    __threadfence();
    __syncthreads();
    if (tid < 2 && (tid == 0 || nruns > 1)) {
        const Run& r = runs[tid == 0 ? 0 : nruns - 1];
        if (r.cta0 != r.cta1 && atomicAdd(&a.counters[r.cta0], 1) == r.cta1 - r.cta0) {
            a.counters[r.cta0] = 0;
            last_flag[tid] = 1;
        }
        __threadfence();
    }
    __syncthreads();
    // few values: several threads share one, each a stretch of the partial results
    const int parts = nv < THREADS ? THREADS / nv : 1;
    const int part = parts > 1 ? tid / nv : 0;
    Partial* jp = reinterpret_cast<Partial*>(scratch);  // [threads]
#pragma unroll 1
    for (int f = 0; f < 2; ++f) {
        if (!last_flag[f]) continue;
        const Run r = runs[f == 0 ? 0 : nruns - 1];
        const int n = r.cta1 - r.cta0 + 1, i0 = n * part / parts, i1 = n * (part + 1) / parts;
#pragma unroll 1
        for (int v = parts > 1 ? tid % nv : tid; v < nv && part < parts; v += THREADS) {
            const int row = v / (D / 4), d = (v % (D / 4)) * 4;
            Partial acc;
#pragma unroll 1
            for (int i = i0; i < i1; i += kJoin) {
                // the loads of kJoin partial results at once; of the first CTA its last run,
                // of the others their first
                float2 ml[kJoin];
                float4 x[kJoin];
#pragma unroll
                for (int k = 0; k < kJoin; ++k) {
                    ml[k] = make_float2(-INFINITY, 0.f);
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i + k < i1) {
                        const long slot = (2L * (r.cta0 + i + k) + (i + k == 0 ? 1 : 0)) * a.M + row;
                        ml[k] = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot);
                        x[k] = __ldcg(reinterpret_cast<const float4*>(a.part + slot * D + d));
                    }
                }
#pragma unroll
                for (int k = 0; k < kJoin; ++k) acc.add(ml[k], x[k]);
            }
            if (parts > 1) {
                jp[tid] = acc;
            } else {
                store_partial(a, acc, (long)r.b * a.T * a.hq + r.h * a.G + q_row[row], D, d);
            }
        }
        if (parts > 1) {
            __syncthreads();
            if (tid < nv) {
                Partial acc = jp[tid];
#pragma unroll 1
                for (int i = 1; i < parts; ++i) acc.add(jp[i * nv + tid].ml, jp[i * nv + tid].v);
                const int row = tid / (D / 4), d = (tid % (D / 4)) * 4;
                store_partial(a, acc, (long)r.b * a.T * a.hq + r.h * a.G + q_row[row], D, d);
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- host side

// Calls launch(args) for at most `most` rows at a time: what the prefix sums hold, and a tile list
// of fewer than 2^31.
template <class Launch>
inline int launch_rows(const rssm_attn_dims* d, const DecArgs& a, int most, Launch launch) {
    const int64_t row_tiles = (int64_t)d->max_pages * (d->page_size / kTok) * a.hkv;
    int64_t per_launch = (((int64_t)1 << 31) - 1) / row_tiles;
    if (per_launch < 1) return RSSM_ERR_UNSUPPORTED;
    if (per_launch > most) per_launch = most;
    for (int b = 0; b < d->batch; b += (int)per_launch) {
        DecArgs x = a;
        x.batch = d->batch - b < per_launch ? d->batch - b : (int)per_launch;
        x.ci = a.ci + b;
        x.q = static_cast<const char*>(a.q) + (long)b * a.T * a.q_stride * (d->act_dtype == RSSM_F32 ? 4 : 2);
        x.o = static_cast<char*>(a.o) + (long)b * a.T * a.hq * d->head_dim * (a.obf ? 2 : 4);
        if (a.lse) x.lse = a.lse + (long)b * a.T * a.hq;
        launch(x);
    }
    return launch_status();
}

// attn_wide.cu
int decode_wide(const rssm_attn_dims* d, const DecArgs& a, const DeviceInfo& di, cudaStream_t st);

}  // namespace attn
}  // namespace rssm
