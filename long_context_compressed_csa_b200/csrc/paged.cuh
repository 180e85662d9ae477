// The paged key-value cache of the full-attention layers: arguments, visibility, and the
// device-side schedule that the attention kernels share.
#pragma once
#include <atomic>

#include "common.cuh"

namespace csa {

constexpr int kPagedMaxD = 256;    // widest head the kernels hold on chip

// Pools of K and V rows: row (p, r, h) of d elements starts p * ld_page + r * ld_row + h * ld_head
// elements after the base; K and V have the same strides.
struct PagedPool {
    int64_t ld_page, ld_row, ld_head;
    int64_t n_pages;
    int page;
    const int32_t* table;  // [B][max_pages]
    int max_pages;
};

// Element offset of cached token j of sequence b (head 0), or -1 when the table has no page
// of the pool there.  0 <= j < max_pages * page.
CSA_DEV int64_t paged_row(const PagedPool& pl, int b, int j)
{
    const int p = (int)((unsigned)j / (unsigned)pl.page);
    const int64_t id = pl.table[(int64_t)b * pl.max_pages + p];
    if ((uint64_t)id >= (uint64_t)pl.n_pages) return -1;
    return id * pl.ld_page + (int64_t)(j - p * pl.page) * pl.ld_row;
}

struct PagedAttnArgs {
    const void *q, *K, *V;
    PagedPool pl;
    const int64_t* t;      // [B][nq]
    int B, nq, n_h, n_kv, d;
    int G;                 // query heads per key head
    int n_win, n_sink;     // n_win = 0: every token up to t
    int cap;               // max_pages * page
    float scale_log2;      // softmax scale * log2(e)
    void* out;
    int out_bf16;
    float* lse;            // [B][nq][n_h] or null
    // Packed rows of one (sequence, key head): row i * G + g is head g of query i.  They are
    // cut into tiles of R rows; an entry e = b * n_tiles + tile and a key head make one item.
    int R, n_tiles;
    int unit;              // cached tokens of a schedule unit
    int min_units;         // places a run has at least
    int item_units;        // what an item costs beside its units, in units
    int runs;              // runs of the schedule
    int heads;             // lists of runs: worker w has run w / heads (prompt and CUDA-core kernels: one list, a worker
                           // is a CTA; decode kernels: a list for each key head, a worker is a group of warps)
    int per_cta;           // decode kernels: workers of a CTA
    long long wait_budget; // clocks, of the prompt kernel's waits
    // workspace
    uint32_t* status;      // 1 after a timeout
    int4* desc;            // [workers]: the split item that begins in this worker's run {entry, head, runs that have a
                           // part of it, 1 after a timeout}, entry -1: none
    float* part_o;         // [2 * workers][R][d] unnormalised partial outputs
    float2* part_ml;       // [2 * workers][R] their (running maximum, sum), base 2
    // accumulated weights: scaled base-2 logits [B][n_kv][nq * G][cap] and the final base-2
    // log-sum-exp [B][n_kv][nq * G], both in the workspace; null: none asked for
    float* logits;
    float* lse2;
    const float* acc;
    float* acc_out;
    bool may_have_holes() const { return n_win > 0 && nq > 1; }
};

// Tokens [0, sink) and [lo, hi) are visible to query i of sequence b, sink <= lo <= hi (empty: hi = 0).
struct RowBounds { int lo, hi, sink; };
CSA_DEV RowBounds paged_bounds_at(const PagedAttnArgs& a, int64_t t)
{
    RowBounds r;
    r.hi = t < 0 ? 0 : t >= a.cap ? a.cap : (int)t + 1;
    r.lo = a.n_win > 0 ? (int)min(max(t - a.n_win + 1, (int64_t)0), (int64_t)r.hi) : 0;
    r.sink = min(a.n_sink, r.lo);
    return r;
}
CSA_DEV RowBounds paged_bounds(const PagedAttnArgs& a, int b, int i)
{
    return paged_bounds_at(a, a.t[(int64_t)b * a.nq + i]);
}
CSA_DEV bool paged_visible(const RowBounds& r, int j) { return j < r.hi && (j >= r.lo || j < r.sink); }

// What an entry reads: units [0, s1) and [w0, ...), n units in all.  Every row of the entry sees all
// of [lo_max, hi_min); none sees a token outside [0, sink) and [lo_min, hi_max).
struct PagedEntry {
    int b, tile;
    int s1, w0, n;
    int lo_max, hi_min;
    int lo_min, hi_max, sink;
    CSA_DEV int first_token(int u, int unit) const { return (u < s1 ? u : u - s1 + w0) * unit; }
};

// Queries whose windows lie apart leave holes in [lo_min, hi_max): tokens that no row of the entry sees.  There is none if
// the queries that are not padding follow one another in steps of up to n_win, rising or falling; else there may be
// (`apart`: begins of such a sequence, and two for a larger step).  LANES as in paged_entry.  Only kernels of calls with a
// window and several queries (PagedAttnArgs::may_have_holes) have code for them, 2 to 5% of their time (8192 queries through
// a window of 2048: 328 -> 334 us; 2 a sequence of 32, window 1024: 45 -> 46); in all kernels it cost the others up to 7%.
template <int LANES>
CSA_DEV bool paged_holes(const PagedAttnArgs& a, const PagedEntry& e)
{
    const int row0 = e.tile * a.R, i0 = row0 / a.G, i1 = (min(row0 + a.R, a.nq * a.G) - 1) / a.G;
    const int64_t* ts = a.t + (int64_t)e.b * a.nq;
    const int64_t far = (int64_t)a.cap + a.n_win;  // past it one t is as good as another
    int apart = 0;
#pragma unroll 1
    for (int i = i0 + (LANES > 1 ? (int)(threadIdx.x & (LANES - 1)) : 0); i <= i1; i += LANES) {
        const int64_t t = min(ts[i], far), before = i > i0 ? min(ts[i - 1], far) : -1;
        if (t >= 0) apart += before < 0 ? 1 : t - before > a.n_win || before - t > a.n_win ? 2 : 0;
    }
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) apart += __shfl_xor_sync(0xffffffffu, apart, o);
    return apart > 1;
}

// Does some row of the entry see token j?  The K and V rows of a token that none sees may hold anything, and a weight of 0
// does not keep a NaN out of a product: they are not read, or set to zero before.
CSA_DEV bool paged_seen(const PagedAttnArgs& a, const PagedEntry& e, bool holes, int j)
{
    if (j >= e.hi_max || (j < e.lo_min && j >= e.sink)) return false;
    if (!holes || j < e.sink) return true;
    const int row0 = e.tile * a.R, i1 = (min(row0 + a.R, a.nq * a.G) - 1) / a.G;
    const int64_t* ts = a.t + (int64_t)e.b * a.nq;
#pragma unroll 1
    for (int i = row0 / a.G; i <= i1; ++i) {
        const int64_t t = ts[i];
        if (j <= t && j > t - a.n_win) return true;
    }
    return false;
}

// LANES neighbouring lanes of a converged warp share the queries of the entry (a tile of many); 1: the
// calling thread reads them all.  Bounds rise with t, so an entry's follow from its smallest and
// largest t.
template <int LANES>
CSA_DEV PagedEntry paged_entry(const PagedAttnArgs& a, int e)
{
    PagedEntry r;
    r.b = e / a.n_tiles;
    r.tile = e - r.b * a.n_tiles;
    const int row0 = r.tile * a.R, row1 = min(row0 + a.R, a.nq * a.G) - 1;
    const int i0 = row0 / a.G, i1 = row1 / a.G;
    const int64_t* ts = a.t + (int64_t)r.b * a.nq;
    constexpr int kAhead = LANES > 1 ? 8 : 1;  // loads under way at once
    // t + 1 in 32 bits, 0 for padding: past the last window that reaches the cache one t is as good as another
    const int64_t far = (int64_t)a.cap + a.n_win;
    uint32_t t_min = UINT32_MAX, t_max = 0, t_seen = UINT32_MAX;  // t_seen: the smallest t >= 0
    for (int i = i0 + (LANES > 1 ? (int)(threadIdx.x & (LANES - 1)) : 0); i <= i1; i += LANES * kAhead) {
        int64_t t[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) t[k] = ts[min(i + k * LANES, i1)];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const uint32_t x = t[k] < 0 ? 0u : (uint32_t)min(t[k], far) + 1;
            t_min = min(t_min, x);
            t_max = max(t_max, x);
            t_seen = min(t_seen, x - 1);  // padding: the largest
        }
    }
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) {
        t_min = min(t_min, __shfl_xor_sync(0xffffffffu, t_min, o));
        t_max = max(t_max, __shfl_xor_sync(0xffffffffu, t_max, o));
        t_seen = min(t_seen, __shfl_xor_sync(0xffffffffu, t_seen, o));
    }
    const RowBounds from = paged_bounds_at(a, (int64_t)t_min - 1), to = paged_bounds_at(a, (int64_t)t_max - 1);
    r.lo_max = to.lo;
    r.hi_min = from.hi;
    r.lo_min = t_max > 0 ? paged_bounds_at(a, t_seen).lo : INT32_MAX;
    r.hi_max = to.hi;
    r.sink = to.sink;
    r.w0 = r.hi_max > 0 ? r.lo_min / a.unit : 0;
    r.s1 = (r.sink + a.unit - 1) / a.unit;
    if (r.s1 >= r.w0) r.s1 = r.w0 = 0;  // the first tokens reach the window: one range from 0
    // a row tile that sees nothing still takes one (masked) unit: its outputs are written there
    r.n = max(1, r.s1 + (r.hi_max + a.unit - 1) / a.unit - r.w0);
    return r;
}

// The schedule.  The units of all items, in the order (entry, key head, unit), are one list
// that is cut into equal runs, whatever the sequences' lengths: a ragged batch and one long sequence both
// fill the GPU.  (Decode kernels have a list (entry, unit) of each key head, cut alike, so that the heads of a
// token, which lie together in a [row][head] page, are read at about one time.)  An item begins with
// item_units places that hold no unit: what it costs to begin and end one, so that a run of many short items
// (the first rows of a prompt) is no longer than one of few long ones.  Only the first and the last item of a
// run can be cut, so a run writes at most two partial results; paged_attn_combine joins them in
// the order of the runs.  The lengths are read on the device, so a captured graph follows them.
struct PagedCursor {
    int64_t at, end;       // this run of the list
    int64_t W;
    int runs;              // that are not empty
    int e, h, u;           // entry, key head and place within the item of `at`
    PagedEntry en;
};

// Shared memory of paged_schedule.
template <int T, int LANES>
struct PagedScratch {
    int64_t sums[T / 32];
    int64_t upto[T];
    int places[LANES > 1 ? T : 1];
};

// Places of entry base + tid in the list of a key head (0 past the last entry).  All T threads.
template <int T, int LANES>
CSA_DEV int paged_places(const PagedAttnArgs& a, int base, int NB, PagedScratch<T, LANES>& sc)
{
    const int tid = threadIdx.x;
    if (LANES == 1) return base + tid < NB ? paged_entry<1>(a, base + tid).n + a.item_units : 0;
    __syncthreads();
    const int n = min(T, NB - base);
    for (int k0 = 0; k0 < n; k0 += T / LANES) {  // whole warps: the last ones repeat the last entry
        const int k = k0 + tid / LANES;
        const int m = paged_entry<LANES>(a, base + min(k, n - 1)).n + a.item_units;
        if (k < n && tid % LANES == 0) sc.places[k] = m;
    }
    __syncthreads();
    return tid < n ? sc.places[tid] : 0;
}

CSA_DEV PagedEntry shfl_entry(const PagedEntry& e, int lane)
{
    PagedEntry r;
    auto get = [&](int x) { return __shfl_sync(0xffffffffu, x, lane); };
    r.b = get(e.b); r.tile = get(e.tile);
    r.s1 = get(e.s1); r.w0 = get(e.w0); r.n = get(e.n);
    r.lo_max = get(e.lo_max); r.hi_min = get(e.hi_min);
    r.lo_min = get(e.lo_min); r.hi_max = get(e.hi_max); r.sink = get(e.sink);
    return r;
}

// The run's first item from its place in the list; `start`: places of a key head before entry c.e.
CSA_DEV void paged_locate(const PagedAttnArgs& a, PagedCursor& c, int64_t start, int H)
{
    const int64_t off = c.at - start * H;
    const int places = c.en.n + a.item_units;
    c.h = (int)(off / places);
    c.u = (int)(off - (int64_t)c.h * places);
}

// paged_schedule with a run for each warp, 32 entries at most: each warp has them in its lanes and waits for no
// other (17 sequences of up to 289 tokens, width 256: 17.4 -> 16.3 us).
CSA_DEV bool paged_schedule_few(const PagedAttnArgs& a, int run, PagedCursor& c)
{
    const int lane = threadIdx.x & 31, NB = a.B * a.n_tiles;
    const PagedEntry en = paged_entry<1>(a, min(lane, NB - 1));
    const int n = lane < NB ? en.n + a.item_units : 0;
    int64_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    c.W = __shfl_sync(0xffffffffu, inc, 31);
    c.runs = (int)max((int64_t)1, min((int64_t)a.runs, c.W / a.min_units));
    if (run >= c.runs) return false;
    c.at = run * c.W / c.runs;
    c.end = (run + 1) * c.W / c.runs;
    c.e = __ffs(__ballot_sync(0xffffffffu, c.at < inc)) - 1;
    c.en = shfl_entry(en, c.e);
    paged_locate(a, c, __shfl_sync(0xffffffffu, inc - n, c.e), 1);
    return true;
}

// T threads call it together, each with the run of its warp (PER_WARP) or of the CTA.  False: that run is empty.
template <int T, int LANES, bool PER_WARP>
CSA_DEV bool paged_schedule(const PagedAttnArgs& a, int run, PagedScratch<T, LANES>& sc, PagedCursor& c)
{
    int64_t* sh = sc.sums;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int NB = a.B * a.n_tiles, H = PER_WARP ? 1 : a.n_kv;  // heads in a list
    if (PER_WARP && NB <= 32) return paged_schedule_few(a, run, c);
    int64_t sum = 0;
    int n0 = 0;
    for (int base = 0; base < NB; base += T) {
        const int n = paged_places<T, LANES>(a, base, NB, sc);
        if (base == 0) n0 = n;
        sum += n;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sh[warp] = sum;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) total += sh[w];
    c.W = total * H;
    c.runs = (int)max((int64_t)1, min((int64_t)a.runs, c.W / a.min_units));
    const bool some = run < c.runs;
    if (!PER_WARP && !some) return false;
    c.at = run * c.W / c.runs;
    c.end = (run + 1) * c.W / c.runs;
    int64_t before = 0, start = 0;  // places (of one key head) before the block of T entries, and before entry c.e
    c.e = -1;
    for (int base = 0; base < NB; base += T) {
        const int n = base == 0 ? n0 : paged_places<T, LANES>(a, base, NB, sc);
        int64_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        __syncthreads();
        if (lane == 31) sh[warp] = inc;
        sc.upto[tid] = inc;  // places of the warp's entries up to and with this one
        __syncthreads();
        for (int w = 0; w < T / 32 && c.e < 0; ++w) {
            // each warp looks for its own run's start
            if (c.at < (before + sh[w]) * H) {
                const int64_t to = before + sc.upto[w * 32 + lane];
                const int k = __ffs(__ballot_sync(0xffffffffu, c.at < to * H)) - 1;
                c.e = base + w * 32 + k;
                start = k > 0 ? __shfl_sync(0xffffffffu, to, k - 1) : before;
            }
            before += sh[w];
        }
        if (!PER_WARP && c.e >= 0) break;  // alike in all threads; else every warp stays to the end
    }
    __syncthreads();  // sc may be reused
    if (!some) return false;
    c.en = paged_entry<(LANES > 1 ? 32 : 1)>(a, c.e);
    paged_locate(a, c, start, H);
    return true;
}

// The part of the current item that this run has, and where its result goes.
struct PagedSegment {
    int places;
    int u0, u1;  // units; empty where the run ends before the item's first unit
    bool whole;
    int slot;    // of a partial result
};
CSA_DEV PagedSegment paged_segment(const PagedAttnArgs& a, const PagedCursor& c, int worker)
{
    PagedSegment s;
    const int all = c.en.n + a.item_units, p1 = (int)min((int64_t)all, c.u + (c.end - c.at));
    s.places = p1 - c.u;
    s.u0 = max(0, c.u - a.item_units);
    s.u1 = max(0, p1 - a.item_units);
    s.whole = s.u0 == 0 && s.u1 == c.en.n;
    s.slot = 2 * worker + (s.u0 == 0 ? 1 : 0);
    return s;
}
// The combine's description of an item whose first units, but not its last, are this worker's.  One thread.
CSA_DEV void paged_describe(const PagedAttnArgs& a, const PagedCursor& c, const PagedSegment& s, int worker)
{
    if (s.whole || s.u0 > 0 || s.u1 == 0) return;
    // the run that has the item's last unit: place x lies in run ((x + 1) runs - 1) / W
    const int64_t last = c.at - c.u + c.en.n + a.item_units - 1;
    a.desc[worker] = make_int4(c.e, c.h, (int)(((last + 1) * c.runs - 1) / c.W) - worker / a.heads + 1, 0);
}
// On to the next item; false at the end of the run.  PER_WARP: of the same key head.
template <int LANES, bool PER_WARP>
CSA_DEV bool paged_next(const PagedAttnArgs& a, PagedCursor& c, const PagedSegment& s)
{
    c.at += s.places;
    if (c.at >= c.end) return false;
    c.u = 0;
    if (PER_WARP || ++c.h == a.n_kv) {
        if (!PER_WARP) c.h = 0;
        c.en = paged_entry<LANES>(a, ++c.e);
    }
    return true;
}

// out / lse element of packed row r of tile `tile`: index of the (query, head) pair, or -1.
CSA_DEV int64_t paged_out_row(const PagedAttnArgs& a, int b, int tile, int h, int r)
{
    const int row = tile * a.R + r;
    if (row >= a.nq * a.G) return -1;
    const int i = row / a.G;
    return ((int64_t)b * a.nq + i) * a.n_h + h * a.G + (row - i * a.G);
}

CSA_DEV uint32_t pack2(float x, float y)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Stores of one result: element `at` of out, and a row's log-sum-exp (natural for the caller,
// base 2 for the accumulated weights) from its running maximum and sum.
CSA_DEV void paged_store(const PagedAttnArgs& a, int64_t at, float v)
{
    if (a.out_bf16)
        static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(a.out)[at] = v;
}
CSA_DEV void paged_store_lse(const PagedAttnArgs& a, int64_t o, int b, int tile, int h, int r, float m, float l)
{
    const float z = l == 0.f ? -INFINITY : m + log2f(l);  // a NaN stays one
    if (a.lse) a.lse[o] = z * 0.6931471805599453f;
    if (a.lse2) a.lse2[((int64_t)b * a.n_kv + h) * (a.nq * a.G) + tile * a.R + r] = z;
}

// A piece in which a row saw nothing, or logits of -inf alone.  One of NaN logits has the maximum -inf too (maxima pass a
// NaN over), but a sum that is NaN, and the joins keep it.
CSA_DEV bool paged_empty(float m, float l) { return m == -INFINITY && l == 0.f; }

// Rows of tile `tile` that are rows of the call.
CSA_DEV int paged_rows(const PagedAttnArgs& a, int tile) { return min(a.R, a.nq * a.G - tile * a.R); }

// The end of a segment: so [NW][R][ld] and sm_m, sm_l [NW][R] hold the warps' results.  Joins them
// and writes the item's output, or a partial result for paged_attn_combine.  All T threads.
template <int T, int NW, int R>
CSA_DEV void paged_finish_segment(const PagedAttnArgs& a, const PagedCursor& c, const PagedSegment& sg, const float* so,
                                  int ld, const float* sm_m, const float* sm_l)
{
    const int n = paged_rows(a, c.en.tile) * a.d;
    for (int x = threadIdx.x; x < n; x += T) {
        const int r = x / a.d, col = x - r * a.d;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, sm_m[w * R + r]);
        float L = 0.f, v = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float m = sm_m[w * R + r], l = sm_l[w * R + r];
            if (paged_empty(m, l)) continue;
            const float f = exp2f(m - M);
            L = fmaf(f, l, L);
            v = fmaf(f, so[(w * R + r) * ld + col], v);
        }
        if (sg.whole) {
            const int64_t o = paged_out_row(a, c.en.b, c.en.tile, c.h, r);
            paged_store(a, o * a.d + col, L == 0.f ? 0.f : v / L);
            if (col == 0) paged_store_lse(a, o, c.en.b, c.en.tile, c.h, r, M, L);
        } else {
            const int64_t at = (int64_t)sg.slot * R + r;
            a.part_o[at * a.d + col] = v;
            if (col == 0) a.part_ml[at] = make_float2(M, L);
        }
    }
}

// Which kernel a call runs on, its row tile, and the units and CTAs of its schedule.
enum PagedKind { kPagedSimt, kPagedFew, kPagedMma, kPagedF32, kPagedPrompt };
struct PagedShape {
    PagedKind kind;
    int DP;         // head width rounded up to a kernel's
    int WR;         // kPagedMma: row groups of 16; kPagedF32: rows
    int R, unit, min_units, item_units;
    int workers;    // of a full GPU
    bool by_head;   // a list of runs for each key head
};
// Runs of each of `lists` lists: what fills the GPU, and no more than the capacity has use for.
inline int paged_runs(const PagedShape& s, int64_t lists, int64_t places)
{
    int64_t n = s.workers / lists;
    if (places / s.min_units < n) n = places / s.min_units;
    return n < 1 ? 1 : (int)n;
}
PagedShape paged_decode_shape(int dtype, int rows, int d);
int launch_paged_decode(const PagedAttnArgs& a, const PagedShape& s, cudaStream_t stream);

// Lets a kernel have `smem` bytes of dynamic shared memory, once on each device (the call costs as much as a tenth of
// a decode step's host time).
template <auto kKernel>
inline bool paged_allow_smem(int smem)
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return true;
    if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return true;
}

bool paged_prompt_takes(const PagedPool& pl, int n_kv, int d);
PagedShape paged_prompt_shape(int d);
int launch_paged_prompt(const PagedAttnArgs& a, const PagedShape& s, cudaStream_t stream);

}  // namespace csa
