// paged_attn: grouped-query attention over the paged cache.  Host path, the CUDA-core kernel
// (any head width and layout), the join of partial results and the accumulated weights.
//
// For query i of sequence b at cache position t, query head x and its key head h = x / G:
//   s_j = scale * q . K_j            over the visible tokens j (paged_bounds)
//   o   = sum_j exp(s_j - lse) V_j,  lse = log sum_j exp(s_j)
// in one pass over K and V with a running maximum and sum (base 2, fp32).
#include <algorithm>

#include "paged.cuh"
#include "tc_utils.cuh"

namespace csa {

int paged_pool_check(const PagedPool& pl, int B, int n_kv, int d);

namespace {

constexpr int kSimtThreads = 128;
constexpr int kSimtWarps = kSimtThreads / 32;
constexpr int kSimtRows = 8;
constexpr int kSimtUnit = 32;  // cached tokens of a schedule unit: one for each lane

// The plain kernel.  A warp takes a unit of 32 cached tokens: lane = token for the logits, lane =
// column for the products with V.  Element-wise loads, so every layout is right; the tensor-core
// kernel takes the layouts that it can load 16 bytes at a time.
template <typename T>
__global__ void __launch_bounds__(kSimtThreads) paged_attn_simt(PagedAttnArgs a)
{
    constexpr int R = kSimtRows, U = kSimtUnit, NC = kPagedMaxD / 32;
    extern __shared__ float smem[];
    __shared__ PagedScratch<kSimtThreads, 1> sh;
    __shared__ float sm_m[kSimtWarps][R], sm_l[kSimtWarps][R];
    const int d = a.d, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    float* sq = smem;                      // [R][d]
    float* sp = sq + R * d + warp * U * R; // [U][R] of this warp
    float* so = sq + R * d;                // [warps][R][d] at the end of a segment (over sp)
    pdl_launch_dependents();
    pdl_wait();
    if (tid == 0) a.desc[cta] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    PagedCursor c;
    if (!paged_schedule<kSimtThreads, 1, false>(a, cta, sh, c)) return;
    const T* K = static_cast<const T*>(a.K);
    const T* V = static_cast<const T*>(a.V);
    while (true) {
        const PagedSegment sg = paged_segment(a, c, cta);
        if (sg.u0 == sg.u1) break;  // the run ends before the item's first unit
        if (tid == 0) paged_describe(a, c, sg, cta);
        const PagedEntry en = c.en;
        for (int x = tid; x < R * d; x += kSimtThreads) {
            const int64_t o = paged_out_row(a, en.b, en.tile, c.h, x / d);
            sq[x] = o < 0 ? 0.f : to_f32(static_cast<const T*>(a.q)[o * d + x % d]);
        }
        __syncthreads();
        float m[R], l[R], acc[R][NC];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i) acc[r][i] = 0.f;
        }
        for (int u = sg.u0 + warp; u < sg.u1; u += kSimtWarps) {
            const int j = en.first_token(u, U) + lane;
            int64_t off = j < a.cap ? paged_row(a.pl, en.b, j) : -1;
            float s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = 0.f;
            if (off >= 0) {
                off += c.h * a.pl.ld_head;
                for (int x = 0; x < d; ++x) {
                    const float k = to_f32(K[off + x]);
#pragma unroll
                    for (int r = 0; r < R; ++r) s[r] = fmaf(sq[r * d + x], k, s[r]);
                }
            }
            bool any = false;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = en.tile * R + r;
                const bool vis = off >= 0 && row < a.nq * a.G &&
                                 paged_visible(paged_bounds(a, en.b, row / a.G), j);
                any |= vis;
                s[r] = vis ? s[r] * a.scale_log2 : -INFINITY;
                if (a.logits && j < a.cap && row < a.nq * a.G)
                    a.logits[(((int64_t)en.b * a.n_kv + c.h) * (a.nq * a.G) + row) * a.cap + j] = s[r];
                float top = s[r];
#pragma unroll
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float mn = fmaxf(m[r], top);
                const float shrink = mn == -INFINITY ? 1.f : exp2f(m[r] - mn);
                // logits of -inf alone leave mn there, and weigh nothing
                const float p = vis ? exp2f(s[r] - (mn == -INFINITY ? 0.f : mn)) : 0.f;
                m[r] = mn;
                l[r] = l[r] * shrink + p;
#pragma unroll
                for (int i = 0; i < NC; ++i) acc[r][i] *= shrink;
                sp[lane * R + r] = p;
            }
            const unsigned live = __ballot_sync(0xffffffffu, any);
            __syncwarp();
            for (int kk = 0; kk < U; ++kk) {
                const int64_t o = __shfl_sync(0xffffffffu, off, kk);
                if (!(live >> kk & 1)) continue;  // a row that nothing sees is not read: it may hold anything
                float p[R];
#pragma unroll
                for (int r = 0; r < R; ++r) p[r] = sp[kk * R + r];
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int x = lane + 32 * i;
                    if (x < d) {
                        const float v = to_f32(V[o + x]);
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            if (p[r] != 0.f) acc[r][i] = fmaf(p[r], v, acc[r][i]);
                    }
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int o = 16; o; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
            if (lane == 0) {
                sm_m[warp][r] = m[r];
                sm_l[warp][r] = l[r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (lane + 32 * i < d) so[(warp * R + r) * d + lane + 32 * i] = acc[r][i];
        }
        __syncthreads();
        paged_finish_segment<kSimtThreads, kSimtWarps, R>(a, c, sg, so, d, &sm_m[0][0], &sm_l[0][0]);
        __syncthreads();
        if (!paged_next<1, false>(a, c, sg)) break;
    }
}

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

// Pieces p0, p0 + step, ... of a row, four under way at once: their running maximum, sum and weighted sum.
// slot(p): where piece p lies.
template <int NC, typename F>
CSA_DEV void join_pieces(const PagedAttnArgs& a, F slot, int p0, int step, int np, float& M, float& L, float (&acc)[NC])
{
    constexpr int kAhead = 4;
    const int lane = threadIdx.x & 31;
    M = -INFINITY;
    L = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) acc[i] = 0.f;
    for (; p0 < np; p0 += step * kAhead) {
        float2 ml[kAhead];
        float v[kAhead][NC];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t at = slot(min(p0 + k * step, np - 1));
            ml[k] = a.part_ml[at];
#pragma unroll
            for (int i = 0; i < NC; ++i) v[k][i] = lane + 32 * i < a.d ? a.part_o[at * a.d + lane + 32 * i] : 0.f;
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (p0 + k * step < np) top = fmaxf(top, ml[k].x);
        const float f = top == M ? 1.f : exp2f(M - top);
        M = top;
        L *= f;
#pragma unroll
        for (int i = 0; i < NC; ++i) acc[i] *= f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (p0 + k * step >= np || paged_empty(ml[k].x, ml[k].y)) continue;
            const float w = exp2f(ml[k].x - M);  // a piece far below the others may still hold a NaN
            L = fmaf(w, ml[k].y, L);
#pragma unroll
            for (int i = 0; i < NC; ++i) acc[i] = fmaf(w, v[k][i], acc[i]);
        }
    }
}

// Joins the partial results of the runs that had a part of an item.  A CTA looks at 32 descriptions together (most
// workers describe none).  An item of few pieces has a warp for each row; one of many (a long sequence of a
// small batch) the whole CTA.  NC: columns of a lane.
template <int NC>
__global__ void __launch_bounds__(kJoinThreads) paged_attn_combine(PagedAttnArgs a)
{
    constexpr int kMany = 16;  // pieces that a warp takes by itself: four rounds
    __shared__ float2 sh[kJoinWarps];  // of a warp's pieces: maximum and sum
    __shared__ float so[kJoinWarps][NC * 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, workers = a.runs * a.heads;
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) {
        int late = 0;
#pragma unroll 4
        for (int i = tid; i < workers; i += kJoinThreads) late |= a.desc[i].w;
        late = __syncthreads_or(late);
        if (tid == 0) *a.status = late ? 1u : 0u;
    }
    for (int base = blockIdx.x; base < workers; base += 32 * gridDim.x) {
        const int mine = base + lane * gridDim.x;
        const int4 ds = mine < workers ? a.desc[mine] : make_int4(-1, 0, 0, 0);
        const unsigned many = __ballot_sync(0xffffffffu, ds.x >= 0 && ds.z > kMany);
        const unsigned few = __ballot_sync(0xffffffffu, ds.x >= 0 && ds.z <= kMany);
        int c0, b, tile, h, np;
        auto item = [&](int k) {
            c0 = base + k * gridDim.x;
            const int entry = __shfl_sync(0xffffffffu, ds.x, k);
            h = __shfl_sync(0xffffffffu, ds.y, k);
            np = __shfl_sync(0xffffffffu, ds.z, k);
            b = entry / a.n_tiles;
            tile = entry - b * a.n_tiles;
        };
        // piece p lies in slot 2 c0 + 1 for p = 0, 2 (c0 + p heads) after that
        int r;
        auto slot = [&](int p) { return (int64_t)(p == 0 ? 2 * c0 + 1 : 2 * (c0 + p * a.heads)) * a.R + r; };
        float M, L, acc[NC];
        auto store = [&] {
            const int64_t o = paged_out_row(a, b, tile, h, r);
            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (lane + 32 * i < a.d) paged_store(a, o * a.d + lane + 32 * i, acc[i] * inv);
            if (lane == 0) paged_store_lse(a, o, b, tile, h, r, M, L);
        };
        for (unsigned todo = many; todo; todo &= todo - 1) {
            item(__ffs(todo) - 1);
            for (r = blockIdx.y; r < paged_rows(a, tile); r += gridDim.y) {
                join_pieces<NC>(a, slot, warp, kJoinWarps, np, M, L, acc);
                __syncthreads();  // the row before
                if (lane == 0) sh[warp] = make_float2(M, L);
#pragma unroll
                for (int i = 0; i < NC; ++i) so[warp][lane + 32 * i] = acc[i];
                __syncthreads();
                if (warp > 0) continue;
                float2 ml = lane < kJoinWarps ? sh[lane] : make_float2(-INFINITY, 0.f);
                M = ml.x;
#pragma unroll
                for (int x = kJoinWarps / 2; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
                M = __shfl_sync(0xffffffffu, M, 0);
                const float f = exp2f(ml.x - M);
                const unsigned some = __ballot_sync(0xffffffffu, !paged_empty(ml.x, ml.y));
                L = 0.f;
#pragma unroll
                for (int i = 0; i < NC; ++i) acc[i] = 0.f;
#pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) {
                    const float fw = __shfl_sync(0xffffffffu, f, w);
                    if (!(some >> w & 1)) continue;
                    L = fmaf(fw, sh[w].y, L);
#pragma unroll
                    for (int i = 0; i < NC; ++i) acc[i] = fmaf(fw, so[w][lane + 32 * i], acc[i]);
                }
                store();
            }
        }
        // rows of the other items: task t of all of theirs goes to warp t of the CTAs of this column
        int t = blockIdx.y * kJoinWarps + warp;
        for (unsigned todo = few; todo; todo &= todo - 1) {
            item(__ffs(todo) - 1);
            for (; t < paged_rows(a, tile); t += gridDim.y * kJoinWarps) {
                r = t;
                join_pieces<NC>(a, slot, 0, 1, np, M, L, acc);
                store();
            }
            t -= paged_rows(a, tile);
        }
    }
}

constexpr int kWeightThreads = 256;
constexpr int kWeightRows = 1024;  // rows whose log-sum-exp is held at a time

// acc_out[b][h][j] = acc[b][h][j] + the sum over the key head's queries of exp(s_j - lse), from the
// logits that the attention kernel left: a thread has V neighbouring tokens and all rows in order, so the sum has
// one order.  Reads 4 bytes a (token, row), mostly from L2; bound by the launch and those reads.
template <int V>
__global__ void __launch_bounds__(kWeightThreads) paged_weights_kernel(PagedAttnArgs a)
{
    __shared__ float z[kWeightRows];
    const int tid = threadIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int j = (blockIdx.x * kWeightThreads + tid) * V;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t g = (int64_t)b * a.n_kv + h, at = g * a.cap + j;
    const int rows = a.nq * a.G, step = max(1, kWeightRows / a.G);  // queries at a time
    float w[V] = {};
    for (int i0 = 0; i0 < a.nq; i0 += step) {
        const int i1 = min(a.nq, i0 + step);
        // held in parts where one query has more rows than that
        for (int g0 = 0; g0 < a.G; g0 += kWeightRows) {
            const int gn = min(kWeightRows, a.G - g0), r0 = i0 * a.G + g0, n = step > 1 ? (i1 - i0) * a.G : gn;
            __syncthreads();
            for (int r = tid; r < n; r += kWeightThreads) {
                // a row that sees nothing has lse = -inf: its logits, all -inf, weigh nothing
                const float x = a.lse2[g * rows + r0 + r];
                z[r] = x == -INFINITY ? INFINITY : x;
            }
            __syncthreads();
            if (j >= a.cap) continue;
            for (int i = i0; i < i1; ++i) {
                const RowBounds rb = paged_bounds(a, b, i);
                bool see[V], any = false;
#pragma unroll
                for (int x = 0; x < V; ++x) any |= see[x] = paged_visible(rb, j + x);
                if (!any) continue;  // logits that were never written
                const float* s = a.logits + (g * rows + i * a.G + g0) * a.cap + j;
#pragma unroll 8
                for (int r = 0; r < gn; ++r) {
                    float x[V];
                    if constexpr (V == 4) {
                        const float4 y = __ldcs(reinterpret_cast<const float4*>(s + (int64_t)r * a.cap));
                        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
                    } else {
                        x[0] = s[(int64_t)r * a.cap];
                    }
                    const float zr = z[(i - i0) * a.G + r];
#pragma unroll
                    for (int k = 0; k < V; ++k) w[k] += see[k] ? tc::ex2_approx(x[k] - zr) : 0.f;
                }
            }
        }
    }
    if (j >= a.cap) return;
#pragma unroll
    for (int i = 0; i < V; ++i) a.acc_out[at + i] = a.acc[at + i] + w[i];
}

}  // namespace

// The kernel of a call, by its rows (queries x heads of a key head), type and layout.  `wide`: every
// row can be loaded 16 bytes at a time; what cannot takes the CUDA-core kernel.  `boxes`: the pools can be
// read by TMA.  A tile of 128 rows costs the prompt kernel the same however few of them there are.  d = 128, pages of 16,
// prompt kernel against decode kernel: 16 sequences of 8K tokens, 24 rows of 8 key heads 117 and 117 us, 32 of 2 key
// heads 49 and 50, 64 50 and 71, 128 53 and 121; 24 rows of 64 sequences of 500 67 and 58, of one of 8K 26 and 23.
constexpr int kPromptRows = 33;
static PagedShape paged_shape(int dtype, bool wide, bool boxes, int rows, int d)
{
    if (wide && boxes && dtype == CSA_BF16 && rows >= kPromptRows && d <= 128) return paged_prompt_shape(d);
    if (wide) return paged_decode_shape(dtype, rows, d);
    PagedShape s{};
    s.kind = kPagedSimt;
    s.R = kSimtRows;
    s.unit = kSimtUnit;
    s.min_units = kSimtWarps;
    s.item_units = 2;
    s.workers = 2 * kNumSMs;
    return s;
}

// Places of a list of the schedule, at most.
static int64_t paged_places(const PagedShape& s, int B, int nq, int G, int n_kv, int64_t cap)
{
    const int64_t tiles = ((int64_t)nq * G + s.R - 1) / s.R;
    return (std::max<int64_t>(1, (cap + s.unit - 1) / s.unit) + s.item_units) * B * tiles * (s.by_head ? 1 : n_kv);
}

// A budget that the test hook set; negative: the one of every other device wait.
static std::atomic<int64_t> g_wait_budget{-1};

// Workspace layout, from the sizes alone: room for every kernel that a call of these sizes may run on.
struct PagedPlan {
    size_t part_o, part_ml, logits, lse2, bytes;  // offsets; before them the 256-byte status block and desc
};

static PagedPlan paged_plan(int B, int nq, int G, int n_kv, int d, int64_t cap, bool weights)
{
    PagedPlan p{};
    size_t slots = 0, workers = 0;  // rows of partial results, descriptions
    for (int dtype : {CSA_BF16, CSA_F32})
        for (int way = 0; way < 3; ++way) {
            const PagedShape s = paged_shape(dtype, way > 0, way > 1, nq * G, d);
            const size_t lists = s.by_head ? n_kv : 1, runs = paged_runs(s, lists, paged_places(s, B, nq, G, n_kv, cap));
            workers = std::max(workers, runs * lists);
            if (runs > 1) slots = std::max(slots, 2 * runs * lists * s.R);  // a single run cuts nothing
        }
    size_t at = 256 + align_up(sizeof(int4) * workers, 256);
    p.part_ml = at;
    at += align_up(slots * sizeof(float2), 256);
    p.part_o = at;
    at += align_up(slots * d * sizeof(float), 256);
    if (weights) {
        const size_t rows = (size_t)B * n_kv * nq * G;
        p.lse2 = at;
        at += align_up(rows * sizeof(float), 256);
        p.logits = at;
        at += align_up(rows * (size_t)cap * sizeof(float), 256);
    }
    p.bytes = at;
    return p;
}

}  // namespace csa

extern "C" size_t paged_attn_workspace_size(int B, int nq, int n_h, int n_kv, int d, int64_t cap, int weights)
{
    using namespace csa;
    if (B <= 0 || nq <= 0 || n_h <= 0 || n_kv <= 0 || n_h % n_kv || d <= 0 || d > kPagedMaxD || cap < 0 ||
        cap > INT32_MAX || (int64_t)nq * n_h > INT32_MAX / 2 || (int64_t)B * nq > INT32_MAX / 2)
        return 0;
    return paged_plan(B, nq, n_h / n_kv, n_kv, d, cap, weights != 0).bytes;
}

extern "C" int paged_attn_set_wait_budget(int64_t cycles)
{
    csa::g_wait_budget.store(cycles, std::memory_order_relaxed);
    return CSA_OK;
}

extern "C" int paged_attn(const void* q, const void* K, const void* V, int64_t pool_ld_page, int64_t pool_ld_row,
                          int64_t pool_ld_head, int64_t n_pages, int page, const int32_t* table, int max_pages,
                          const int64_t* t, int B, int nq, int n_h, int n_kv, int d, int n_win, int n_sink, float scale,
                          void* out, float* lse, const float* acc, float* acc_out, void* workspace, size_t ws_bytes,
                          int dtype, int out_bf16, csa_stream_t stream)
{
    using namespace csa;
    if (dtype != CSA_BF16 && dtype != CSA_F32) return CSA_ERR_DTYPE;
    if (out_bf16 && dtype != CSA_BF16) return CSA_ERR_DTYPE;
    if (B < 0 || nq < 0 || n_h <= 0 || n_kv <= 0 || n_h % n_kv || n_win < 0 || n_sink < 0) return CSA_ERR_ARG;
    PagedPool pl{pool_ld_page, pool_ld_row, pool_ld_head, n_pages, page, table, max_pages};
    int st = paged_pool_check(pl, B, n_kv, d);
    if (st != CSA_OK) return st;
    if (d > kPagedMaxD) return CSA_ERR_UNSUPPORTED;
    if (B == 0 || nq == 0) return CSA_OK;
    if ((int64_t)nq * n_h > INT32_MAX / 2 || (int64_t)B * nq > INT32_MAX / 2 || B > 65535 || n_kv > 65535)
        return CSA_ERR_UNSUPPORTED;
    const int64_t cap = (int64_t)max_pages * page;
    if (!q || !out || !t || (cap > 0 && (!K || !V || !table)) || (!acc != !acc_out)) return CSA_ERR_ARG;
    const uintptr_t eb = (uintptr_t)elem_bytes(dtype) - 1;
    if ((((uintptr_t)q | (uintptr_t)K | (uintptr_t)V) & eb) || ((uintptr_t)out & (out_bf16 ? 1 : 3)) ||
        (((uintptr_t)lse | (uintptr_t)acc | (uintptr_t)acc_out | (uintptr_t)table) & 3) || ((uintptr_t)t & 7))
        return CSA_ERR_ALIGN;
    const int G = n_h / n_kv;
    const PagedPlan p = paged_plan(B, nq, G, n_kv, d, cap, acc != nullptr);
    if (!workspace || ws_bytes < p.bytes) return CSA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return CSA_ERR_ALIGN;

    PagedAttnArgs a{};
    a.q = q; a.K = K; a.V = V; a.pl = pl; a.t = t;
    a.B = B; a.nq = nq; a.n_h = n_h; a.n_kv = n_kv; a.d = d; a.G = G;
    a.n_win = n_win; a.n_sink = n_win > 0 ? n_sink : 0; a.cap = (int)cap;
    a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)d)) * kLog2e;
    a.out = out; a.out_bf16 = out_bf16; a.lse = lse;
    // 16-byte loads and stores: every row starts on a 16-byte boundary and is whole 16-byte words
    const int64_t lds = pool_ld_page | pool_ld_row | (n_kv > 1 ? pool_ld_head : 0) | d;
    // (without a capacity the pools may be null: the CUDA-core kernel forms no address from them)
    const bool wide = cap > 0 && aligned16(q) && aligned16(K) && aligned16(V) && aligned16(out) &&
                      lds * elem_bytes(dtype) % 16 == 0;
    const PagedShape sp = paged_shape(dtype, wide, paged_prompt_takes(pl, n_kv, d), nq * G, d);
    a.R = sp.R; a.unit = sp.unit; a.min_units = sp.min_units; a.item_units = sp.item_units;
    a.n_tiles = (nq * G + sp.R - 1) / sp.R;
    a.heads = sp.by_head ? n_kv : 1;
    a.runs = paged_runs(sp, a.heads, paged_places(sp, B, nq, G, n_kv, cap));
    const int64_t budget = g_wait_budget.load(std::memory_order_relaxed);
    a.wait_budget = budget < 0 ? tc::kWaitBudget : budget;
    char* ws = static_cast<char*>(workspace);
    a.status = reinterpret_cast<uint32_t*>(ws);
    a.desc = reinterpret_cast<int4*>(ws + 256);
    a.part_ml = reinterpret_cast<float2*>(ws + p.part_ml);
    a.part_o = reinterpret_cast<float*>(ws + p.part_o);
    if (acc) {
        a.lse2 = reinterpret_cast<float*>(ws + p.lse2);
        a.logits = reinterpret_cast<float*>(ws + p.logits);
        a.acc = acc;
        a.acc_out = acc_out;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (sp.kind == kPagedSimt) {
        const size_t smem =
            ((size_t)a.R * d + std::max<size_t>((size_t)kSimtWarps * a.R * d, kSimtWarps * kSimtUnit * a.R)) * sizeof(float);
        if (dtype == CSA_BF16)
            launch_pdl(paged_attn_simt<__nv_bfloat16>, dim3(a.runs), dim3(kSimtThreads), smem, s, a);
        else
            launch_pdl(paged_attn_simt<float>, dim3(a.runs), dim3(kSimtThreads), smem, s, a);
        st = launch_status();
    } else {
        st = sp.kind == kPagedPrompt ? launch_paged_prompt(a, sp, s) : launch_paged_decode(a, sp, s);
    }
    if (st != CSA_OK) return st;
    // a CTA for each row of a decode call, eight rows of a prompt's tile for each CTA; nothing is cut into a single
    // run, but the status is written
    const int rows = std::min(a.R, nq * G), columns = std::min(a.runs * a.heads, kNumSMs);
    const dim3 grid = a.runs == 1 ? dim3(1) : dim3(columns, std::min(rows, 32));
    if (d <= 128)
        launch_pdl(paged_attn_combine<4>, grid, dim3(kJoinThreads), 0, s, a);
    else
        launch_pdl(paged_attn_combine<8>, grid, dim3(kJoinThreads), 0, s, a);
    st = launch_status();
    if (st != CSA_OK || !acc || cap == 0) return st;
    const int wide_v = cap % 4 == 0 ? 4 : 1;  // rows of logits start on 16 bytes
    const dim3 tokens((unsigned)((cap + wide_v * kWeightThreads - 1) / (wide_v * kWeightThreads)), n_kv, B);
    if (wide_v == 4)
        launch_pdl(paged_weights_kernel<4>, tokens, dim3(kWeightThreads), 0, s, a);
    else
        launch_pdl(paged_weights_kernel<1>, tokens, dim3(kWeightThreads), 0, s, a);
    return launch_status();
}
