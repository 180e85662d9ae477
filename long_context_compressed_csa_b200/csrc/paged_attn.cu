// paged_attn: grouped-query attention over the paged cache.  Host path, the CUDA-core kernel
// (any head width and layout), the join of partial results and the accumulated weights.
//
// For query i of sequence b at cache position t, query head x and its key head h = x / G:
//   s_j = scale * q . K_j            over the visible tokens j (paged_bounds)
//   o   = sum_j exp(s_j - lse) V_j,  lse = log sum_j exp(s_j)
// in one pass over K and V with a running maximum and sum (base 2, fp32).
#include <algorithm>

#include "paged.cuh"

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
    if (!paged_schedule<kSimtThreads, 1>(a, cta, sh, c)) return;
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
                const float p = vis ? exp2f(s[r] - mn) : 0.f;
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
        if (!paged_next<1>(a, c, sg)) break;
    }
}

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

// Joins the partial results of the CTAs that had a part of an item: PS warps of a CTA share the pieces
// of a row.  A decode call may cut an item into many pieces and has few rows (PS = 4); a prompt's
// items are cut in two or three and have many (PS = 1).
template <int PS>
__global__ void __launch_bounds__(kJoinThreads) paged_attn_combine(PagedAttnArgs a)
{
    constexpr int NC = kPagedMaxD / 32, RW = kJoinWarps / PS;
    __shared__ float sh[kJoinWarps][2];
    __shared__ float so[PS > 1 ? kJoinWarps : 1][kPagedMaxD];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c0 = blockIdx.x;
    const int r = blockIdx.y * RW + warp / PS, ps = warp % PS;
    pdl_launch_dependents();
    pdl_wait();
    if (c0 == 0 && blockIdx.y == 0 && warp == 0) {
        int late = 0;
        for (int i = lane; i < a.grid; i += 32) late |= a.desc[i].w;
        late = __any_sync(0xffffffffu, late);
        if (lane == 0) *a.status = late ? 1u : 0u;
    }
    const int4 ds = a.desc[c0];
    if (ds.x < 0) return;
    const int b = ds.x / a.n_tiles, tile = ds.x - b * a.n_tiles, h = ds.y;
    const int np = ds.z - c0 + 1;
    const bool in = r < paged_rows(a, tile);
    // piece p lies in slot 2 c0 + 1 for p = 0, 2 (c0 + p) after that
    auto slot = [&](int p) { return (int64_t)(p == 0 ? 2 * c0 + 1 : 2 * (c0 + p)) * a.R + r; };
    float M = -INFINITY, L = 0.f, acc[NC];
    if (in)
        for (int p = lane; p < np; p += 32) M = fmaxf(M, a.part_ml[slot(p)].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
#pragma unroll
    for (int i = 0; i < NC; ++i) acc[i] = 0.f;
    if (in) {
#pragma unroll 2
        for (int p = ps; p < np; p += PS) {
            const float2 ml = a.part_ml[slot(p)];
            const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
            L = fmaf(w, ml.y, L);
            const float* src = a.part_o + slot(p) * a.d;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (lane + 32 * i < a.d) acc[i] = fmaf(w, src[lane + 32 * i], acc[i]);
        }
    }
    const int64_t o = in ? paged_out_row(a, b, tile, h, r) : -1;
    if (PS > 1) {
        if (lane == 0) sh[warp][0] = L;
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (lane + 32 * i < a.d) so[warp][lane + 32 * i] = acc[i];
        __syncthreads();
        if (ps > 0) return;
#pragma unroll
        for (int w = 1; w < PS; ++w) {
            L += sh[warp + w][0];
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (lane + 32 * i < a.d) acc[i] += so[warp + w][lane + 32 * i];
        }
    }
    if (o < 0) return;
    const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
        if (lane + 32 * i < a.d) paged_store(a, o * a.d + lane + 32 * i, acc[i] * inv);
    if (lane == 0) paged_store_lse(a, o, b, tile, h, r, M, L);
}

constexpr int kWeightThreads = 256;

// acc_out[b][h][j] = acc[b][h][j] + the sum over the key head's queries of exp(s_j - lse), from the
// logits that the attention kernel left: one thread per cached token, so the sum has one order.
__global__ void __launch_bounds__(kWeightThreads) paged_weights_kernel(PagedAttnArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int j = blockIdx.x * kWeightThreads + threadIdx.x, h = blockIdx.y, b = blockIdx.z;
    if (j >= a.cap) return;
    const int64_t g = (int64_t)b * a.n_kv + h, at = g * a.cap + j;
    const int rows = a.nq * a.G;
    const float* s = a.logits + g * rows * a.cap + j;
    const float* z = a.lse2 + g * rows;
    float w = 0.f;
    for (int i = 0; i < a.nq; ++i) {
        if (!paged_visible(paged_bounds(a, b, i), j)) continue;
        for (int r = i * a.G; r < (i + 1) * a.G; ++r) {
            // every visible logit was written; -inf (a token without a page) weighs nothing,
            // and with no visible row at all lse is -inf too
            const float x = s[(int64_t)r * a.cap];
            if (x != -INFINITY) w += exp2f(x - z[r]);
        }
    }
    a.acc_out[at] = a.acc[at] + w;
}

}  // namespace

// The kernel of a call, by its rows (queries x heads of a key head), type and layout.  `wide`: every
// row can be loaded 16 bytes at a time; what cannot takes the CUDA-core kernel.  `boxes`: the pools can be
// read by TMA.  A tile of 128 rows costs the prompt kernel the same however few of them there are.
constexpr int kPromptRows = 17;
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
    s.grid = 2 * kNumSMs;
    return s;
}

// Workspace layout, from the sizes alone: room for every kernel that a call of these sizes may run on.
struct PagedPlan {
    size_t part_o, part_ml, logits, lse2, bytes;  // offsets; before them the 256-byte status block and desc
};

static PagedPlan paged_plan(int B, int nq, int G, int n_kv, int d, int64_t cap, bool weights)
{
    PagedPlan p{};
    size_t slots = 0;  // rows of partial results
    for (int dtype : {CSA_BF16, CSA_F32})
        for (int way = 0; way < 3; ++way) {
            const PagedShape s = paged_shape(dtype, way > 0, way > 1, nq * G, d);
            slots = std::max(slots, (size_t)2 * s.grid * s.R);
        }
    size_t at = 256 + align_up(sizeof(int4) * kPagedMaxCtas, 256);
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
    // 16-byte loads: every row starts on a 16-byte boundary and is whole 16-byte words
    const int64_t lds = pool_ld_page | pool_ld_row | (n_kv > 1 ? pool_ld_head : 0) | d;
    const bool wide = aligned16(q) && aligned16(K) && aligned16(V) && lds * elem_bytes(dtype) % 16 == 0;
    const PagedShape sp = paged_shape(dtype, wide, paged_prompt_takes(pl, n_kv, d), nq * G, d);
    a.R = sp.R; a.unit = sp.unit; a.min_units = sp.min_units; a.item_units = sp.item_units;
    a.n_tiles = (nq * G + sp.R - 1) / sp.R;
    // no more CTAs than the capacity has units
    const int64_t units = std::max<int64_t>(1, (cap + sp.unit - 1) / sp.unit) * B * n_kv * a.n_tiles;
    a.grid = (int)std::max<int64_t>(1, std::min<int64_t>(sp.grid, units / sp.min_units));
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
            launch_pdl(paged_attn_simt<__nv_bfloat16>, dim3(a.grid), dim3(kSimtThreads), smem, s, a);
        else
            launch_pdl(paged_attn_simt<float>, dim3(a.grid), dim3(kSimtThreads), smem, s, a);
        st = launch_status();
    } else {
        st = sp.kind == kPagedPrompt ? launch_paged_prompt(a, sp, s) : launch_paged_decode(a, sp, s);
    }
    if (st != CSA_OK) return st;
    const int rows = std::min(a.R, nq * G);
    if (sp.kind == kPagedPrompt)
        launch_pdl(paged_attn_combine<1>, dim3(a.grid, (rows + 7) / 8), dim3(kJoinThreads), 0, s, a);
    else
        launch_pdl(paged_attn_combine<4>, dim3(a.grid, (rows + 1) / 2), dim3(kJoinThreads), 0, s, a);
    st = launch_status();
    if (st != CSA_OK || !acc || cap == 0) return st;
    launch_pdl(paged_weights_kernel, dim3((unsigned)((cap + kWeightThreads - 1) / kWeightThreads), n_kv, B),
               dim3(kWeightThreads), 0, s, a);
    return launch_status();
}
