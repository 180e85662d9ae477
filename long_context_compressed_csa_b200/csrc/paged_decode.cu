// paged_attn for few query rows: the decode kernels, bound by the bytes of the cache.
//
// A CTA has 8 warps (4 for wide heads), each a worker of its own with a run of units (a few cached tokens) of one
// key head and a ring of stages that its lanes fill with 16-byte cp.async, two units ahead of the one being used; a
// token that no row sees, or without a page, is zero-filled and not read.  The warps of a CTA have the same run of
// neighbouring heads, whose rows lie together in a [row][head] page.  No warp waits for another: a run's
// output, or its partial result, goes from the warp's registers to memory.
//   bf16: the rows are the 16-row operand of mma.sync (m16n8k16), K is its B operand as stored,
//         V through transposing ldmatrix.  The weights go to the second product as two bf16
//         parts (hi + lo), which keeps 16 bits of them at the price of tensor work that is idle anyway.
//         WR > 1: WR warps have 16 rows each and share a ring; they are one worker, and round the weights once.
//   fp32: packed FMAs, a token spread over LT lanes, RT rows in registers.
#include "cluster.cuh"
#include "paged.cuh"
#include "tc_utils.cuh"

namespace csa {
namespace {

CSA_DEV void cp16(uint32_t dst, const void* src, bool take)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
CSA_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
CSA_DEV void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
CSA_DEV void ldsm4(uint32_t (&r)[4], uint32_t p)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(p));
}
CSA_DEV void ldsm4_t(uint32_t (&r)[4], uint32_t p)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(p));
}
CSA_DEV void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
CSA_DEV float lo16(uint32_t u) { return __uint_as_float(u << 16); }
CSA_DEV float hi16(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Byte offset of 16-byte chunk c of row r of a stage's K or V block; the XOR spreads the 8 rows
// that an ldmatrix (or the lanes of an fp32 load) touches over the banks.
template <int ROWB>
CSA_DEV uint32_t at16(int r, int c) { return r * ROWB + ((c ^ (r & 7)) << 4); }

template <int WR>
CSA_DEV void group_sync(int group)
{
    if (WR == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * WR) : "memory");
}

// The filling side of a group's ring: ROWB bytes a row, U rows of K and of V a stage.
template <int ROWB, int U, int WR>
struct Ring {
    static constexpr int kChunks = ROWB / 16, kLanes = 32 * WR;
    static constexpr int kStage = 2 * U * ROWB;
    uint32_t base;          // shared address of the group's ring
    uint32_t* masks;        // [stages]: bit r of a word: row r has a token
    const char *K, *V;      // of this key head
    int row_bytes;          // d elements
    bool one_page;          // a unit never lies in two pages, and has no holes
    int lane;               // within the group
    bool holes;             // of the item

    // Start of the loads of unit u into `stage`; every lane of the group.
    CSA_DEV void load(const PagedAttnArgs& a, const PagedEntry& en, int u, int stage, int eb)
    {
        const int j0 = en.first_token(u, U), l = lane & 31;
        const uint32_t s = base + stage * kStage;
        // a pass takes kLanes chunks: kLanes / kChunks rows, or a part of one row
        constexpr int kPasses = U * kChunks / kLanes;
        static_assert(U * kChunks % kLanes == 0, "whole passes");
        // Nearly every unit lies in one page and is wholly visible to some row: one look at the table, and rows
        // at a fixed distance (a third of the instructions of the way below).
        if (one_page && j0 >= en.lo_min && j0 + U <= en.hi_max) {
            const int64_t first = paged_row(a.pl, en.b, j0);
            if (first >= 0) {
                if (lane == 0) masks[stage] = U == 32 ? ~0u : (1u << (U & 31)) - 1;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int x = i * kLanes + lane, r = x / kChunks, c = x % kChunks;
                    const bool take = c * 16 < row_bytes;
                    const int64_t at = take ? (first + r * a.pl.ld_row) * eb + c * 16 : 0;
                    cp16(s + at16<ROWB>(r, c), K + at, take);
                    cp16(s + U * ROWB + at16<ROWB>(r, c), V + at, take);
                }
                return;
            }
        }
        int64_t off = -1;
        if (l < U && j0 + l < a.cap && paged_seen(a, en, holes, j0 + l)) off = paged_row(a.pl, en.b, j0 + l);
        const unsigned have = __ballot_sync(0xffffffffu, off >= 0);
        if (lane == 0) masks[stage] = have;
        off *= eb;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int x = i * kLanes + lane, r = x / kChunks, c = x % kChunks;
            const int64_t o = __shfl_sync(0xffffffffu, off, r);
            const bool take = o >= 0 && c * 16 < row_bytes;
            const int64_t at = take ? o + c * 16 : 0;
            cp16(s + at16<ROWB>(r, c), K + at, take);
            cp16(s + U * ROWB + at16<ROWB>(r, c), V + at, take);
        }
    }
};

template <int DP, int WR>
struct MmaShape {
    // Wide heads: two warps have the same 16 rows, both their logits and each half of the output columns, since a
    // ring of 16 tokens is too large for eight groups and four warps do not hide their latencies
    static constexpr int kWC = DP == 256 && WR == 1 ? 2 : 1;
    static constexpr int kWarps = DP == 256 && WR > 1 ? 4 : 8, kThreads = 32 * kWarps;
    static constexpr int kGW = WR * kWC;                           // warps of a group (a worker)
    static constexpr int kGroups = kWarps / kGW;
    static constexpr int kU = DP == 64 || (WR > 1 && DP == 128) ? 32 : 16;
    static constexpr int kStages = DP == 256 && WR == 2 ? 2 : DP < 256 && WR == 4 ? 6 : 3;
    static constexpr int kCtas = DP == 256 && WR > 1 ? 2 : 1;      // on an SM
    // Many rows are bound by the tensor cores, not by the cache's bytes: the weights are rounded once then, as in
    // the prompt kernel (half a step is 2^-9 to 2^-8 of a weight)
    static constexpr bool kSplit = WR == 1;
    static constexpr int kRows = 16 * WR;
    static constexpr int kRing = kGroups * kStages * 2 * kU * DP * 2;    // bytes
    static constexpr int kQ = DP == 256 ? kGroups * kRows * DP * 2 : 0;  // wide heads: q in shared memory
    static constexpr int kSmem = kQ + kRing;
};

template <int DP, int WR, bool kHoles>
__global__ void __launch_bounds__(MmaShape<DP, WR>::kThreads, MmaShape<DP, WR>::kCtas) paged_attn_mma(PagedAttnArgs a)
{
    using S = MmaShape<DP, WR>;
    constexpr int U = S::kU, R = S::kRows, NS = S::kStages, KS = DP / 16, NT = U / 8, ROWB = DP * 2;
    constexpr int WC = S::kWC, GW = S::kGW, ON = DP / 8 / WC;  // ON: output tiles of 8 columns of a warp
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ PagedScratch<S::kThreads, 1> sh;
    __shared__ uint32_t masks[S::kGroups * NS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = warp / GW, wr = warp % GW / WC, wc = warp % WC, worker = blockIdx.x * a.per_cta + group;
    const bool first = warp % GW == 0 && lane == 0;  // of the worker's threads
    const int run = group < a.per_cta ? worker / a.heads : a.runs;  // a.runs: none
    uint8_t* sring = smem + S::kQ;
    pdl_launch_dependents();
    pdl_wait();
    if (run < a.runs && first) a.desc[worker] = make_int4(-1, 0, 0, 0);
    PagedCursor c;
    if (!paged_schedule<S::kThreads, 1, true>(a, run, sh, c)) return;
    c.h = worker - run * a.heads;
    Ring<ROWB, U, GW> ring;
    ring.base = tc::smem_u32(sring) + group * (NS * ring.kStage);
    ring.masks = masks + group * NS;
    ring.row_bytes = a.d * 2;
    ring.one_page = a.pl.page % U == 0;
    ring.lane = warp % GW * 32 + lane;
    ring.K = static_cast<const char*>(a.K) + c.h * a.pl.ld_head * 2;
    ring.V = static_cast<const char*>(a.V) + c.h * a.pl.ld_head * 2;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    uint8_t* my_q = smem + (group * R + wr * 16) * ROWB;  // this warp's rows (wide heads)
    const uint32_t sq = tc::smem_u32(my_q);
    const int r0 = wr * 16 + (lane >> 2);  // this lane's rows: r0 and r0 + 8
    while (true) {
        const PagedSegment sg = paged_segment(a, c, worker);
        if (sg.u0 == sg.u1) break;  // the run ends before the item's first unit
        if (first) paged_describe(a, c, sg, worker);
        const PagedEntry en = c.en;
        ring.holes = kHoles && paged_holes<1>(a, en);
        if (kHoles) ring.one_page = a.pl.page % U == 0 && !ring.holes;
        const int n_u = sg.u1 - sg.u0;
#pragma unroll
        for (int s = 0; s < NS - 1; ++s) {
            if (s < n_u) ring.load(a, en, sg.u0 + s, s, 2);
            cp_commit();
        }
        uint32_t qf[DP == 256 ? 1 : KS][4];
        if constexpr (DP == 256) {
            for (int x = wc * 32 + lane; x < 16 * (DP / 8); x += 32 * WC) {
                const int r = x / (DP / 8), ch = x % (DP / 8);
                const int64_t o = paged_out_row(a, en.b, en.tile, c.h, wr * 16 + r);
                const bool in = o >= 0 && ch * 8 < a.d;
                const uint4 v = in ? *reinterpret_cast<const uint4*>(q + o * a.d + ch * 8) : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(my_q + at16<ROWB>(r, ch)) = v;
            }
            group_sync<GW>(group);
        } else {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int64_t o = paged_out_row(a, en.b, en.tile, c.h, r0 + 8 * half);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int col = k * 16 + p * 8 + 2 * (lane & 3);
                        qf[k][2 * p + half] =
                            o >= 0 && col < a.d ? *reinterpret_cast<const uint32_t*>(q + o * a.d + col) : 0u;
                    }
            }
        }
        RowBounds rb[2];
        bool row_in[2];
        float* lg[2];  // the rows' logits, when they are asked for
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = en.tile * R + r0 + 8 * half;
            row_in[half] = row < a.nq * a.G;
            rb[half] = row_in[half] ? paged_bounds(a, en.b, row / a.G) : RowBounds{0, 0, 0};
            lg[half] = a.logits && row_in[half] && wc == 0
                           ? a.logits + (((int64_t)en.b * a.n_kv + c.h) * (a.nq * a.G) + row) * a.cap
                           : nullptr;
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[ON][4];
#pragma unroll
        for (int i = 0; i < ON; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
        int st = 0;
        for (int i = 0; i < n_u; ++i) {
            cp_wait<NS - 2>();
            group_sync<GW>(group);
            const int u = sg.u0 + i;
            {
                const int nx = st == 0 ? NS - 1 : st - 1;
                if (i + NS - 1 < n_u) ring.load(a, en, u + NS - 1, nx, 2);
                cp_commit();
            }
            const uint32_t sk = ring.base + st * ring.kStage, sv = sk + U * ROWB;
            const unsigned have = ring.masks[st];
            st = st == NS - 1 ? 0 : st + 1;
            float s[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[t][x] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t qk[4];
                if constexpr (DP == 256)
                    ldsm4(qk, sq + at16<ROWB>((lane & 7) + (lane & 8), 2 * k + (lane >> 4)));
                else {
#pragma unroll
                    for (int x = 0; x < 4; ++x) qk[x] = qf[k][x];
                }
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    uint32_t b[4];  // tokens t*8 .. +15, k16 step k: {n0 k0, n0 k8, n8 k0, n8 k8}
                    ldsm4(b, sk + at16<ROWB>(t * 8 + (lane & 7) + ((lane & 16) >> 1), 2 * k + ((lane >> 3) & 1)));
                    mma16816(s[t], qk, b[0], b[1]);
                    mma16816(s[t + 1], qk, b[2], b[3]);
                }
            }
            const int j0 = en.first_token(u, U);
            const bool clear = j0 >= en.lo_max && j0 + U <= en.hi_min && have == (U == 32 ? ~0u : (1u << (U & 31)) - 1);
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int r = t * 8 + 2 * (lane & 3) + (x & 1);
                    float v = s[t][x] * a.scale_log2;
                    if (!clear && !((have >> r & 1) && paged_visible(rb[x >> 1], j0 + r))) v = -INFINITY;
                    s[t][x] = v;
                    top[x >> 1] = fmaxf(top[x >> 1], v);
                }
                if (a.logits) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int j = j0 + t * 8 + 2 * (lane & 3) + (x & 1);
                        if (lg[x >> 1] && j < a.cap) lg[x >> 1][j] = s[t][x];
                    }
                }
            }
            float shrink[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                top[half] = fmaxf(top[half], __shfl_xor_sync(0xffffffffu, top[half], 1));
                top[half] = fmaxf(top[half], __shfl_xor_sync(0xffffffffu, top[half], 2));
                const float mn = fmaxf(m[half], top[half]);
                shrink[half] = mn == m[half] ? 1.f : exp2f(m[half] - mn);  // m = -inf: 0
                m[half] = mn;
                l[half] *= shrink[half];
            }
            if (__any_sync(0xffffffffu, shrink[0] != 1.f || shrink[1] != 1.f)) {
#pragma unroll
                for (int i2 = 0; i2 < ON; ++i2)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[i2][x] *= shrink[x >> 1];
            }
            const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    s[t][x] = tc::ex2_approx(s[t][x] - base[x >> 1]);
                    l[x >> 1] += s[t][x];
                }
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float p = s[t + (x >> 1)][2 * (x & 1)], p1 = s[t + (x >> 1)][2 * (x & 1) + 1];
                    hi[x] = pack2(p, p1);
                    if (S::kSplit) lo[x] = pack2(p - lo16(hi[x]), p1 - hi16(hi[x]));
                }
#pragma unroll
                for (int n = 0; n < ON; n += 2) {
                    uint32_t b[4];  // tokens t*8 .. +15, 16 columns: {k0 n0, k8 n0, k0 n8, k8 n8}
                    ldsm4_t(b, sv + at16<ROWB>(t * 8 + (lane & 15), wc * ON + n + (lane >> 4)));
                    mma16816(o[n], hi, b[0], b[1]);
                    mma16816(o[n + 1], hi, b[2], b[3]);
                    if constexpr (S::kSplit) {
                        mma16816(o[n], lo, b[0], b[1]);
                        mma16816(o[n + 1], lo, b[2], b[3]);
                    }
                }
            }
        }
        cp_wait<0>();
        group_sync<GW>(group);  // the ring is filled anew
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = r0 + 8 * half;
            l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
            l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
            if (!row_in[half]) continue;
            if (sg.whole) {
                const int64_t at = paged_out_row(a, en.b, en.tile, c.h, r);
                const float inv = l[half] == 0.f ? 0.f : 1.f / l[half];
#pragma unroll
                for (int n = 0; n < ON; ++n) {
                    const int col = (wc * ON + n) * 8 + 2 * (lane & 3);
                    const float x = o[n][2 * half] * inv, y = o[n][2 * half + 1] * inv;
                    if (col >= a.d) continue;
                    if (a.out_bf16)
                        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + at * a.d + col) = pack2(x, y);
                    else
                        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at * a.d + col) = make_float2(x, y);
                }
                if ((lane & 3) == 0 && wc == 0) paged_store_lse(a, at, en.b, en.tile, c.h, r, m[half], l[half]);
            } else {
                const int64_t at = (int64_t)sg.slot * R + r;
#pragma unroll
                for (int n = 0; n < ON; ++n) {
                    const int col = (wc * ON + n) * 8 + 2 * (lane & 3);
                    if (col < a.d)
                        *reinterpret_cast<float2*>(a.part_o + at * a.d + col) =
                            make_float2(o[n][2 * half], o[n][2 * half + 1]);
                }
                if ((lane & 3) == 0 && wc == 0) a.part_ml[at] = make_float2(m[half], l[half]);
            }
        }
        if (!paged_next<1, true>(a, c, sg)) break;
    }
}

// The two 8 x 8 blocks of 16-bit values of a fragment, transposed.
CSA_DEV uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int DP>
struct FewShape {
    static constexpr int kU = DP == 64 ? 32 : 16, kStages = 3, kRows = 8;
    static constexpr int kWC = DP == 256 ? 2 : 1;                  // warps of a worker, each half of the columns
    static constexpr int kWarps = 8, kThreads = 32 * kWarps, kGroups = kWarps / kWC;
    static constexpr int kSmem = kGroups * kStages * 2 * kU * DP * 2;
};

// Eight rows or fewer (a decode step of most head layouts): the products the other way round, so that the rows are
// the 8-wide side of m16n8k16 and no row of it is padding:
//   S^T (16 tokens x 8 rows) = K Q^T,   O^T (16 columns x 8 rows) += V^T P^T.
// A lane has two rows (2 (lane mod 4) and the next) and tokens, or columns, lane / 4 and 8 more.  P^T becomes the
// second product's operand by a transposition of its 8 x 8 blocks.  Half the tensor work and half the logits a
// lane of the 16-row kernel, whose time and power (not the cache's bytes alone) bounded long decodes: two
// sequences of 256K tokens, width 64: 185 us, now 166 to 177 (6.1 to 6.5 TB/s); 16 of up to 128K, 8 rows: 322 to 330 us,
// 6.5 to 6.7 TB/s, at the power cap too, where the 16-row kernel took 372.
template <int DP, bool kHoles>
__global__ void __launch_bounds__(FewShape<DP>::kThreads, 1) paged_attn_few(PagedAttnArgs a)
{
    using S = FewShape<DP>;
    constexpr int U = S::kU, NS = S::kStages, KS = DP / 16, NT = U / 16, ROWB = DP * 2, WC = S::kWC, ON = DP / 16 / WC;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ PagedScratch<S::kThreads, 1> sh;
    __shared__ uint32_t masks[S::kGroups * NS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = warp / WC, wc = warp % WC, worker = blockIdx.x * a.per_cta + group;
    const int run = group < a.per_cta ? worker / a.heads : a.runs;  // a.runs: none
    const bool first = wc == 0 && lane == 0;
    pdl_launch_dependents();
    pdl_wait();
    if (run < a.runs && first) a.desc[worker] = make_int4(-1, 0, 0, 0);
    PagedCursor c;
    if (!paged_schedule<S::kThreads, 1, true>(a, run, sh, c)) return;
    c.h = worker - run * a.heads;
    Ring<ROWB, U, WC> ring;
    ring.base = tc::smem_u32(smem) + group * (NS * ring.kStage);
    ring.masks = masks + group * NS;
    ring.row_bytes = a.d * 2;
    ring.one_page = a.pl.page % U == 0;
    ring.lane = wc * 32 + lane;
    ring.K = static_cast<const char*>(a.K) + c.h * a.pl.ld_head * 2;
    ring.V = static_cast<const char*>(a.V) + c.h * a.pl.ld_head * 2;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    const int r0 = 2 * (lane & 3), k0 = lane >> 2;  // this lane's first row; its token, or column, of a block
    while (true) {
        const PagedSegment sg = paged_segment(a, c, worker);
        if (sg.u0 == sg.u1) break;  // the run ends before the item's first unit
        if (first) paged_describe(a, c, sg, worker);
        const PagedEntry en = c.en;
        ring.holes = kHoles && paged_holes<1>(a, en);
        if (kHoles) ring.one_page = a.pl.page % U == 0 && !ring.holes;
        const int n_u = sg.u1 - sg.u0;
#pragma unroll
        for (int s = 0; s < NS - 1; ++s) {
            if (s < n_u) ring.load(a, en, sg.u0 + s, s, 2);
            cp_commit();
        }
        uint32_t qf[KS][2];
        {
            const int64_t o = paged_out_row(a, en.b, en.tile, c.h, k0);
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const int col = k * 16 + p * 8 + 2 * (lane & 3);
                    qf[k][p] = o >= 0 && col < a.d ? *reinterpret_cast<const uint32_t*>(q + o * a.d + col) : 0u;
                }
        }
        RowBounds rb[2];
        bool row_in[2];
        float* lg[2];  // the rows' logits, when they are asked for
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int row = en.tile * S::kRows + r0 + x;
            row_in[x] = row < a.nq * a.G;
            rb[x] = row_in[x] ? paged_bounds(a, en.b, row / a.G) : RowBounds{0, 0, 0};
            lg[x] = a.logits && row_in[x] && wc == 0
                        ? a.logits + (((int64_t)en.b * a.n_kv + c.h) * (a.nq * a.G) + row) * a.cap
                        : nullptr;
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[ON][4];
#pragma unroll
        for (int i = 0; i < ON; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
        int st = 0;
        for (int i = 0; i < n_u; ++i) {
            cp_wait<NS - 2>();
            group_sync<WC>(group);
            const int u = sg.u0 + i;
            {
                const int nx = st == 0 ? NS - 1 : st - 1;
                if (i + NS - 1 < n_u) ring.load(a, en, u + NS - 1, nx, 2);
                cp_commit();
            }
            const uint32_t sk = ring.base + st * ring.kStage, sv = sk + U * ROWB;
            const unsigned have = ring.masks[st];
            st = st == NS - 1 ? 0 : st + 1;
            // two partial sums a tile: a chain of KS products is the longest wait of a unit
            float s[NT][4], s2[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[t][x] = s2[t][x] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; k += 2)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    uint32_t f[4];  // tokens t*16 .. +15, k16 step: {m0 k0, m8 k0, m0 k8, m8 k8}
                    ldsm4(f, sk + at16<ROWB>(t * 16 + (lane & 15), 2 * k + (lane >> 4)));
                    mma16816(s[t], f, qf[k][0], qf[k][1]);
                    ldsm4(f, sk + at16<ROWB>(t * 16 + (lane & 15), 2 * k + 2 + (lane >> 4)));
                    mma16816(s2[t], f, qf[k + 1][0], qf[k + 1][1]);
                }
            const int j0 = en.first_token(u, U);
            const bool clear = j0 >= en.lo_max && j0 + U <= en.hi_min && have == (U == 32 ? ~0u : (1u << (U & 31)) - 1);
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int r = t * 16 + k0 + 8 * (x >> 1);
                    float v = (s[t][x] + s2[t][x]) * a.scale_log2;
                    if (!clear && !((have >> r & 1) && paged_visible(rb[x & 1], j0 + r))) v = -INFINITY;
                    s[t][x] = v;
                    top[x & 1] = fmaxf(top[x & 1], v);
                }
            if (a.logits) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int j = j0 + t * 16 + k0 + 8 * (x >> 1);
                        if (lg[x & 1] && j < a.cap) lg[x & 1][j] = s[t][x];
                    }
            }
            float shrink[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], y));
                const float mn = fmaxf(m[x], top[x]);
                shrink[x] = mn == m[x] ? 1.f : tc::ex2_approx(m[x] - mn);  // m = -inf: 0
                m[x] = mn;
                l[x] *= shrink[x];
            }
            if (__any_sync(0xffffffffu, shrink[0] != 1.f || shrink[1] != 1.f)) {
#pragma unroll
                for (int n = 0; n < ON; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[n][x] *= shrink[x & 1];
            }
            const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float p = tc::ex2_approx(s[t][2 * x] - base[0]), p1 = tc::ex2_approx(s[t][2 * x + 1] - base[1]);
                    l[0] += p;
                    l[1] += p1;
                    hi[x] = pack2(p, p1);
                    lo[x] = transpose8(pack2(p - lo16(hi[x]), p1 - hi16(hi[x])));
                    hi[x] = transpose8(hi[x]);
                }
#pragma unroll
                for (int n = 0; n < ON; ++n) {
                    uint32_t f[4];  // columns n*16 .. +15, tokens t*16 .. +15: {m0 k0, m8 k0, m0 k8, m8 k8}
                    ldsm4_t(f, sv + at16<ROWB>(t * 16 + (lane & 7) + ((lane >> 4) << 3),
                                               2 * (wc * ON + n) + ((lane >> 3) & 1)));
                    mma16816(o[n], f, hi[0], hi[1]);
                    mma16816(o[n], f, lo[0], lo[1]);
                }
            }
        }
        cp_wait<0>();
        group_sync<WC>(group);  // the ring is filled anew
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], y);
            if (!row_in[x]) continue;
            const int64_t at = sg.whole ? paged_out_row(a, en.b, en.tile, c.h, r0 + x) : (int64_t)sg.slot * S::kRows + r0 + x;
            const float inv = sg.whole ? (l[x] == 0.f ? 0.f : 1.f / l[x]) : 1.f;
#pragma unroll
            for (int n = 0; n < ON; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int col = (wc * ON + n) * 16 + 8 * y + k0;
                    const float v = o[n][2 * y + x] * inv;
                    if (col >= a.d) continue;
                    if (sg.whole)
                        paged_store(a, at * a.d + col, v);
                    else
                        a.part_o[at * a.d + col] = v;
                }
            if (k0 == 0 && wc == 0) {
                if (sg.whole)
                    paged_store_lse(a, at, en.b, en.tile, c.h, r0 + x, m[x], l[x]);
                else
                    a.part_ml[at] = make_float2(m[x], l[x]);
            }
        }
        __syncwarp();
        if (!paged_next<1, true>(a, c, sg)) break;
    }
}

// fp32 rows: RT of them in registers, EL = 64 / RT elements of a row a lane, so that q and the output take 128
// registers for either RT.  Bound by FMA and shuffle issue at 8 rows (16 sequences of 8K tokens, 537 MB: 128 us, 4.2 TB/s;
// 4 rows: 105 us, 5.1 TB/s), by latency in small calls (8 of up to 4K, 69 MB: 30 us).
template <int DP, int RT>
struct F32Shape {
    static constexpr int kEL = 64 / RT;      // elements of a row that a lane has
    static constexpr int kLT = DP / kEL;     // lanes of a token
    static constexpr int kNG = 32 / kLT;     // tokens at a time
    static constexpr int kU = 1024 / DP;     // tokens of a unit: 8 KB of K and V
    static constexpr int kStages = 3;
    static constexpr int kWarps = 8, kThreads = 32 * kWarps;
    static constexpr int kSmem = kWarps * kStages * 2 * kU * DP * 4;
};

template <int DP, int RT, bool kHoles>
__global__ void __launch_bounds__(F32Shape<DP, RT>::kThreads, 1) paged_attn_f32(PagedAttnArgs a)
{
    using S = F32Shape<DP, RT>;
    constexpr int U = S::kU, NS = S::kStages, EL = S::kEL, LT = S::kLT, NG = S::kNG, TG = U / NG, ROWB = DP * 4;
    // N logits of a token group at a time; NV of them a lane, or SH lanes with the same one
    constexpr int N = TG * RT, NV = N > LT ? N / LT : 1, SH = LT > N ? LT / N : 1;
    static_assert(RT % NV == 0 && TG * NG == U, "a lane's logits are of one token");
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ PagedScratch<S::kThreads, 1> sh;
    __shared__ uint32_t masks[S::kWarps * NS];
    __shared__ RowBounds bounds[S::kWarps][RT];  // of the rows of each warp's item
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, worker = blockIdx.x * a.per_cta + warp;
    const int run = warp < a.per_cta ? worker / a.heads : a.runs;  // a.runs: none
    const int g = lane / LT, e = lane % LT;
    pdl_launch_dependents();
    pdl_wait();
    if (run < a.runs && lane == 0) a.desc[worker] = make_int4(-1, 0, 0, 0);
    PagedCursor c;
    if (!paged_schedule<S::kThreads, 1, true>(a, run, sh, c)) return;
    c.h = worker - run * a.heads;
    Ring<ROWB, U, 1> ring;
    ring.base = tc::smem_u32(smem) + warp * (NS * ring.kStage);
    ring.masks = masks + warp * NS;
    ring.row_bytes = a.d * 4;
    ring.one_page = a.pl.page % U == 0;
    ring.lane = lane;
    ring.K = static_cast<const char*>(a.K) + c.h * a.pl.ld_head * 4;
    ring.V = static_cast<const char*>(a.V) + c.h * a.pl.ld_head * 4;
    const uint8_t* my = smem + warp * (NS * ring.kStage);
    const float* q = static_cast<const float*>(a.q);
    while (true) {
        const PagedSegment sg = paged_segment(a, c, worker);
        if (sg.u0 == sg.u1) break;  // the run ends before the item's first unit
        if (lane == 0) paged_describe(a, c, sg, worker);
        const PagedEntry en = c.en;
        ring.holes = kHoles && paged_holes<1>(a, en);
        if (kHoles) ring.one_page = a.pl.page % U == 0 && !ring.holes;
        const int n_u = sg.u1 - sg.u0;
#pragma unroll
        for (int s = 0; s < NS - 1; ++s) {
            if (s < n_u) ring.load(a, en, sg.u0 + s, s, 4);
            cp_commit();
        }
        __syncwarp();
        if (lane < RT) {
            const int row = en.tile * RT + lane;
            bounds[warp][lane] = row < a.nq * a.G ? paged_bounds(a, en.b, row / a.G) : RowBounds{0, 0, 0};
        }
        __syncwarp();
        float2 qr[RT][EL / 2], o[RT][EL / 2];
        float m_own[NV], l_own[NV];  // of this lane's rows
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            m_own[i] = -INFINITY;
            l_own[i] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int64_t at = paged_out_row(a, en.b, en.tile, c.h, r);
#pragma unroll
            for (int x = 0; x < EL / 2; ++x) {
                const int col = (e + LT * (x / 2)) * 4 + 2 * (x & 1);
                qr[r][x] = o[r][x] = make_float2(0.f, 0.f);
                if (at >= 0 && col < a.d) {
                    qr[r][x].x = q[at * a.d + col];
                    if (col + 1 < a.d) qr[r][x].y = q[at * a.d + col + 1];
                }
            }
        }
        int st = 0;
        for (int i = 0; i < n_u; ++i) {
            cp_wait<NS - 2>();
            __syncwarp();
            const int u = sg.u0 + i;
            {
                const int nx = st == 0 ? NS - 1 : st - 1;
                if (i + NS - 1 < n_u) ring.load(a, en, u + NS - 1, nx, 4);
                cp_commit();
            }
            const uint8_t *sk = my + st * ring.kStage, *sv = sk + U * ROWB;
            const unsigned have = ring.masks[st];
            st = st == NS - 1 ? 0 : st + 1;
            const int j0 = en.first_token(u, U);
            const bool clear = j0 >= en.lo_max && j0 + U <= en.hi_min && have == (U == 32 ? ~0u : (1u << (U & 31)) - 1);
            // this lane's part of the N logits of its token group, (token, row) in the order token * RT + row
            float s[N];
#pragma unroll
            for (int t = 0; t < TG; ++t) {
                const int r8 = t * NG + g;
                float2 k[EL / 2];
#pragma unroll
                for (int x = 0; x < EL / 4; ++x) {
                    const float4 v = *reinterpret_cast<const float4*>(sk + at16<ROWB>(r8, e + LT * x));
                    k[2 * x] = make_float2(v.x, v.y);
                    k[2 * x + 1] = make_float2(v.z, v.w);
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    float2 dot = make_float2(0.f, 0.f);
#pragma unroll
                    for (int x = 0; x < EL / 2; ++x) dot = tc::fma2(qr[r][x], k[x], dot);
                    s[t * RT + r] = dot.x + dot.y;
                }
            }
            // Summed over the LT lanes so that each ends with NV whole logits: in a step a lane keeps half of its
            // values and hands the other half to its partner (30 shuffles for 32 logits instead of 128)
            int n = N;
#pragma unroll
            for (int y = LT / 2; y; y >>= 1) {
                if (n > 1) {
                    n >>= 1;
                    const bool up = e & y;
#pragma unroll
                    for (int x = 0; x < N / 2; ++x)
                        if (x < n) {
                            const float keep = up ? s[x + n] : s[x], give = up ? s[x] : s[x + n];
                            s[x] = keep + __shfl_xor_sync(0xffffffffu, give, y);
                        }
                } else {
                    s[0] += __shfl_xor_sync(0xffffffffu, s[0], y);
                }
            }
            float shrink[NV];
            bool grew = false;
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                const int at = e / SH * NV + x, r = at % RT, r8 = at / RT * NG + g;
                s[x] *= a.scale_log2;
                if (!clear && !((have >> r8 & 1) && paged_visible(bounds[warp][r], j0 + r8))) s[x] = -INFINITY;
                const int row = en.tile * RT + r;
                if (a.logits && e % SH == 0 && j0 + r8 < a.cap && row < a.nq * a.G)
                    a.logits[(((int64_t)en.b * a.n_kv + c.h) * (a.nq * a.G) + row) * a.cap + j0 + r8] = s[x];
                float top = s[x];  // over the tokens of the row
#pragma unroll
                for (int y = RT * SH / NV; y < LT; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
                const float mn = fmaxf(m_own[x], top);
                shrink[x] = mn == m_own[x] ? 1.f : tc::ex2_approx(m_own[x] - mn);
                grew |= shrink[x] != 1.f;
                m_own[x] = mn;
                s[x] = tc::ex2_approx(s[x] - (mn == -INFINITY ? 0.f : mn));
                l_own[x] = l_own[x] * shrink[x] + s[x];
            }
            const int lane0 = lane - e;  // of the token group
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float f = __shfl_sync(0xffffffffu, shrink[r % NV], lane0 + r / NV * SH);
#pragma unroll
                    for (int x = 0; x < EL / 2; ++x) {
                        o[r][x].x *= f;
                        o[r][x].y *= f;
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < TG; ++t) {
                const int r8 = t * NG + g;
                float4 v[EL / 4];
#pragma unroll
                for (int x = 0; x < EL / 4; ++x) v[x] = *reinterpret_cast<const float4*>(sv + at16<ROWB>(r8, e + LT * x));
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const int at = t * RT + r;
                    const float w = __shfl_sync(0xffffffffu, s[at % NV], lane0 + at / NV * SH);
                    const float2 p = make_float2(w, w);
#pragma unroll
                    for (int x = 0; x < EL / 4; ++x) {
                        o[r][2 * x] = tc::fma2(p, make_float2(v[x].x, v[x].y), o[r][2 * x]);
                        o[r][2 * x + 1] = tc::fma2(p, make_float2(v[x].z, v[x].w), o[r][2 * x + 1]);
                    }
                }
            }
        }
        cp_wait<0>();
        __syncwarp();  // the ring is filled anew
        // join the NG token groups of the warp
#pragma unroll
        for (int x = 0; x < NV; ++x)
#pragma unroll
            for (int y = RT * SH / NV; y < LT; y <<= 1) l_own[x] += __shfl_xor_sync(0xffffffffu, l_own[x], y);
        float m[RT], l[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            m[r] = __shfl_sync(0xffffffffu, m_own[r % NV], lane - e + r / NV * SH);
            l[r] = __shfl_sync(0xffffffffu, l_own[r % NV], lane - e + r / NV * SH);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float M = m[r];
#pragma unroll
            for (int y = LT; y < 32; y <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, y));
            const float f = m[r] == -INFINITY ? 0.f : exp2f(m[r] - M);
            l[r] *= f;
#pragma unroll
            for (int y = LT; y < 32; y <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], y);
#pragma unroll
            for (int x = 0; x < EL / 2; ++x) {
                o[r][x].x *= f;
                o[r][x].y *= f;
#pragma unroll
                for (int y = LT; y < 32; y <<= 1) {
                    o[r][x].x += __shfl_xor_sync(0xffffffffu, o[r][x].x, y);
                    o[r][x].y += __shfl_xor_sync(0xffffffffu, o[r][x].y, y);
                }
            }
            if (g == 0 && r < paged_rows(a, en.tile)) {
                const int64_t at = sg.whole ? paged_out_row(a, en.b, en.tile, c.h, r) : (int64_t)sg.slot * RT + r;
                float* to = (sg.whole ? static_cast<float*>(a.out) : a.part_o) + at * a.d;
                const float inv = sg.whole ? (l[r] == 0.f ? 0.f : 1.f / l[r]) : 1.f;
#pragma unroll
                for (int x = 0; x < EL / 4; ++x) {
                    const int col = (e + LT * x) * 4;
                    if (col < a.d)
                        *reinterpret_cast<float4*>(to + col) = make_float4(o[r][2 * x].x * inv, o[r][2 * x].y * inv,
                                                                           o[r][2 * x + 1].x * inv, o[r][2 * x + 1].y * inv);
                }
                if (e == 0) {
                    if (sg.whole)
                        paged_store_lse(a, at, en.b, en.tile, c.h, r, M, l[r]);
                    else
                        a.part_ml[at] = make_float2(M, l[r]);
                }
            }
            __syncwarp();
        }
        if (!paged_next<1, true>(a, c, sg)) break;
    }
}

template <auto kKernel>
int launch_one(int threads, int smem, const PagedAttnArgs& a, cudaStream_t stream)
{
    if (!paged_allow_smem<kKernel>(smem)) return CSA_ERR_CUDA;
    launch_pdl(kKernel, dim3((a.runs * a.heads + a.per_cta - 1) / a.per_cta), dim3(threads), smem, stream, a);
    return launch_status();
}
template <auto kKernel, auto kWithHoles>
int launch(int threads, int groups, int smem, PagedAttnArgs a, cudaStream_t stream)
{
    // few workers: one or two on every SM, not eight on a few
    a.per_cta = (a.runs * a.heads + kNumSMs - 1) / kNumSMs;
    if (a.per_cta > groups) a.per_cta = groups;
    return a.may_have_holes() ? launch_one<kWithHoles>(threads, smem, a, stream) : launch_one<kKernel>(threads, smem, a, stream);
}

template <int DP, int WR>
int launch_mma(const PagedAttnArgs& a, cudaStream_t stream)
{
    using S = MmaShape<DP, WR>;
    return launch<paged_attn_mma<DP, WR, false>, paged_attn_mma<DP, WR, true>>(S::kThreads, S::kGroups, S::kSmem, a, stream);
}
template <int DP>
int launch_few(const PagedAttnArgs& a, cudaStream_t stream)
{
    using S = FewShape<DP>;
    return launch<paged_attn_few<DP, false>, paged_attn_few<DP, true>>(S::kThreads, S::kGroups, S::kSmem, a, stream);
}
template <int DP, int RT>
int launch_f32(const PagedAttnArgs& a, cudaStream_t stream)
{
    using S = F32Shape<DP, RT>;
    return launch<paged_attn_f32<DP, RT, false>, paged_attn_f32<DP, RT, true>>(S::kThreads, S::kWarps, S::kSmem, a, stream);
}

}  // namespace

// Rows, units and CTAs of a decode call.
PagedShape paged_decode_shape(int dtype, int rows, int d)
{
    PagedShape s{};
    s.DP = d <= 64 ? 64 : d <= 128 ? 128 : 256;
    s.by_head = true;
    if (dtype == CSA_BF16 && rows <= 8) {
        s.kind = kPagedFew;
        s.R = 8;
        s.unit = s.DP == 64 ? 32 : 16;
        s.min_units = 4;  // as below
        s.item_units = 4;
        s.workers = (s.DP == 256 ? 4 : 8) * kNumSMs;
    } else if (dtype == CSA_BF16) {
        s.kind = kPagedMma;
        s.WR = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
        s.R = 16 * s.WR;
        s.unit = s.DP == 64 || (s.WR > 1 && s.DP == 128) ? 32 : 16;
        // short runs fill the GPU, long ones leave fewer pieces to join (one 8K sequence, 8 key heads: 3 units 21.6 us, 4
        // 19.4, 6 21.5, 8 24.0)
        s.min_units = 4;
        s.item_units = 4;
        s.workers = (s.DP == 256 && s.WR == 1 ? 4 : 8) / s.WR * kNumSMs;
    } else {
        s.kind = kPagedF32;
        s.WR = s.R = rows <= 4 ? 4 : 8;
        s.unit = 1024 / s.DP;
        s.min_units = 3;  // 15 sequences of up to 700 tokens: 8 units 33 us, 4 27, 3 23
        s.item_units = 4;
        s.workers = 8 * kNumSMs;
    }
    return s;
}

int launch_paged_decode(const PagedAttnArgs& a, const PagedShape& s, cudaStream_t stream)
{
    if (s.kind == kPagedFew)
        return s.DP == 64 ? launch_few<64>(a, stream) : s.DP == 128 ? launch_few<128>(a, stream) : launch_few<256>(a, stream);
    if (s.kind == kPagedF32) {
        if (s.DP == 64) return s.WR == 4 ? launch_f32<64, 4>(a, stream) : launch_f32<64, 8>(a, stream);
        if (s.DP == 128) return s.WR == 4 ? launch_f32<128, 4>(a, stream) : launch_f32<128, 8>(a, stream);
        return s.WR == 4 ? launch_f32<256, 4>(a, stream) : launch_f32<256, 8>(a, stream);
    }
#define PAGED_MMA(DP) \
    (s.WR == 1 ? launch_mma<DP, 1>(a, stream) : s.WR == 2 ? launch_mma<DP, 2>(a, stream) : launch_mma<DP, 4>(a, stream))
    if (s.DP == 64) return PAGED_MMA(64);
    if (s.DP == 128) return PAGED_MMA(128);
    return PAGED_MMA(256);
#undef PAGED_MMA
}

}  // namespace csa
