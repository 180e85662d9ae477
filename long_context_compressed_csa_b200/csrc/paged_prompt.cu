// paged_attn for many query rows: a prompt, a chunk of one, or a decode step whose query rows fill a tile.
//
// Packed rows (query, head of the key head's group) are the M dimension of tcgen05: both products
//   S = Q K^T (128 rows x 128 tokens)   and   O += P V (128 rows x d)
// are bf16 tensor-core work with fp32 accumulators in TMEM.  A CTA has two tiles of 128 rows
// that share every K and V tile, and takes a run of the schedule (paged.cuh):
//   warps 0-3, 4-7  softmax of tile 0 and tile 1, one thread per row: S from TMEM to registers,
//                   running maximum and sum, P (bf16) over S in TMEM; q -> shared memory before, O ->
//                   memory after a segment
//   warps 8, 10     TMA loads of K and of V, one box of up to 128 rows of one page per lane; a page that is
//                   not there, or that no row sees, is a box outside the tensor: zeros
//   warp 9          MMA issue
// One tile's softmax runs while the other's products do.  Where every item is one tile (kOne) both warpgroups work on it:
// they take its units in turn, each with its own S, O, maximum and sum, and warps 0-3 join the two at the end: 40 rows
// of 8 key heads, 16 sequences of 8K tokens in pages of 64, d = 128 and 64: 122 -> 100 us and 98 -> 71 (64 of 400: 63 ->
// 57 and 47 -> 43).  A kernel of its own: in one kernel with the two-tile form the added registers cost prompts 4 to 9%.
// P replaces S in TMEM, half by half, so the first half's product with V starts under the second's exponentials, and
// the next S of the same place follows P(j) V.
// (Two S of 64 tokens a tile, so that S(j+1) is there before P(j), measured slower: a product of
// N = 64 takes as long as one of 128, since the operand q is read from shared memory either way.)
// O is rescaled only when the running maximum grew by more than 2^8 (P stays below 2^8).  S(j) is
// issued after the P V before it of its O, so once S(j) is there O is at rest, and the softmax thread rescales its
// row in TMEM by itself.  P is rounded to bf16 (half a step is 2^-9 to 2^-8 of a weight), as the
// operand of the tensor core has to be; the row sum takes the weights before the rounding.
// The masks (positions, window, first tokens, missing pages) are applied to S only in units that
// are not wholly visible; there the rows of V that no query sees are set to zero too, since 0 x NaN
// would reach the sums.  Bounded waits: a timeout ends the CTA and sets its status.
// 2 x 1024 queries over 15-16K tokens, 64 / 8 heads, d = 128: 1010 to 1100 us by the power cap (926 to 1008 TFLOP/s, 0.68 to
// 0.74 of the sustained GEMM); 1 x 1024 over 8K, 32 heads, d = 128: 154 us, below the cap.  d = 64, 2 x 1024 over 8K, 32 / 8
// heads: 214 us, 0.60 PFLOP/s.  A unit of both tiles takes 3500 clocks, 2048 of which are products: a tile's
// softmax (2100) and its products (1100 with their barriers) take turns, and there is no TMEM for a second S.
#include "paged.cuh"
#include "tc_utils.cuh"

namespace csa {
namespace {

constexpr int kM = 128;             // rows of a tile
constexpr int kT = 128;             // cached tokens of a unit
constexpr int kH = 64;              // of a half: P is handed over in two
constexpr int kThreads = 384;       // two softmax warpgroups, and one of which three warps work
constexpr int kKWarp = 8, kMmaWarp = 9, kVWarp = 10;
// Registers of a thread: launched with 168, then split between the warpgroups (a row of S is 128 of them).
constexpr int kRegs = 168, kSoftmaxRegs = 216, kOtherRegs = 72;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kRegs, "no more than the CTA was launched with");
constexpr float kRescale = 8.0f;    // log2 units

template <int DP>
struct PromptShape {
    static constexpr int kPanels = DP / 64;
    static constexpr int kTile = kT * DP * 2;           // bytes of a K or V tile (and of a q tile)
    static constexpr int kStages = DP == 64 ? 4 : 2;
    static constexpr int kStage = 8 * 32 * 128;         // 128 bytes of an output row for each softmax thread
    static constexpr int kSmem = 1024 + 2 * kTile + 2 * kStages * kTile + kStage;
};

// D[tmem] (+)= A[tmem] * B[smem], bf16 inputs (A: two values a 32-bit column), fp32 accumulate.
CSA_DEV void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
CSA_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
CSA_DEV void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int h, int r, int p)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(h), "r"(r), "r"(p)
        : "memory");
}

// One lane of a converged warp.
CSA_DEV bool elect()
{
    uint32_t x;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(x));
    return x != 0;
}
CSA_DEV float max3(float x, float y, float z)
{
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
    return m;
}
// Bit i: token j + i is visible to the row (paged_visible), i < 32.
CSA_DEV uint32_t below32(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }
CSA_DEV uint32_t visible32(const RowBounds& r, int j)
{
    return below32(r.hi - j) & (~below32(r.lo - j) | below32(r.sink - j));
}
// Bits 4 x .. 4 x + 3 of `have`, each for 8 tokens.
CSA_DEV uint32_t pages32(uint32_t have, int x)
{
    const uint32_t h = have >> (4 * x);
    return (h & 1) * 0xffu | (h >> 1 & 1) * 0xff00u | (h >> 2 & 1) * 0xff0000u | (h >> 3 & 1) * 0xff000000u;
}

template <int DP, bool kOne, bool kHoles>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_prompt(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ PagedAttnArgs a, const int box_rows)
{
    using S = PromptShape<DP>;
    constexpr int NS = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sQ = smem;                    // two tiles
    uint8_t* sK = smem + 2 * S::kTile;     // [NS]
    uint8_t* sV = sK + NS * S::kTile;      // [NS]
    uint8_t* sO = sV + NS * S::kTile;      // [8 warps][32 rows][128 bytes]
    __shared__ uint64_t Qfull[2], Sfull[2], Pready[2][2], Ofull[2], Joined, Kfull[NS], Kempty[NS], Vfull[NS], Vempty[NS], drained;
    // Of a unit: bit i: rows 8 i .. 8 i + 7 have a page.  Written before its K, read after its S, before its P; K of
    // unit n is written once S(n - NS) is done, which follows P(n - NS - 2), so unit n - 2 NS has been read.
    __shared__ uint32_t have[2 * NS];
    __shared__ uint32_t tmem_slot;
    // before the first tiles arrive
    PagedScratch<kThreads, 8>& sh = *reinterpret_cast<PagedScratch<kThreads, 8>*>(sK);
    __shared__ PagedCursor cursors[8];     // of the softmax warps, whose registers hold S
    __shared__ volatile int failed;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&Qfull[i], kM / 32);
            tc::mbar_init(&Sfull[i], 1);
            for (int half = 0; half < 2; ++half) tc::mbar_init(&Pready[i][half], kM / 32);
            tc::mbar_init(&Ofull[i], 1);
        }
        tc::mbar_init(&Joined, kM / 32);
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&Kfull[i], 1);
            tc::mbar_init(&Kempty[i], 1);
            tc::mbar_init(&Vfull[i], 1);
            tc::mbar_init(&Vempty[i], 1);
        }
        tc::mbar_init(&drained, 1);
        failed = 0;
        tc::tma_prefetch_desc(&map_k);
        tc::tma_prefetch_desc(&map_v);
        tc::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    pdl_launch_dependents();  // with the TMEM in hand: no later kernel of the stream can wait for it and hold it up
    // S of tile w at column w kT, O at 2 kT + w DP
    auto tS = [&](int w) { return tmem + w * kT; };
    auto tO = [&](int w) { return tmem + 2 * kT + w * DP; };
    pdl_wait();
    if (tid == 0) a.desc[cta] = make_int4(-1, 0, 0, 0);
    PagedCursor c;
    const bool some = paged_schedule<kThreads, 8, false>(a, cta, sh, c);
    // false after a timeout; the caller leaves its loops
    auto wait_for = [&](uint64_t* bar, uint32_t phase, long long budget) {
        // no sleep between the polls: a wake-up costs more than the waits of this kernel last
        if (tc::mbar_test(bar, phase & 1)) return true;
        const long long t0 = clock64();
        do {
            if (clock64() - t0 > budget) {
                failed = 1;
                return false;
            }
        } while (!tc::mbar_try_wait(bar, phase & 1));
        return true;
    };
    auto wait = [&](uint64_t* bar, uint32_t phase) { return wait_for(bar, phase, a.wait_budget); };
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };  // a warp gives up as one

    if (some && warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ------------------------------------------------------------ softmax
        const int w = warp >> 2, r = tid & (kM - 1);  // tile, row in it
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tS(w) + quarter, o_at = tO(w) + quarter;
        constexpr int kStep = kOne ? 2 : 1;                     // of a warpgroup's units
        const int row0 = kOne ? 0 : w * kM, unit0 = kOne ? w : 0;  // its first row and unit
        const bool has_q = !kOne || w == 0;
        // units and segments (and joins) of this warpgroup, V tiles: the barriers' phases
        uint32_t n_s = 0, n_o = 0, n_v = 0;
        // A row's part of a segment: loaded while the last product of the segment before runs
        struct Row {
            bool tile, in;  // the warpgroup's tile has rows; this is one
            bool holes;     // of the item
            int64_t at;
            RowBounds rb;
        };
        // one arrival a warp: 32 on one barrier take their turns, about 400 clocks a half unit
        auto arrive = [&](uint64_t* bar) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar);
        };
        auto row_of = [&](const PagedEntry& en, int h) {
            Row x;
            const int n_rows = paged_rows(a, en.tile);
            x.tile = kOne || row0 < n_rows;
            x.in = row0 + r < n_rows;
            x.holes = kHoles && paged_holes<32>(a, en);
            x.at = x.in ? paged_out_row(a, en.b, en.tile, h, row0 + r) : 0;
            x.rb = x.in ? paged_bounds(a, en.b, (en.tile * a.R + row0 + r) / a.G) : RowBounds{0, 0, 0};
            return x;
        };
        // q of the warp's 32 rows, kC lanes to a row
        constexpr int kC = DP / 8, kRowsAtOnce = 32 / kC;
        const int qc = lane % kC, qr = lane / kC;
        auto load_q = [&](const Row& x) {
            const char* mine = static_cast<const char*>(a.q) + x.at * a.d * 2;
            const uint32_t ins = __ballot_sync(0xffffffffu, x.in);
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const int rr = i * kRowsAtOnce + qr;
                const char* from = reinterpret_cast<const char*>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), rr));
                const bool in = (ins >> rr & 1) && qc * 8 < a.d;
                const uint32_t to = tc::smem_u32(sQ) + w * S::kTile + (qc >> 3) * (kM * 128) +
                                    tc::sw128_offset((r & ~31) + rr, qc & 7);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from + (in ? qc * 16 : 0)),
                             "r"(in ? 16 : 0)
                             : "memory");
            }
        };
        auto give_q = [&] {
            asm volatile("cp.async.wait_all;" ::: "memory");
            tc::fence_proxy_async_smem();
            arrive(&Qfull[w]);
        };
        PagedCursor& cur = cursors[warp];
        if (lane == 0) cur = c;
        __syncwarp();
        auto next = [&](const PagedSegment& sg) {
            const int64_t at = cur.at + sg.places;
            if (at >= cur.end) return false;
            int h = cur.h + 1;
            PagedEntry en;
            const bool other = h == a.n_kv;
            if (other) {
                h = 0;
                en = paged_entry<32>(a, cur.e + 1);
            }
            __syncwarp();
            if (lane == 0) {
                cur.at = at;
                cur.u = 0;
                cur.h = h;
                if (other) {
                    ++cur.e;
                    cur.en = en;
                }
            }
            __syncwarp();
            return true;
        };
        PagedSegment sg = paged_segment(a, cur, cta);
        bool ok = true, more = sg.u0 < sg.u1;
        Row row;
        if (more) {
            row = row_of(cur.en, cur.h);
            if (has_q && row.tile) {
                load_q(row);
                give_q();
            }
        }
        while (more) {
            if (tid == 0) paged_describe(a, cur, sg, cta);
            const int b = cur.en.b, tile = cur.en.tile, h = cur.h;
            float m = -INFINITY, l = 0.f;  // m: what the weights in O and l are relative to
            if (row.tile) {
                float* lg = a.logits && row.in ? a.logits + (((int64_t)b * a.n_kv + h) * (a.nq * a.G) +
                                                             tile * a.R + row0 + r) * a.cap
                                               : nullptr;
                for (int u = sg.u0 + unit0; u < sg.u1; u += kStep, ++n_s) {
                    const uint32_t vt = n_v + (uint32_t)(u - sg.u0), vs = vt % NS;
                    ok = all(wait(&Sfull[w], n_s));
                    if (!ok) break;
                    tc::fence_after_sync();
                    const PagedEntry& en = cur.en;
                    const int j0 = en.first_token(u, kT);
                    const uint32_t hv = have[vt % (2 * NS)];
                    const bool clear = j0 >= en.lo_max && j0 + kT <= en.hi_min && hv == 0xffffu;
                    if (!clear) {
                        // rows of V that no query sees: thread r has row r
                        ok = all(wait(&Vfull[vs], vt / NS));
                        if (!ok) break;
                        if (!paged_seen(a, en, row.holes, j0 + r)) {
#pragma unroll
                            for (int x = 0; x < DP / 8; ++x)
                                *reinterpret_cast<uint4*>(sV + vs * S::kTile + (x >> 3) * (kT * 128) +
                                                          tc::sw128_offset(r, x & 7)) = make_uint4(0, 0, 0, 0);
                        }
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                    }
                    uint32_t s[4][32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tc::tmem_ld32_async(s_at + 32 * i, s[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) tc::tmem_wait_ld_regs(s[i]);  // all have landed; each names its registers
                    if (!clear) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t see = visible32(row.rb, j0 + 32 * x) & pages32(hv, x);
                            if (__any_sync(0xffffffffu, see != ~0u)) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (!(see >> i & 1)) s[x][i] = __float_as_uint(-INFINITY);
                            }
                        }
                    }
                    if (lg) {
#pragma unroll
                        for (int i = 0; i < kT; ++i)
                            if (j0 + i < a.cap) lg[j0 + i] = __uint_as_float(s[i >> 5][i & 31]) * a.scale_log2;
                    }
                    __syncwarp();
                    float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < kT; i += 8)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            t4[x] = max3(t4[x], __uint_as_float(s[i >> 5][(i + 2 * x) & 31]),
                                         __uint_as_float(s[i >> 5][(i + 2 * x + 1) & 31]));
                    float top = max3(t4[0], t4[1], fmaxf(t4[2], t4[3]));
                    top *= a.scale_log2;
                    const bool grow = top > m + kRescale;  // m = -inf: as soon as anything is visible
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = grow ? exp2f(m - top) : 1.f;
                        if (grow) m = top;
                        l *= f;
                        if (u > sg.u0 + unit0) {  // before the first product O holds nothing of this segment
#pragma unroll 1
                            for (int x = 0; x < DP; x += 32) {
                                uint32_t o[16], o1[16];
                                tc::tmem_ld16_async(o_at + x, o);
                                tc::tmem_ld16_async(o_at + x + 16, o1);
                                tc::tmem_wait_ld_regs16(o, o1);
#pragma unroll
                                for (int y = 0; y < 16; ++y) {
                                    o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                                    o1[y] = __float_as_uint(__uint_as_float(o1[y]) * f);
                                }
                                tmem_st16(o_at + x, o);
                                tmem_st16(o_at + x + 16, o1);
                            }
                        }
                    }
                    const float neg = m == -INFINITY ? 0.f : -m;
                    const float2 sc = make_float2(a.scale_log2, a.scale_log2), sb = make_float2(neg, neg);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t p[16];
                    auto weights = [&](const uint32_t (&v)[32]) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 x = tc::fma2(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sc, sb);
                            x.x = tc::ex2_approx(x.x);
                            x.y = tc::ex2_approx(x.y);
                            sum[i & 1] = tc::fma2(x, make_float2(1.f, 1.f), sum[i & 1]);
                            p[i] = pack2(x.x, x.y);
                        }
                    };
                    auto hand_over = [&](int half) {
                        tc::tmem_wait_st();
                        tc::fence_before_sync();
                        arrive(&Pready[w][half]);
                    };
                    weights(s[0]);
                    tmem_st16(s_at, p);
                    weights(s[1]);
                    tmem_st16(s_at + 16, p);
                    weights(s[2]);
                    hand_over(0);  // its stores were done under the third quarter's exponentials
                    tmem_st16(s_at + 32, p);
                    weights(s[3]);
                    tmem_st16(s_at + 48, p);
                    hand_over(1);
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                }
            }
            n_v += (uint32_t)(sg.u1 - sg.u0);
            const PagedSegment done = sg;
            const Row out = row;
            more = ok && next(sg);
            if (more) {
                sg = paged_segment(a, cur, cta);
                more = sg.u0 < sg.u1;
            }
            if (more) {
                row = row_of(cur.en, cur.h);
                // S of the last unit was there: no product reads q any more, but the other warpgroup's of the same tile
                if (!kOne && row.tile) load_q(row);
            }
            if (out.tile && ok) ok = all(wait(&Ofull[w], n_o++));
            if (!ok) break;
            // every product of the segment is done
            if (more && has_q && row.tile) {
                if (kOne) load_q(row);
                give_q();
            }
            // Warps 4-7 leave their maximum and sum in their part of sO.  Warps 0-3 have read it, and O of both, before
            // they hand over the first P of the next segment, which its products and Ofull follow.
            if (kOne && w == 1) {
                reinterpret_cast<float2*>(sO + warp * (32 * 128))[lane] = make_float2(m, l);
                arrive(&Joined);
            } else if (out.tile) {
                float fa = 1.f, fb = 0.f;
                if constexpr (kOne) {
                    ok = all(wait(&Joined, n_o - 1));
                    if (!ok) break;
                    const float2 ml = reinterpret_cast<const float2*>(sO + (warp + 4) * (32 * 128))[lane];
                    const float top = fmaxf(m, ml.x);
                    fa = m == -INFINITY ? 0.f : exp2f(m - top);
                    fb = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
                    m = top;
                    l = l * fa + ml.y * fb;
                }
                const bool two = kOne && done.u1 - done.u0 > 1;  // else nothing was written to the other O
                tc::fence_after_sync();
                const int64_t slot = (int64_t)done.slot * a.R + row0 + r;
                const float inv = done.whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                fa *= inv;
                fb *= inv;
                // through shared memory, so that a warp writes whole lines: 128 bytes of each of its rows at a time,
                // 16-byte chunks swizzled by the row
                uint8_t* so = sO + warp * (32 * 128);
                const bool bf16 = done.whole && a.out_bf16;
                char* mine = bf16         ? static_cast<char*>(a.out) + out.at * a.d * 2
                             : done.whole ? static_cast<char*>(a.out) + out.at * a.d * 4
                                          : reinterpret_cast<char*>(a.part_o + slot * a.d);
                const uint32_t ins = __ballot_sync(0xffffffffu, out.in);
                const int row_bytes = a.d * (bf16 ? 2 : 4);
                auto flush = [&](int byte) {  // 8 lanes to a row
                    __syncwarp();
                    const int k = lane & 7, at = byte + k * 16;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = 4 * i + (lane >> 3);
                        char* to = reinterpret_cast<char*>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), rr));
                        if ((ins >> rr & 1) && at < row_bytes)
                            *reinterpret_cast<uint4*>(to + at) =
                                *reinterpret_cast<const uint4*>(so + rr * 128 + ((k ^ (rr & 7)) << 4));
                    }
                    __syncwarp();
                };
#pragma unroll
                for (int x = 0; x < DP; x += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32_async(o_at + x, o);
                    tc::tmem_wait_ld_regs(o);
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * fa);
                    if (two) {
                        uint32_t o1[32];
                        tc::tmem_ld32_async(tO(1) + quarter + x, o1);
                        tc::tmem_wait_ld_regs(o1);
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            o[y] = __float_as_uint(fmaf(__uint_as_float(o1[y]), fb, __uint_as_float(o[y])));
                    }
                    if (bf16) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float* v = reinterpret_cast<const float*>(o) + 8 * k;
                            *reinterpret_cast<uint4*>(so + lane * 128 + (((x / 8 % 8 + k) ^ (lane & 7)) << 4)) =
                                make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
                        }
                        if (x % 64 == 32) flush((x - 32) * 2);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<uint4*>(so + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                                make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                        flush(x * 4);
                    }
                }
                if (out.in) {
                    if (done.whole)
                        paged_store_lse(a, out.at, b, tile, h, row0 + r, m, l);
                    else
                        a.part_ml[slot] = make_float2(m, l);
                }
                __syncwarp();
                tc::fence_before_sync();  // these loads, before the next segment's products write O
            }
        }
    } else if (some) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kKWarp || warp == kVWarp) {
            // ------------------------------------------------------------ K or V
            // a warp each: K of the units ahead does not wait for a free stage of V, and twice as many small boxes are
            // asked for (one tile by one warpgroup, pages of 16, d = 128: 141 -> 124 us; pages of 64: the same within 3%)
            const bool is_v = warp == kVWarp;
            const CUtensorMap* const map = is_v ? &map_v : &map_k;
            uint64_t *const fulls = is_v ? Vfull : Kfull, *const empties = is_v ? Vempty : Kempty;
            uint8_t* const tiles = is_v ? sV : sK;
            tc::fence_proxy_async_smem();  // the schedule's scratch, before the tiles over it
            uint32_t n = 0;  // tiles begun
            bool ok = true;
            const int boxes = kT / box_rows, none = (int)a.pl.n_pages;
            while (ok) {
                const PagedSegment sg = paged_segment(a, c, cta);
                if (sg.u0 == sg.u1) break;
                for (int u = sg.u0; u < sg.u1; ++u, ++n) {
                    const int j = c.en.first_token(u, kT) + lane * box_rows;
                    int page = none, in = 0;
                    const bool any = j < c.en.hi_max && (j < c.en.sink || j + box_rows > c.en.lo_min);
                    if (lane < boxes && any && j < a.cap) {
                        const int p = j / a.pl.page;
                        const int id = a.pl.table[(int64_t)c.en.b * a.pl.max_pages + p];
                        if ((uint32_t)id < (uint32_t)none) {
                            page = id;
                            in = j - p * a.pl.page;
                        }
                    }
                    const unsigned there = __ballot_sync(0xffffffffu, page != none);
                    uint32_t hv = 0;
                    for (int i = 0; i < kT / 8; ++i) hv |= (there >> (i * 8 / box_rows) & 1u) << i;
                    const uint32_t st = n % NS;
                    ok = all(wait(&empties[st], n / NS + 1));  // of the first round: passes at once
                    if (!ok) break;
                    if (lane == 0) {
                        if (!is_v) have[n % (2 * NS)] = hv;
                        tc::mbar_arrive_expect_tx(&fulls[st], S::kTile);
                    }
                    __syncwarp();
                    if (lane < boxes) {
                        uint8_t* dst = tiles + st * S::kTile + lane * box_rows * 128;
#pragma unroll
                        for (int x = 0; x < S::kPanels; ++x)
                            tma_load_4d(dst + x * (kT * 128), map, &fulls[st], x * 64, c.h, in, page);
                    }
                }
                if (!ok || !paged_next<32, false>(a, c, sg)) break;
            }
            // No copy is in flight when the CTA ends, whichever warp gave up: on the normal path the products wait for them,
            // but after a timeout elsewhere they may not have.
            for (uint32_t k = n >= NS ? n - NS : 0; k < n; ++k) wait_for(&fulls[k % NS], k / NS, tc::kWaitBudget);
        } else if (warp == kMmaWarp) {
            // ------------------------------------------------------------ products
            constexpr uint32_t kIdescS = tc::idesc_bf16_f32(kM, kT, false, false);
            constexpr uint32_t kIdescO = tc::idesc_bf16_f32(kM, DP, false, true);
            uint32_t n = 0;                     // tiles used
            uint32_t n_p[2] = {0, 0}, n_q[2] = {0, 0};  // phases of Pready and Qfull
            bool ok = true;
            // The issue is on the path between a tile's P and its next S.  The whole warp runs these loops, so that
            // descriptors stay in uniform registers, and one lane is elected to issue; a descriptor is one addition:
            // the low words of the tiles' descriptors (16-byte address units), and their common high words.
            const uint64_t dk = tc::smem_desc_sw128(0, 16, 1024), dv = tc::smem_desc_sw128(0, kT * 128, 1024);
            const uint32_t q0 = (uint32_t)dk + (tc::smem_u32(sQ) >> 4), k0 = (uint32_t)dk + (tc::smem_u32(sK) >> 4),
                           v0 = (uint32_t)dv + (tc::smem_u32(sV) >> 4);
            const uint32_t dk_hi = (uint32_t)(dk >> 32), dv_hi = (uint32_t)(dv >> 32);
            constexpr uint32_t kTileStep = S::kTile >> 4;
            auto desc = [](uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; };
            // by the elected lane
            auto mma_s = [&](int w, uint32_t st) {
                const uint32_t q = q0 + (kOne ? 0 : w * kTileStep), k = k0 + st * kTileStep;
#pragma unroll
                for (int x = 0; x < DP / 16; ++x) {
                    const uint32_t at = ((x >> 2) * (kM * 128) + (x & 3) * 32) >> 4;
                    tc::mma_bf16_ss(tS(w), desc(q + at, dk_hi), desc(k + at, dk_hi), kIdescS, x ? 1u : 0u);
                }
                tc::mma_commit(&Sfull[w]);
            };
            auto mma_o = [&](int w, uint32_t st, int half, bool more) {
                const uint32_t v = v0 + st * kTileStep;
#pragma unroll
                for (int x = half * (kH / 16); x < (half + 1) * (kH / 16); ++x)
                    mma_bf16_ts(tO(w), tS(w) + x * 8, desc(v + (x * 16 * 128 >> 4), dv_hi), kIdescO,
                                more || x ? 1u : 0u);
            };
            while (ok) {
                const PagedSegment sg = paged_segment(a, c, cta);
                if (sg.u0 == sg.u1) break;
                const int n_u = sg.u1 - sg.u0;
                if constexpr (kOne) {
                    // The units in turn, S two units ahead.  No wait is for a K or V that needs a later step: K(u + 2)
                    // takes a stage that S(u) has left at the latest, V(u) one that P(u - 2) V has (NS >= 2).
                    ok = all(wait(&Qfull[0], n_q[0]++));
                    for (int w = 0; w < 2 && w < n_u && ok; ++w) {
                        const uint32_t st = (n + w) % NS;
                        ok = all(wait(&Kfull[st], (n + w) / NS));
                        if (!ok) break;
                        tc::fence_after_sync();
                        if (elect()) {
                            mma_s(w, st);
                            tc::mma_commit(&Kempty[st]);
                        }
                        __syncwarp();
                    }
                    for (int u = 0; u < n_u && ok; ++u, ++n) {
                        const uint32_t st = n % NS, nx = (n + 2) % NS;
                        const bool more = u + 2 < n_u;
                        const int w = u & 1;
                        const uint32_t ph = w ? n_p[1] : n_p[0];
                        ok = all(wait(&Vfull[st], n / NS)) && all(wait(&Pready[w][0], ph));
                        if (!ok) break;
                        tc::fence_after_sync();
                        if (elect()) mma_o(w, st, 0, u > 1);
                        __syncwarp();
                        if (more) ok = all(wait(&Kfull[nx], (n + 2) / NS));
                        ok = ok && all(wait(&Pready[w][1], ph));
                        if (!ok) break;
                        ++(w ? n_p[1] : n_p[0]);
                        tc::fence_after_sync();
                        if (elect()) {
                            mma_o(w, st, 1, true);
                            if (more) {
                                mma_s(w, nx);
                                tc::mma_commit(&Kempty[nx]);
                            }
                            tc::mma_commit(&Vempty[st]);
                            if (u + 1 == n_u) {
                                tc::mma_commit(&Ofull[0]);
                                tc::mma_commit(&Ofull[1]);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok || !paged_next<32, false>(a, c, sg)) break;
                    continue;
                }
                const int tiles = paged_rows(a, c.en.tile) > kM ? 2 : 1;
                ok = all(wait(&Kfull[n % NS], n / NS));
                for (int w = 0; w < tiles && ok; ++w) {
                    ok = all(wait(&Qfull[w], n_q[w]++));
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (elect()) {
                        mma_s(w, n % NS);
                        if (w == tiles - 1) tc::mma_commit(&Kempty[n % NS]);
                    }
                    __syncwarp();
                }
                for (int u = 0; u < n_u && ok; ++u, ++n) {
                    const uint32_t st = n % NS, nx = (n + 1) % NS;
                    const bool more = u + 1 < n_u;
                    ok = all(wait(&Vfull[st], n / NS));
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        if (!ok || w >= tiles) continue;
                        ok = all(wait(&Pready[w][0], n_p[w]));
                        if (!ok) continue;
                        tc::fence_after_sync();
                        if (elect()) mma_o(w, st, 0, u > 0);
                        __syncwarp();
                        if (w == 0 && more) ok = all(wait(&Kfull[nx], (n + 1) / NS));
                        ok = ok && all(wait(&Pready[w][1], n_p[w]));
                        if (!ok) continue;
                        ++n_p[w];
                        tc::fence_after_sync();
                        if (elect()) {
                            mma_o(w, st, 1, true);
                            if (more)
                                mma_s(w, nx);  // over the P that was just used
                            else
                                tc::mma_commit(&Ofull[w]);
                            if (w == tiles - 1) {
                                tc::mma_commit(&Vempty[st]);
                                if (more) tc::mma_commit(&Kempty[nx]);
                            }
                        }
                        __syncwarp();
                    }
                }
                if (!ok || !paged_next<32, false>(a, c, sg)) break;
            }
            // nor a product: they read shared memory and write TMEM
            if (elect()) tc::mma_commit(&drained);
            __syncwarp();
            wait_for(&drained, 0, tc::kWaitBudget);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && failed) a.desc[cta].w = 1;
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int DP, bool kOne, bool kHoles>
int launch_one(const PagedAttnArgs& a, const CUtensorMap& k, const CUtensorMap& v, int box_rows, cudaStream_t stream)
{
    constexpr int smem = PromptShape<DP>::kSmem;
    if (!paged_allow_smem<paged_attn_prompt<DP, kOne, kHoles>>(smem)) return CSA_ERR_CUDA;
    launch_pdl(paged_attn_prompt<DP, kOne, kHoles>, dim3(a.runs), dim3(kThreads), smem, stream, k, v, a, box_rows);
    return launch_status();
}

template <int DP, bool kOne>
int launch(const PagedAttnArgs& a, const CUtensorMap& k, const CUtensorMap& v, int box_rows, cudaStream_t stream)
{
    return a.may_have_holes() ? launch_one<DP, kOne, true>(a, k, v, box_rows, stream)
                              : launch_one<DP, kOne, false>(a, k, v, box_rows, stream);
}

}  // namespace

bool paged_prompt_takes(const PagedPool& pl, int n_kv, int d)
{
    // TMA: boxes of 8 rows or more that lie in one page, strides that a tensor map can hold
    constexpr int64_t kMaxStride = (int64_t)1 << 38;  // elements
    return d <= 128 && pl.page % 8 == 0 && pl.n_pages >= 1 && pl.n_pages < INT32_MAX &&
           (pl.n_pages == 1 || pl.ld_page > 0) && pl.ld_page < kMaxStride && pl.ld_row < kMaxStride &&
           (n_kv == 1 || pl.ld_head < kMaxStride);
}

PagedShape paged_prompt_shape(int d)
{
    PagedShape s{};
    s.kind = kPagedPrompt;
    s.DP = d <= 64 ? 64 : 128;
    s.R = 2 * kM;
    s.unit = kT;
    s.min_units = 2;
    s.item_units = 2;
    s.workers = kNumSMs;
    return s;
}

int launch_paged_prompt(const PagedAttnArgs& a, const PagedShape& s, cudaStream_t stream)
{
    const PagedPool& pl = a.pl;
    int rows = 128;  // of a box: the largest power of two that divides the page
    while (pl.page % rows) rows >>= 1;
    // strides of dimensions of size 1 are never used, but have to be valid
    const int64_t ld_head = a.n_kv > 1 ? pl.ld_head : align_up(a.d, 8);
    const int64_t ld_page = pl.n_pages > 1 ? pl.ld_page : pl.ld_row;
    CUtensorMap k, v;
    for (int i = 0; i < 2; ++i)
        if (!make_tmap_bf16_4d(i ? &v : &k, i ? a.V : a.K, a.d, a.n_kv, pl.page, pl.n_pages, ld_head, pl.ld_row, ld_page,
                               64, rows))
            return CSA_ERR_CUDA;
    // every item has one tile
    if (a.nq * a.G <= kM)
        return s.DP == 64 ? launch<64, true>(a, k, v, rows, stream) : launch<128, true>(a, k, v, rows, stream);
    return s.DP == 64 ? launch<64, false>(a, k, v, rows, stream) : launch<128, false>(a, k, v, rows, stream);
}

}  // namespace csa
