// paged_evict: cuts a cache back to its heaviest tokens.
//
// For every (sequence, key head) with n cached tokens, min(n, keep) stay: the first n_sink, the last
// n_recent, and of the others those with the largest accumulated weight (ties: the lower index).
// They keep their order and move to the pages of new_table.  Two kernels: the selection, and
// the copy of the selected rows, which is what the call's bytes are.
#include "paged.cuh"

namespace csa {

int paged_pool_check(const PagedPool& pl, int B, int n_kv, int d);

namespace {

struct EvictArgs {
    char *K, *V;
    PagedPool from, to;    // strides in bytes
    const int64_t* lens;   // [B]
    const float* acc;      // [B][n_kv][cap]
    int64_t* new_lens;     // [B]
    float* new_acc;        // [B][n_kv][new_cap]
    int32_t* idx;          // [B][n_kv][keep]
    int B, n_kv, keep, n_sink, n_recent, cap, new_cap;
    int words;             // words of VT in a row
};

CSA_DEV int evict_len(const EvictArgs& a, int b)
{
    return (int)min(max(a.lens[b], (int64_t)0), (int64_t)a.cap);
}

constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;

// Order of the weights; a NaN goes below every number (and is evicted first).
CSA_DEV uint32_t weight_key(float x) { return x != x ? 0u : order_key(x); }

// Inclusive prefix sum over the CTA; sh has kSelThreads / 32 elements.  All threads get the total.
CSA_DEV int block_scan(int v, int* sh, int& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
        const int x = sh[w];
        if (w < warp) before += x;
        total += x;
    }
    return v + before;
}

// One CTA per (sequence, key head).  The keep-th largest weight is found by radix: 11, 11 and 10
// bits of the order key, a histogram of the keys that match the bits found so far in each pass.
__global__ void __launch_bounds__(kSelThreads) paged_evict_select(EvictArgs a)
{
    __shared__ int hist[kSelBins];
    __shared__ int sh[kSelThreads / 32];
    __shared__ uint32_t s_digit;
    __shared__ int s_above;
    const int tid = threadIdx.x, h = blockIdx.x, b = blockIdx.y;
    pdl_launch_dependents();
    pdl_wait();
    const int n = evict_len(a, b), kept = min(n, a.keep);
    const int64_t g = (int64_t)b * a.n_kv + h;
    const float* acc = a.acc + g * a.cap;
    float* new_acc = a.new_acc + g * a.new_cap;
    int32_t* idx = a.idx + g * a.keep;
    if (h == 0 && tid == 0) a.new_lens[b] = kept;
    if (n <= a.keep) {
        for (int j = tid; j < a.keep; j += kSelThreads) idx[j] = j < n ? j : -1;
        for (int j = tid; j < a.new_cap; j += kSelThreads) new_acc[j] = j < n ? acc[j] : 0.f;
        return;
    }
    // n > keep >= n_sink + n_recent: `want` of the tokens [first, last) stay
    const int first = a.n_sink, last = n - a.n_recent;
    int want = a.keep - a.n_sink - a.n_recent;
    uint32_t prefix = 0;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int x = tid; x < kSelBins; x += kSelThreads) hist[x] = 0;
        __syncthreads();
        for (int j = first + tid; j < last; j += kSelThreads) {
            const uint32_t k = weight_key(acc[j]);
            if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
        }
        __syncthreads();
        // digits from the top: thread x has digits 2047 - 2 x and 2046 - 2 x
        const int hi = hist[kSelBins - 1 - 2 * tid], lo = hist[kSelBins - 2 - 2 * tid];
        int total;
        const int inc = block_scan(hi + lo, sh, total), exc = inc - hi - lo;
        if (tid == 0) {
            s_digit = 0;
            s_above = 0;
        }
        __syncthreads();
        // the digit at which the count from the top reaches `want` (want = 0: above every digit)
        if (want > exc && want <= exc + hi) {
            s_digit = kSelBins - 1 - 2 * tid;
            s_above = exc;
        } else if (want > exc + hi && want <= inc) {
            s_digit = kSelBins - 2 - 2 * tid;
            s_above = exc + hi;
        }
        __syncthreads();
        prefix = (prefix << bits) | s_digit;
        want -= s_above;
        __syncthreads();
    }
    // keys above `prefix` stay, and the first `want` of those equal to it
    const bool none = a.keep == a.n_sink + a.n_recent;
    int out = 0, equal = 0;
    for (int base = 0; base < n; base += kSelThreads) {
        const int j = base + tid;
        bool above = false, tie = false;
        if (j < n) {
            if (j < first || j >= last)
                above = true;
            else if (!none) {
                const uint32_t k = weight_key(acc[j]);
                above = k > prefix;
                tie = k == prefix;
            }
        }
        int ties, n_ties, n_out;
        ties = block_scan(tie, sh, n_ties);
        const bool stay = above || (tie && equal + ties <= want);
        const int at = out + block_scan(stay, sh, n_out) - 1;
        if (stay) {
            idx[at] = j;
            new_acc[at] = acc[j];
        }
        out += n_out;
        equal += n_ties;
    }
    for (int j = a.keep + tid; j < a.new_cap; j += kSelThreads) new_acc[j] = 0.f;
}

constexpr int kMoveThreads = 256;

// One thread moves one word of a K row and of a V row.  The pages of new_table are not among those
// that the call reads, so the words may move in any order.
template <typename VT>
__global__ void __launch_bounds__(kMoveThreads) paged_evict_move(EvictArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t x = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x;
    // words of one kept slot of all key heads lie together, as they do in a page
    const int64_t per_slot = (int64_t)a.n_kv * a.words, per_seq = per_slot * a.keep;
    const int b = (int)(x / per_seq);
    if (b >= a.B) return;
    const int64_t in = x - b * per_seq;
    const int s = (int)(in / per_slot);
    const int hw = (int)(in - s * per_slot), h = hw / a.words, w = hw - h * a.words;
    const int j = a.idx[((int64_t)b * a.n_kv + h) * a.keep + s];
    if (j < 0) return;
    const int64_t src = paged_row(a.from, b, j), dst = paged_row(a.to, b, s);
    if (dst < 0) return;
    VT kx{}, vx{};  // a token without a page reads as zeros
    if (src >= 0) {
        const int64_t o = src + h * a.from.ld_head + (int64_t)w * sizeof(VT);
        kx = *reinterpret_cast<const VT*>(a.K + o);
        vx = *reinterpret_cast<const VT*>(a.V + o);
    }
    const int64_t o = dst + h * a.to.ld_head + (int64_t)w * sizeof(VT);
    *reinterpret_cast<VT*>(a.K + o) = kx;
    *reinterpret_cast<VT*>(a.V + o) = vx;
}

}  // namespace
}  // namespace csa

extern "C" int paged_evict(void* K, void* V, int64_t pool_ld_page, int64_t pool_ld_row, int64_t pool_ld_head,
                           int64_t n_pages, int page, const int32_t* table, int max_pages, const int64_t* lens,
                           const float* acc, int B, int n_kv, int d, int keep, int n_sink, int n_recent,
                           const int32_t* new_table, int new_max_pages, int64_t* new_lens, float* new_acc,
                           int32_t* idx_out, int dtype, csa_stream_t stream)
{
    using namespace csa;
    if (dtype != CSA_BF16 && dtype != CSA_F32) return CSA_ERR_DTYPE;
    PagedPool from{pool_ld_page, pool_ld_row, pool_ld_head, n_pages, page, table, max_pages};
    PagedPool to = from;
    to.table = new_table;
    to.max_pages = new_max_pages;
    int st = paged_pool_check(from, B, n_kv, d);
    if (st == CSA_OK) st = paged_pool_check(to, B, n_kv, d);
    if (st != CSA_OK) return st;
    if (keep < 1 || n_sink < 0 || n_recent < 0 || (int64_t)n_sink + n_recent > keep ||
        (int64_t)new_max_pages * page < keep)
        return CSA_ERR_ARG;
    if (B > 65535) return CSA_ERR_UNSUPPORTED;
    if (B == 0) return CSA_OK;
    if (!K || !V || !lens || !new_table || !new_lens || !new_acc || !idx_out || (max_pages > 0 && (!table || !acc)))
        return CSA_ERR_ARG;
    // in place is refused: the rows move in any order
    if (table == new_table || lens == new_lens || acc == new_acc) return CSA_ERR_ARG;
    const int eb = elem_bytes(dtype);
    const uintptr_t ptrs = (uintptr_t)K | (uintptr_t)V;
    if ((ptrs & (eb - 1)) ||
        (((uintptr_t)table | (uintptr_t)new_table | (uintptr_t)acc | (uintptr_t)new_acc | (uintptr_t)idx_out) & 3) ||
        (((uintptr_t)lens | (uintptr_t)new_lens) & 7))
        return CSA_ERR_ALIGN;
    EvictArgs a{};
    a.K = static_cast<char*>(K);
    a.V = static_cast<char*>(V);
    a.from = from;
    a.to = to;
    for (PagedPool* p : {&a.from, &a.to}) {
        p->ld_page *= eb;
        p->ld_row *= eb;
        p->ld_head *= eb;
    }
    a.lens = lens; a.acc = acc; a.new_lens = new_lens; a.new_acc = new_acc; a.idx = idx_out;
    a.B = B; a.n_kv = n_kv; a.keep = keep; a.n_sink = n_sink; a.n_recent = n_recent;
    a.cap = max_pages * page;
    a.new_cap = new_max_pages * page;
    const int64_t lds = a.from.ld_page | a.from.ld_row | a.from.ld_head | (d * eb);
    const bool wide = (ptrs & 15) == 0 && (lds & 15) == 0;
    const int wb = wide ? 16 : eb;
    a.words = d * eb / wb;
    const int64_t n = (int64_t)B * keep * n_kv * a.words, ctas = (n + kMoveThreads - 1) / kMoveThreads;
    if (ctas > INT32_MAX || (int64_t)n_kv * a.words > INT32_MAX) return CSA_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    launch_pdl(paged_evict_select, dim3(n_kv, B), dim3(kSelThreads), 0, s, a);
    st = launch_status();
    if (st != CSA_OK) return st;
    const dim3 grid((unsigned)ctas), block(kMoveThreads);
    if (wide)
        launch_pdl(paged_evict_move<uint4>, grid, block, 0, s, a);
    else if (eb == 2)
        launch_pdl(paged_evict_move<uint16_t>, grid, block, 0, s, a);
    else
        launch_pdl(paged_evict_move<uint32_t>, grid, block, 0, s, a);
    return launch_status();
}
