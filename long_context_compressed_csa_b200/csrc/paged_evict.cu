// paged_evict: cuts a cache back to its heaviest tokens.
//
// For every (sequence, key head) with n cached tokens, min(n, keep) stay: the first n_sink, the last
// n_recent, and of the others those with the largest accumulated weight (ties: the lower index).
// They keep their order and move to the pages of new_table.  Two kernels: the selection, and
// the copy of the selected rows, which is what the call's bytes are.
#include "cluster.cuh"
#include "paged.cuh"
#include "tc_utils.cuh"

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
    int cluster;           // CTAs that share the selection of a key head
};

CSA_DEV int evict_len(const EvictArgs& a, int b)
{
    return (int)min(max(a.lens[b], (int64_t)0), (int64_t)a.cap);
}

constexpr int kSelBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kKeys = 16;  // of a thread's registers

// Order of the weights; a NaN goes below every number (and is evicted first).
CSA_DEV uint32_t weight_key(float x) { return x != x ? 0u : order_key(x); }

// Inclusive prefix sum over the T threads of the CTA; sh has T / 32 elements.  All threads get the total.
template <int T>
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
    for (int w = 0; w < T / 32; ++w) {
        const int x = sh[w];
        if (w < warp) before += x;
        total += x;
    }
    return v + before;
}

// Elements of a shared array of CTA `rank` of the cluster.
CSA_DEV int remote(const int* p, uint32_t rank)
{
    int v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cl::peer_addr(tc::smem_u32(p), rank)) : "memory");
    return v;
}
CSA_DEV int2 remote2(const int* p, uint32_t rank, bool far)
{
    if (!far) return *reinterpret_cast<const int2*>(p);
    int2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "r"(cl::peer_addr(tc::smem_u32(p), rank))
                 : "memory");
    return v;
}

// One cluster of CTAs per (sequence, key head), its tokens cut into one run for each CTA.  The keep-th
// largest weight is found by radix: 11, 11 and 10 bits of the order key, a histogram of the keys that match the
// bits found so far in each pass.  A CTA sums its part of the digits over the cluster through distributed shared
// memory, and the one whose part holds the threshold tells the others its digit (each CTA reading all
// histograms took 10,000 clocks a pass with 8 CTAs).  Then each warp counts what stays of its own
// neighbouring tokens, and a prefix sum over the CTA and the CTAs before it gives their places in the output.
// Keys stay in registers when a run is no longer than T * kKeys, else each pass reads them again.
// Bound by latency, a chain of reads, shared-memory atomics and eleven cluster barriers (three a pass, two about the
// counts): 8 heads of 128K tokens take 45 us (384 with one CTA a head), 16 sequences of 8K about 27.
template <int T>
__global__ void __launch_bounds__(T, 1024 / T) paged_evict_select(EvictArgs a)
{
    __shared__ __align__(16) int hist[2][kSelBins];  // of even and odd lanes: weights share few exponents
    __shared__ int sh[T / 32];
    __shared__ int total_of, found[2];  // this CTA's part of the histogram; the digit, and the keys above it
    __shared__ int counts[2];           // of this CTA: keys above the threshold (and the safe ones), keys equal to it
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = a.cluster;
    const uint32_t rank = blockIdx.x % C;
    const int h = blockIdx.x / C, b = blockIdx.y;
    pdl_launch_dependents();
    pdl_wait();
    const int n = evict_len(a, b), kept = min(n, a.keep);
    const int64_t g = (int64_t)b * a.n_kv + h;
    const float* acc = a.acc + g * a.cap;
    float* new_acc = a.new_acc + g * a.new_cap;
    int32_t* idx = a.idx + g * a.keep;
    const int all = C * T, me = rank * T + tid;
    if (h == 0 && me == 0) a.new_lens[b] = kept;
    if (n <= a.keep) {
        for (int j = me; j < a.keep; j += all) idx[j] = j < n ? j : -1;
        for (int j = me; j < a.new_cap; j += all) new_acc[j] = j < n ? acc[j] : 0.f;
        return;  // the whole cluster
    }
    // n > keep >= n_sink + n_recent: `want` of the tokens [first, last) stay
    const int first = a.n_sink, last = n - a.n_recent;
    int want = a.keep - a.n_sink - a.n_recent;
    const bool none = want == 0;
    // this CTA's tokens [r0, r1), in chunks; of a chunk each warp has `rows` rows of 32 neighbouring ones
    const int run = (n + C - 1) / C, r0 = min(n, (int)rank * run), len = min(n - r0, run);
    const int rows = min(kKeys, (run + T - 1) / T), chunk = rows * T;
    uint32_t key[kKeys];
    auto token = [&](int64_t c0, int i) { return c0 + (warp * rows + i) * 32 + lane; };  // from r0
    // no branch around a load, so that all are under way at once: those past the run repeat its last token
    auto load = [&](int64_t c0) {
        float x[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) x[i] = acc[max((int64_t)0, r0 + min(token(c0, min(i, rows - 1)), (int64_t)len - 1))];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) key[i] = weight_key(x[i]);
    };
    load(0);
    const bool reload = len > chunk;
    uint32_t prefix = 0;
    for (int pass = 0; pass < 3 && !none; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int x = tid; x < 2 * kSelBins; x += T) hist[0][x] = 0;
        __syncthreads();
        for (int64_t c0 = 0; c0 < len; c0 += chunk) {
            if (reload) load(c0);
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                if (i >= rows) break;
                const int64_t x = token(c0, i), j = r0 + x;
                if (x < len && j >= first && j < last && (pass == 0 || (key[i] >> (shift + bits)) == prefix))
                    atomicAdd(&hist[lane & 1][(key[i] >> shift) & ((1u << bits) - 1)], 1);
            }
        }
        if (C > 1)
            cl::cluster_sync();
        else
            __syncthreads();
        // digits from the top: this CTA has kSelBins / C of them, thread x the x-th kD
        constexpr int kD = kSelBins / T;
        const int part = kSelBins / C, at = kSelBins - (int)rank * part - kD * (tid + 1);
        int digit[kD] = {}, mine = 0;  // rising
        if (kD * tid < part) {
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r)
                if (r < C)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int d = 0; d < kD; d += 2) {
                            const int2 v = remote2(&hist[x][at + d], r, C > 1);
                            digit[d] += v.x;
                            digit[d + 1] += v.y;
                        }
#pragma unroll
            for (int d = 0; d < kD; ++d) mine += digit[d];
        }
        int total;
        const int inc = block_scan<T>(mine, sh, total);
        int before = 0, owner = 0;  // keys in the parts of the CTAs before the threshold's, and that CTA
        if (C > 1) {
            if (tid == 0) total_of = total;
            cl::cluster_sync();
            const int t = lane < C ? remote(&total_of, lane) : 0;
            int up = t;
#pragma unroll
            for (int o = 1; o < kMaxCluster; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += u;
            }
            owner = __ffs(__ballot_sync(0xffffffffu, lane < C && want <= up)) - 1;
            before = __shfl_sync(0xffffffffu, up - t, owner);
        }
        if (C == 1 || (int)rank == owner) {
            // the digit at which the count from the top reaches `want`
            int above = before + inc - mine;
#pragma unroll
            for (int d = kD - 1; d >= 0; --d) {
                if (want > above && want <= above + digit[d]) {
                    found[0] = at + d;
                    found[1] = above;
                }
                above += digit[d];
            }
        }
        if (C > 1)
            cl::cluster_sync();
        else
            __syncthreads();
        prefix = (prefix << bits) | (uint32_t)(C > 1 ? remote(&found[0], owner) : found[0]);
        want -= C > 1 ? remote(&found[1], owner) : found[1];
        if (C == 1) __syncthreads();  // found and hist are written again
    }
    // keys above `prefix` stay, and the first `want` of those equal to it
    auto rows_of = [&](int64_t c0, auto use) {  // use(token, key, tokens that stay, tokens equal) for each row of the warp
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            if (i >= rows) break;
            const int64_t x = token(c0, i), j = r0 + x;
            const bool safe = j < first || j >= last;
            const unsigned up = __ballot_sync(0xffffffffu, x < len && (safe || (!none && key[i] > prefix)));
            const unsigned eq = __ballot_sync(0xffffffffu, x < len && !safe && !none && key[i] == prefix);
            use((int)j, key[i], up, eq);
        }
    };
    int n_above = 0, n_tie = 0;
    for (int64_t c0 = 0; c0 < len; c0 += chunk) {
        if (reload) load(c0);
        rows_of(c0, [&](int, uint32_t, unsigned up, unsigned eq) {
            n_above += __popc(up);
            n_tie += __popc(eq);
        });
    }
    // by the last lane of each warp, so that the prefix sums over the threads are sums over the warps
    int all_above, all_tie;
    block_scan<T>(lane == 31 ? n_above : 0, sh, all_above);
    block_scan<T>(lane == 31 ? n_tie : 0, sh, all_tie);
    int above = 0, ties = 0;  // before the chunk
    if (C > 1) {
        if (tid == 0) {
            counts[0] = all_above;
            counts[1] = all_tie;
        }
        cl::cluster_sync();
        if (lane < (int)rank) {
            above = remote(&counts[0], lane);
            ties = remote(&counts[1], lane);
        }
        above = __reduce_add_sync(0xffffffffu, above);
        ties = __reduce_add_sync(0xffffffffu, ties);
        cl::cluster_sync();  // no CTA ends while its shared memory is read
    }
    for (int64_t c0 = 0; c0 < len; c0 += chunk) {
        if (reload) {
            load(c0);
            n_above = n_tie = 0;
            rows_of(c0, [&](int, uint32_t, unsigned up, unsigned eq) {
                n_above += __popc(up);
                n_tie += __popc(eq);
            });
        }
        const int own_above = lane == 31 ? n_above : 0, own_tie = lane == 31 ? n_tie : 0;
        int w_above = above + block_scan<T>(own_above, sh, all_above) - own_above;
        int w_tie = ties + block_scan<T>(own_tie, sh, all_tie) - own_tie;
        w_above = __shfl_sync(0xffffffffu, w_above, 0);
        w_tie = __shfl_sync(0xffffffffu, w_tie, 0);
        rows_of(c0, [&](int j, uint32_t k, unsigned up, unsigned eq) {
            const unsigned below = (1u << lane) - 1;
            const int at_tie = w_tie + __popc(eq & below);
            if ((up >> lane & 1) || ((eq >> lane & 1) && at_tie < want)) {
                const int at = w_above + __popc(up & below) + min(at_tie, want);  // those before it that stay
                idx[at] = j;
                // the key is the weight, but for a NaN and a zero of either sign
                new_acc[at] = k == 0 || k == 0x80000000u ? acc[j] : key_to_float(k);
            }
            w_above += __popc(up);
            w_tie += __popc(eq);
        });
        above += all_above;
        ties += all_tie;
    }
    for (int j = a.keep + me; j < a.new_cap; j += all) new_acc[j] = 0.f;
}

// Bound by HBM: 530 MB (65 thousand tokens of 8 heads of 128 bf16, read and written) in 83 us, 6.4 TB/s.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 128;  // (slot, key head) pairs of a CTA

// A CTA moves the K and V rows of kMoveRows neighbouring (slot, head) pairs of a sequence, which lie together
// in a page of [row][head] order: their places first, once a row, then the words, four of K and
// of V under way in each thread.  The pages of new_table are not among those that the call reads, so the words
// may move in any order.
template <typename VT>
__global__ void __launch_bounds__(kMoveThreads) paged_evict_move(EvictArgs a)
{
    __shared__ int64_t src[kMoveRows], dst[kMoveRows];
    pdl_launch_dependents();
    const int b = blockIdx.y, tid = threadIdx.x;
    const unsigned row0 = blockIdx.x * kMoveRows, rows = min((unsigned)kMoveRows, (unsigned)a.keep * a.n_kv - row0);
    pdl_wait();
    if (tid < rows) {
        const unsigned s = (row0 + tid) / (unsigned)a.n_kv, h = row0 + tid - s * a.n_kv;
        const int j = a.idx[((int64_t)b * a.n_kv + h) * a.keep + s];
        const int64_t from = j < 0 ? -1 : paged_row(a.from, b, j), to = j < 0 ? -1 : paged_row(a.to, b, s);
        src[tid] = from < 0 ? -1 : from + h * a.from.ld_head;  // a token without a page reads as zeros
        dst[tid] = to < 0 ? -1 : to + h * a.to.ld_head;
    }
    __syncthreads();
    const unsigned n = rows * a.words;
    constexpr int U = 4;
    for (unsigned x0 = tid; x0 < n; x0 += U * kMoveThreads) {
        VT k[U], v[U];
        int64_t to[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const unsigned x = x0 + i * kMoveThreads, r = x / (unsigned)a.words;
            const int64_t w = (int64_t)(x - r * a.words) * sizeof(VT);
            to[i] = -1;
            k[i] = v[i] = VT{};
            if (x < n && dst[r] >= 0) {
                to[i] = dst[r] + w;
                if (src[r] >= 0) {
                    k[i] = *reinterpret_cast<const VT*>(a.K + src[r] + w);
                    v[i] = *reinterpret_cast<const VT*>(a.V + src[r] + w);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (to[i] >= 0) {
                *reinterpret_cast<VT*>(a.K + to[i]) = k[i];
                *reinterpret_cast<VT*>(a.V + to[i]) = v[i];
            }
    }
}

// launch_pdl in clusters of `size` CTAs along x.
template <typename... P, typename... A>
void launch_pdl_cluster(void (*kern)(P...), dim3 grid, dim3 block, int size, cudaStream_t stream, A&&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = size > 1 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
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
    const int64_t rows = (int64_t)keep * n_kv, ctas = (rows + kMoveRows - 1) / kMoveRows;
    if (rows > INT32_MAX || n_kv > INT32_MAX / 8 || a.words > INT32_MAX / (2 * kMoveRows)) return CSA_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // CTAs to a selection: as many as fill the GPU, while each has 2048 tokens or more
    a.cluster = 1;
    while (a.cluster < kMaxCluster && (int64_t)B * n_kv * a.cluster * 2 <= kNumSMs && a.cap / (2 * a.cluster) >= 2048)
        a.cluster *= 2;
    // a CTA of 1024 threads has an SM for itself; two of 512 share one where there are more CTAs than SMs (64
    // sequences of 4096 tokens, 8 key heads: 130 instead of 163 us)
    if ((int64_t)B * n_kv * a.cluster > kNumSMs)
        launch_pdl_cluster(paged_evict_select<512>, dim3(n_kv * a.cluster, B), dim3(512), a.cluster, s, a);
    else
        launch_pdl_cluster(paged_evict_select<1024>, dim3(n_kv * a.cluster, B), dim3(1024), a.cluster, s, a);
    st = launch_status();
    if (st != CSA_OK) return st;
    const dim3 grid((unsigned)ctas, B), block(kMoveThreads);
    if (wide)
        launch_pdl(paged_evict_move<uint4>, grid, block, 0, s, a);
    else if (eb == 2)
        launch_pdl(paged_evict_move<uint16_t>, grid, block, 0, s, a);
    else
        launch_pdl(paged_evict_move<uint32_t>, grid, block, 0, s, a);
    return launch_status();
}
