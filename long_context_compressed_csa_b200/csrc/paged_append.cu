// paged_append: new tokens' keys and values into the pages of their sequences.
//
// A copy: K[page(t)][t mod page][h] = k[b][i][h], the same for V.  It moves 2 x 2 rows of
// d elements per (token, head) and is bound by HBM for prompts, by the launch for a decode step: four
// prompts of 4099 tokens, 8 heads of 128 bf16 (134 MB) take 24.4 us, 0.84 of the copy rate; 64 single tokens 2.2 us.
// (Four words a thread and one 64-bit division a CTA measured the same.)
#include "paged.cuh"

namespace csa {
namespace {

struct AppendArgs {
    const char *k, *v;
    char *K, *V;
    int64_t ld_batch, ld_tok, ld_head;  // of k and v, bytes
    PagedPool pl;                       // strides in bytes
    const int64_t* t;
    int B, nq, n_kv;
    int words;                          // words of VT in a row
};

constexpr int kAppendThreads = 256;

// One thread copies one word (16 bytes, or one element where a layout is not 16-byte aligned)
// of the key row and of the value row.
template <typename VT>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(AppendArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t per_tok = (int64_t)a.n_kv * a.words;
    const int64_t n = (int64_t)a.B * a.nq * per_tok;
    const int64_t x = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x;
    if (x >= n) return;
    const int64_t tok = x / per_tok;
    const int in = (int)(x - tok * per_tok), h = in / a.words, w = in - h * a.words;
    const int b = (int)(tok / a.nq), i = (int)(tok - (int64_t)b * a.nq);
    const int64_t src = b * a.ld_batch + i * a.ld_tok + h * a.ld_head + (int64_t)w * sizeof(VT);
    const VT kx = *reinterpret_cast<const VT*>(a.k + src), vx = *reinterpret_cast<const VT*>(a.v + src);
    const int64_t t = a.t[tok];
    if (t < 0 || t >= (int64_t)a.pl.max_pages * a.pl.page) return;
    const int64_t row = paged_row(a.pl, b, (int)t);
    if (row < 0) return;
    const int64_t dst = row + h * a.pl.ld_head + (int64_t)w * sizeof(VT);
    *reinterpret_cast<VT*>(a.K + dst) = kx;
    *reinterpret_cast<VT*>(a.V + dst) = vx;
}

}  // namespace

int paged_pool_check(const PagedPool& pl, int B, int n_kv, int d)
{
    if (pl.n_pages < 0 || pl.page < 1 || pl.max_pages < 0 || B < 0 || n_kv < 1 || d < 1) return CSA_ERR_ARG;
    if (pl.ld_page < 0 || pl.ld_row < d || pl.ld_head < 0 || (n_kv > 1 && pl.ld_head < d)) return CSA_ERR_ARG;
    if ((int64_t)pl.max_pages * pl.page > INT32_MAX - 1024) return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

}  // namespace csa

extern "C" int paged_append(const void* k, const void* v, int64_t ld_batch, int64_t ld_tok, int64_t ld_head, void* K,
                            void* V, int64_t pool_ld_page, int64_t pool_ld_row, int64_t pool_ld_head, int64_t n_pages,
                            int page, const int32_t* table, int max_pages, const int64_t* t, int B, int nq, int n_kv,
                            int d, int dtype, csa_stream_t stream)
{
    using namespace csa;
    if (dtype != CSA_BF16 && dtype != CSA_F32) return CSA_ERR_DTYPE;
    PagedPool pl{pool_ld_page, pool_ld_row, pool_ld_head, n_pages, page, table, max_pages};
    const int st = paged_pool_check(pl, B, n_kv, d);
    if (st != CSA_OK) return st;
    if (nq < 0 || ld_batch < 0 || ld_tok < 0 || ld_head < 0) return CSA_ERR_ARG;
    if (B == 0 || nq == 0 || max_pages == 0) return CSA_OK;
    if (!k || !v || !K || !V || !table || !t) return CSA_ERR_ARG;
    const int eb = elem_bytes(dtype);
    const uintptr_t ptrs = (uintptr_t)k | (uintptr_t)v | (uintptr_t)K | (uintptr_t)V;
    if ((ptrs & (eb - 1)) || ((uintptr_t)table & 3) || ((uintptr_t)t & 7)) return CSA_ERR_ALIGN;
    AppendArgs a{static_cast<const char*>(k), static_cast<const char*>(v), static_cast<char*>(K),
                 static_cast<char*>(V), ld_batch * eb, ld_tok * eb, ld_head * eb, pl, t, B, nq, n_kv, 0};
    a.pl.ld_page *= eb;
    a.pl.ld_row *= eb;
    a.pl.ld_head *= eb;
    // 16-byte words when every row starts on a 16-byte boundary and is whole 16-byte words
    const int64_t lds = a.ld_batch | a.ld_tok | a.ld_head | a.pl.ld_page | a.pl.ld_row | a.pl.ld_head | (d * eb);
    const bool wide = (ptrs & 15) == 0 && (lds & 15) == 0;
    const int wb = wide ? 16 : eb;
    a.words = d * eb / wb;
    const int64_t n = (int64_t)B * nq * n_kv * a.words, ctas = (n + kAppendThreads - 1) / kAppendThreads;
    if (ctas > INT32_MAX) return CSA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)ctas), block(kAppendThreads);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (wide)
        e = launch_pdl(paged_append_kernel<uint4>, grid, block, 0, s, a);
    else if (eb == 2)
        e = launch_pdl(paged_append_kernel<uint16_t>, grid, block, 0, s, a);
    else
        e = launch_pdl(paged_append_kernel<uint32_t>, grid, block, 0, s, a);
    (void)e;
    return launch_status();
}
