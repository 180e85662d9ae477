"""Paged cache on the GPU against the fp64 oracle.

Bounds, per output element, with u = 2^-24.  Logits are fp32 sums of d products (each product
and addition rounded; a tensor-core sum may truncate, which doubles the step): their error is at
most es = (d + 4) 2u M, M = max_j scale sum_x |q_x K_jx|, plus the scale's own 4u M.  A weight
p_j = exp(s_j - lse) is then off by a factor of at most exp(2 es + 8u (1 + M)) (both exponentials,
ex2 within 2^-22), and sums over n tokens and their joins by (n + 64) 2u.  So out is off by at most
  E = (2 es + 16u (1 + M) + (n + 64) 2u + P) sum_j p_j |V_j|
where P covers weights that go to the tensor cores in bf16: 2^-16 where they are split into two
parts, 2^-8 where they are not.  A bf16 output adds its rounding, 2^-8 |out|; an fp32 output u |out|.
lse is off by es + 8u (1 + M) + (n + 64) 2u + 2u |lse|.
"""
import math

import numpy as np
import pytest
import torch

import long_context_compressed_csa_b200 as lib
from long_context_compressed_csa_b200.synth import randn, to_f64
from oracle import paged as O

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_compressed_csa_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def pools(n_pages, page, n_kv, d, dtype, seed, layout="nhd"):
    """K and V pools [n_pages, page, n_kv, d] in one of three memory layouts."""
    K, V = (randn((n_pages, page, n_kv, d), seed + i, dtype) for i in range(2))
    if layout == "hnd":
        return [x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) for x in (K, V)]
    if layout == "both":  # one tensor [n_pages, 2, page, n_kv, d]
        kv = torch.stack([K, V], 1).to(DEV)
        return [kv[:, 0], kv[:, 1]]
    if layout == "odd":  # rows that do not start on 16 bytes
        wide = torch.zeros(2, n_pages, page, n_kv, d + 1, dtype=dtype, device=DEV)
        wide[0, ..., :d], wide[1, ..., :d] = K.to(DEV), V.to(DEV)
        return [wide[0, ..., :d], wide[1, ..., :d]]
    return [K.to(DEV), V.to(DEV)]


def tables(B, max_pages, n_pages, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(n_pages, generator=g)[:B * max_pages].reshape(B, max_pages).to(torch.int32)


def positions(lens, nq):
    t = torch.tensor(lens)[:, None] - nq + torch.arange(nq)[None]
    return torch.clamp(t, min=-1).to(torch.int64)


def weight_bits(nq, n_h, n_kv, d, dtype, acc):
    """P of the module's bound: how exactly the call keeps the softmax weights (17 rows or more of a key
    head take the kernels that round them once)."""
    return 2.0 ** -8 if dtype == torch.bfloat16 and nq * n_h // n_kv >= 17 else 2.0 ** -16


def check_attn(q, K, V, table, t, out, lse, P, n_win=0, n_sink=0, scale=None, acc=None, acc_out=None):
    ref, rl, w, (n, M, pv) = O.attn(to_f64(q), to_f64(K), to_f64(V), table.cpu().numpy(), t.cpu().numpy(), scale, n_win,
                                    n_sink)
    d = q.shape[-1]
    es = (d + 6) * 2 * U * M
    rel = 2 * es + 16 * U * (1 + M) + (n + 64) * 2 * U
    step = 2.0 ** -8 if out.dtype == torch.bfloat16 else U
    got = to_f64(out)
    assert np.all(np.isfinite(got))
    off = np.abs(got - ref) - (step * np.abs(ref) + (rel + P)[..., None] * pv * (1 + step))
    assert off.max() <= 0, "out off its bound by %g" % off.max()
    gl = to_f64(lse)
    empty = n == 0
    assert np.all(gl[empty] == -np.inf) and np.all(got[empty] == 0)
    gl, rl, room = gl[~empty], rl[~empty], (es + 8 * U * (1 + M) + (n + 64) * 2 * U)[~empty]
    off = np.abs(gl - rl) - (room + 2 * U * np.abs(rl))
    assert off.size == 0 or off.max() <= 0, "lse off its bound by %g" % off.max()
    if acc is not None:
        a = to_f64(acc)
        rows = q.shape[1] * q.shape[2] // K.shape[2]
        worst = rel.max() + rows * 2 * U
        np.testing.assert_array_less(np.abs(to_f64(acc_out) - (a + w)), worst * w + 2 * U * np.abs(a + w) + 1e-30)


def run_attn(q, K, V, table, t, n_win=0, n_sink=0, scale=0.0, acc=None, out_dtype=None, ws=None):
    B, nq, n_h, d = q.shape
    out = torch.full(q.shape, float("nan"), dtype=out_dtype or q.dtype, device=DEV)
    lse = torch.full((B, nq, n_h), float("nan"), device=DEV)
    acc_out = None if acc is None else torch.full_like(acc, float("nan"))
    if ws is None:
        size = lib.paged_attn_workspace_size(B, nq, n_h, K.shape[2], d, table.shape[1] * K.shape[1], acc is not None)
        ws = torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)  # whatever an earlier call left
    lib.paged_attn(q, K, V, table, t, out, ws, lse=lse, n_win=n_win, n_sink=n_sink, scale=scale, acc=acc,
                   acc_out=acc_out)
    torch.cuda.synchronize()
    return out, lse, acc_out


def case(lens, nq=1, n_h=8, n_kv=2, d=64, page=16, dtype=torch.bfloat16, n_win=0, n_sink=0, layout="nhd", acc=False,
         out_dtype=None, scale=None, seed=0, spare=1):
    B = len(lens)
    max_pages = max(-(-max(lens) // page), 0) + spare
    n_pages = B * max_pages + 2
    K, V = pools(n_pages, page, n_kv, d, dtype, 100 + seed, layout)
    table = tables(B, max_pages, n_pages, seed)
    t = positions(lens, nq)
    # rows that no token has hold NaN: tails of the last pages, and pages that no table names
    used = torch.zeros(n_pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        j = torch.arange(n)
        used[table[b].long()[j // page], j % page] = True
    K[~used.to(DEV)] = float("nan")
    V[~used.to(DEV)] = float("nan")
    table, t = table.to(DEV), t.to(DEV)
    q = randn((B, nq, n_h, d), 7 + seed, dtype, scale=2.0).to(DEV)
    a = torch.rand(B, n_kv, max_pages * page, device=DEV) if acc else None
    out, lse, acc_out = run_attn(q, K, V, table, t, n_win, n_sink, scale or 0.0, a, out_dtype)
    check_attn(q, torch.nan_to_num(K), torch.nan_to_num(V), table, t, out, lse,
               weight_bits(nq, n_h, n_kv, d, dtype, acc), n_win, n_sink, scale, a, acc_out)


# ==================================================================================
# attention
# ==================================================================================
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 300, 1025])
def test_attn_lengths(n, dtype):
    case([n], dtype=dtype, seed=n)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_h,n_kv", [(1, 1), (3, 3), (8, 1), (7, 1), (10, 2), (16, 1), (24, 1), (33, 3), (64, 1), (128, 1)])
def test_attn_head_layouts(n_h, n_kv, dtype):
    case([70, 1, 200], n_h=n_h, n_kv=n_kv, dtype=dtype, seed=n_h)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [1, 7, 8, 40, 64, 80, 96, 128, 192, 255, 256])
def test_attn_head_widths(d, dtype):
    case([45, 130], d=d, dtype=dtype, seed=d)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 32, 48, 64, 100, 128, 256])
def test_attn_page_sizes(page):
    case([50, 257, 1], page=page, d=128, seed=page)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "both", "odd"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attn_pool_layouts(layout, d, dtype):
    case([90, 33], layout=layout, d=d, dtype=dtype)


@pytest.mark.parametrize("n_win,n_sink", [(1, 0), (1, 1), (5, 2), (16, 4), (32, 0), (33, 40), (100, 4), (128, 16), (1000, 4)])
@pytest.mark.parametrize("nq", [1, 3])
def test_attn_window_and_first_tokens(n_win, n_sink, nq):
    case([300, 40, 3, 129], nq=nq, n_win=n_win, n_sink=n_sink, d=128, seed=n_win)
    case([300, 40, 3, 129], nq=nq, n_win=n_win, n_sink=n_sink, dtype=torch.float32, seed=n_win)


@pytest.mark.parametrize("nq,n_h,n_kv", [(2, 4, 4), (5, 8, 2), (17, 6, 2), (64, 8, 2), (150, 4, 1), (300, 16, 2)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_win,n_sink", [(0, 0), (50, 3)])
def test_attn_several_queries(nq, n_h, n_kv, d, n_win, n_sink):
    case([nq, nq + 100, max(1, nq // 2)], nq=nq, n_h=n_h, n_kv=n_kv, d=d, n_win=n_win, n_sink=n_sink, seed=nq)


@pytest.mark.parametrize("page", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "both"])
def test_attn_prompt_pages(page, layout):
    case([100, 413], nq=100, n_h=8, n_kv=2, d=128, page=page, layout=layout, seed=page)


def test_attn_many_sequences_and_heads():
    # more (sequence, tile) entries than the schedule's threads scan at once
    lens = [(37 * i) % 90 + 1 for i in range(300)]
    case(lens, n_h=4, n_kv=2, page=8)
    case(lens[:200], nq=9, n_h=8, n_kv=2, page=8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attn_long_and_ragged_is_split_and_joined(dtype):
    case([20000, 1, 37, 5000], n_h=4, n_kv=1, d=128, dtype=dtype)
    case([30011], n_h=16, n_kv=2, d=64, dtype=dtype, page=64)
    case([9000, 12], n_h=64, n_kv=1, d=128, dtype=dtype, page=64)


def test_attn_fp32_output_of_bf16_inputs_and_scale():
    case([500, 3], out_dtype=torch.float32, d=128)
    case([500, 3], scale=0.25, d=128)
    case([260, 200], nq=40, out_dtype=torch.float32, d=128)


def test_attn_queries_that_see_nothing_and_positions_past_the_capacity():
    K, V = pools(6, 16, 2, 64, torch.bfloat16, 5)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device=DEV)
    q = randn((3, 2, 4, 64), 9).to(DEV)
    for t in ([[-1, -5], [0, -1], [31, 1000]], [[-1, -1]] * 3, [[2**40, 3], [-2**40, 40], [32, 31]]):
        t = torch.tensor(t, dtype=torch.int64, device=DEV)
        for n_win, n_sink in ((0, 0), (4, 2), (2**31 - 1, 2**31 - 1)):
            out, lse, _ = run_attn(q, K, V, table, t, n_win, n_sink)
            check_attn(q, K, V, table, t, out, lse, 2.0 ** -16, n_win, n_sink)


@pytest.mark.parametrize("nq", [1, 70])
def test_attn_pages_that_are_not_there(nq):
    # entries outside the pool: their tokens are not seen, whatever lies beyond
    K, V = pools(8, 16, 2, 128, torch.bfloat16, 6)
    table = torch.tensor([[3, -1, 7, 8], [-2**31, 2**31 - 1, -1, 99], [0, 1, 2, -7]], dtype=torch.int32, device=DEV)
    t = positions([64, 64, 61], nq).to(DEV)
    q = randn((3, nq, 8, 128), 9).to(DEV)
    P = weight_bits(nq, 8, 2, 128, torch.bfloat16, False)
    for n_win, n_sink in ((0, 0), (20, 18)):
        out, lse, _ = run_attn(q, K, V, table, t, n_win, n_sink)
        check_attn(q, K, V, table, t, out, lse, P, n_win, n_sink)
    none = torch.zeros(3, 0, dtype=torch.int32, device=DEV)  # no pages at all
    out, lse, _ = run_attn(q, K, V, none, t)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_attn_equal_and_extreme_logits():
    # equal logits give the mean exactly enough; one far above the rest gives its value
    K, V = pools(4, 16, 1, 64, torch.bfloat16, 3)
    K.zero_()
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=DEV)
    t = torch.tensor([[44]], dtype=torch.int64, device=DEV)
    q = torch.ones(1, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, lse, _ = run_attn(q, K, V, table, t)
    check_attn(q, K, V, table, t, out, lse, 2.0 ** -16)
    K[0, 5] = 1000.0
    out, lse, _ = run_attn(q, K, V, table, t)
    assert torch.equal(out[0, 0], V[0, 5, 0].expand(2, 64))
    K[0, 5] = -1e30  # far below the rest
    out, lse, _ = run_attn(q, K, V, table, t)
    check_attn(q, K, V, table, t, out, lse, 2.0 ** -16)


def test_attn_offsets_past_32_bits():
    # a pool of 2^32 + elements; the sequence's pages lie at its end
    page, n_kv, d = 16, 8, 128
    n_pages = (2**32) // (page * n_kv * d) + 40
    K = torch.empty(n_pages, page, n_kv, d, dtype=torch.bfloat16, device=DEV)
    V = torch.empty_like(K)
    K[-4:], V[-4:] = (randn((4, page, n_kv, d), 3 + i).to(DEV) for i in range(2))
    K[:2], V[:2] = 7.0, 7.0
    table = torch.tensor([[n_pages - 1, n_pages - 3, n_pages - 4, n_pages - 2]], dtype=torch.int32, device=DEV)
    near = torch.tensor([[3, 1, 0, 2]], dtype=torch.int32, device=DEV)
    for nq in (1, 60):
        q = randn((1, nq, 16, d), 5).to(DEV)
        t = positions([62], nq).to(DEV)
        out, lse, _ = run_attn(q, K, V, table, t)
        want, want_lse, _ = run_attn(q, K[-4:], V[-4:], near, t)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    new = torch.tensor([[n_pages - 9, n_pages - 8]], dtype=torch.int32, device=DEV)
    k = randn((1, 1, n_kv, d), 8).to(DEV)
    lib.paged_append(k, k, K, V, table, torch.tensor([[63]], device=DEV))
    assert torch.equal(K[n_pages - 2, 15], k[0, 0]) and torch.equal(V[n_pages - 2, 15], k[0, 0])
    acc = torch.rand(1, n_kv, 64, device=DEV)
    idx, _, _ = run_evict(K, V, table, torch.tensor([64], device=DEV), acc, 32, new, 1, 2)
    rows = K[table[0].long()].flatten(0, 1)  # [64, n_kv, d]
    got = K[new[0].long()].flatten(0, 1)
    for h in range(n_kv):
        assert torch.equal(got[:, h], rows[idx[0, h].long(), h])


# ==================================================================================
# accumulated weights
# ==================================================================================
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nq,n_h,n_kv,d", [(1, 8, 2, 64), (1, 16, 1, 128), (3, 5, 5, 128), (9, 12, 3, 256), (20, 8, 1, 40)])
@pytest.mark.parametrize("n_win,n_sink", [(0, 0), (40, 5)])
def test_weights(nq, n_h, n_kv, d, n_win, n_sink, dtype):
    case([nq, 300, 77], nq=nq, n_h=n_h, n_kv=n_kv, d=d, n_win=n_win, n_sink=n_sink, dtype=dtype, acc=True)


def test_weights_long():
    case([10000, 1, 444], n_h=16, n_kv=2, d=128, acc=True, page=64)


def test_weights_in_place_sum_to_the_heads_and_skip_padding():
    K, V = pools(9, 16, 2, 128, torch.bfloat16, 5)
    table = tables(2, 4, 9, 1).to(DEV)
    q = randn((2, 2, 8, 128), 9).to(DEV)
    t = torch.tensor([[50, -1], [-1, -1]], dtype=torch.int64, device=DEV)
    acc = torch.ones(2, 2, 64, device=DEV)
    out = torch.empty_like(q)
    ws = torch.zeros(lib.paged_attn_workspace_size(2, 2, 8, 2, 128, 64, True), dtype=torch.uint8, device=DEV)
    lib.paged_attn(q, K, V, table, t, out, ws, acc=acc)
    got = (acc - 1).double().cpu()
    np.testing.assert_allclose(got[0].sum(-1), [4.0, 4.0], atol=64 * 2 * 2 * U)
    assert bool((got[0, :, 51:] == 0).all()) and bool((got[1] == 0).all())


# ==================================================================================
# append
# ==================================================================================
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "both", "odd"])
@pytest.mark.parametrize("n_kv,d,page", [(1, 1, 1), (2, 64, 16), (3, 40, 7), (8, 128, 32), (5, 7, 3)])
def test_append(n_kv, d, page, layout, dtype):
    B, nq, max_pages = 3, 6, 4
    n_pages = B * max_pages + 2
    K, V = pools(n_pages, page, n_kv, d, dtype, 20, layout)
    table = tables(B, max_pages, n_pages, 3)
    table[1, 0], table[2, 1] = -1, n_pages
    cap = max_pages * page
    t = torch.tensor([[0, 1, 2, 3, cap - 1, cap], [-1, -9, 3, 0, 2, 1], [2**40, 2, 1, -2**40, 0, 3]], dtype=torch.int64)
    t[0, 3] = min(3, cap - 2)  # one place for each token, the smallest cache's too
    if cap < 6:
        t[0, 2:] = torch.tensor([2, -1, 3, cap])
    qkv = randn((B, nq, 2 * n_kv + 1, d), 30, dtype).to(DEV)  # k and v are parts of one projection's output
    k, v = qkv[:, :, :n_kv], qkv[:, :, n_kv:2 * n_kv]
    wk, wv = to_f64(K), to_f64(V)
    O.append(to_f64(k), to_f64(v), wk, wv, table.numpy(), t.numpy())
    lib.paged_append(k, v, K, V, table.to(DEV), t.to(DEV))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(to_f64(K), wk)
    np.testing.assert_array_equal(to_f64(V), wv)


# ==================================================================================
# eviction
# ==================================================================================
def run_evict(K, V, table, lens, acc, keep, new_table, n_sink=0, n_recent=0):
    B, n_kv = acc.shape[:2]
    idx = torch.full((B, n_kv, keep), -77, dtype=torch.int32, device=DEV)
    new_lens = torch.full((B,), -77, dtype=torch.int64, device=DEV)
    new_acc = torch.full((B, n_kv, new_table.shape[1] * K.shape[1]), float("nan"), device=DEV)
    lib.paged_evict(K, V, table, lens, acc, keep, new_table, new_lens, new_acc, idx, n_sink=n_sink, n_recent=n_recent)
    torch.cuda.synchronize()
    return idx, new_lens, new_acc


def evict_case(lens, keep, n_sink=0, n_recent=0, n_kv=2, d=64, page=16, dtype=torch.bfloat16, layout="nhd", values="rand",
               seed=0):
    B, max_pages, new_pages = len(lens), max(1, -(-max(lens) // page)) + 1, -(-keep // page) + 1
    n_pages = B * (max_pages + new_pages) + 1
    K, V = pools(n_pages, page, n_kv, d, dtype, 40 + seed, layout)
    both = tables(B, max_pages + new_pages, n_pages, seed)
    table, new_table = both[:, :max_pages].contiguous(), both[:, max_pages:].contiguous()
    g = torch.Generator().manual_seed(seed)
    shape = (B, n_kv, max_pages * page)
    acc = torch.rand(shape, generator=g)
    if values == "ties":
        acc = torch.randint(0, 3, shape, generator=g).float() - 1  # and both zeros
        acc = torch.where(torch.rand(shape, generator=g) < 0.3, -acc * 0, acc)
    elif values == "equal":
        acc = torch.full(shape, 0.25)
    elif values == "special":
        pick = torch.randint(0, 6, shape, generator=g)
        special = torch.tensor([math.nan, math.inf, -math.inf, 1e-42, -0.0, 3e38])
        acc = torch.where(torch.rand(shape, generator=g) < 0.5, special[pick], acc)
        acc[0, 0, :3] = -math.nan
    wk, wv = to_f64(K), to_f64(V)
    want = O.evict(wk, wv, table.numpy(), np.array(lens), acc.numpy(), keep, new_table.numpy(), n_sink, n_recent)
    idx, new_lens, new_acc = run_evict(K, V, table.to(DEV), torch.tensor(lens, device=DEV), acc.to(DEV), keep,
                                       new_table.to(DEV), n_sink, n_recent)
    np.testing.assert_array_equal(new_lens.cpu().numpy(), want[0])
    np.testing.assert_array_equal(idx.cpu().numpy(), want[2])
    np.testing.assert_array_equal(new_acc.cpu().numpy(), want[1])
    np.testing.assert_array_equal(to_f64(K), wk)
    np.testing.assert_array_equal(to_f64(V), wv)


@pytest.mark.parametrize("values", ["rand", "ties", "equal", "special"])
@pytest.mark.parametrize("lens,keep,n_sink,n_recent", [
    ([100, 3, 0, 40], 40, 4, 8), ([1, 2, 3], 1, 0, 0), ([50, 60], 17, 17, 0), ([50, 60], 17, 0, 17), ([50, 17], 17, 9, 8),
    ([3000, 1500, 2049], 1024, 1, 100), ([5000], 4999, 0, 0), ([5000], 1, 0, 0), ([7, 9], 100, 4, 4)])
def test_evict(lens, keep, n_sink, n_recent, values):
    evict_case(lens, keep, n_sink, n_recent, values=values)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "both", "odd"])
@pytest.mark.parametrize("n_kv,d,page", [(1, 1, 1), (3, 40, 7), (8, 128, 32), (5, 7, 3), (2, 300, 16)])
def test_evict_layouts(n_kv, d, page, layout, dtype):
    evict_case([90, 20, 61], 33, 2, 5, n_kv=n_kv, d=d, page=page, layout=layout, dtype=dtype)


def test_evict_long():
    evict_case([70000, 66000], 30000, 4, 1000, n_kv=1, d=8, page=64, values="ties")
    evict_case([70001], 3, 1, 1, n_kv=3, d=8, page=64)


def test_evict_lengths_out_of_range_and_missing_pages():
    K, V = pools(12, 4, 1, 8, torch.float32, 1)
    table = torch.tensor([[0, 1, 2], [3, -1, 12], [4, 5, 6]], dtype=torch.int32)
    new = torch.tensor([[7, 8], [9, 10], [11, -1]], dtype=torch.int32)
    lens, acc = torch.tensor([2**40, 12, -5]), torch.rand(3, 1, 12)
    lens[2] = 12
    wk, wv = to_f64(K), to_f64(V)
    want = O.evict(wk, wv, table.numpy(), lens.numpy(), acc.numpy(), 7, new.numpy(), 1, 2)
    got = run_evict(K, V, table.to(DEV), lens.to(DEV), acc.to(DEV), 7, new.to(DEV), 1, 2)
    np.testing.assert_array_equal(got[1].cpu().numpy(), want[0])
    np.testing.assert_array_equal(got[0].cpu().numpy(), want[2])
    np.testing.assert_array_equal(to_f64(K), wk)
    np.testing.assert_array_equal(to_f64(V), wv)
    lens = torch.tensor([-5, 0, 1])
    idx, new_lens, new_acc = run_evict(K, V, table.to(DEV), lens.to(DEV), acc.to(DEV), 7, new.to(DEV), 1, 2)
    assert new_lens.tolist() == [0, 0, 1] and idx[2, 0].tolist() == [0] + [-1] * 6
    assert bool((idx[:2] == -1).all()) and bool((new_acc[:2] == 0).all())


# ==================================================================================
# refusals of the binding, streams, graphs, and the operators together
# ==================================================================================
def test_binding_refuses_what_does_not_fit():
    K, V = pools(4, 16, 2, 64, torch.bfloat16, 1)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    t = torch.tensor([[5]], dtype=torch.int64, device=DEV)
    q = randn((1, 1, 4, 64), 1).to(DEV)
    out, ws = torch.empty_like(q), torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    acc = torch.zeros(1, 2, 32, device=DEV)
    bad = [dict(table=table.long()), dict(t=t.int()), dict(K_pages=K.float()), dict(V_pages=V[:, :8]),
           dict(V_pages=V.transpose(1, 2).contiguous().transpose(1, 2)), dict(q=q[..., :32]), dict(out=out[..., :32]),
           dict(acc=acc[..., :16]), dict(acc_out=acc), dict(lse=torch.zeros(1, 1, 3, device=DEV)), dict(t=t.expand(1, 2))]
    for kw in bad:
        args = dict(q=q, K_pages=K, V_pages=V, table=table, t=t, out=out, workspace=ws)
        args.update(kw)
        with pytest.raises((AssertionError, TypeError)):
            lib.paged_attn(**args)
    with pytest.raises(lib.CSAError):
        lib.paged_attn(q, K, V, table, t, out, ws[:64])
    with pytest.raises(lib.CSAError):
        lib.paged_attn(randn((1, 1, 3, 64), 1).to(DEV), K, V, table, t, out[:, :, :3].contiguous(), ws)
    k = randn((1, 1, 2, 64), 2).to(DEV)
    for kk, vv in ((k, k.float()), (k.float(), k.float()), (k[:, :, :1], k[:, :, :1])):
        with pytest.raises(AssertionError):
            lib.paged_append(kk, vv, K, V, table, t)


def test_other_stream():
    K, V = pools(9, 16, 2, 128, torch.bfloat16, 5)
    table = tables(2, 4, 9, 1).to(DEV)
    q = randn((2, 1, 8, 128), 9).to(DEV)
    t = positions([60, 33], 1).to(DEV)
    want = run_attn(q, K, V, table, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(q), torch.empty(2, 1, 8, device=DEV)
    ws = torch.empty(lib.paged_attn_workspace_size(2, 1, 8, 2, 128, 64), dtype=torch.uint8, device=DEV)
    lib.paged_attn(q, K, V, table, t, out, ws, lse=lse, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("nq", [1, 40])
def test_graphs_follow_the_lengths_and_share_a_workspace(nq):
    K, V = pools(70, 16, 2, 128, torch.bfloat16, 5)
    table = tables(2, 30, 70, 1).to(DEV)
    qs = [randn((2, nq, 8, 128), 9 + i).to(DEV) for i in range(2)]
    ts = [positions([100, 70], nq).to(DEV), positions([400, 90], nq).to(DEV)]
    outs = [torch.empty_like(q) for q in qs]
    lses = [torch.empty(2, nq, 8, device=DEV) for _ in qs]
    accs = [torch.zeros(2, 2, 480, device=DEV) for _ in qs]
    ws = torch.empty(lib.paged_attn_workspace_size(2, nq, 8, 2, 128, 480, True), dtype=torch.uint8, device=DEV)
    graphs = []
    for i in range(2):
        lib.paged_attn(qs[i], K, V, table, ts[i], outs[i], ws, lse=lses[i], n_win=64 * i, n_sink=4)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lib.paged_attn(qs[i], K, V, table, ts[i], outs[i], ws, lse=lses[i], n_win=64 * i, n_sink=4, acc=accs[i])
            lib.paged_attn(qs[i], K, V, table, ts[i], outs[i], ws, lse=lses[i], n_win=64 * i, n_sink=4)
        graphs.append(g)
    P = weight_bits(nq, 8, 2, 128, torch.bfloat16, False)
    for lens in ([100, 70], [480, nq], [max(nq, 33), 470]):
        for i in range(2):
            ts[i].copy_(positions(lens, nq))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            check_attn(qs[i], K, V, table, ts[i], outs[i], lses[i], P, 64 * i, 4)


def test_results_do_not_depend_on_the_run():
    K, V = pools(400, 16, 2, 128, torch.bfloat16, 5)
    table = tables(3, 130, 400, 1).to(DEV)
    for nq in (1, 33):
        q = randn((3, nq, 16, 128), 9).to(DEV)
        t = positions([2000, 77, 900], nq).to(DEV)
        acc = torch.rand(3, 2, 2080, device=DEV)
        first = run_attn(q, K, V, table, t, acc=acc)
        for _ in range(3):
            again = run_attn(q, K, V, table, t, acc=acc)
            assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_a_serving_run():
    """A prompt, decode steps with a window, steps that accumulate weights, an eviction, and steps on
    the smaller cache: every call against the oracle on the same cache."""
    B, n_h, n_kv, d, page, max_pages = 2, 8, 2, 64, 16, 12
    n_pages = 2 * B * max_pages
    K, V = (torch.full((n_pages, page, n_kv, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    both = tables(B, 2 * max_pages, n_pages, 2).to(DEV)
    table, new_table = both[:, :max_pages].contiguous(), both[:, max_pages:max_pages + 6].contiguous()
    cap = max_pages * page
    acc = torch.zeros(B, n_kv, cap, device=DEV)
    ws = torch.empty(lib.paged_attn_workspace_size(B, 90, n_h, n_kv, d, cap, True), dtype=torch.uint8, device=DEV)
    ok, ov = np.zeros(K.shape), np.zeros(V.shape)
    seed = [1000]

    def step(nq, lens, tab, weights=None, n_win=0, n_sink=0):
        seed[0] += 3
        k, v = (randn((B, nq, n_kv, d), seed[0] + i).to(DEV) for i in range(2))
        q = randn((B, nq, n_h, d), seed[0] + 2, scale=2.0).to(DEV)
        t = positions(lens, nq).to(DEV)
        lib.paged_append(k, v, K, V, tab, t)
        O.append(to_f64(k), to_f64(v), ok, ov, tab.cpu().numpy(), t.cpu().numpy())
        out, lse = torch.empty_like(q), torch.empty(B, nq, n_h, device=DEV)
        before = None if weights is None else weights.clone()
        lib.paged_attn(q, K, V, tab, t, out, ws, lse=lse, n_win=n_win, n_sink=n_sink, acc=weights)
        torch.cuda.synchronize()
        check_attn(q, torch.tensor(ok), torch.tensor(ov), tab, t, out, lse,
                   weight_bits(nq, n_h, n_kv, d, torch.bfloat16, weights is not None), n_win, n_sink, acc=before,
                   acc_out=weights)

    lens = [90, 71]
    step(90, lens, table)
    for i in range(4):
        lens = [n + 1 for n in lens]
        step(1, lens, table, n_win=32 if i == 0 else 0, n_sink=4)
    for _ in range(4):
        lens = [n + 1 for n in lens]
        step(1, lens, table, acc)
    new_lens = torch.zeros(B, dtype=torch.int64, device=DEV)
    new_acc = torch.zeros(B, n_kv, 6 * page, device=DEV)
    idx = torch.zeros(B, n_kv, 64, dtype=torch.int32, device=DEV)
    lib.paged_evict(K, V, table, torch.tensor(lens, device=DEV), acc, 64, new_table, new_lens, new_acc, idx, n_sink=2,
                    n_recent=8)
    want = O.evict(ok, ov, table.cpu().numpy(), np.array(lens), acc.cpu().numpy(), 64, new_table.cpu().numpy(), 2, 8)
    np.testing.assert_array_equal(new_lens.cpu().numpy(), want[0])
    np.testing.assert_array_equal(idx.cpu().numpy(), want[2])
    np.testing.assert_array_equal(new_acc.cpu().numpy(), want[1])
    lens = new_lens.tolist()
    for i in range(3):
        lens = [n + 1 for n in lens]
        step(1, lens, new_table, new_acc if i else None, n_win=0 if i else 16, n_sink=2)


# ==================================================================================
# the borders of the kernels: row tiles, boxes of pages, halves, runs and clusters
# ==================================================================================
@pytest.mark.parametrize("nq,G", [(16, 1), (17, 1), (4, 4), (6, 3), (127, 1), (32, 4), (43, 3), (64, 4), (257, 1), (86, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_attn_row_tiles(nq, G, d):
    case([nq, nq + 70], nq=nq, n_h=G, n_kv=1, d=d, seed=nq)


@pytest.mark.parametrize("page", [4, 7, 8, 24, 40, 56, 80, 96, 100, 192])
def test_attn_prompt_page_boxes(page):
    case([60, 300], nq=60, n_h=6, n_kv=2, d=128, page=page, seed=page)
    case([60, 300], nq=60, n_h=6, n_kv=2, d=128, page=page, n_win=70, n_sink=9, seed=page)


@pytest.mark.parametrize("d", [8, 24, 40, 72, 96, 104, 120, 192])
def test_attn_prompt_head_widths(d):
    case([50, 190], nq=50, n_h=4, n_kv=2, d=d, seed=d)


@pytest.mark.parametrize("n_win", [1, 2, 63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("n_sink", [0, 1, 64, 130])
def test_attn_prompt_window_borders(n_win, n_sink):
    case([130, 460], nq=130, n_h=2, n_kv=1, d=64, n_win=n_win, n_sink=n_sink, seed=n_win)


def test_attn_prompts_ragged():
    case([(53 * i) % 200 + 1 for i in range(40)], nq=30, n_h=4, n_kv=2, d=64, page=8)
    case([900, 1, 40, 333], nq=200, n_h=8, n_kv=2, d=128, page=32)
    case([2500], nq=70, n_h=2, n_kv=2, d=128, page=16)


@pytest.mark.parametrize("nq,G", [(33, 1), (13, 8), (128, 1), (50, 6)])
@pytest.mark.parametrize("strong", [0, 1])
def test_attn_units_of_one_tile_in_turn(nq, G, strong):
    """Of one row tile the units of 128 tokens are taken in turn by two halves of the kernel: either may hold
    nearly all of the weight, nothing that a row sees, or no unit at all."""
    lens = [nq, 129, 256, 257, 1024, 1500, 2900]
    lens = [max(n, nq) for n in lens]
    page, d, n_kv = 32, 128, 2
    B, max_pages = len(lens), -(-max(lens) // page) + 1
    n_pages = B * max_pages + 2
    K, V = pools(n_pages, page, n_kv, d, torch.bfloat16, 3)
    table = tables(B, max_pages, n_pages, 5)
    for b in range(B):
        for x in range(max_pages):
            K[table[b, x].item()] *= 8.0 if x * page // 128 % 2 == strong else 0.125
    table, t = table.to(DEV), positions(lens, nq).to(DEV)
    q = randn((B, nq, G * n_kv, d), nq, torch.bfloat16).to(DEV)
    for n_win, n_sink in ((0, 0), (100, 0), (129, 3)):
        out, lse, _ = run_attn(q, K, V, table, t, n_win, n_sink)
        check_attn(q, K, V, table, t, out, lse, weight_bits(nq, G * n_kv, n_kv, d, torch.bfloat16, False), n_win, n_sink)


def test_attn_more_key_heads_than_workers():
    case([20, 3], n_h=1300, n_kv=1300, d=8)
    case([20, 3], n_h=1300, n_kv=1300, d=8, dtype=torch.float32)


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attn_outputs_that_do_not_start_on_16_bytes(nq, dtype):
    K, V = pools(9, 16, 2, 64, dtype, 5)
    table = tables(2, 4, 9, 1).to(DEV)
    t = positions([60, 45], nq).to(DEV)
    q = randn((2, nq, 8, 64), 9, dtype).to(DEV)
    ws = torch.empty(lib.paged_attn_workspace_size(2, nq, 8, 2, 64, 64), dtype=torch.uint8, device=DEV)
    for odd_q in (False, True):
        flat = torch.zeros(q.numel() + 1, dtype=dtype, device=DEV)
        out = flat[1:].view(q.shape) if not odd_q else torch.empty_like(q)
        flat_q = torch.zeros(q.numel() + 1, dtype=dtype, device=DEV)
        flat_q[1:] = q.flatten()
        lse = torch.empty(2, nq, 8, device=DEV)
        lib.paged_attn(flat_q[1:].view(q.shape) if odd_q else q, K, V, table, t, out, ws, lse=lse)
        check_attn(q, K, V, table, t, out, lse, 2.0 ** -16)
        assert flat[0] == 0


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attn_nan_that_is_seen_is_told(nq, dtype):
    K, V = pools(9, 16, 2, 64, dtype, 5)
    table = tables(2, 4, 9, 1).to(DEV)
    t = positions([60, 60], nq).to(DEV)
    q = randn((2, nq, 8, 64), 9, dtype).to(DEV)
    K[table[0, 0].long(), 3, 1, 5] = float("nan")  # token 3 of sequence 0, key head 1
    out, lse, _ = run_attn(q, K, V, table, t)
    bad = torch.zeros(2, 8, dtype=torch.bool, device=DEV)
    bad[0, 4:] = True
    assert torch.equal(lse.isnan(), bad[:, None].expand(2, nq, 8))
    assert torch.equal(out.isnan().all(-1), out.isnan().any(-1)) and torch.equal(out.isnan().all(-1), lse.isnan())


def test_attn_positions_in_any_order():
    # padding among the queries, a position twice, falling positions
    K, V = pools(20, 16, 2, 128, torch.bfloat16, 5)
    table = tables(2, 9, 20, 1).to(DEV)
    g = torch.Generator().manual_seed(3)
    t = torch.randint(-3, 150, (2, 50), generator=g)
    t[0, 7], t[0, 8], t[1, 20:30] = 77, 77, -1
    t = t.to(torch.int64).to(DEV)
    q = randn((2, 50, 8, 128), 9).to(DEV)
    for n_win, n_sink in ((0, 0), (20, 3)):
        out, lse, _ = run_attn(q, K, V, table, t, n_win, n_sink)
        check_attn(q, K, V, table, t, out, lse, 2.0 ** -8, n_win, n_sink)


@pytest.mark.parametrize("nq", [1, 40])
def test_attn_pages_shared_by_sequences(nq):
    K, V = pools(9, 16, 2, 128, torch.bfloat16, 5)
    table = torch.tensor([[1, 2, 3, 8], [1, 2, 5, 6], [1, 1, 1, 1]], dtype=torch.int32, device=DEV)
    t = positions([64, 50, 41], nq).to(DEV)
    q = randn((3, nq, 8, 128), 9).to(DEV)
    out, lse, _ = run_attn(q, K, V, table, t)
    check_attn(q, K, V, table, t, out, lse, weight_bits(nq, 8, 2, 128, torch.bfloat16, False))


@pytest.mark.parametrize("nq,dtype", [(1, torch.bfloat16), (40, torch.bfloat16), (1, torch.float32)])
def test_attn_status_of_an_uncleared_workspace(nq, dtype):
    K, V = pools(9, 16, 2, 64, dtype, 5)
    table = tables(2, 4, 9, 1).to(DEV)
    q = randn((2, nq, 8, 64), 9, dtype).to(DEV)
    ws = torch.full((lib.paged_attn_workspace_size(2, nq, 8, 2, 64, 64),), 0xff, dtype=torch.uint8, device=DEV)
    lib.paged_attn(q, K, V, table, positions([60, 45], nq).to(DEV), torch.empty_like(q), ws)
    assert lib.csa_workspace_status(ws) == 0


def test_prompt_on_another_stream():
    K, V = pools(9, 16, 2, 128, torch.bfloat16, 5)
    table = tables(2, 4, 9, 1).to(DEV)
    q = randn((2, 33, 8, 128), 9).to(DEV)
    t = positions([60, 33], 33).to(DEV)
    want = run_attn(q, K, V, table, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    ws = torch.empty(lib.paged_attn_workspace_size(2, 33, 8, 2, 128, 64), dtype=torch.uint8, device=DEV)
    with torch.cuda.stream(side):
        lib.paged_attn(q, K, V, table, t, out, ws)
    side.synchronize()
    assert torch.equal(out, want[0])


def test_two_prompts_at_once():
    # two streams, each with its own workspace, many calls under way
    K, V = pools(40, 16, 2, 128, torch.bfloat16, 5)
    table = tables(2, 18, 40, 1).to(DEV)
    qs = [randn((2, nq, 8, 128), 9 + nq).to(DEV) for nq in (70, 1)]
    ts = [positions([280, 90], nq).to(DEV) for nq in (70, 1)]
    want = [run_attn(q, K, V, table, t) for q, t in zip(qs, ts)]
    streams = [torch.cuda.Stream() for _ in qs]
    wss = [torch.empty(lib.paged_attn_workspace_size(2, q.shape[1], 8, 2, 128, 288), dtype=torch.uint8, device=DEV) for q in qs]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, t, o, w, s in zip(qs, ts, outs, wss, streams):
            lib.paged_attn(q, K, V, table, t, o, w, stream=s)
    torch.cuda.synchronize()
    for o, (x, _, _) in zip(outs, want):
        assert torch.equal(o, x)


@pytest.mark.parametrize("values", ["rand", "ties"])
@pytest.mark.parametrize("B,n_kv,long,keep", [
    (1, 160, 700, 300),    # more key heads than SMs: two selections an SM
    (1, 150, 9000, 100),   # ... with runs that its registers do not hold
    (1, 80, 17000, 5000),  # a CTA for each, too long for its registers
    (1, 30, 9000, 3001),   # clusters of 4
    (2, 15, 5000, 77),     # of 2
])
def test_evict_clusters(B, n_kv, long, keep, values):
    evict_case([long, long // 2][:B], keep, 3, 20, n_kv=n_kv, d=8, page=64, values=values)


def test_counts_that_do_not_fit_are_refused():
    K, V = pools(4, 16, 2, 64, torch.bfloat16, 1)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    t = torch.tensor([[5]], dtype=torch.int64, device=DEV)
    q = randn((1, 1, 4, 64), 1).to(DEV)
    out, ws = torch.empty_like(q), torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    for kw in (dict(n_win=2**32 + 4), dict(n_win=4, n_sink=2**31)):
        with pytest.raises(ValueError):
            lib.paged_attn(q, K, V, table, t, out, ws, **kw)
    with pytest.raises(lib.CSAError):
        lib.paged_attn(q, K, V, table, t, out, ws, n_win=-1)


@pytest.mark.parametrize("nq", [2, 40])
def test_attn_positions_at_the_ends_of_64_bits(nq):
    K, V = pools(6, 16, 2, 64, torch.bfloat16, 5)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device=DEV)
    q = randn((3, nq, 4, 64), 9).to(DEV)
    t = torch.full((3, nq), 2**63 - 1, dtype=torch.int64)
    t[1, 0], t[2] = 5, -2**63
    t = t.to(DEV)
    P = weight_bits(nq, 4, 2, 64, torch.bfloat16, False)
    for n_win, n_sink in ((0, 0), (4, 2)):
        out, lse, _ = run_attn(q, K, V, table, t, n_win, n_sink)
        check_attn(q, K, V, table, t, out, lse, P, n_win, n_sink)


# ==================================================================================
# values that are not finite: what is seen is told, what is not seen reaches nothing
# ==================================================================================
KINDS = [  # a call of each kernel: queries, query heads (two key heads), width, type, layout
    (1, 8, 64, torch.bfloat16, "nhd"), (1, 8, 256, torch.bfloat16, "nhd"), (2, 16, 128, torch.bfloat16, "nhd"),
    (3, 16, 128, torch.bfloat16, "nhd"), (12, 8, 256, torch.bfloat16, "nhd"), (10, 8, 128, torch.bfloat16, "hnd"),
    (90, 8, 64, torch.bfloat16, "nhd"), (1, 4, 64, torch.float32, "nhd"), (2, 8, 128, torch.float32, "hnd"),
    (1, 4, 256, torch.float32, "nhd"), (2, 6, 64, torch.bfloat16, "odd"), (1, 6, 40, torch.float32, "odd")]


@pytest.mark.parametrize("nq,n_h,d,dtype,layout", KINDS)
def test_attn_logits_of_minus_infinity(nq, n_h, d, dtype, layout):
    """Weigh nothing: the first tokens, which a kernel meets before any other, and a run of them further on."""
    lens, page = [40000 if layout == "odd" else 400, 333], 16  # a warp of the CUDA-core kernel has several units
    max_pages = lens[0] // page + 1
    K, V = pools(2 * max_pages + 4, page, 2, d, dtype, 11, layout)
    table = tables(2, max_pages, 2 * max_pages + 4, 4).to(DEV)
    t = positions(lens, nq).to(DEV)
    q = randn((2, nq, n_h, d), 9, dtype).abs().clamp(min=2.0 ** -6).to(DEV)
    hidden = torch.zeros(2, max_pages, dtype=torch.bool, device=DEV)
    hidden[:, :9], hidden[0, max_pages // 2:max_pages * 3 // 4] = True, True
    for b in range(2):
        K[table[b, hidden[b]].long(), :, :, d // 2] = -math.inf
    out, lse, _ = run_attn(q, K, V, table, t)
    # the same as if those pages were not there
    there = torch.where(hidden, -1, table)
    P = 2.0 ** -16 if layout == "odd" else weight_bits(nq, n_h, 2, d, dtype, False)
    check_attn(q, torch.nan_to_num(K, neginf=0.0), V, there, t, out, lse, P)


@pytest.mark.parametrize("what", ["query", "pages", "faint"])
@pytest.mark.parametrize("nq,n_h,d,dtype,layout", KINDS)
def test_attn_nan_in_an_item_that_is_cut(nq, n_h, d, dtype, layout, what):
    """A row whose logits are NaN, all of them or a long run of them, or one far below the row's largest: its out and
    lse are NaN however its tokens are cut into pieces, and no other row changes."""
    lens, page = [9000, 90, 9000], 16
    max_pages = 564
    K, V = pools(3 * max_pages + 2, page, 2, d, dtype, 11, layout)
    table = tables(3, max_pages, 3 * max_pages + 2, 4).to(DEV)
    t = positions(lens, nq).to(DEV)
    q = randn((3, nq, n_h, d), 9, dtype).to(DEV)
    bad = torch.zeros(3, nq, n_h, dtype=torch.bool, device=DEV)
    if what == "faint":  # token 20 has nearly all of the weight
        q[2, :, n_h // 2:] = 1.0
        K[table[2, 1].long(), 4, 1] = 40.0
    want, want_lse, _ = run_attn(q, K, V, table, t)
    if what == "query":
        q[0, nq - 1, 1] = float("nan")
        bad[0, nq - 1, 1] = True
    else:
        bad[2, :, n_h // 2:] = True
        if what == "pages":
            K[table[2, 100:300].long(), :, 1] = float("nan")
        else:
            K[table[2, 400].long(), 7, 1, 3] = float("nan")
    out, lse, _ = run_attn(q, K, V, table, t)
    assert torch.equal(lse.isnan(), bad)
    assert torch.equal(out.isnan(), bad[..., None].expand_as(out))
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])


def spread(nq, n_win, cap, seed):
    """Positions whose windows leave holes: falling and far apart; in any order, with padding among them; and at the two
    steps where a hole of one token ends: n_win + 1 and n_win."""
    g = torch.Generator().manual_seed(seed)
    t = torch.full((4, nq), -1, dtype=torch.int64)
    t[0] = torch.linspace(cap - 1, 5, nq).long() if nq > 1 else cap - 1
    t[1] = torch.randint(-cap // 4, cap, (nq,), generator=g).clamp(min=-1)
    at = 7
    for i in range(nq):
        t[2, i] = min(at, cap - 1)
        at += n_win + 1 if i % 3 == 1 else n_win if i % 3 == 0 else 1
    t[3, 0], t[3, nq - 1], t[3, nq // 2] = 30, cap + 3, 30 + n_win // 2
    return t


@pytest.mark.parametrize("n_win,n_sink", [(1, 0), (16, 3), (50, 70)])
@pytest.mark.parametrize("nq,n_h,d,dtype,layout", [
    (2, 4, 64, torch.bfloat16, "nhd"), (4, 4, 256, torch.bfloat16, "hnd"), (8, 4, 128, torch.bfloat16, "nhd"),
    (15, 4, 64, torch.bfloat16, "nhd"), (33, 2, 256, torch.bfloat16, "nhd"), (50, 4, 128, torch.bfloat16, "nhd"),
    (50, 2, 64, torch.bfloat16, "hnd"), (150, 4, 128, torch.bfloat16, "nhd"), (3, 2, 64, torch.float32, "nhd"),
    (20, 4, 128, torch.float32, "hnd"), (9, 2, 256, torch.float32, "nhd"), (7, 4, 40, torch.bfloat16, "odd")])
@pytest.mark.parametrize("page", [16, 24])
def test_attn_rows_between_windows_reach_nothing(nq, n_h, d, dtype, layout, n_win, n_sink, page):
    cap = page * (912 // page)
    B, max_pages = 4, cap // page
    n_pages = B * max_pages + 1
    K, V = pools(n_pages, page, 2, d, dtype, 21, layout)
    table = tables(B, max_pages, n_pages, 6)
    t = spread(nq, n_win, cap, nq)
    j = torch.arange(cap)
    seen = ((j <= t[..., None]) & ((j > t[..., None] - n_win) | (j < n_sink))).any(1)  # [B, cap]
    used = torch.zeros(n_pages, page, dtype=torch.bool)
    for b in range(B):
        used[table[b].long()[j // page], j % page] = seen[b]
    K[~used.to(DEV)], V[~used.to(DEV)] = float("nan"), float("nan")
    table, t = table.to(DEV), t.to(DEV)
    q = randn((B, nq, n_h, d), 9, dtype, scale=2.0).to(DEV)
    acc = torch.rand(B, 2, cap, device=DEV)
    out, lse, acc_out = run_attn(q, K, V, table, t, n_win, n_sink, acc=acc)
    P = 2.0 ** -16 if layout == "odd" else weight_bits(nq, n_h, 2, d, dtype, True)
    check_attn(q, torch.nan_to_num(K), torch.nan_to_num(V), table, t, out, lse, P, n_win, n_sink, acc=acc, acc_out=acc_out)


# ==================================================================================
# waits that run out
# ==================================================================================
@pytest.mark.parametrize("budget", [0, 100, 500, 2000, 8000])
@pytest.mark.parametrize("nq,d,n_win", [(40, 128, 0), (33, 64, 50), (150, 128, 0), (300, 64, 70)])
def test_prompt_waits_that_run_out_are_reported(nq, d, n_win, budget):
    """Failure detection without a GPU fault: with a budget of a few clocks the prompt kernel's bounded waits run out,
    wherever its warps happen to be; the call says so through the workspace's status, and the next call is right."""
    K, V = pools(140, 16, 2, d, torch.bfloat16, 5)
    table = tables(2, 66, 140, 1).to(DEV)
    q = randn((2, nq, 8, d), 9).to(DEV)
    t = positions([1050, 400], nq).to(DEV)
    ws = torch.empty(lib.paged_attn_workspace_size(2, nq, 8, 2, d, 1056, True), dtype=torch.uint8, device=DEV)
    acc = torch.zeros(2, 2, 1056, device=DEV)
    want = run_attn(q, K, V, table, t, n_win, 4, acc=acc, ws=ws)
    assert lib.csa_workspace_status(ws) == 0
    try:
        lib.paged_attn_set_wait_budget(budget)
        got = run_attn(q, K, V, table, t, n_win, 4, acc=acc, ws=ws)
    finally:
        lib.paged_attn_set_wait_budget(-1)
    status = lib.csa_workspace_status(ws)
    assert status in ((-7,) if budget == 0 else (0, -7))
    again = run_attn(q, K, V, table, t, n_win, 4, acc=acc, ws=ws)
    assert lib.csa_workspace_status(ws) == 0
    for x, y, z in zip(want, got, again):
        assert torch.equal(x, z) and (status != 0 or torch.equal(x, y))


@pytest.mark.parametrize("nq", [1, 40])
def test_no_capacity_needs_no_pools(nq):
    """The C call with max_pages = 0: the pools and the table may be null, and every query sees nothing."""
    import ctypes
    q = randn((2, nq, 8, 128), 9).to(DEV)
    out, lse = torch.full_like(q, 7.0), torch.full((2, nq, 8), 7.0, device=DEV)
    t = positions([60, 45], nq).to(DEV)
    ws = torch.empty(lib.paged_attn_workspace_size(2, nq, 8, 2, 128, 0), dtype=torch.uint8, device=DEV)
    p = lambda x: ctypes.c_void_p(x.data_ptr())  # noqa: E731
    assert lib.library().paged_attn(p(q), None, None, 16 * 256, 256, 128, 4, 16, None, 0, p(t), 2, nq, 8, 2, 128, 0, 0, 0.0,
                                    p(out), p(lse), None, None, p(ws), ws.nbytes, 0, 1,
                                    ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


# ==================================================================================
# accumulated weights of every kernel, and in captured calls
# ==================================================================================
@pytest.mark.parametrize("n_win,n_sink", [(0, 0), (40, 5)])
@pytest.mark.parametrize("nq,n_h,n_kv,d,page", [
    (1, 8, 2, 256, 16), (2, 6, 2, 256, 16),         # 8 rows or fewer of wide heads: two warps a worker
    (3, 16, 2, 128, 16), (2, 24, 2, 64, 32),        # 17 to 32 rows
    (4, 16, 2, 256, 16), (5, 24, 2, 256, 16),       # ... of wide heads, and 60
    (5, 32, 2, 128, 16), (40, 2, 2, 64, 64), (5, 16, 1, 96, 8),  # one tile of the prompt kernel
    (60, 8, 2, 128, 16), (140, 4, 2, 64, 32),       # two tiles, and a third
    (1, 8, 2, 64, 3), (50, 4, 2, 64, 7)])           # a capacity that is no multiple of 4
def test_weights_of_every_kernel(nq, n_h, n_kv, d, page, n_win, n_sink):
    case([nq, 300, 2999], nq=nq, n_h=n_h, n_kv=n_kv, d=d, page=page, n_win=n_win, n_sink=n_sink, acc=True, seed=nq)


@pytest.mark.parametrize("nq,n_h", [(1, 8), (3, 16), (40, 8)])
def test_graphs_accumulate_the_weights_of_their_lengths(nq, n_h):
    """Two captured graphs share a workspace; in each a call that accumulates and one that does not. Every replay's
    increment, outputs and log-sum-exps are those of the lengths that it finds."""
    K, V = pools(70, 16, 2, 128, torch.bfloat16, 5)
    table = tables(2, 30, 70, 1).to(DEV)
    qs = [randn((2, nq, n_h, 128), 9 + i).to(DEV) for i in range(2)]
    ts = [positions([100, 70], nq).to(DEV) for _ in qs]
    outs = [[torch.empty_like(q) for _ in range(2)] for q in qs]
    lses = [[torch.empty(2, nq, n_h, device=DEV) for _ in range(2)] for _ in qs]
    accs = [torch.rand(2, 2, 480, device=DEV) for _ in qs]
    ws = torch.empty(lib.paged_attn_workspace_size(2, nq, n_h, 2, 128, 480, True), dtype=torch.uint8, device=DEV)
    lib.paged_attn(qs[0], K, V, table, ts[0], outs[0][0], ws)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for x in range(2):
                lib.paged_attn(qs[i], K, V, table, ts[i], outs[i][x], ws, lse=lses[i][x], n_win=64 * i, n_sink=4,
                               acc=None if x else accs[i])
        graphs.append(g)
    P = weight_bits(nq, n_h, 2, 128, torch.bfloat16, True)
    for lens in ([100, 70], [480, nq], [max(nq, 33), 470], [nq, 2 * nq]):
        before = [a.clone() for a in accs]
        for i in range(2):
            ts[i].copy_(positions(lens, nq))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for x in range(2):
                check_attn(qs[i], K, V, table, ts[i], outs[i][x], lses[i][x], P, 64 * i, 4, acc=None if x else before[i],
                           acc_out=None if x else accs[i])


# ==================================================================================
# captured serving steps, and calls with nothing to do
# ==================================================================================
def test_a_captured_step_appends_attends_and_evicts():
    """One graph: append, attention that accumulates, eviction to other pages. Every replay is right for the tokens,
    positions and lengths that it finds, and leaves the old pages as they were."""
    B, n_h, n_kv, d, page, max_pages, keep = 3, 8, 2, 64, 16, 20, 64
    n_pages = B * (max_pages + 4)
    K, V = pools(n_pages, page, n_kv, d, torch.bfloat16, 31)
    both = tables(B, max_pages + 4, n_pages, 2).to(DEV)
    table, new_table = both[:, :max_pages].contiguous(), both[:, max_pages:].contiguous()
    cap = max_pages * page
    k, v = (torch.empty(B, 1, n_kv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.empty(B, 1, n_h, d, dtype=torch.bfloat16, device=DEV)
    t, lens = torch.zeros(B, 1, dtype=torch.int64, device=DEV), torch.ones(B, dtype=torch.int64, device=DEV)
    acc, out, lse = torch.zeros(B, n_kv, cap, device=DEV), torch.empty_like(q), torch.empty(B, 1, n_h, device=DEV)
    new_lens, idx = torch.zeros_like(lens), torch.zeros(B, n_kv, keep, dtype=torch.int32, device=DEV)
    new_acc = torch.zeros(B, n_kv, 4 * page, device=DEV)
    ws = torch.empty(lib.paged_attn_workspace_size(B, 1, n_h, n_kv, d, cap, True), dtype=torch.uint8, device=DEV)

    def step():
        lib.paged_append(k, v, K, V, table, t)
        lib.paged_attn(q, K, V, table, t, out, ws, lse=lse, acc=acc)
        lib.paged_evict(K, V, table, lens, acc, keep, new_table, new_lens, new_acc, idx, n_sink=2, n_recent=8)

    for x in (k, v, q):
        x.zero_()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, ns in enumerate(([300, 65, 1], [64, 320, 200], [301, 66, 2])):
        for j, x in enumerate((k, v, q)):
            x.copy_(randn(tuple(x.shape), 50 + 3 * i + j))
        lens.copy_(torch.tensor(ns))
        t.copy_(positions(ns, 1))
        acc.copy_(torch.rand(B, n_kv, cap))
        before, wk, wv = acc.clone(), to_f64(K), to_f64(V)
        graph.replay()
        torch.cuda.synchronize()
        O.append(to_f64(k), to_f64(v), wk, wv, table.cpu().numpy(), t.cpu().numpy())
        check_attn(q, torch.tensor(wk), torch.tensor(wv), table, t, out, lse, 2.0 ** -16, acc=before, acc_out=acc)
        want = O.evict(wk, wv, table.cpu().numpy(), np.array(ns), acc.cpu().numpy(), keep, new_table.cpu().numpy(), 2, 8)
        np.testing.assert_array_equal(new_lens.cpu().numpy(), want[0])
        np.testing.assert_array_equal(new_acc.cpu().numpy(), want[1])
        np.testing.assert_array_equal(idx.cpu().numpy(), want[2])
        np.testing.assert_array_equal(to_f64(K), wk)
        np.testing.assert_array_equal(to_f64(V), wv)


def test_calls_with_nothing_to_do():
    K, V = pools(6, 16, 2, 64, torch.bfloat16, 5)
    wk, wv = K.clone(), V.clone()
    i32, i64 = dict(dtype=torch.int32, device=DEV), dict(dtype=torch.int64, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    for B, nq in ((0, 1), (2, 0)):  # no sequences, no queries
        x = torch.empty(B, nq, 2, 64, dtype=torch.bfloat16, device=DEV)
        table, t = torch.zeros(B, 2, **i32), torch.zeros(B, nq, **i64)
        lib.paged_append(x, x, K, V, table, t)
        lib.paged_attn(x, K, V, table, t, torch.empty_like(x), ws)
    none = torch.zeros(0, 2, **i32)
    lib.paged_evict(K, V, none, torch.zeros(0, **i64), torch.zeros(0, 2, 32, device=DEV), 4, none[:, :1].contiguous(),
                    torch.zeros(0, **i64), torch.zeros(0, 2, 16, device=DEV), torch.zeros(0, 2, 4, **i32))
    # a cache without pages: nothing is kept, whatever its lengths say
    new = torch.tensor([[3], [4]], **i32)
    idx, new_lens, new_acc = run_evict(K, V, torch.zeros(2, 0, **i32), torch.tensor([5, 0], **i64),
                                       torch.zeros(2, 2, 0, device=DEV), 4, new)
    assert new_lens.tolist() == [0, 0] and bool((idx == -1).all()) and bool((new_acc == 0).all())
    ones = torch.ones(2, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    lib.paged_append(ones, ones, K, V, torch.zeros(2, 0, **i32), torch.zeros(2, 1, **i64))
    torch.cuda.synchronize()
    assert torch.equal(K, wk) and torch.equal(V, wv)
