"""Paged cache, without a GPU: the oracle against closed forms, and the refusals of the C ABI
(every call below fails its host checks, or has nothing to do, before any launch)."""
import ctypes
import math

import numpy as np
import pytest

from oracle import paged as O

vp = ctypes.c_void_p
FAKE = vp(0x10000)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from long_context_compressed_csa_b200 import build
    build.build()
    from long_context_compressed_csa_b200._binding import library
    return library()


def test_oracle_visibility():
    assert O.visible(5, 100, 0, 3) == [0, 1, 2, 3, 4, 5]
    assert O.visible(9, 100, 3, 2) == [0, 1, 7, 8, 9]
    assert O.visible(9, 100, 9, 2) == list(range(10))
    assert O.visible(-1, 100, 4, 2) == []
    assert O.visible(9, 8, 3, 0) == [7]
    assert O.visible(0, 8, 1, 4) == [0]


def test_oracle_attention_closed_forms():
    # one visible token: its value, and its logit; equal logits: the mean; a missing page is not seen
    K = np.zeros((3, 2, 1, 2))
    V = np.arange(12, dtype=float).reshape(3, 2, 1, 2)
    q = np.ones((1, 1, 2, 2))
    table = np.array([[2, -1, 0]])
    out, lse, w, _ = O.attn(q, K, V, table, np.array([[0]]))
    np.testing.assert_array_equal(out[0, 0], [[8, 9], [8, 9]])
    np.testing.assert_array_equal(lse[0, 0], [0, 0])
    np.testing.assert_array_equal(w[0, 0], [2, 0, 0, 0, 0, 0])
    out, lse, w, _ = O.attn(q, K, V, table, np.array([[5]]))  # tokens 0, 1 (page 2) and 4, 5 (page 0)
    np.testing.assert_allclose(out[0, 0, 0], [(8 + 10 + 0 + 2) / 4, (9 + 11 + 1 + 3) / 4])
    np.testing.assert_allclose(lse[0, 0], math.log(4))
    np.testing.assert_allclose(w[0, 0], [0.5, 0.5, 0, 0, 0.5, 0.5])
    K[2, 1] = [1.0, 2.0]
    out, lse, _, _ = O.attn(q, K, V, table, np.array([[1]]), scale=0.5)
    p = math.exp(1.5) / (1 + math.exp(1.5))
    np.testing.assert_allclose(out[0, 0, 0], [8 * (1 - p) + 10 * p, 9 * (1 - p) + 11 * p])
    np.testing.assert_allclose(lse[0, 0], math.log(1 + math.exp(1.5)))


def test_oracle_eviction():
    acc = np.array([0.0, 5.0, 1.0, 5.0, math.nan, 3.0, -math.inf, 0.0])
    assert O.evict_keep(acc, 8, 3, 0, 0) == [1, 3, 5]
    assert O.evict_keep(acc, 8, 1, 0, 0) == [1]
    assert O.evict_keep(acc, 8, 4, 1, 2) == [0, 1, 6, 7]
    assert O.evict_keep(acc, 8, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 7]
    assert O.evict_keep(acc, 3, 3, 1, 2) == [0, 1, 2]
    assert O.evict_keep(acc, 0, 3, 1, 2) == []


def append_args(**kw):
    a = dict(k=FAKE, v=FAKE, lb=64, lt=64, lh=8, K=FAKE, V=FAKE, lp=256, lr=16, lhd=8, n_pages=4, page=16, table=FAKE,
             max_pages=2, t=FAKE, B=1, nq=1, n_kv=2, d=8, dtype=0, stream=None)
    a.update(kw)
    return list(a.values())


def attn_args(**kw):
    a = dict(q=FAKE, K=FAKE, V=FAKE, lp=256, lr=16, lhd=8, n_pages=4, page=16, table=FAKE, max_pages=2, t=FAKE, B=1,
             nq=1, n_h=4, n_kv=2, d=8, n_win=0, n_sink=0, scale=0.0, out=FAKE, lse=None, acc=None, acc_out=None,
             ws=FAKE, ws_bytes=1 << 40, dtype=0, out_bf16=1, stream=None)
    a.update(kw)
    return list(a.values())


def evict_args(**kw):
    a = dict(K=FAKE, V=FAKE, lp=256, lr=16, lhd=8, n_pages=4, page=16, table=FAKE, max_pages=2, lens=FAKE, acc=FAKE,
             B=1, n_kv=2, d=8, keep=8, n_sink=1, n_recent=2, new_table=vp(0x20000), new_max_pages=1,
             new_lens=vp(0x20000), new_acc=vp(0x20000), idx=FAKE, dtype=0, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(k=None), -1), (dict(table=None), -1), (dict(t=None), -1), (dict(V=None), -1),
    (dict(B=-1), -1), (dict(nq=-1), -1), (dict(n_kv=0), -1), (dict(d=0), -1), (dict(page=0), -1), (dict(n_pages=-1), -1),
    (dict(max_pages=-1), -1), (dict(lr=7), -1), (dict(lhd=4), -1), (dict(lt=-8), -1), (dict(k=vp(0x10001)), -2),
    (dict(t=vp(0x10004)), -2), (dict(table=vp(0x10002)), -2), (dict(page=1 << 30, max_pages=2), -6),
    (dict(B=0), 0), (dict(nq=0), 0), (dict(max_pages=0), 0)])
def test_append_refusals(lib, kw, status):
    assert lib.paged_append(*append_args(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(dtype=1, out_bf16=1), -3), (dict(n_h=5), -1), (dict(n_h=0), -1), (dict(n_win=-1), -1),
    (dict(n_sink=-1), -1), (dict(q=None), -1), (dict(K=None), -1), (dict(table=None), -1), (dict(t=None), -1),
    (dict(out=None), -1), (dict(acc=FAKE), -1), (dict(acc_out=FAKE), -1), (dict(ws=None), -4), (dict(ws_bytes=64), -4),
    (dict(ws=vp(0x10004)), -2), (dict(q=vp(0x10001)), -2), (dict(lse=vp(0x10002)), -2), (dict(t=vp(0x10004)), -2),
    (dict(acc=vp(0x10002), acc_out=FAKE), -2), (dict(d=257, lr=600, lhd=257), -6), (dict(page=1 << 30), -6),
    (dict(nq=1 << 30), -6), (dict(B=70000), -6), (dict(B=0), 0), (dict(nq=0), 0), (dict(page=-1), -1), (dict(lr=4), -1)])
def test_attn_refusals(lib, kw, status):
    assert lib.paged_attn(*attn_args(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(K=None), -1), (dict(lens=None), -1), (dict(acc=None), -1), (dict(idx=None), -1),
    (dict(keep=0), -1), (dict(n_sink=-1), -1), (dict(n_recent=-1), -1), (dict(n_sink=4, n_recent=5), -1),
    (dict(n_sink=2**31 - 1, n_recent=2**31 - 1), -1), (dict(keep=17), -1), (dict(new_table=FAKE), -1),
    (dict(new_lens=FAKE), -1), (dict(new_acc=FAKE), -1), (dict(K=vp(0x10001)), -2), (dict(lens=vp(0x10004)), -2),
    (dict(idx=vp(0x10002)), -2), (dict(new_max_pages=1 << 28), -6), (dict(B=0), 0)])
def test_evict_refusals(lib, kw, status):
    assert lib.paged_evict(*evict_args(**kw)) == status


def test_workspace_size(lib):
    size = lib.paged_attn_workspace_size
    assert size(1, 1, 8, 8, 64, 1 << 20, 0) > 0
    assert size(0, 1, 8, 8, 64, 100, 0) == size(1, 1, 9, 8, 64, 100, 0) == size(1, 1, 8, 8, 257, 100, 0) == 0
    # the weights' logits: fp32 for every (token, query row)
    assert size(2, 1, 64, 8, 128, 8192, 1) >= size(2, 1, 64, 8, 128, 8192, 0) + 2 * 64 * 8192 * 4


def test_binding_refuses_host_tensors():
    import torch

    import long_context_compressed_csa_b200 as lib
    K = torch.zeros(2, 4, 1, 8, dtype=torch.bfloat16)
    table, t = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int64)
    x = torch.zeros(1, 1, 1, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.paged_append(x, x, K, K, table, t)
    with pytest.raises(ValueError):
        lib.paged_attn(x, K, K, table, t, x, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        lib.paged_evict(K, K, table, t[0], torch.zeros(1, 1, 4), 2, table, t[0], torch.zeros(1, 1, 4), table)
