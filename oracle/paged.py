"""fp64 oracle of the paged key-value cache: plain loops over sequences, heads and queries.

Test infrastructure, numpy only; it shares no code with the CUDA path.  A token whose table entry
lies outside the pool is cached nowhere: it is neither read nor written, and no query sees it.
"""
import numpy as np


def page_of(table, b, j, page, n_pages):
    p = int(table[b, j // page])
    return p if 0 <= p < n_pages else -1


def visible(t, cap, n_win, n_sink):
    """The tokens that a query at position t sees, rising."""
    out = []
    for j in range(min(t + 1, cap) if t >= 0 else 0):
        if n_win == 0 or j > t - n_win or j < n_sink:
            out.append(j)
    return out


def append(k, v, K, V, table, t):
    """K, V [pages, page, n_kv, d] in place."""
    n_pages, page = K.shape[:2]
    cap = table.shape[1] * page
    B, nq = t.shape
    for b in range(B):
        for i in range(nq):
            if 0 <= t[b, i] < cap:
                p = page_of(table, b, int(t[b, i]), page, n_pages)
                if p >= 0:
                    K[p, t[b, i] % page] = k[b, i]
                    V[p, t[b, i] % page] = v[b, i]


def attn(q, K, V, table, t, scale=None, n_win=0, n_sink=0):
    """out [B, nq, n_h, d], lse [B, nq, n_h], weights [B, n_kv, cap] (summed over the queries and the
    query heads of a key head), and for the error bounds per (b, i, x): the number of visible
    tokens, max_j scale * sum |q K_j|, and sum_j p_j |V_j| [.., d]."""
    q, K, V = (np.asarray(x, np.float64) for x in (q, K, V))
    B, nq, n_h, d = q.shape
    n_pages, page, n_kv, _ = K.shape
    cap, G = table.shape[1] * page, n_h // n_kv
    scale = scale or d ** -0.5
    out = np.zeros((B, nq, n_h, d))
    lse = np.full((B, nq, n_h), -np.inf)
    w = np.zeros((B, n_kv, cap))
    n_vis, mag, pv = np.zeros((B, nq, n_h)), np.zeros((B, nq, n_h)), np.zeros((B, nq, n_h, d))
    for b in range(B):
        for i in range(nq):
            js = [j for j in visible(int(t[b, i]), cap, n_win, n_sink) if page_of(table, b, j, page, n_pages) >= 0]
            if not js:
                continue
            js = np.array(js)
            ps, rs = table[b, js // page], js % page
            for h in range(n_kv):
                k, v = K[ps, rs, h], V[ps, rs, h]
                x = slice(h * G, (h + 1) * G)
                s = scale * (q[b, i, x] @ k.T)
                top = s.max(-1, keepdims=True)
                e = np.exp(s - top)
                p = e / e.sum(-1, keepdims=True)
                out[b, i, x] = p @ v
                lse[b, i, x] = top[:, 0] + np.log(e.sum(-1))
                w[b, h, js] += p.sum(0)
                n_vis[b, i, x] = len(js)
                mag[b, i, x] = scale * (np.abs(q[b, i, x]) @ np.abs(k).T).max(-1)
                pv[b, i, x] = p @ np.abs(v)
    return out, lse, w, (n_vis, mag, pv)


def evict_keep(acc, n, keep, n_sink, n_recent):
    """Positions that stay of n tokens with weights acc (NaN: lowest), rising."""
    if n <= keep:
        return list(range(n))
    safe = list(range(n_sink)) + list(range(n - n_recent, n))
    value = [-np.inf if np.isnan(a) else a for a in acc[:n]]
    # a NaN goes below -inf too
    rest = sorted(range(n_sink, n - n_recent), key=lambda j: (np.isnan(acc[j]), -value[j], j))
    return sorted(safe + rest[:keep - len(safe)])


def evict(K, V, table, lens, acc, keep, new_table, n_sink=0, n_recent=0):
    """K, V in place; returns new_lens, new_acc, idx."""
    n_pages, page, n_kv, _ = K.shape
    B, new_cap = table.shape[0], new_table.shape[1] * page
    new_lens = np.zeros(B, np.int64)
    new_acc = np.zeros((B, n_kv, new_cap), acc.dtype)
    idx = np.full((B, n_kv, keep), -1, np.int32)
    for b in range(B):
        n = int(min(max(lens[b], 0), table.shape[1] * page))
        new_lens[b] = min(n, keep)
        for h in range(n_kv):
            for s, j in enumerate(evict_keep(acc[b, h], n, keep, n_sink, n_recent)):
                idx[b, h, s] = j
                new_acc[b, h, s] = acc[b, h, j]
                src, dst = page_of(table, b, j, page, n_pages), page_of(new_table, b, s, page, n_pages)
                if dst >= 0:
                    K[dst, s % page, h] = K[src, j % page, h] if src >= 0 else 0
                    V[dst, s % page, h] = V[src, j % page, h] if src >= 0 else 0
    return new_lens, new_acc, idx
