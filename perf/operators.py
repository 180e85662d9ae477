"""What is measured of the paged key-value cache of the stack's full-attention layers.

Four operators: `append` writes new tokens' keys and values into pages, `attn` is grouped-query
attention of one or many query tokens over the pages (every earlier token, or a sliding window
and a few first tokens), `weights` is the same attention that also accumulates each cached
token's attention weight, and `evict` keeps the heaviest tokens and moves them to new pages.

Layouts: q, out [B, nq, n_h, d]; new keys and values [B, nq, n_kv, d]; pools
[pages, page, n_kv, d]; table int32 [B, max_pages]; t int64 [B, nq] (the cache position of each
query token, which sees the tokens up to its own); accumulated weights fp32 [B, n_kv, cap] with
cap = max_pages * page.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------- cases
def _case(name, op, B, long, short, nq=1, n_h=32, n_kv=8, d=128, page=16, dtype="bf16", n_win=0, n_sink=0, keep=0,
          n_recent=0):
    return dict(name=name, op=op, B=B, long=long, short=short, nq=nq, n_h=n_h, n_kv=n_kv, d=d, page=page, dtype=dtype,
                n_win=n_win, n_sink=n_sink, keep=keep, n_recent=n_recent)


def listed():
    return [
        # one decode step's new row of each of 64 sequences
        _case("append_b64", "append", 64, 8192, 1, page=16),
        # a prompt of four ragged sequences enters the cache
        _case("append_prompt_4x8k", "append", 4, 8192, 4099, nq=4099, page=64),
        # a single user's decode step at the 8K context: latency counts
        _case("attn_b1_8k", "attn", 1, 8191, 8191, n_h=64),
        # a serving batch with contexts from one token to 128K
        _case("attn_b16_128k", "attn", 16, 131072, 1, n_h=32, n_kv=4, page=64),
        # two sequences at 256K with one key head per query head, narrow heads
        _case("attn_b2_256k_mha", "attn", 2, 262139, 262001, n_h=8, n_kv=8, d=64, page=128),
        # the fp32 form
        _case("attn_b8_4k_fp32", "attn", 8, 4097, 100, n_h=16, n_kv=4, d=128, dtype="fp32"),
        # streaming decode: 1024 recent tokens and 4 first ones of long contexts
        _case("window_b64_32k", "attn", 64, 32768, 500, n_h=64, n_win=1024, n_sink=4),
        # a prompt through the window: 8192 query tokens, each with 2048 recent tokens and 4 first ones
        _case("window_prompt_8k", "attn", 1, 8192, 8192, nq=8192, n_win=2048, n_sink=4, page=64),
        # a chunk of a long prompt against everything before it
        _case("chunk_2x1k_of_16k", "attn", 2, 16384, 15001, nq=1024, n_h=64, page=64),
        # a decode step that accumulates the weights eviction goes by
        _case("weights_b16_8k", "weights", 16, 8193, 4097, n_h=64),
        # the cache of 16 sequences cut back to 4096 tokens a head
        _case("evict_b16_8k", "evict", 16, 8193, 3001, keep=4096, n_sink=4, n_recent=512),
        # one long sequence cut back to a quarter
        _case("evict_b1_128k", "evict", 1, 131072, 131072, keep=32768, n_sink=4, n_recent=4096, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """Batches of 1 to 64, contexts of 1 to 262144 tokens, one query token to a long prompt, both types."""
    op = rng.choice(["append", "attn", "attn", "attn", "window", "window", "chunk", "weights", "evict", "evict"])
    B, n_kv, G = _log(rng, 1, 64), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
    d, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 48, 64, 128])
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    nq, n_win, n_sink, keep, n_recent = 1, 0, 0, 0, 0
    long = _log(rng, 1, 262144)
    if op == "append":
        nq = _log(rng, 1, 4096)
    elif op in ("attn", "weights"):
        nq = rng.choice([1, 1, 1, 2, 3, 5])
    elif op == "window":
        n_win, n_sink = _log(rng, 1, 4096), rng.choice([0, 1, 4, 16])
    elif op == "chunk":
        B, nq, dtype, d = rng.choice([1, 2, 3]), _log(rng, 32, 4096), "bf16", rng.choice([64, 128])
        n_win, n_sink = rng.choice([(0, 0), (_log(rng, 16, 4096), 4)])
        long = _log(rng, nq, 16384)
    room = 1.2e8 if op == "evict" else 5.0e8  # cached elements of both pools: no more bytes than the largest listed case's
    long = max(1, min(long, int(room / (2 * B * n_kv * d))))
    nq = min(nq, long)
    while op == "chunk" and B * nq * n_kv * G * long * d > 2.0e11:
        nq, long = max(1, nq // 2), max(1, long // 2)
    short = rng.choice([long, max(1, long // 2), max(1, long // 7), 1])
    if op == "evict":
        long = max(long, 2)
        keep = max(1, _log(rng, 1, long))
        n_sink = min(rng.choice([0, 1, 4]), keep // 2)
        n_recent = min(_log(rng, 1, 4096), keep - n_sink)
    if op == "chunk":
        short = max(nq, short)
    c = _case("", {"window": "attn", "chunk": "attn"}.get(op, op), B, long, short, nq, n_kv * G, n_kv, d, page, dtype,
              n_win, n_sink, keep, n_recent)
    del c["name"]
    return c


def _lens(case):
    """Cached tokens of each sequence, the new ones included: from `short` to `long`, out of order."""
    B = case["B"]
    return [case["long"] - (case["long"] - case["short"]) * ((5 * b + 3) % B if B > 1 else 0) // max(1, B - 1)
            for b in range(B)]


def _visible(case, t):
    """How many tokens a query at position t sees."""
    if t < 0 or not case["n_win"]:
        return max(0, t + 1)
    first = max(0, t - case["n_win"] + 1)
    return t + 1 - first + min(first, case["n_sink"])


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    dtype = DTYPES[case["dtype"]]
    B, nq, n_h, n_kv, d, page = (case[x] for x in ("B", "nq", "n_h", "n_kv", "d", "page"))
    lens = _lens(case)

    def normal(*shape, dtype=dtype, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    max_pages = -(-case["long"] // page) + 1  # room for the tokens to come
    new_pages = -(-case["keep"] // page) + 1 if case["keep"] else 0
    pages = B * (max_pages + new_pages) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)  # pages of a pool in use lie anywhere
    s["table"] = order[:B * max_pages].reshape(B, max_pages).contiguous()
    s["K"], s["V"] = (normal(pages, page, n_kv, d) for _ in range(2))
    s["lens"] = torch.tensor(lens, dtype=torch.int64, device="cuda")
    # the last nq positions of each sequence; a shorter one's rows before its first token are padding
    s["t"] = torch.clamp(s["lens"][:, None] - nq + torch.arange(nq, device="cuda")[None], min=-1).contiguous()
    cap = max_pages * page
    if case["op"] == "append":
        s["k"], s["v"] = (normal(B, nq, n_kv, d) for _ in range(2))
        return s
    if case["op"] in ("weights", "evict"):
        s["acc"] = torch.rand(B, n_kv, cap, generator=g, device="cuda") ** 4  # few tokens carry most of the weight
    if case["op"] == "evict":
        s["new_table"] = order[B * max_pages:B * (max_pages + new_pages)].reshape(B, new_pages).contiguous()
        s["new_lens"] = torch.zeros(B, dtype=torch.int64, device="cuda")
        s["new_acc"] = torch.zeros(B, n_kv, new_pages * page, device="cuda")
        s["idx"] = torch.zeros(B, n_kv, case["keep"], dtype=torch.int32, device="cuda")
        return s
    s["q"] = normal(B, nq, n_h, d, scale=2.0)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(B, nq, n_h, device="cuda")
    s["acc_out"] = torch.zeros_like(s["acc"]) if case["op"] == "weights" else None
    # what a call may need at most: kept by the program from step to step
    if own:
        import long_context_compressed_csa_b200 as lib
        s["ws"] = torch.zeros(lib.paged_attn_workspace_size(B, nq, n_h, n_kv, d, cap, weights=case["op"] == "weights"),
                              dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms
def _rows(pool, table):
    """The cached rows of every sequence in order, [B, n_kv, cap, d]."""
    x = pool[table.long()]
    return x.flatten(1, 2).transpose(1, 2)


def _plain_append(s):
    t = s["t"]
    page_of = torch.gather(s["table"].long(), 1, t.clamp(min=0) // s["page"])
    row = t.clamp(min=0) % s["page"]
    keep = t >= 0
    for pool, x in ((s["K"], s["k"]), (s["V"], s["v"])):
        pool[page_of[keep], row[keep]] = x[keep]
    return {"K": s["K"], "V": s["V"]}


def _plain_attn(s):
    q, n_kv, d, t = s["q"], s["n_kv"], s["d"], s["t"]
    B, nq, n_h, _ = q.shape
    K, V = _rows(s["K"], s["table"]).float(), _rows(s["V"], s["table"]).float()
    cap = K.shape[2]
    # query heads h * G .. h * G + G - 1 share key head h
    rows = q.float().reshape(B, nq, n_kv, n_h // n_kv, d).permute(0, 2, 3, 1, 4).reshape(B, n_kv, -1, d)
    x = torch.matmul(rows, K.transpose(2, 3)) / math.sqrt(d)
    at = torch.arange(cap, device=q.device)
    see = at <= t[:, :, None]
    if s["n_win"]:
        see = see & ((at > t[:, :, None] - s["n_win"]) | (at < s["n_sink"]))
    x = x.reshape(B, n_kv, n_h // n_kv, nq, cap).masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp_(x.sub_(top))
    total = p.sum(-1, keepdim=True)
    p = p.div_(total.clamp(min=torch.finfo(torch.float32).tiny))
    o = torch.matmul(p.reshape(B, n_kv, -1, cap), V).reshape(B, n_kv, -1, nq, d)
    back = lambda y: y.permute(0, 3, 1, 2, 4).reshape(B, nq, n_h, -1)  # noqa: E731
    res = {"out": back(o).to(q.dtype), "lse": back(top + torch.log(total))[..., 0]}
    if s["op"] == "weights":
        res["acc"] = s["acc"] + p.sum((2, 3))
    return res


def _plain_evict(s):
    acc, lens, keep = s["acc"], s["lens"][:, None, None], s["keep"]
    at = torch.arange(acc.shape[2], device=acc.device)
    held = at < lens
    safe = held & ((at < s["n_sink"]) | (at >= lens - s["n_recent"]))
    key = acc.masked_fill(safe, math.inf).masked_fill(~held, -math.inf)
    by_weight = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :keep]
    n = torch.clamp(lens, max=keep)
    slot = torch.arange(by_weight.shape[2], device=acc.device)
    none = acc.shape[2]
    idx = torch.sort(by_weight.masked_fill(slot >= n, none), dim=2).values
    idx = torch.nn.functional.pad(idx, (0, keep - idx.shape[2]), value=none)
    slot = torch.arange(keep, device=acc.device)
    full = slot < n
    src = idx.clamp(max=none - 1)
    page = s["page"]
    b = torch.arange(acc.shape[0], device=acc.device)[:, None, None]
    h = torch.arange(acc.shape[1], device=acc.device)[None, :, None]
    from_page, from_row = s["table"].long()[b, src // page], src % page
    to_page, to_row = s["new_table"].long()[b, (slot // page).expand_as(src)], (slot % page).expand_as(src)
    for pool in (s["K"], s["V"]):
        pool[to_page, to_row, h] = torch.where(full[..., None], pool[from_page, from_row, h], pool[to_page, to_row, h])
    new_acc = torch.nn.functional.pad(torch.gather(acc, 2, src).masked_fill(~full, 0.0),
                                      (0, s["new_acc"].shape[2] - keep))
    return {"idx": idx.masked_fill(~full, -1).to(torch.int32), "lens": n[:, 0, 0], "acc": new_acc,
            "K": s["K"], "V": s["V"]}


# ---------------------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return {"append": _plain_append, "attn": _plain_attn, "weights": _plain_attn, "evict": _plain_evict}[s["op"]](s)
    import long_context_compressed_csa_b200 as lib
    if s["op"] == "append":
        lib.paged_append(s["k"], s["v"], s["K"], s["V"], s["table"], s["t"])
        return {"K": s["K"], "V": s["V"]}
    if s["op"] == "evict":
        lib.paged_evict(s["K"], s["V"], s["table"], s["lens"], s["acc"], s["keep"], s["new_table"], s["new_lens"],
                        s["new_acc"], s["idx"], n_sink=s["n_sink"], n_recent=s["n_recent"])
        return {"idx": s["idx"], "lens": s["new_lens"], "acc": s["new_acc"], "K": s["K"], "V": s["V"]}
    lib.paged_attn(s["q"], s["K"], s["V"], s["table"], s["t"], s["out"], s["ws"], lse=s["lse"], n_win=s["n_win"],
                   n_sink=s["n_sink"], acc=s.get("acc"), acc_out=s["acc_out"])
    res = {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "weights":
        res["acc"] = s["acc_out"]
    return res


def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    B, nq, n_h, n_kv, d, page = (case[x] for x in ("B", "nq", "n_h", "n_kv", "d", "page"))
    lens, row = _lens(case), n_kv * d * eb
    if case["op"] == "append":
        rows = sum(min(n, nq) for n in lens)
        return {"bytes": 4 * rows * row + 8 * B * nq, "flops": 0}
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        new_cap = (-(-case["keep"] // page) + 1) * page
        return {"bytes": 4 * kept * row + 4 * n_kv * (sum(lens) + B * case["keep"] + B * new_cap), "flops": 0}
    read = pairs = 0
    for n in lens:
        ts = range(max(0, n - nq), n)
        pairs += sum(_visible(case, t) for t in ts)
        # the cached rows that at least one of the queries sees
        first = max(0, ts[0] - case["n_win"] + 1) if case["n_win"] else 0
        read += n - first + min(first, case["n_sink"])
    moved = 2 * read * row + 2 * B * nq * n_h * d * eb + 4 * B * nq * n_h + 8 * B * nq + 4 * B * (-(-case["long"] // page))
    if case["op"] == "weights":
        moved += 8 * B * n_kv * (-(-case["long"] // page) + 1) * page
    return {"bytes": moved, "flops": 4 * d * n_h * pairs}


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    if case["op"] == "append":
        return None  # copies alone
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(case, s)
    B, nq, n_h, n_kv, d, page = (case[x] for x in ("B", "nq", "n_h", "n_kv", "d", "page"))
    G = n_h // n_kv
    out = torch.zeros(B, nq, n_h, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, nq, n_h), -math.inf, dtype=torch.float64, device="cuda")
    acc = s["acc"].double() if case["op"] == "weights" else None
    step = max(1, int(2.0e8 / (G * case["long"])))  # queries at a time: the logits of a block stay below 2 GB
    for b, n in enumerate(_lens(case)):
        where = torch.arange(n, device="cuda")
        page_of, row = s["table"][b].long()[where // page], where % page
        for h in range(n_kv):
            k, v = s["K"][page_of, row, h].double(), s["V"][page_of, row, h].double()
            for i in range(0, nq, step):
                t = s["t"][b, i:i + step]
                q = s["q"][b, i:i + step, h * G:(h + 1) * G].double()
                x = torch.einsum("igd,nd->ign", q, k) * d ** -0.5
                hidden = where > t[:, None]
                if case["n_win"]:
                    hidden |= (where <= t[:, None] - case["n_win"]) & (where >= case["n_sink"])
                x[hidden[:, None].expand_as(x)] = -math.inf
                some = (t >= 0)
                z = torch.logsumexp(x[some], -1)
                w = torch.exp(x[some] - z[..., None])
                lse[b, i:i + step, h * G:(h + 1) * G][some] = z
                out[b, i:i + step, h * G:(h + 1) * G][some] = torch.einsum("ign,nd->igd", w, v)
                if acc is not None:
                    acc[b, h, :n] += w.sum((0, 1))
                del x, w
    res = {"out": out, "lse": lse}
    if acc is not None:
        res["acc"] = acc
    return res


def _exact_evict(case, s):
    keep, lens = case["keep"], _lens(case)
    acc = s["acc"].double().cpu().numpy()
    idx = torch.full(s["idx"].shape, -1, dtype=torch.int32)
    new_acc = torch.zeros(s["new_acc"].shape, dtype=torch.float64)
    for b, n in enumerate(lens):
        last = min(n, case["n_recent"])
        for h in range(case["n_kv"]):
            first = range(min(case["n_sink"], n - last))
            safe = list(first) + list(range(n - last, n))
            middle = range(len(first), n - last)
            rest = sorted(middle, key=lambda j, a=acc[b, h]: (-a[j], j))[:max(0, min(n, keep) - len(safe))]
            kept = sorted(safe + rest)
            idx[b, h, :len(kept)] = torch.tensor(kept, dtype=torch.int32)
            new_acc[b, h, :len(kept)] = torch.from_numpy(acc[b, h, kept])
    return {"idx": idx.cuda(), "lens": torch.tensor([min(n, keep) for n in lens], device="cuda"), "acc": new_acc.cuda(),
            "K": None, "V": None}
