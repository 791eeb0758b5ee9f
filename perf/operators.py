"""Performance cases of the paged-cache operators: page bookkeeping and data movement
(append, free + fork, compact, copy), single-token decode attention over paged keys and
values, and decode attention for batches whose rows share a long prefix.

`run` computes a case in plain torch operations, or (with `own` set) through the
package's paged cache and decoder.  A paged cache keeps its keys and values in pools
[n_pages, Hkv, blk, d] and its bookkeeping in one int32 array:

    header[8] (header[0] = free pages), lengths[B], table[B, max_pages], ref[n_pages],
    free_list[n_pages], each section padded to a multiple of 4 words

table[b, j] is the page of block j of row b (-1: none), ref counts the rows that hold a
page, and free_list[0 .. header[0]) is a stack of free pages, the next one on top.
"""
import math
import random

import torch

own = False

DEV = "cuda"
PAGE_KINDS = ("append", "beam", "compact", "copy")


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # chunked prefill beside running decodes: some rows bring a prompt chunk of up to
        # 1024 tokens, the others their one new token
        dict(name="append chunk+decode", kind="append", B=64, Hkv=4, d=128, blk=64,
             ctx=8192, n_pages=8192, chunk=1024),
        # one beam-search or best-of-n step on a small cache: latency of the bookkeeping
        dict(name="beam small", kind="beam", B=8, Hkv=1, d=64, blk=64, ctx=4096,
             n_pages=640, fan=4),
        # sampling 7 more continuations of each of 8 long prompts (128K tokens)
        dict(name="beam long", kind="beam", B=64, Hkv=4, d=128, blk=128, ctx=131072,
             n_pages=10000, fan=8),
        # a small pool after half of its requests left
        dict(name="compact small", kind="compact", B=16, Hkv=1, d=64, blk=64, ctx=16384,
             n_pages=4096, live=0.5),
        # a large pool before its upper part is handed back: ~1.4 GB moves
        dict(name="compact large", kind="compact", B=64, Hkv=4, d=128, blk=64, ctx=32768,
             n_pages=32768, live=0.6),
        # duplicating resident prompt pages for requests that will overwrite them
        dict(name="copy pages", kind="copy", B=1, Hkv=4, d=128, blk=64, ctx=64,
             n_pages=6000, n_copy=1777),
        # the smallest decode: one row, 38% of the blocks, hard gate
        dict(name="paged tiny", kind="paged", B=1, Hq=4, Hkv=1, d=64, blk=64, ctx=4096,
             density=0.38, T=0.0, out="bf16"),
        # ragged dense decode without a gate, one KV head per query head, 128-token pages
        dict(name="paged dense ragged", kind="paged", B=13, Hq=8, Hkv=8, d=128, blk=128,
             ctx=20011, density=1.0, T=-1.0, out="f32"),
        # the block-sparse decode of long contexts: 16% of the blocks of 128K tokens
        dict(name="paged long", kind="paged", B=32, Hq=16, Hkv=4, d=128, blk=64, ctx=131072,
             density=0.16, T=0.05, out="bf16"),
        # four continuations of one short prompt: latency
        dict(name="shared small", kind="shared", B=4, Hq=16, Hkv=4, d=128, blk=64,
             groups=1, prefix=2048, suffix=64, T=0.0, out="bf16"),
        # several prompts of different lengths, each continued by a few rows; d = 64
        dict(name="shared groups", kind="shared", B=37, Hq=16, Hkv=2, d=64, blk=64,
             groups=5, prefix=16384, suffix=700, T=0.05, out="f32"),
        # 64 requests over one 128K-token document
        dict(name="shared long", kind="shared", B=64, Hq=16, Hkv=4, d=128, blk=64,
             groups=1, prefix=131072, suffix=1024, T=-1.0, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("append", "beam", "compact", "copy", "paged", "paged", "shared",
                       "shared"))
    d = rng.choice((64, 128, 128))
    blk = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4))
    if kind in PAGE_KINDS:
        c = dict(kind=kind, B=_log_int(rng, 2, 64), Hkv=Hkv, d=d, blk=blk,
                 ctx=_log_int(rng, 200, 32768), n_pages=0)
        per_row = -(-c["ctx"] // blk) + 1
        if kind == "append":
            c["chunk"] = _log_int(rng, 1, 1024)
            c["n_pages"] = c["B"] * (per_row + -(-c["chunk"] // blk) + 1) + rng.randint(0, 500)
        elif kind == "beam":
            c["fan"] = rng.randint(2, 8)
            c["n_pages"] = c["B"] * (per_row + 1) + rng.randint(0, 500)
        elif kind == "compact":
            c["live"] = round(rng.uniform(0.2, 0.9), 3)
            c["n_pages"] = _log_int(rng, 300, 16000)
        else:
            c["B"], c["ctx"] = 1, 64
            c["n_copy"] = _log_int(rng, 1, 1500)
            c["n_pages"] = 2 * c["n_copy"] + rng.randint(1, 1000)
        return c
    G = rng.choice((1, 2, 4, 8))
    T = rng.choice((-1.0, 0.0, 0.05, 0.3))
    out = rng.choice(("bf16", "f32"))
    if kind == "paged":
        return dict(kind=kind, B=_log_int(rng, 1, 48), Hq=G * Hkv, Hkv=Hkv, d=d, blk=blk,
                    ctx=_log_int(rng, 1, 65536), density=round(rng.uniform(0.1, 1.0), 3), T=T,
                    out=out)
    B = _log_int(rng, 2, 64)
    return dict(kind=kind, B=B, Hq=G * Hkv, Hkv=Hkv, d=d, blk=blk,
                groups=rng.randint(1, max(1, min(6, B // 2))),
                prefix=_log_int(rng, 64, 65536), suffix=_log_int(rng, 1, 2048), T=T, out=out)


# ------------------------------------------------------------- sizes fixed by the case
def _rng_of(case):
    return random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))


def _lengths(case):
    """Tokens of each row: ragged between half of ctx and ctx, the first row full."""
    r = _rng_of(case)
    ctx = case["ctx"]
    return [ctx if b == 0 else r.randint(max(1, ctx // 2), ctx) for b in range(case["B"])]


def _new_tokens(case):
    """Tokens each row appends: a chunk for about a quarter of the rows, one for the rest."""
    r = _rng_of(case)
    return [r.randint(1, case["chunk"]) if r.random() < 0.25 else 1 for _ in range(case["B"])]


def _blocks(n, blk):
    return -(-n // blk)


def _union_counts(case):
    return [[max(1, round(case["density"] * _blocks(n, case["blk"])))
             for _ in range(case["Hkv"])] for n in _lengths(case)]


def _groups(case):
    """Row offsets, shared whole-page prefix and row lengths of a shared-prefix batch."""
    r = _rng_of(case)
    B, n, blk = case["B"], case["groups"], case["blk"]
    cuts = sorted(r.sample(range(1, B), n - 1)) if n > 1 else []
    off = [0] + cuts + [B]
    pre = [max(1, _blocks(case["prefix"] if g == 0 else
                          r.randint(max(1, case["prefix"] // 2), case["prefix"]), blk)) * blk
           for g in range(n)]
    lens = []
    for g in range(n):
        lens += [pre[g] + r.randint(1, case["suffix"]) for _ in range(off[g], off[g + 1])]
    return off, pre, lens


# ------------------------------------------------------------------- the cache's state
def _pad4(n):
    return (n + 3) // 4 * 4


def _sections(B, max_pages, n_pages):
    at, x = {}, 0
    for name, n in (("header", 8), ("lengths", B), ("table", B * max_pages), ("ref", n_pages),
                    ("free_list", n_pages)):
        at[name] = (x, n)
        x += _pad4(n)
    return at, x


def _views(state, B, max_pages, n_pages):
    at, _ = _sections(B, max_pages, n_pages)
    v = {k: state[a:a + n] for k, (a, n) in at.items()}
    v["table"] = v["table"].view(B, max_pages)
    return v


def _pools(case, n_pages, gen, scale=1.0):
    """Key and value pools, filled in pieces (one random fp32 tensor of the whole pool
    would take twice its size)."""
    shape = (n_pages, case["Hkv"], case["blk"], case["d"])
    out = []
    for _ in range(2):
        t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        step = max(1, (1 << 28) // (shape[1] * shape[2] * shape[3]))
        for a in range(0, n_pages, step):
            t[a:a + step].normal_(0.0, scale, generator=gen)
        out.append(t)
    return out


def _fill_state(case, lens, max_pages, n_pages, perm, shared=None):
    """Rows' pages taken from `perm`, in row order; shared[b] = (row, pages) of the row
    whose first pages row b holds too.  The rest of `perm` is the free list."""
    B, blk = len(lens), case["blk"]
    _, words = _sections(B, max_pages, n_pages)
    state = torch.zeros(words, dtype=torch.int32)
    v = _views(state, B, max_pages, n_pages)
    v["table"].fill_(-1)
    k = 0
    for b, n in enumerate(lens):
        row, nsh = (shared or {}).get(b, (b, 0))
        nb = _blocks(n, blk)
        if nsh:
            v["table"][b, :nsh] = v["table"][row, :nsh]
        v["table"][b, nsh:nb] = perm[k:k + nb - nsh]
        k += nb - nsh
        v["lengths"][b] = n
    ids = v["table"][v["table"] >= 0].long()
    v["ref"].copy_(torch.bincount(ids, minlength=n_pages).int())
    n_free = n_pages - k
    v["free_list"][:n_free] = perm[k:]
    v["header"][0] = n_free
    return state.to(DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def prepare(case, seed):
    gen = _gen(seed)
    cpu = torch.Generator().manual_seed(int(seed))
    kind, blk = case["kind"], case["blk"]
    s = {"case": case}
    if kind in ("paged", "shared"):
        B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
        shared = None
        if kind == "paged":
            lens = _lengths(case)
        else:
            off, pre, lens = _groups(case)
            shared = {b: (off[g], pre[g] // blk) for g in range(case["groups"])
                      for b in range(off[g] + 1, off[g + 1])}
        max_pages = max(_blocks(n, blk) for n in lens)
        used = sum(_blocks(n, blk) - (shared or {}).get(b, (b, 0))[1]
                   for b, n in enumerate(lens))
        n_pages = used + 7
        perm = torch.randperm(n_pages, generator=cpu).int()
        s["K"], s["V"] = _pools(case, n_pages, gen)
        s["state"] = _fill_state(case, lens, max_pages, n_pages, perm, shared)
        s["q"] = torch.randn(B, Hq, d, generator=gen, device=DEV).to(torch.bfloat16)
        # thresholds inside the range of the scores, which are close to N(0, 1)
        s["tau"] = 0.3 + 0.5 * torch.randn(B, Hq, generator=gen, device=DEV)
        if kind == "paged":
            cnt = torch.tensor(_union_counts(case), dtype=torch.int32, device=DEV)
            nb = torch.tensor([_blocks(n, blk) for n in lens], device=DEV)
            # a random subset of every row's blocks that holds the newest one, ascending
            key = torch.rand(B, Hkv, max_pages, generator=gen, device=DEV)
            j = torch.arange(max_pages, device=DEV)
            key = torch.where(j == nb[:, None, None] - 1, -1.0, key)
            key = torch.where(j >= nb[:, None, None], 2.0, key)
            order = key.argsort(dim=-1)
            order = torch.where(j < cnt[..., None], order, max_pages).sort(dim=-1).values
            s["union_idx"] = torch.where(j < cnt[..., None], order, 0).int().contiguous()
            s["union_cnt"] = cnt.contiguous()
            s["U"] = int(cnt.max())
        else:
            s["off"] = torch.tensor(off, dtype=torch.int32, device=DEV)
            s["pre"] = torch.tensor(pre, dtype=torch.int32, device=DEV)
            s["lens"], s["off_h"], s["pre_h"] = lens, off, pre
        s["dims"] = (B, max_pages, n_pages)
        if own:
            from long_context_decoding_eta_b200.paged import PagedEtaDecoder, PagedKVCache
            cache = PagedKVCache(B, Hkv, d, blk, max_pages, n_pages, K=s["K"], V=s["V"])
            cache.state.copy_(s["state"])
            dec = PagedEtaDecoder(cache, Hq, T=None if case["T"] < 0 else case["T"],
                                  out_dtype=_OUT[case["out"]])
            if kind == "paged":
                dec.union_idx.copy_(s["union_idx"])
                dec.union_cnt.copy_(s["union_cnt"])
            s["dec"] = dec
        return s
    # page operations
    B, Hkv, d, n_pages = case["B"], case["Hkv"], case["d"], case["n_pages"]
    perm = torch.randperm(n_pages, generator=cpu).int()
    if kind == "append":
        new = _new_tokens(case)
        lens = _lengths(case)
        max_pages = max(_blocks(a + n, blk) for a, n in zip(lens, new))
        lens[1:2] = [0]                       # a request that has just arrived
        total = sum(new)
        s["k_new"] = torch.randn(total, Hkv, d, generator=gen, device=DEV).to(torch.bfloat16)
        s["v_new"] = torch.randn(total, Hkv, d, generator=gen, device=DEV).to(torch.bfloat16)
        s["cu"] = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).int().to(DEV)
        s["state"] = _fill_state(case, lens, max_pages, n_pages, perm)
    elif kind == "beam":
        # every fan-th row survives; the rows after it held another beam's pages
        lens = _lengths(case)
        max_pages = max(_blocks(n, blk) for n in lens)
        fan = case["fan"]
        keep = [b for b in range(B) if b % fan == 0]
        lose = [b for b in range(B) if b % fan]
        # every losing row shares its survivor's first half, as after an earlier fork
        shared = {b: (b - b % fan, min(lens[b - b % fan], lens[b]) // blk // 2) for b in lose}
        s["rows"] = torch.tensor(lose, dtype=torch.int32, device=DEV)
        s["src"] = torch.tensor([b - b % fan for b in lose], dtype=torch.int32, device=DEV)
        s["dst"] = s["rows"]
        while sum(_blocks(n, blk) - shared.get(b, (b, 0))[1]
                  for b, n in enumerate(lens)) > n_pages:
            lens = [max(1, n * 3 // 4) for n in lens]
            shared = {b: (b - b % fan, min(lens[b - b % fan], lens[b]) // blk // 2)
                      for b in lose}
        assert len(keep) + len(lose) == B
        s["state"] = _fill_state(case, lens, max_pages, n_pages, perm, shared)
    elif kind == "compact":
        live = int(case["live"] * n_pages)
        per = max(1, live // B)
        lens = [min(per, _blocks(case["ctx"], blk)) * blk - (b % blk) for b in range(B)]
        max_pages = max(_blocks(n, blk) for n in lens)
        s["state"] = _fill_state(case, lens, max_pages, n_pages, perm)
    else:
        lens, max_pages = [case["ctx"]], 1
        s["src"] = perm[:case["n_copy"]].to(DEV)
        s["dst"] = perm[case["n_copy"]:2 * case["n_copy"]].to(DEV)
        s["state"] = _fill_state(case, lens, max_pages, n_pages, perm[-n_pages:])
    s["K"], s["V"] = _pools(case, n_pages, gen)
    s["dims"] = (B, max_pages, n_pages)
    if own:
        from long_context_decoding_eta_b200.paged import PagedKVCache
        s["cache"] = PagedKVCache(B, Hkv, d, blk, max_pages, n_pages, K=s["K"], V=s["V"])
    else:
        s["work"] = torch.empty_like(s["state"])
    return s


_OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------- run
def run(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "paged":
        if own:
            return s["dec"].decode(s["q"], tau=s["tau"], all_blocks=case["density"] >= 1.0)
        return _plain_paged(s)
    if kind == "shared":
        if own:
            return s["dec"].shared_decode(s["q"], s["off"], s["pre"], tau=s["tau"])
        return _plain_shared(s)
    # every pass starts from the same bookkeeping
    if own:
        c = s["cache"]
        if kind == "copy":
            c.copy_pages(s["src"], s["dst"])
            return c.K, c.V
        c.state.copy_(s["state"])
        if kind == "append":
            c.append(s["k_new"], s["v_new"], s["cu"])
        elif kind == "beam":
            c.free(s["rows"])
            c.fork(s["src"], s["dst"])
        else:
            c.compact()
        return c.state, c.K, c.V
    if kind == "copy":
        s["K"][s["dst"].long()] = s["K"][s["src"].long()]
        s["V"][s["dst"].long()] = s["V"][s["src"].long()]
        return s["K"], s["V"]
    s["work"].copy_(s["state"])
    v = _views(s["work"], *s["dims"])
    if kind == "append":
        _plain_append(s, v)
    elif kind == "beam":
        _plain_free(s, v)
        _plain_fork(s, v)
    else:
        _plain_compact(s, v)
    return s["work"], s["K"], s["V"]


# ------------------------------------------------------------------ plain page operations
def _plain_append(s, v):
    blk = s["case"]["blk"]
    len0 = v["lengths"].clone()
    cu = s["cu"]
    len1 = len0 + (cu[1:] - cu[:-1])
    col = torch.arange(v["table"].shape[1], device=DEV)
    fresh = (col >= ((len0 + blk - 1) // blk)[:, None]) & (col < ((len1 + blk - 1) // blk)[:, None])
    rank = fresh.view(-1).cumsum(0).view(fresh.shape) - 1
    n_free = v["header"][0].long()
    page = v["free_list"][(n_free - 1 - rank).clamp(min=0)]
    v["table"].copy_(torch.where(fresh, page, v["table"]))
    v["ref"][page[fresh].long()] = 1
    v["header"][0] -= fresh.sum().int()
    v["lengths"].copy_(len1)
    t = torch.arange(s["k_new"].shape[0], device=DEV)
    row = torch.searchsorted(cu, t.int(), right=True) - 1
    pos = len0[row] + t - cu[row]
    at = v["table"][row, pos // blk].long()
    s["K"][at, :, pos % blk] = s["k_new"]
    s["V"][at, :, pos % blk] = s["v_new"]


def _plain_free(s, v):
    rows = s["rows"].long()
    ids = v["table"][rows]
    held = torch.bincount(ids[ids >= 0].long(), minlength=s["dims"][2])
    v["ref"].sub_(held.int())
    gone = ((held > 0) & (v["ref"] == 0)).nonzero().view(-1).flip(0)
    n_free = v["header"][0].long()
    v["free_list"][n_free + torch.arange(gone.numel(), device=DEV)] = gone.int()
    v["header"][0] += gone.numel()
    v["table"][rows] = -1
    v["lengths"][rows] = 0


def _plain_fork(s, v):
    blk = s["case"]["blk"]
    src, dst = s["src"].long(), s["dst"].long()
    n = v["lengths"][src]
    full, part = n // blk, n % blk
    col = torch.arange(v["table"].shape[1], device=DEV)
    t = torch.where(col < full[:, None], v["table"][src], -1)
    ids = t[t >= 0].long()
    v["ref"].add_(torch.bincount(ids, minlength=s["dims"][2]).int())
    last = part > 0
    rank = last.cumsum(0) - 1
    n_free = v["header"][0].long()
    page = v["free_list"][(n_free - 1 - rank).clamp(min=0)]
    t = torch.where((col == full[:, None]) & last[:, None], page[:, None], t)
    v["ref"][page[last].long()] = 1
    v["header"][0] -= last.sum().int()
    old = v["table"][src, full.clamp(max=t.shape[1] - 1).long()][last].long()
    new = page[last].long()
    tok = (torch.arange(blk, device=DEV) < part[last][:, None])[:, None, :, None]
    s["K"][new] = torch.where(tok, s["K"][old], s["K"][new])
    s["V"][new] = torch.where(tok, s["V"][old], s["V"][new])
    v["table"][dst] = t
    v["lengths"][dst] = n


def _plain_compact(s, v):
    n_pages = s["dims"][2]
    live = v["ref"] > 0
    n_live = live.sum()
    ids = torch.arange(n_pages, device=DEV)
    holes = (~live & (ids < n_live)).nonzero().view(-1)
    moved = (live & (ids >= n_live)).nonzero().view(-1)
    to = ids.clone()
    to[moved] = holes
    s["K"][holes] = s["K"][moved]
    s["V"][holes] = s["V"][moved]
    v["ref"][holes] = v["ref"][moved]
    v["ref"][moved] = 0
    t = v["table"]
    t.copy_(torch.where(t >= 0, to[t.clamp(min=0).long()].int(), t))
    k = torch.arange(n_pages, device=DEV)
    v["free_list"].copy_(torch.where(k < n_pages - n_live, n_pages - 1 - k,
                                     v["free_list"]).int())


# ------------------------------------------------------------------- plain attention
def _gate(x, tau, T):
    if T < 0:
        return x
    if T == 0:
        return torch.where(x >= tau, x, torch.zeros_like(x))
    return x * torch.sigmoid((x - tau) / T)


def _softmax_parts(x, valid, V):
    """Running statistics of softmax(x) V over the last axis of x: max, sum, weighted sum."""
    x = torch.where(valid, x, -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    return m, p.sum(-1, keepdim=True), p @ V


def _finish(m, l, acc, out):
    empty = l == 0
    o = torch.where(empty, 0.0, acc / torch.where(empty, 1.0, l))
    lse = torch.where(empty, -math.inf, m + torch.log(torch.where(empty, 1.0, l)))
    return o.to(_OUT[out]), lse.squeeze(-1)


def _plain_paged(s):
    c = s["case"]
    B, Hq, Hkv, d, blk = c["B"], c["Hq"], c["Hkv"], c["d"], c["blk"]
    G, U = Hq // Hkv, s["U"]
    v = _views(s["state"], *s["dims"])
    idx = s["union_idx"][..., :U].long()
    row = torch.arange(B, device=DEV)[:, None, None]
    page = v["table"][row, idx].clamp(min=0).long()
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    K = s["K"][page, head].view(B, Hkv, U * blk, d).float()
    pos = idx[..., None] * blk + torch.arange(blk, device=DEV)
    ok = (pos < v["lengths"][:, None, None, None]) & \
        (torch.arange(U, device=DEV)[:, None] < s["union_cnt"][..., None, None])
    ok = ok.view(B, Hkv, 1, U * blk)
    q = s["q"].view(B, Hkv, G, d).float()
    x = (q @ K.transpose(-1, -2)) / math.sqrt(d)
    del K
    x = _gate(x, s["tau"].view(B, Hkv, G, 1), c["T"])
    V = s["V"][page, head].view(B, Hkv, U * blk, d).float()
    V = torch.where(ok.view(B, Hkv, U * blk, 1), V, 0.0)
    m, l, acc = _softmax_parts(x, ok, V)
    o, lse = _finish(m, l, acc, c["out"])
    return o.view(B, Hq, d), lse.view(B, Hq)


def _plain_shared(s):
    """The prefixes once per group, the suffixes per row, joined by their maxima and sums."""
    c = s["case"]
    B, Hq, Hkv, d, blk = c["B"], c["Hq"], c["Hkv"], c["d"], c["blk"]
    G, n = Hq // Hkv, c["groups"]
    v = _views(s["state"], *s["dims"])
    off, pre = s["off"].long(), s["pre"].long()
    rows_most = max(b - a for a, b in zip(s["off_h"], s["off_h"][1:]))
    P = max(s["pre_h"])
    q = s["q"].view(B, Hkv, G, d).float()
    tau = s["tau"].view(B, Hkv, G, 1)
    # prefixes: [group, KV head, rows * G, tokens]
    member = off[:-1, None] + torch.arange(rows_most, device=DEV)
    real = member < off[1:, None]
    member = member.clamp(max=B - 1)
    qg = q[member].permute(0, 2, 1, 3, 4).reshape(n, Hkv, rows_most * G, d)
    tg = tau[member].permute(0, 2, 1, 3, 4).reshape(n, Hkv, rows_most * G, 1)
    page = v["table"][off[:-1], :P // blk].clamp(min=0).long()
    K = s["K"][page].permute(0, 2, 1, 3, 4).reshape(n, Hkv, P, d).float()
    x = _gate((qg @ K.transpose(-1, -2)) / math.sqrt(d), tg, c["T"])
    del K
    ok = (torch.arange(P, device=DEV) < pre[:, None])[:, None, None]
    V = s["V"][page].permute(0, 2, 1, 3, 4).reshape(n, Hkv, P, d).float()
    parts = [t.view(n, Hkv, rows_most, G, -1).permute(0, 2, 1, 3, 4)[real]
             for t in _softmax_parts(x, ok, V)]
    del x, V
    # suffixes: [row, KV head, G, tokens]
    group = torch.searchsorted(off, torch.arange(B, device=DEV), right=True) - 1
    start = pre[group]
    most = max(b - s["pre_h"][g] for g in range(n)
               for b in s["lens"][s["off_h"][g]:s["off_h"][g + 1]])
    nb = _blocks(most, blk)
    col = start[:, None] // blk + torch.arange(nb, device=DEV)
    page = v["table"].gather(1, col.clamp(max=s["dims"][1] - 1)).clamp(min=0).long()
    K = s["K"][page].permute(0, 2, 1, 3, 4).reshape(B, Hkv, nb * blk, d).float()
    V = s["V"][page].permute(0, 2, 1, 3, 4).reshape(B, Hkv, nb * blk, d).float()
    ok = (start[:, None] + torch.arange(nb * blk, device=DEV) < v["lengths"][:, None])
    x = _gate((q @ K.transpose(-1, -2)) / math.sqrt(d), tau, c["T"])
    m2, l2, a2 = _softmax_parts(x, ok[:, None, None], V)
    m1, l1, a1 = parts
    m = torch.maximum(m1, m2)
    w1, w2 = torch.exp(m1 - m), torch.exp(m2 - m)
    o, lse = _finish(m, l1 * w1 + l2 * w2, a1 * w1 + a2 * w2, c["out"])
    return o.view(B, Hq, d), lse.view(B, Hq)


# -------------------------------------------------------------------------------- work
def work(case):
    kind, blk = case["kind"], case["blk"]
    Hkv, d = case["Hkv"], case["d"]
    tok = Hkv * d * 2 * 2                       # K and V of one token
    if kind == "paged":
        keys = 0
        for n, cnt in zip(_lengths(case), _union_counts(case)):
            tail = n - (_blocks(n, blk) - 1) * blk
            keys += sum((c - 1) * blk + tail for c in cnt)      # of one KV head each
        rows, G = case["B"] * case["Hq"], case["Hq"] // Hkv
        ob = 2 if case["out"] == "bf16" else 4
        lists = 4 * sum(map(sum, _union_counts(case)))
        return {"bytes": keys * d * 4 + rows * (d * (2 + ob) + 8) + lists,
                "flops": 4.0 * d * G * keys}
    if kind == "shared":
        off, pre, lens = _groups(case)
        keys = sum(pre)
        pairs = 0
        for g in range(case["groups"]):
            for n in lens[off[g]:off[g + 1]]:
                keys += n - pre[g]
                pairs += n
        rows = case["B"] * case["Hq"]
        ob = 2 if case["out"] == "bf16" else 4
        return {"bytes": keys * tok + rows * (d * (2 + ob) + 8) + keys // blk * 4,
                "flops": 4.0 * d * case["Hq"] * pairs}
    if kind == "append":
        n = sum(_new_tokens(case))
        return {"bytes": 2 * n * tok + 8 * case["B"], "flops": 0}
    if kind == "copy":
        return {"bytes": 2 * case["n_copy"] * blk * tok + 8 * case["n_copy"], "flops": 0}
    if kind == "beam":
        # what the fork copies of each partly filled page, and the table rows: read and
        # rewritten for the rows freed, read and written again for the rows forked
        lens = _lengths(case)
        fan = case["fan"]
        lose = [b for b in range(case["B"]) if b % fan]
        part = sum(lens[b - b % fan] % blk for b in lose)
        words = sum(2 * _blocks(lens[b], blk) + 4 * _blocks(lens[b - b % fan], blk) for b in lose)
        return {"bytes": 2 * part * tok + 4 * words, "flops": 0}
    live = int(case["live"] * case["n_pages"])
    used = min(max(1, live // case["B"]), _blocks(case["ctx"], blk)) * case["B"]
    moved = used * (1 - used / case["n_pages"])          # expected, of a random placement
    return {"bytes": 2 * moved * blk * tok + 8.0 * case["n_pages"], "flops": 0}


# ------------------------------------------------------------------------------- exact
def exact(case, seed):
    """Attention outputs from the definition in 64 bits, one row at a time over the row's
    own tokens; the page operations only move data and have no such value."""
    if case["kind"] in PAGE_KINDS:
        return None
    s = prepare(case, seed)
    B, Hq, Hkv, d, blk = (case[k] for k in ("B", "Hq", "Hkv", "d", "blk"))
    _, max_pages, n_pages = s["dims"]
    at, _ = _sections(B, max_pages, n_pages)
    host = s["state"].cpu()
    table = host[at["table"][0]:][:B * max_pages].view(B, max_pages)
    lens = host[at["lengths"][0]:][:B].tolist()
    o = torch.zeros(B, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
    G = Hq // Hkv
    for b in range(B):
        if case["kind"] == "paged":
            picks = [s["union_idx"][b, g, :int(s["union_cnt"][b, g])].cpu() for g in range(Hkv)]
        else:
            picks = [torch.arange(_blocks(lens[b], blk))] * Hkv
        for g in range(Hkv):
            j = picks[g].long()
            pages = table[b, j].long().to(DEV)
            pos = (j[:, None] * blk + torch.arange(blk)).view(-1).to(DEV)
            inside = pos < lens[b]
            k = s["K"][pages, g].reshape(-1, d)[inside].double()
            w = s["V"][pages, g].reshape(-1, d)[inside].double()
            for h in range(g * G, (g + 1) * G):
                x = (k @ s["q"][b, h].double()) * (1.0 / math.sqrt(d))
                t = s["tau"][b, h].double()
                if case["T"] == 0:
                    x = x * (x >= t)
                elif case["T"] > 0:
                    x = x / (1.0 + torch.exp((t - x) / case["T"]))
                z = torch.logsumexp(x, 0)
                lse[b, h] = z
                o[b, h] = torch.exp(x - z) @ w
    return o, lse
