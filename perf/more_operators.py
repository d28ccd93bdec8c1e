"""The pages of the paged 8-bit cache (free, reserve, fork, compact, copy) and attention over packed documents: cases,
inputs and plain forms.

Pages: a pool has a table [rows, max_pages] with the pages of each sequence in order (-1: none) and refs [n_pages], how
many table entries hold each page (0: free).  New pages are the lowest-numbered free ones, in the order of the call's
list and of the positions.  A page holds `page` tokens: E4M3 codes [heads, page, 128] of keys and values, one scale per
head, the rotary key in bf16 [page, 64].

Documents: the rows of q are the new tokens of several documents one after the other, the rows of the dense caches
[64, rows, 192] and [64, rows, 128] their keys and values.  Query t of a document with n queries and L keys sits at
position i = L - n + t and sees key j < L iff j < prefix, or j <= i and (window = 0 or i - j < window or j < sinks).
"""
import math
import random

import numpy as np
import torch

own = False

NOPE, ROPE, V = 128, 64, 128
QK = NOPE + ROPE
DENSE_HEADS = 64          # the dense caches' head count
SCALE = 1.0 / math.sqrt(QK)
TENSORS = ["k_codes", "v_codes", "k_pe", "k_scales", "v_scales"]


# ---- the cases ----------------------------------------------------------------------------------------------
def listed():
    return [
        # four answers are drawn from one conversation: the last ones are dropped, its pages shared anew
        {"name": "fork 1 into 4", "op": "fork", "n": 4, "parents": 1, "lo": 1000, "hi": 1000, "page": 64, "heads": 64},
        # a beam step of a whole batch on small pages
        {"name": "fork 64 beams", "op": "fork", "n": 64, "parents": 64, "lo": 1, "hi": 2047, "page": 16, "heads": 64},
        # a decode batch: rejected drafts are given back, room for the next four tokens is taken
        {"name": "regrow 64x4", "op": "regrow", "n": 64, "T": 4, "lo": 1, "hi": 2000, "page": 16},
        # whole prompts come in where others have ended
        {"name": "regrow 600x2048", "op": "regrow", "n": 600, "T": 2048, "lo": 0, "hi": 777, "page": 16},
        # a small pool after a few conversations have ended
        {"name": "compact 333", "op": "compact", "n_pages": 333, "rows": 16, "live": 0.5, "page": 32, "heads": 16},
        # a pool of 2 GB, half of it in use
        {"name": "compact 8192", "op": "compact", "n_pages": 8192, "rows": 64, "live": 0.5, "page": 16, "heads": 64},
        # one short conversation goes to another pool
        {"name": "copy 3", "op": "copy", "n": 3, "page": 64, "heads": 64},
        # a prefill pool hands a batch of prompts to a decode pool
        {"name": "copy 1531", "op": "copy", "n": 1531, "page": 32, "heads": 64},
        # single new tokens of a few conversations, each behind its cached ones
        {"name": "documents 4x1", "op": "documents", "n": 4, "lo": 1, "hi": 1, "past": 500, "prefix": 0, "window": 0,
         "sinks": 0},
        # a step of ragged prompts
        {"name": "documents 16x1531", "op": "documents", "n": 16, "lo": 17, "hi": 1531, "past": 0, "prefix": 0,
         "window": 0, "sinks": 0},
        # pieces of prompts behind cached tokens, each with a prefix that is seen from both sides
        {"name": "documents 8x777 prefix", "op": "documents", "n": 8, "lo": 50, "hi": 777, "past": 2048, "prefix": 300,
         "window": 0, "sinks": 0},
        # long documents packed for one pass
        {"name": "documents 5x4096", "op": "documents", "n": 5, "lo": 2000, "hi": 4096, "past": 0, "prefix": 0,
         "window": 0, "sinks": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fork", "regrow", "compact", "copy", "documents", "documents"])
    page, heads = rng.choice([16, 32, 64, 128]), rng.choice([4, 8, 12, 16, 32, 64])
    if op == "fork":
        n = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 2047)
        return {"op": op, "n": n, "parents": rng.randint(1, n), "lo": rng.randint(0, hi), "hi": hi, "page": page,
                "heads": heads}
    if op == "regrow":
        hi = _log_int(rng, 1, 2000)
        return {"op": op, "n": _log_int(rng, 1, 600), "T": _log_int(rng, 1, 2048), "lo": rng.randint(0, hi), "hi": hi,
                "page": page}
    if op == "compact":
        n_pages = _log_int(rng, 2, 8192 * 1024 // (page * heads))
        return {"op": op, "n_pages": n_pages, "rows": _log_int(rng, 1, 64), "live": rng.choice([0.0, 0.1, 0.5, 0.9, 1.0]),
                "page": page, "heads": heads}
    if op == "copy":
        return {"op": op, "n": _log_int(rng, 1, 1531 * 2048 // (page * heads)), "page": page, "heads": heads}
    n, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 2048)
    hi = min(hi, 16384 // n)
    past = rng.choice([0, _log_int(rng, 1, 2048)])
    past = min(past, 16384 // n)
    window = rng.choice([0, 0, _log_int(rng, 1, 1024)])
    return {"op": op, "n": n, "lo": rng.randint(0, hi), "hi": hi, "past": past,
            "prefix": rng.choice([0, rng.randint(1, 300)]), "window": window,
            "sinks": rng.randint(0, 130) if window else 0}


def _numbers(case, n, lo, hi, salt):
    """n whole numbers in [lo, hi], the ends among them, the same for every seed."""
    rng = random.Random("%s %s %s %s %s" % (case["op"], n, lo, hi, salt))
    x = [hi] + [lo] * (n > 1) + [rng.randint(lo, hi) for _ in range(n - 2)]
    rng.shuffle(x)
    return x


def _pages(positions, page):
    return -(-positions // page)


def _page_bytes(case):
    return case["page"] * (case["heads"] * 256 + 128) + case["heads"] * 8


def _forks(case):
    """Positions of each parent, and for each fork its parent, child and the positions it takes."""
    n, parents = case["n"], case["parents"]
    lengths = _numbers(case, parents, case["lo"], case["hi"], "lengths")
    parent = [i % parents for i in range(n)]
    rng = random.Random("%s %s %s" % (n, parents, case["hi"]))
    # most forks take all of the parent, some go back a little
    at = [lengths[p] - (rng.randint(0, min(lengths[p], 40)) if rng.random() < 0.25 else 0) for p in parent]
    return lengths, parent, [parents + i for i in range(n)], at


def _compaction(case):
    """Pages of each row; a tenth of the rows share their first half with the row before."""
    live = max(1, int(case["n_pages"] * case["live"])) if case["live"] else 0
    rows = case["rows"]
    rng = random.Random("%s %s %s" % (case["n_pages"], rows, live))
    cuts = sorted(rng.randint(0, live) for _ in range(rows - 1))
    own_pages = [b - a for a, b in zip([0] + cuts, cuts + [live])]
    shared = [own_pages[i - 1] // 2 if i and rng.random() < 0.1 else 0 for i in range(rows)]
    return own_pages, shared


def _documents(case):
    """New tokens, keys and prefix of each document."""
    n = case["n"]
    new = _numbers(case, n, case["lo"], case["hi"], "new")
    past = _numbers(case, n, 0, case["past"], "past") if case["past"] else [0] * n
    keys = [a + b for a, b in zip(new, past)]
    prefix = [min(p, k) for p, k in zip(_numbers(case, n, 0, case["prefix"], "prefix"), keys)] if case["prefix"] else \
        [0] * n
    return new, keys, prefix


def _seen(new, keys, prefix, window, sinks):
    """Keys that one of a document's queries sees, and (query, key) pairs."""
    i = np.arange(keys - new, keys, dtype=np.int64)
    first = np.maximum(i - window + 1, 0) if window else np.zeros_like(i)   # the window's first key
    ahead = max(prefix, sinks if window else 0)                             # keys before it that are seen
    pairs = i + 1 - first + np.minimum(first, ahead) + np.maximum(prefix - (i + 1), 0)
    start = max(0, keys - new - window + 1) if window else 0
    return (keys - start + min(start, ahead) if new else 0), int(pairs.sum())


def work(case):
    op = case["op"]
    if op == "fork":
        lengths, parent, child, at = _forks(case)
        shared = sum(p // case["page"] for p in at)
        tails = sum((p % case["page"]) * (case["heads"] * 256 + 128) + case["heads"] * 8 for p in at if p % case["page"])
        # entries dropped and shared (table and refs both ways), the copied tails
        return {"bytes": shared * 4 * 7 + 2 * tails, "flops": 0}
    if op == "regrow":
        P = _numbers(case, case["n"], case["lo"], case["hi"], "P")
        new = sum(_pages(p + case["T"], case["page"]) - _pages(p, case["page"]) for p in P)
        return {"bytes": new * 4 * 7 + case["n"] * 12, "flops": 0}
    if op == "compact":
        own_pages, shared = _compaction(case)
        live = sum(own_pages)
        moves = live * (case["n_pages"] - live) // case["n_pages"]  # expected, of a random layout
        return {"bytes": moves * 2 * _page_bytes(case) + 12 * case["n_pages"] + 8 * (live + sum(shared)), "flops": 0}
    if op == "copy":
        return {"bytes": case["n"] * (2 * _page_bytes(case) + 8), "flops": 0}
    new, keys, prefix = _documents(case)
    seen = [_seen(*d, case["window"], case["sinks"]) for d in zip(new, keys, prefix)]
    return {"bytes": DENSE_HEADS * (QK + V) * 2 * (sum(k for k, _ in seen) + sum(new)),
            "flops": DENSE_HEADS * 2 * (QK + V) * sum(p for _, p in seen)}


# ---- the inputs ---------------------------------------------------------------------------------------------
def _cache(g, n_pages, page, heads):
    """Pages of random codes, scales and rotary keys."""
    def codes():
        x = torch.empty((n_pages, heads, page, 128), dtype=torch.bfloat16, device="cuda").normal_(0, 100, generator=g)
        return x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def scales():
        return torch.exp2(torch.randint(-12, -5, (n_pages, heads), generator=g, device="cuda").float())

    pe = torch.empty((n_pages, page, ROPE), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    return {"k_codes": codes(), "v_codes": codes(), "k_pe": pe, "k_scales": scales(), "v_scales": scales()}


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _book(rows, max_pages, lists, n_pages, order, width=0):
    """Table and refs, in one buffer, of rows that hold lists of indexes into `order`."""
    book = np.zeros(rows * max_pages + n_pages, dtype=np.int32)
    table, refs = book[:rows * max_pages].reshape(rows, max_pages), book[rows * max_pages:]
    table[:] = -1
    for r, pages in enumerate(lists):
        table[r, :len(pages)] = order[pages]
        np.add.at(refs, order[pages], 1)
    book = torch.from_numpy(book).cuda()
    return book, book[:rows * max_pages].view(rows, max_pages), book[rows * max_pages:]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = dict(case)
    op = case["op"]

    if op == "documents":
        def normal(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)

        new, keys, prefix = _documents(case)
        s["new"], s["keys"], s["first"] = new, keys, prefix
        N, L = sum(new), sum(keys)
        s["q"] = normal(max(N, 1), DENSE_HEADS * QK)
        s["k"], s["v"] = normal(DENSE_HEADS, max(L, 1), QK), normal(DENSE_HEADS, max(L, 1), V)
        s["cu_q"], s["cu_k"] = _ints([0] + list(np.cumsum(new))), _ints([0] + list(np.cumsum(keys)))
        s["prefix"] = _ints(prefix) if case["prefix"] else None
        s["out"] = torch.zeros((max(N, 1), DENSE_HEADS * V), dtype=torch.bfloat16, device="cuda")
        if own:
            import mla_gb300 as m
            s["workspace"] = m.alloc_workspace(m.MODE_DOCUMENTS, case["n"], max(N, 1))
        return s

    page = case["page"]
    if op == "copy":
        s["from"], s["to"] = (_cache(g, case["n"] + extra, page, case["heads"]) for extra in (7, 3))
        src = torch.randperm(case["n"] + 7, generator=g, device="cuda")[:case["n"]]
        dst = torch.randperm(case["n"] + 3, generator=g, device="cuda")[:case["n"]]
        s["src"], s["dst"] = src.to(torch.int32), dst.to(torch.int32)
        if own:
            import mla_gb300 as m
            for name in ("from", "to"):
                s[name]["table"] = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
                s[name + "_handle"] = m.make_paged_cache(s[name])
            s["workspace"] = m.alloc_workspace(m.MODE_PAGES, case["n"], case["n"] + 3)
        return s

    if op == "fork":
        lengths, parent, child, at = _forks(case)
        parents, n = case["parents"], case["n"]
        counts = [_pages(p, page) for p in lengths]
        total = sum(counts)
        n_pages, wide, rows = total + n + total // 3 + 1, max(counts) + 1, parents + n
        order = rng.permutation(n_pages).astype(np.int32)
        starts = np.cumsum([0] + counts)
        lists = [np.arange(a, b) for a, b in zip(starts[:-1], starts[1:])]
        # the children hold what the last pass gave them: all shared pages
        lists += [lists[p][:a // page] for p, a in zip(parent, at)]
        s["parent"], s["child"], s["at"] = _ints(parent), _ints(child), _ints(at)
        s["zero"] = _ints([0] * n)
        tails = [i for i in range(n) if at[i] % page]
        s["tails"] = torch.tensor(tails, dtype=torch.int64, device="cuda")
    elif op == "regrow":
        P = _numbers(case, case["n"], case["lo"], case["hi"], "P")
        rows, counts = case["n"] + 1, [_pages(p + case["T"], page) for p in P]
        total = sum(counts)
        n_pages, wide = total + total // 3 + 5, max(counts)
        order = rng.permutation(n_pages).astype(np.int32)
        starts = np.cumsum([0] + counts)
        # the last pass's pages are held; one more row is not part of the call
        lists = [np.arange(a, b) for a, b in zip(starts[:-1], starts[1:])] + [np.arange(total, total + min(3, wide))]
        s["rows_of"] = _ints(rng.permutation(case["n"]))
        kept = np.asarray(P, dtype=np.int32)[s["rows_of"].cpu().numpy()]
        s["keep"], s["grow"] = _ints(kept.tolist()), _ints((kept + case["T"]).tolist())
    else:
        own_pages, shared = _compaction(case)
        n_pages, rows = case["n_pages"], case["rows"]
        order = rng.permutation(n_pages).astype(np.int32)
        lists, at = [], 0
        for r in range(rows):
            mine = np.arange(at, at + own_pages[r])
            at += own_pages[r]
            lists.append(np.concatenate([lists[r - 1][:shared[r]], mine]) if shared[r] else mine)
        wide = max(1, max(len(x) for x in lists))
        live = np.zeros(n_pages, dtype=bool)
        live[order[:at]] = True
        s["moves"] = int(live[at:].sum())
        s["moved"] = torch.empty(n_pages, dtype=torch.int32, device="cuda")
        s["n_live"] = torch.empty(1, dtype=torch.int32, device="cuda")
    s["book"], s["table"], s["refs"] = _book(rows, wide, lists, n_pages, order)
    if op == "compact":
        s["scattered"] = s["book"].clone()   # what the pool looks like before each pass
    if op != "regrow":
        s["cache"] = _cache(g, n_pages, page, case["heads"])
    if own:
        import mla_gb300 as m
        s["pool"] = m.make_page_pool(s["table"], s["refs"], page)
        if op != "regrow":
            s["handle"] = m.make_paged_cache(dict(s["cache"], table=s["table"]))
        s["workspace"] = m.alloc_workspace(m.MODE_PAGES, case.get("n", 1), n_pages, cap=rows)
    return s


# ---- one pass -----------------------------------------------------------------------------------------------
def _values(cache):
    """A cache's tensors, the codes as the numbers they stand for."""
    return {n: cache[n].view(torch.float8_e4m3fn) if n.endswith("codes") else cache[n] for n in TENSORS}


def run(s):
    if own:
        import mla_gb300 as m
    op = s["op"]
    if op == "documents":
        if own:
            m.mla_document_attention(s["q"], s["cu_q"], s["k"], s["v"], s["out"], s["workspace"], cu_k=s["cu_k"],
                                     prefix=s["prefix"], window=s["window"], sinks=s["sinks"])
        else:
            _plain_documents(s)
        return s["out"]
    if op == "copy":
        if own:
            m.mla_pages_copy(s["from_handle"], s["to_handle"], s["src"], s["dst"], s["workspace"])
        else:
            _plain_copy(s)
        return _values(s["to"])
    if op == "regrow":
        if own:
            m.mla_pages_free(s["pool"], s["rows_of"], s["keep"], s["workspace"])
            m.mla_pages_reserve(s["pool"], s["rows_of"], s["grow"], s["workspace"])
        else:
            _plain_free(s, s["rows_of"], s["keep"])
            _plain_reserve(s)
        return {"table": s["table"], "refs": s["refs"]}
    if op == "fork":
        if own:
            m.mla_pages_free(s["pool"], s["child"], s["zero"], s["workspace"])
            m.mla_pages_fork(s["handle"], s["pool"], s["parent"], s["child"], s["at"], s["workspace"])
        else:
            _plain_free(s, s["child"], s["zero"])
            _plain_fork(s)
        return dict(_values(s["cache"]), table=s["table"], refs=s["refs"])
    s["book"].copy_(s["scattered"])
    if own:
        m.mla_pages_compact(s["handle"], s["pool"], s["moved"], s["n_live"], s["workspace"])
    else:
        _plain_compact(s)
    return dict(_values(s["cache"]), table=s["table"], refs=s["refs"], moved=s["moved"], n_live=s["n_live"])


def _first(flags, n):
    """The first n indexes whose flag is set."""
    return torch.sort(flags.logical_not().to(torch.uint8), stable=True).indices[:n]


def _plain_free(s, rows, keep):
    table, refs, page = s["table"], s["refs"], s["page"]
    rows = rows.long()
    held = table[rows]
    col = torch.arange(table.shape[1], device="cuda")
    drop = (col >= ((keep + page - 1) // page)[:, None]) & (held >= 0)
    refs.scatter_add_(0, held.clamp_min(0).flatten().long(), -drop.flatten().to(torch.int32))
    table[rows] = torch.where(drop, -1, held)


def _plain_reserve(s):
    table, refs, page = s["table"], s["refs"], s["page"]
    rows = s["rows_of"].long()
    held = table[rows]
    col = torch.arange(table.shape[1], device="cuda")
    add = (col < ((s["grow"] + page - 1) // page)[:, None]) & (held < 0)
    free = _first(refs == 0, refs.shape[0])
    which = free[(torch.cumsum(add.flatten().to(torch.int32), 0) - 1).clamp_min(0)]
    refs.scatter_add_(0, which, add.flatten().to(torch.int32))
    table[rows] = torch.where(add, which.view(add.shape).to(torch.int32), held)


def _plain_fork(s):
    table, refs, page, c = s["table"], s["refs"], s["page"], s["cache"]
    held = table[s["parent"].long()]
    full, rest = s["at"] // page, s["at"] % page
    col = torch.arange(table.shape[1], device="cuda")
    shared, tail = col < full[:, None], (col == full[:, None]) & (rest > 0)[:, None]
    free = _first(refs == 0, rest.shape[0])
    new = free[(torch.cumsum((rest > 0).to(torch.int32), 0) - 1).clamp_min(0)]
    child = torch.where(shared, held, torch.where(tail, new[:, None].to(torch.int32), -1))
    table[s["child"].long()] = child
    refs.scatter_add_(0, child.clamp_min(0).flatten().long(), (child >= 0).flatten().to(torch.int32))
    t = s["tails"]
    src, dst = held[t, full[t].long()].long(), new[t]
    older = torch.arange(page, device="cuda")[None, :] < rest[t][:, None]
    for name in ("k_codes", "v_codes"):
        c[name][dst] = torch.where(older[:, None, :, None], c[name][src], c[name][dst])
    c["k_pe"][dst] = torch.where(older[:, :, None], c["k_pe"][src], c["k_pe"][dst])
    for name in ("k_scales", "v_scales"):
        c[name][dst] = c[name][src]


def _plain_compact(s):
    table, refs, c, moves = s["table"], s["refs"], s["cache"], s["moves"]
    live = refs > 0
    n_live = live.sum()
    number = torch.arange(refs.shape[0], device="cuda")
    src = _first(live & (number >= n_live), moves)
    dst = _first(~live & (number < n_live), moves)
    moved = torch.where(live, number, -1).to(torch.int32)
    moved[src] = dst.to(torch.int32)
    for name in TENSORS:
        c[name][dst] = c[name][src]
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, moved[table.clamp_min(0).long()], -1))
    s["moved"].copy_(moved)
    s["n_live"].copy_(n_live.view(1))


def _plain_copy(s):
    for name in TENSORS:
        s["to"][name][s["dst"].long()] = s["from"][name][s["src"].long()]


def _plain_documents(s):
    row = key = 0
    for n, L, prefix in zip(s["new"], s["keys"], s["first"]):
        if n:
            q = s["q"][row:row + n].view(n, DENSE_HEADS, QK).float().transpose(0, 1)
            k, v = s["k"][:, key:key + L].float(), s["v"][:, key:key + L].float()
            i = torch.arange(L - n, L, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")[None, :]
            sees = j <= i
            if s["window"]:
                sees &= (i - j < s["window"]) | (j < s["sinks"])
            sees |= j < prefix
            scores = (torch.matmul(q, k.transpose(-1, -2)) * SCALE).masked_fill_(~sees, -math.inf)
            p = torch.exp(scores - scores.amax(-1, keepdim=True))
            o = torch.matmul(p / p.sum(-1, keepdim=True), v)
            s["out"][row:row + n] = o.transpose(0, 1).reshape(n, DENSE_HEADS * V).to(torch.bfloat16)
        row, key = row + n, key + L


# ---- the same from the definitions: one row, page and document after the other ------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"fork": _exact_fork, "regrow": _exact_regrow, "compact": _exact_compact, "copy": _exact_copy,
            "documents": _exact_documents}[case["op"]](s)


def _exact_drop(table, refs, r, keep):
    for e in range(keep, table.shape[1]):
        if table[r, e] >= 0:
            refs[table[r, e]] -= 1
            table[r, e] = -1


def _exact_regrow(s):
    table, refs, page = s["table"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy(), s["page"]
    rows, keep, grow = (s[n].tolist() for n in ("rows_of", "keep", "grow"))
    for r, p in zip(rows, keep):
        _exact_drop(table, refs, r, math.ceil(p / page))
    free = iter(np.flatnonzero(refs == 0).tolist())
    for r, p in zip(rows, grow):
        for e in range(math.ceil(p / page)):
            if table[r, e] < 0:
                table[r, e] = next(free)
                refs[table[r, e]] = 1
    return {"table": torch.from_numpy(table).cuda(), "refs": torch.from_numpy(refs).cuda()}


def _exact_fork(s):
    table, refs, page = s["table"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy(), s["page"]
    c = {n: x.clone() for n, x in _values(s["cache"]).items()}
    parent, child, at = (s[n].tolist() for n in ("parent", "child", "at"))
    for r in child:
        _exact_drop(table, refs, r, 0)
    free = iter(np.flatnonzero(refs == 0).tolist())
    for p, r, n in zip(parent, child, at):
        whole, rest = divmod(n, page)
        for e in range(whole):
            table[r, e] = table[p, e]
            refs[table[p, e]] += 1
        if rest:
            old, new = int(table[p, whole]), next(free)
            table[r, whole], refs[new] = new, 1
            for name in ("k_codes", "v_codes"):
                c[name].view(torch.uint8)[new, :, :rest] = c[name].view(torch.uint8)[old, :, :rest]
            c["k_pe"][new, :rest] = c["k_pe"][old, :rest]
            for name in ("k_scales", "v_scales"):
                c[name][new] = c[name][old]
    return dict(c, table=torch.from_numpy(table).cuda(), refs=torch.from_numpy(refs).cuda())


def _exact_compact(s):
    table, refs = s["table"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()
    c = {n: x.clone() for n, x in _values(s["cache"]).items()}
    n_live = int(np.count_nonzero(refs))
    holes = [p for p in range(n_live) if refs[p] == 0]
    moved = [p if refs[p] else -1 for p in range(len(refs))]
    for p in range(n_live, len(refs)):
        if refs[p]:
            to = holes.pop(0)
            moved[p] = to
            refs[to], refs[p] = refs[p], 0
            for n in TENSORS:
                bits = c[n].view(torch.uint8) if n.endswith("codes") else c[n]
                bits[to] = bits[p]
    for r in range(table.shape[0]):
        for e in range(table.shape[1]):
            if table[r, e] >= 0:
                table[r, e] = moved[table[r, e]]
    return dict(c, table=torch.from_numpy(table).cuda(), refs=torch.from_numpy(refs).cuda(),
                moved=_ints(moved), n_live=_ints([n_live]))


def _exact_copy(s):
    c = {n: x.clone() for n, x in _values(s["to"]).items()}
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        for n in TENSORS:
            (c[n].view(torch.uint8) if n.endswith("codes") else c[n])[b] = s["from"][n][a]
    return c


def _exact_documents(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    row = key = 0
    for n, L, prefix in zip(s["new"], s["keys"], s["first"]):
        at = np.arange(n)[:, None] + (L - n)
        col = np.arange(L)[None, :]
        hidden = (col > at) if not s["window"] else (col > at) | ((at - col >= s["window"]) & (col >= s["sinks"]))
        hidden = torch.from_numpy(hidden & (col >= prefix)).cuda()
        for h in range(DENSE_HEADS if n else 0):
            score = s["q"][row:row + n, h * QK:(h + 1) * QK].double() @ s["k"][h, key:key + L].double().T * SCALE
            score[hidden] = -math.inf
            w = torch.exp(score - score.max(1, keepdim=True).values)
            out[row:row + n, h * V:(h + 1) * V] = (w @ s["v"][h, key:key + L].double()) / w.sum(1, keepdim=True)
        row, key = row + n, key + L
    return out
