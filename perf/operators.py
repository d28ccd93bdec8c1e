"""The paged 8-bit cache, the attention that reads it and attention under a sliding window: cases, inputs and plain forms.

Shapes: a head has 128 key values without a position, 64 rotated ones (one rotary key per token, shared by all
heads) and 128 values.  Cache: pages of `page` tokens; keys and values as E4M3 codes [n_pages, heads, page, 128]
with one power-of-two scale per page and head, the rotary key in bf16 [n_pages, page, 64], and a table of page
numbers per sequence.
"""
import math
import random

import numpy as np
import torch

own = False

NOPE, ROPE, V = 128, 64, 128
QK = NOPE + ROPE
DENSE_HEADS = 64          # the dense caches' head count
BASE = 10000.0
SCALE = 1.0 / math.sqrt(QK)
FLOOR_EXP, CEIL_EXP = -60, 60


# ---- the cases ----------------------------------------------------------------------------------------------
def listed():
    return [
        # one new token of one sequence: the latency of a chat's decode step
        {"name": "append 1x1", "op": "append", "B": 1, "T": 1, "ragged": False, "lo": 1000, "hi": 1000, "page": 64,
         "heads": 64},
        # one new token of each of 64 sequences of different lengths: a decode batch
        {"name": "append 64x1", "op": "append", "B": 64, "T": 1, "ragged": False, "lo": 1, "hi": 2000, "page": 16,
         "heads": 64},
        # ragged prompts that go on behind cached tokens: a serving step that mixes prompts
        {"name": "append ragged 16x1531", "op": "append", "B": 16, "T": 1531, "ragged": True, "lo": 0, "hi": 777,
         "page": 32, "heads": 64},
        # a whole prefill batch
        {"name": "append 8x4096", "op": "append", "B": 8, "T": 4096, "ragged": False, "lo": 0, "hi": 0, "page": 64,
         "heads": 64},
        # the first token after a short prompt
        {"name": "attend 1x17", "op": "attend", "B": 1, "T": 1, "lo": 16, "hi": 16, "page": 64, "heads": 64,
         "window": 0, "sinks": 0},
        # one long conversation
        {"name": "attend 1x32k", "op": "attend", "B": 1, "T": 1, "lo": 32817, "hi": 32817, "page": 64, "heads": 64,
         "window": 0, "sinks": 0},
        # a decode batch of equal lengths
        {"name": "attend 64x1001", "op": "attend", "B": 64, "T": 1, "lo": 1000, "hi": 1000, "page": 64, "heads": 64,
         "window": 0, "sinks": 0},
        # a ragged batch up to 8192 positions on small pages
        {"name": "attend ragged 32x8192", "op": "attend", "B": 32, "T": 1, "lo": 1, "hi": 8191, "page": 16,
         "heads": 64, "window": 0, "sinks": 0},
        # four drafted tokens verified at once, on a quarter of the heads
        {"name": "attend draft 16x4", "op": "attend", "B": 16, "T": 4, "lo": 100, "hi": 4000, "page": 32, "heads": 16,
         "window": 0, "sinks": 0},
        # a long ragged batch under a sliding window with sinks
        {"name": "attend window 1024", "op": "attend", "B": 64, "T": 1, "lo": 500, "hi": 8191, "page": 16, "heads": 64,
         "window": 1024, "sinks": 20},
        # a chunk of a prompt behind cached positions, under a window
        {"name": "window chunk 2048+2048", "op": "window", "B": 1, "T": 2048, "P0": 2048, "window": 1000, "sinks": 4},
        # whole prompts under a window
        {"name": "window prefill 2x4096", "op": "window", "B": 2, "T": 4096, "P0": 0, "window": 1024, "sinks": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "window"])
    page, heads = rng.choice([16, 32, 64, 128]), rng.choice([4, 8, 12, 16, 32, 64])
    if op == "append":
        B, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 4096)
        T = rng.choice([1, _log_int(rng, 2, 4096)])
        T = min(T, 32768 // B)
        return {"op": op, "B": B, "T": T, "ragged": rng.random() < 0.5, "lo": rng.randint(0, hi), "hi": hi,
                "page": page, "heads": heads}
    if op == "attend":
        B, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 32768)
        hi = min(hi, 2 ** 17 // B * 64 // heads)
        window = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        return {"op": op, "B": B, "T": rng.choice([1, 1, rng.randint(2, 8)]), "lo": rng.randint(0, hi), "hi": hi,
                "page": page, "heads": heads, "window": window, "sinks": rng.randint(0, 130) if window else 0}
    T = _log_int(rng, 1, 4096)
    return {"op": op, "B": rng.choice([1, 2]), "T": T, "P0": rng.choice([0, rng.randint(1, 4097 - T)]),
            "window": _log_int(rng, 1, 1024), "sinks": rng.choice([0, rng.randint(1, 128)])}


def _numbers(case, lo, hi, salt):
    """B whole numbers in [lo, hi], the ends among them, the same for every seed."""
    rng = random.Random("%s %s %s %s" % (case["B"], case["T"], hi, salt))
    x = [hi] + [lo] * (case["B"] > 1) + [rng.randint(lo, hi) for _ in range(case["B"] - 2)]
    rng.shuffle(x)
    return x


def _lengths(case):
    """Positions P of the first new token and counts T of the new tokens, per sequence."""
    P = _numbers(case, case["lo"], case["hi"], "P")
    T = _numbers(case, max(1, case["T"] // 8), case["T"], "T") if case.get("ragged") else [case["T"]] * case["B"]
    return P, T


def _visible(P, T, window, sinks):
    """Keys that one of the queries at positions P .. P + T - 1 sees, and (query, key) pairs."""
    pairs, start = 0, 0
    i = np.arange(P, P + T, dtype=np.int64)
    if window:
        first = np.maximum(i - window + 1, 0)
        pairs = int(np.sum(i + 1 - first + np.minimum(first, sinks)))
        start = max(0, P - window + 1)
        return P + T - start + min(start, sinks), pairs
    return P + T, int(np.sum(i + 1))


def work(case):
    if case["op"] == "append":
        H, n = case["heads"], sum(_lengths(case)[1])
        return {"bytes": n * (H * 256 * 3 + 128 * 2), "flops": n * H * 256 * 2}
    if case["op"] == "attend":
        H, T = case["heads"], case["T"]
        seen = [_visible(p, T, case["window"], case["sinks"]) for p in _lengths(case)[0]]
        return {"bytes": sum(k for k, _ in seen) * (H * 256 + 128) + case["B"] * T * H * (QK + V) * 2,
                "flops": sum(n for _, n in seen) * H * 2 * (QK + V)}
    keys, pairs = _visible(case["P0"], case["T"], case["window"], case["sinks"])
    bh = case["B"] * DENSE_HEADS
    return {"bytes": bh * (keys + case["T"]) * (QK + V) * 2, "flops": bh * pairs * 2 * (QK + V)}


# ---- the inputs ---------------------------------------------------------------------------------------------
def _quantised(g, n_pages, heads, page):
    """Random codes and their scales: values of size about 1, with larger and smaller pages among them."""
    size = torch.exp2(torch.randint(-2, 3, (n_pages, heads, 1, 1), generator=g, device="cuda").float())
    x = torch.empty((n_pages, heads, page, 128), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    top = x.abs().amax((2, 3), keepdim=True).float() * size
    e = torch.ceil(torch.log2(top / 448.0)).clamp_(FLOOR_EXP, CEIL_EXP)
    codes = (x * (size * torch.exp2(-e)).to(torch.bfloat16)).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), torch.exp2(e)[:, :, 0, 0].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)

    if case["op"] == "window":
        B, T, L = case["B"], case["T"], case["P0"] + case["T"]
        s["q"] = normal(B, T, DENSE_HEADS * QK)
        s["k"], s["v"] = normal(B, DENSE_HEADS, L, QK), normal(B, DENSE_HEADS, L, V)
        if own:
            import mla_gb300 as m
            s["out"] = torch.empty((B, T, DENSE_HEADS * V), dtype=torch.bfloat16, device="cuda")
            s["workspace"] = m.alloc_workspace(m.MODE_WINDOW_ATTN, B, T)
        return s

    # a cache whose pages lie in random order, with one spare page
    H, page = case["heads"], case["page"]
    P, T = _lengths(case)
    B, pages = case["B"], [-(-(p + t) // page) for p, t in zip(P, T)]
    n_pages, wide = sum(pages) + 1, max(pages)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    c = {"table": table, "k_pe": normal(n_pages, page, ROPE)}
    c["k_codes"], c["k_scales"] = _quantised(g, n_pages, H, page)
    c["v_codes"], c["v_scales"] = _quantised(g, n_pages, H, page)
    s["cache"] = c
    s["P"], s["P_max"] = torch.tensor(P, dtype=torch.int32, device="cuda"), max(P)
    if case["op"] == "append":
        n = sum(T)
        kv = normal(n, H, NOPE + V)                # a fused projection's output, per head [key | value]
        kv *= torch.exp(normal(n, 1, 1) * 0.5)     # tokens of different size
        s["kv"], s["pe"] = kv, normal(n, 576)      # the rotary key is the last 64 of 576 columns
        s["cu"] = torch.tensor([0] + list(np.cumsum(T)), dtype=torch.int32, device="cuda") if case["ragged"] else None
        if own:
            import mla_gb300 as m
            s["handle"] = m.make_paged_cache(c)
            s["workspace"] = m.alloc_workspace(m.MODE_PAGED_APPEND, B, case["T"])
    else:
        s["q"] = normal(B * case["T"], H * QK)
        if own:
            import mla_gb300 as m
            s["handle"] = m.make_paged_cache(c)
            s["out"] = torch.empty((B * case["T"], H * V), dtype=torch.bfloat16, device="cuda")
            s["workspace"] = m.alloc_workspace(m.MODE_PAGED_ATTN, B, case["T"])
    return s


# ---- one pass -----------------------------------------------------------------------------------------------
def run(s):
    if s["op"] == "append":
        if own:
            import mla_gb300 as m
            m.mla_paged_append(s["handle"], s["kv"][..., :NOPE], s["kv"][..., NOPE:], s["pe"][:, 512:], s["P"],
                               s["T"], s["workspace"], cu=s["cu"])
        else:
            _plain_append(s)
        c = s["cache"]
        return {"k": c["k_codes"].view(torch.float8_e4m3fn), "v": c["v_codes"].view(torch.float8_e4m3fn),
                "k_scales": c["k_scales"], "v_scales": c["v_scales"], "k_pe": c["k_pe"]}
    if s["op"] == "attend":
        if own:
            import mla_gb300 as m
            m.mla_paged_attention(s["handle"], s["q"], s["P"], s["P_max"], s["out"], s["workspace"],
                                  window=s["window"], sinks=s["sinks"])
            return s["out"]
        return _plain_attend(s)
    if own:
        import mla_gb300 as m
        m.mla_window_attention(s["q"], s["P0"], s["k"], s["v"], s["out"], s["workspace"], window=s["window"],
                               sinks=s["sinks"])
        return s["out"]
    return _plain_window(s)


def _exponent(top):
    """The smallest k in [-60, 60] with top <= 448 * 2^k (448 = 0.875 * 2^9)."""
    frac, e = torch.frexp(top)
    k = torch.where(frac <= 0.875, e - 9, e - 8).clamp(FLOOR_EXP, CEIL_EXP)
    return torch.where(top > 0, k, FLOOR_EXP)


def _coded(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    c, page, B = s["cache"], s["page"], s["B"]
    n, dev = s["kv"].shape[0], s["kv"].device
    token = torch.arange(n, device=dev)
    if s["cu"] is None:
        seq, first = token // s["T"], torch.arange(B, device=dev) * s["T"]
    else:
        seq, first = torch.searchsorted(s["cu"], token, right=True, out_int32=False) - 1, s["cu"][:-1].long()
    pos = s["P"][seq].long() + token - first[seq]
    pid, slot = c["table"][seq, pos // page].long(), pos % page
    old_pid, old_n = c["table"][torch.arange(B, device=dev), s["P"].long() // page].long(), s["P"].long() % page
    for name, cols in (("k", slice(0, NOPE)), ("v", slice(NOPE, NOPE + V))):
        x = s["kv"][..., cols].float()
        codes, scales = c[name + "_codes"], c[name + "_scales"]
        exp = torch.full(scales.shape, -1000, dtype=torch.int32, device=dev)
        exp.scatter_reduce_(0, pid[:, None].expand(n, x.shape[1]), _exponent(x.abs().amax(-1)).to(torch.int32), "amax")
        old_exp = torch.frexp(scales[old_pid])[1] - 1
        exp[old_pid] = torch.where(old_n[:, None] > 0, torch.maximum(exp[old_pid], old_exp), exp[old_pid])
        scales.copy_(torch.where(exp > -1000, torch.exp2(exp.float()), scales))
        # the codes that a growing scale re-expresses
        ratio = torch.exp2((old_exp - exp[old_pid]).float())[:, :, None, None]
        kept = codes[old_pid]
        older = torch.arange(page, device=dev)[None, :] < old_n[:, None]
        moved = _coded(kept.view(torch.float8_e4m3fn).float() * ratio)
        codes[old_pid] = torch.where(older[:, None, :, None], moved, kept)
        codes[pid, :, slot] = _coded(x * torch.exp2(-exp[pid].float())[:, :, None])
    # the rotation: pairs (i, i + 32), angles in 64 bits
    angle = pos.double()[:, None] * BASE ** (-torch.arange(32, device=dev, dtype=torch.float64) / 32.0)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    x1, x2 = s["pe"][:, 512:544].float(), s["pe"][:, 544:576].float()
    c["k_pe"][pid, slot] = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], 1).to(torch.bfloat16)


def _softmax(scores, seen):
    """Probabilities over the last axis; a row that sees nothing gets zeros."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isfinite(top), top, 0.0))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _sees(at, keys, window, sinks):
    ahead = at[..., None] - keys
    seen = ahead >= 0
    return seen & ((ahead < window) | (keys < sinks)) if window else seen


def _plain_attend(s):
    c, page, B, T, H = s["cache"], s["page"], s["B"], s["T"], s["heads"]
    n = -(-(s["P_max"] + T) // page)
    pid, L = c["table"][:, :n].clamp_min(0).long(), n * page
    q = s["q"].view(B, T, H, QK).float().transpose(1, 2)

    def dense(name):
        x = c[name + "_codes"][pid].view(torch.float8_e4m3fn).float() * c[name + "_scales"][pid][..., None, None]
        return x.transpose(1, 2).reshape(B, H, L, 128)

    scores = torch.matmul(q[..., :NOPE], dense("k").transpose(-1, -2))
    pe = c["k_pe"][pid].float().reshape(B, 1, L, ROPE)
    scores = (scores + torch.matmul(q[..., NOPE:], pe.transpose(-1, -2))) * SCALE
    at = s["P"].long()[:, None] + torch.arange(T, device=q.device)
    seen = _sees(at, torch.arange(L, device=q.device), s["window"], s["sinks"])
    out = torch.matmul(_softmax(scores, seen[:, None]), dense("v"))
    return out.transpose(1, 2).reshape(B * T, H * V).to(torch.bfloat16)


def _plain_window(s):
    B, T, L = s["B"], s["T"], s["P0"] + s["T"]
    q = s["q"].view(B, T, DENSE_HEADS, QK).float().transpose(1, 2)
    scores = torch.matmul(q, s["k"].float().transpose(-1, -2)) * SCALE
    at = s["P0"] + torch.arange(T, device=q.device)
    seen = _sees(at, torch.arange(L, device=q.device), s["window"], s["sinks"])
    out = torch.matmul(_softmax(scores, seen), s["v"].float())
    return out.transpose(1, 2).reshape(B, T, DENSE_HEADS * V).to(torch.bfloat16)


# ---- the same in 64 bits, from the definitions --------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "window": _exact_window}[case["op"]](case, s)


def _exact_append(case, s):
    """Values in units of their page's scale, before they are rounded to a code."""
    c, page = s["cache"], case["page"]
    got = {n: c[n + "_codes"].view(torch.float8_e4m3fn).double() for n in "kv"}
    scales = {n: c[n + "_scales"].double().cpu().numpy() for n in "kv"}
    pe = c["k_pe"].double()
    table = c["table"].cpu().numpy()
    theta = torch.tensor([BASE ** (-2.0 * i / ROPE) for i in range(ROPE // 2)], dtype=torch.float64, device=pe.device)
    P, T = _lengths(case)
    at = 0
    for b in range(case["B"]):
        done = 0
        while done < T[b]:
            pos = P[b] + done
            slot, n = pos % page, min(page - pos % page, T[b] - done)
            pid = int(table[b, pos // page])
            for name, off in (("k", 0), ("v", NOPE)):
                x = s["kv"][at:at + n, :, off:off + 128].double()
                need = np.exp2(np.clip(np.ceil(np.log2(np.maximum(x.abs().amax((0, 2)).cpu().numpy(), 1e-300) / 448.0)),
                                       FLOOR_EXP, CEIL_EXP))
                old = scales[name][pid].copy()
                new = np.maximum(need, old) if slot else need
                scales[name][pid] = new
                if slot:
                    got[name][pid, :, :slot] *= torch.from_numpy(old / new).to(x.device)[:, None, None]
                got[name][pid, :, slot:slot + n] = x.transpose(0, 1) / torch.from_numpy(new).to(x.device)[:, None, None]
            a = torch.arange(pos, pos + n, device=pe.device).double()[:, None] * theta
            z = torch.complex(s["pe"][at:at + n, 512:544].double(), s["pe"][at:at + n, 544:576].double())
            z = z * torch.polar(torch.ones_like(a), a)
            pe[pid, slot:slot + n] = torch.cat([z.real, z.imag], 1)
            at, done = at + n, done + n
    return {"k": got["k"], "v": got["v"], "k_scales": torch.from_numpy(scales["k"]),
            "v_scales": torch.from_numpy(scales["v"]), "k_pe": pe}


def _exact_keys(i, window, sinks):
    """The keys that the query at position i sees."""
    return [j for j in range(i + 1) if not window or i - j < window or j < sinks]


def _exact_attend(case, s):
    c, page, T, H = s["cache"], case["page"], case["T"], case["heads"]
    out = torch.zeros((case["B"], T, H, V), dtype=torch.float64, device="cuda")
    for b, p in enumerate(_lengths(case)[0]):
        for t in range(T):
            j = torch.tensor(_exact_keys(p + t, case["window"], case["sinks"]), device="cuda")
            pid, slot = c["table"][b][j // page].long(), j % page
            k = c["k_codes"][pid, :, slot].view(torch.float8_e4m3fn).double() * c["k_scales"][pid].double()[..., None]
            v = c["v_codes"][pid, :, slot].view(torch.float8_e4m3fn).double() * c["v_scales"][pid].double()[..., None]
            q = s["q"][b * T + t].view(H, QK).double()
            score = (k * q[:, :NOPE]).sum(-1) + c["k_pe"][pid, slot].double() @ q[:, NOPE:].T
            w = torch.exp((score - score.max(0).values) * SCALE)
            out[b, t] = torch.einsum("jh,jhd->hd", w / w.sum(0), v)
    return out.view(case["B"] * T, H * V)


def _exact_window(case, s):
    B, T = case["B"], case["T"]
    i = np.arange(case["P0"], case["P0"] + T)[:, None]
    j = np.arange(case["P0"] + T)[None, :]
    hidden = torch.from_numpy((j > i) | ((i - j >= case["window"]) & (j >= case["sinks"]))).cuda()
    out = torch.empty((B, T, DENSE_HEADS, V), dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(DENSE_HEADS):
            q = s["q"][b, :, h * QK:(h + 1) * QK].double()
            score = (q @ s["k"][b, h].double().T) * SCALE
            score[hidden] = -math.inf
            w = torch.exp(score - score.max(1, keepdim=True).values)
            out[b, :, h] = (w @ s["v"][b, h].double()) / w.sum(1, keepdim=True)
    return out.view(B, T, DENSE_HEADS * V)
