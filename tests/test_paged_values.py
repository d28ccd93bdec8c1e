"""The paged 8-bit cache at values that its own append does not make, or makes seldom: scales of other quantizers,
pages whose scale no visible key needs, long contexts of small weights, far positions.

References in 64 bits, from the definitions in include/mla.h.  Tolerances count roundings: a value rounded to nearest
in bf16 is off by at most 2^-8 of it, in float16 by 2^-11 (eps/2 of the type)."""

import ctypes
import math

import numpy as np
import pytest

import mla_gb300 as m
from test_paged import f64, filled, ints, normal

gpu = pytest.mark.gpu


def e4m3(x):
    """float64 -> the nearest E4M3 value (ties to even, saturating at 448), as float64: exact, with no rounding in
    between (3 fraction bits from 2^-6 on, steps of 2^-9 below)."""
    with np.errstate(all="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -60)))
    e = np.where(2.0 ** (e + 1) <= np.abs(x), e + 1, np.where(2.0 ** e > np.abs(x), e - 1, e))
    q = 2.0 ** (np.maximum(e, -6) - 3)
    return np.clip(np.round(x / q) * q, -448, 448)


def need_of(x):
    """2^k with the smallest k in [-60, 60] for which amax <= 448 * 2^k"""
    top = np.abs(x).max()
    k = -60
    while k < 60 and top > 448 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def test_rounding_of_this_file():
    import torch
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    every = np.sort(every[np.isfinite(every)])
    assert np.array_equal(e4m3(every), every)
    mid = (every[1:] + every[:-1]) / 2
    assert np.all((e4m3(mid * (1 + 2.0 ** -40)) == np.where(mid > 0, every[1:], every[:-1]))[mid != 0])
    assert e4m3(np.array([500.0, -1e9, 17.0, 19.0])).tolist() == [448, -448, 16, 20] and need_of(np.array([449.0])) == 2


# ---- append --------------------------------------------------------------------------------------------------
FOREIGN = [3.0, 1.5, 0.9, 2.0 ** -70, 1.3 * 2.0 ** -70, 2.0 ** 70, 1.7 * 2.0 ** 64, 448.0 / 449.0, 2.0 ** -3, 2.0 ** 5,
           float(np.float32(0.1)), 2.0 ** 127]


@gpu
@pytest.mark.parametrize("page,T,size", [(16, 1, 1.0), (16, 1, 2.0 ** 20), (64, 1, 700.0), (128, 100, 1.0), (32, 9, 900.0),
                                         (64, 5, 2.0 ** -66)])
def test_append_into_pages_of_other_quantizers(gpu_available, page, T, size):
    """A partly filled page with any positive scale: the scale becomes the larger of it and the new tokens' own, the
    codes there are kept, or re-expressed where the scale grows, and the new ones are x / scale rounded once."""
    import torch
    heads, fill = 12, 7
    t = m.alloc_paged_cache(3, page, heads)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(heads * fill)[:heads * fill * 128]
    codes = torch.where((codes & 0x7F) == 0x7F, torch.zeros_like(codes), codes).view(heads, fill, 128)
    for n in ("k_codes", "v_codes"):
        t[n][1, :, :fill] = codes
    scales = np.array(FOREIGN, dtype=np.float32)
    t["k_scales"][1], t["v_scales"][1] = torch.from_numpy(scales).cuda(), torch.from_numpy(scales[::-1].copy()).cuda()
    t["table"] = ints([[1, 2, 0]])
    n0 = min(T, page - fill)
    kv = (normal(7 + T, T, heads, 256).float() * size).to(torch.bfloat16)
    if T > 1:  # values at and beside halfway points between codes of the scales
        kv[1, :, :4] = torch.tensor([17.0, 1.0625, 19.0, 0.001953125], device="cuda")
    before = {n: f64(t[n + "_codes"].view(torch.float8_e4m3fn))[1] for n in "kv"}
    ws = m.alloc_workspace(m.MODE_PAGED_APPEND, 1, T)
    m.mla_paged_append(m.make_paged_cache(t), kv[..., :128], kv[..., 128:], normal(1, T, 64), ints([fill]), T, ws)
    assert m.mla_device_status(ws) == 0
    for name, x, old in (("k", f64(kv[..., :128]), scales), ("v", f64(kv[..., 128:]), scales[::-1])):
        got = f64(t[name + "_codes"].view(torch.float8_e4m3fn))[1]
        for h in range(heads):
            s0 = float(old[h])
            s = max(s0, need_of(x[:n0, h]))
            assert f64(t[name + "_scales"])[1, h] == s, (name, s0)
            assert np.array_equal(got[h, :fill], e4m3(before[name][h, :fill] * (s0 / s))), (name, s0, "older codes")
            assert np.array_equal(got[h, fill:fill + n0], e4m3(x[:n0, h] / s)), (name, s0, "new codes")
            assert np.all(got[h, fill + n0:] == 0), "slots behind the last token"


# ---- attention -----------------------------------------------------------------------------------------------
def attend(t, q, P, T=1, window=0, sinks=0):
    import torch
    out = torch.full((q.shape[0], q.shape[1] // 192 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = m.alloc_workspace(m.MODE_PAGED_ATTN, len(P), T)
    m.mla_paged_attention(m.make_paged_cache(t), q, ints(P), max(P), out, ws, window=window, sinks=sinks)
    assert m.mla_device_status(ws) == 0
    return f64(out).reshape(len(P), T, -1, 128)


def check_attention(t, q, P, T=1, window=0, sinks=0, what="", scale=1 / math.sqrt(192), rows=4, sums=2.0 ** -14):
    """The first `rows` sequences, element by element, with A = sum p |v| of the element (the weights sum to one): the
    output's own rounding 2^-8 |o|; the weights' rounding to float16, 2^-11 A; float32 scores, exponentials and sums,
    2^-14 A (scores here stay below 2^7 in log2 units, off by 2^-24 of that a few times over: 2^-15; chains of a few
    hundred float32 sums: 2^-16); weights below 2^-29 of the largest of their 32 keys, 2^-40 of it for each of the 32:
    2^-35 p max |v| of its page."""
    import torch
    got = attend(t, q, P, T, window, sinks)
    heads, page = t["k_codes"].shape[1], t["k_codes"].shape[2]
    table, qn = t["table"].cpu().numpy(), f64(q).reshape(len(P), T, heads, 192)
    v_all = t["v_codes"].view(torch.float8_e4m3fn)
    for b, p in enumerate(P[:rows]):
        for i in range(T):
            at = p + i
            j = np.arange(at + 1)
            if window:
                j = j[(at - j < window) | (j < sinks)]
            key, count = np.unique(table[b][j // page].astype(np.int64) * page + j % page, return_counts=True)
            pid, slot = torch.from_numpy(key // page).cuda(), torch.from_numpy(key % page).cuda()
            k = f64(t["k_codes"].view(torch.float8_e4m3fn)[pid, :, slot]) * f64(t["k_scales"][pid])[..., None]
            v = f64(v_all[pid, :, slot]) * f64(t["v_scales"][pid])[..., None]
            s = (np.einsum("hd,jhd->jh", qn[b, i, :, :128], k) + f64(t["k_pe"][pid, slot]) @ qn[b, i, :, 128:].T) * scale
            assert np.abs(s).max() / math.log(2) < 2 ** 7, "scores as the bound has them"
            w = np.exp(s - s.max(0)) * count[:, None]
            w /= w.sum(0)
            page_max = np.zeros((int(key.max()) // page + 1, heads))
            np.maximum.at(page_max, key // page, np.abs(v).max(2))
            ref, A = np.einsum("jh,jhd->hd", w, v), np.einsum("jh,jhd->hd", w, np.abs(v))
            low = (w * page_max[key // page]).sum(0)[:, None]
            bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + sums) * A + 2.0 ** -35 * low
            d = np.abs(got[b, i] - ref)
            assert np.all(d <= bound), f"{what}: sequence {b} query {i}: {np.max(d / np.maximum(bound, 1e-300)):.3g} of the bound"


@gpu
@pytest.mark.parametrize("page,T", [(16, 1), (16, 4), (32, 1), (64, 3), (128, 1), (128, 8)])
@pytest.mark.parametrize("up", [0, 20, 24, 30, 60, 100])
def test_page_scales_that_no_visible_value_needs(gpu_available, page, T, up):
    """Pages whose value scale is far above their values: all zero, or small. The other pages keep their bits."""
    import torch
    P, heads = [700, 45] * 30, 8                  # several tiles a CTA
    t, _ = filled(P, T, page, heads, 3 + up)
    for b in range(len(P)):
        for i, pid in enumerate(t["table"][b].tolist()):
            if pid >= 0 and i % 2 == 0:
                t["v_scales"][pid, ::2] *= 2.0 ** up
                t["v_codes"][pid, ::2] = 0
            elif pid >= 0 and i % 3 == 0:
                t["v_scales"][pid, 1::2] *= 2.0 ** -up
    check_attention(t, normal(5, len(P) * T, heads * 192), P, T, what=f"scales times 2^{up}")


@gpu
@pytest.mark.parametrize("value", [2.0 ** 24, 2.0 ** 50, math.inf])
def test_a_value_that_the_window_has_passed(gpu_available, value):
    """A page keeps the scale that an outlier gave it; once the window has passed the outlier, its page and the others
    answer as if it had not been. The same for a rejected draft that other tokens overwrite."""
    import torch
    heads, page, n = 4, 16, 96
    kv, pe, q = normal(1, n, heads, 256), normal(2, n, 64), normal(3, 1, heads * 192)
    kv[34, :, 128] = value
    t = m.alloc_paged_cache(6, page, heads)
    t["table"] = ints([[2, 0, 1, 5, 3, 4]])
    ws = m.alloc_workspace(m.MODE_PAGED_APPEND, 1, n)

    def put(at, x, y):
        m.mla_paged_append(m.make_paged_cache(t), x[..., :128], x[..., 128:], y, ints([at]), x.shape[0], ws)
        assert m.mla_device_status(ws) == 0

    put(0, kv, pe)
    check_attention(t, q, [n - 1], window=n - 35, what="behind the window")
    draft = kv[66:].clone()
    draft[0, :, 128:] = value
    put(66, draft, pe[66:])
    put(66, kv[66:], pe[66:])
    check_attention(t, q, [n - 1], window=n - 35, what="rejected draft")


@gpu
@pytest.mark.parametrize("page,n,gap", [(128, 1 << 21, 21), (16, 1 << 17, 24), (64, 1 << 20, 33), (32, 5000, 40),
                                        (128, 1 << 24, 30)])
def test_many_keys_of_small_weight(gpu_available, page, n, gap):
    """One key outweighs each other one by 2^gap, and the others are many: together they carry a share of the output
    that float16 steps of the one key's weight would lose. Their pages are shared, so that the cache stays small."""
    import torch
    heads = 4
    t = m.alloc_paged_cache(3, page, heads)
    wide = -(-n // page)
    t["table"] = torch.full((1, wide), 1, dtype=torch.int32, device="cuda")
    t["table"][0, 0] = 0
    for name in ("k", "v"):
        x = normal(4, 3, heads, page, 128, scale=0.25 if name == "k" else 1.0)
        t[name + "_codes"].copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
    t["v_codes"][1] &= 0x7F                       # all of one sign: their sum does not cancel
    t["v_codes"][0, :, :, :64] = 0
    q = normal(6, 1, heads * 192, scale=0.25)
    q[0, 128::192] = 8.0                          # the first rotary value weighs the first key up
    t["k_pe"][:, :, 0] = 0
    t["k_pe"][0, 3, 0] = gap * math.log(2) * math.sqrt(192) / 8
    # 2^24 keys are 2^18 tiles, 1,725 a thread block: as many sums in a row for O and twice as many for the weights'
    # total, each off by up to 2^-24: 2^-11.6
    check_attention(t, q, [n - 1], what=f"{n} keys", **(dict(sums=2.0 ** -11.5) if n > 1 << 21 else {}))


@gpu
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("up", [10, 25, 50])
def test_large_values_of_small_weight(gpu_available, page, up):
    """A page whose weights are 2^-up of the others' and whose values are 2^up of theirs carries half of the output."""
    import torch
    P, heads = [3 * 64 - 1], 4
    t, _ = filled(P, 1, page, heads, 8, spread=0)
    low = t["table"][0, 64 // page:128 // page].long()
    t["v_scales"][low] *= 2.0 ** up
    q = normal(6, 1, heads * 192, scale=0.25)
    q[0, 128::192] = 8.0
    t["k_pe"][:, :, 0] = 0
    t["k_pe"][low, :, 0] = -up * math.log(2) * math.sqrt(192) / 8
    check_attention(t, q, P, what=f"2^{up}")


# ---- the binding ---------------------------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("shape", [(0, 4), (2, 0), (0, 0)])
def test_tables_without_entries_are_refused(gpu_available, shape):
    import torch
    t = m.alloc_paged_cache(2, 16, 4)
    t["table"] = torch.zeros(shape, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="at least one"):
        m.make_paged_cache(t)


# ---- the status word -----------------------------------------------------------------------------------------
@gpu
def test_status_words_end_inside_the_status_region(gpu_available):
    """A workspace that no call has written may hold any count of further status words: no more are read than a call
    writes, one for each of at most 256 thread blocks."""
    import torch
    ws = torch.zeros(8192, dtype=torch.uint8, device="cuda")
    words = ws.view(torch.int32)
    words[64 + 256:] = -1
    for count in (0, 1, 256, 257, 400, 960, 961, 1024, 1025, -1, 2 ** 31 - 1):
        words[1] = count
        assert m.mla_device_status(ws) == 0, count
    words[1], words[64 + 255] = 256, -1
    assert m.mla_device_status(ws) != 0
    words[1] = 255
    assert m.mla_device_status(ws) == 0


# ---- far positions and long, ragged batches ------------------------------------------------------------------
def test_sizes_of_an_append_that_are_taken_and_refused():
    """What mla.h states: 2^24 rows and sequences, T up to 2^30, 2^22 pages where B * T passes 2^24. A call that passes
    these checks meets the next one here, on its workspace (-3): nothing is enqueued."""
    from test_paged import append, fake_cache, FAKE
    far = fake_cache(max_pages=1 << 23, page=128, heads=4)
    assert m.workspace_size(m.MODE_PAGED_APPEND, 600, 32768) > 0
    assert append(far, B=600, T=32768, N=40000, cu=FAKE + 16384, wsb=16) == -3
    assert append(far, B=600, T=32768, N=40000, wsb=16) == -1
    assert append(far, B=2, T=(1 << 30) + 1, N=7, cu=FAKE + 16384, wsb=16) == -1
    assert append(far, B=(1 << 24) + 1, T=1, N=7, cu=FAKE + 16384, wsb=16) == -1
    assert append(far, B=1 << 20, T=1 << 20, N=1 << 24, cu=FAKE + 16384, wsb=16) == -1
    assert append(far, B=1 << 20, T=1 << 20, N=7, cu=FAKE + 16384, wsb=16) == -3      # no sequence has more than 7
    assert append(far, B=512, T=1 << 30, N=(8191 - 1) * 128 + 2, cu=FAKE + 16384, wsb=16) == -3   # 8,192 pages each
    assert append(far, B=512, T=1 << 30, N=(8191 - 1) * 128 + 130, cu=FAKE + 16384, wsb=16) == -1
    assert append(far, B=1 << 24, T=1, N=1 << 24, cu=FAKE + 16384, wsb=16) == -3
    assert append(far, B=(1 << 24) - 1, T=2, N=7, cu=FAKE + 16384, wsb=16) == -1


def test_reaches_that_are_taken_and_refused():
    """What mla.h states: positions up to 2^30, 2^24 visible keys, counts of tiles in 31 bits; else as above."""
    from test_paged import attend, fake_cache, FAKE
    from test_paged_sublayer import fake_weights
    far = fake_cache(max_pages=1 << 23, page=128, heads=4)
    assert attend(far, P_max=(1 << 24) - 1, wsb=16) == -3 and attend(far, P_max=1 << 24, wsb=16) == -1
    assert attend(far, P_max=(1 << 30) - 1, window=1 << 20, sinks=4, wsb=16) == -3
    assert attend(far, P_max=(1 << 30) - 1, window=(1 << 24) - 4, sinks=4, wsb=16) == -3
    assert attend(far, P_max=(1 << 30) - 1, window=(1 << 24) - 3, sinks=4, wsb=16) == -1
    assert attend(far, P_max=1 << 30, window=1 << 20, wsb=16) == -1
    assert attend(far, P_max=(1 << 24) - 1, B=(1 << 13) - 1, wsb=16) == -3
    assert attend(far, P_max=(1 << 24) - 1, B=1 << 13, wsb=16) == -1
    assert m.workspace_size(m.MODE_DECODE_PAGED, 2, (1 << 30) - 1) > 0
    L, w, c = m.lib(), fake_weights(), fake_cache(max_pages=1 << 23, page=128)

    def dec(P_max, window):
        return L.mla_decode_paged(ctypes.byref(w), None, FAKE + (1 << 30), 2, FAKE, P_max, ctypes.byref(c), window, 4,
                                  FAKE + (2 << 30), FAKE + (3 << 30), 64, None)

    assert dec((1 << 30) - 1, 4096) == -3 and dec((1 << 24) - 1, 0) == -3
    assert dec(1 << 24, 0) == -1 and dec(1 << 30, 4096) == -1


@gpu
@pytest.mark.parametrize("T", [1, 3])
def test_window_at_positions_past_24_bits(gpu_available, T):
    """Tokens appended and attended to around positions 2^24, 2^25 and 2^30, under a window with sinks: the pages
    in between are not there."""
    import torch
    heads, page, n = 4, 128, 300
    ends = [2 ** 25 + 77, 2 ** 24 + 5, 2 ** 30 - 128]
    wide = 2 ** 30 // page
    t = m.alloc_paged_cache(16, page, heads)
    table = torch.full((3, wide), -1, dtype=torch.int32)
    at = 0
    for b, e in enumerate(ends):
        for pi in [0] + list(range((e - n) // page, (e + T - 1) // page + 1)):
            table[b, pi] = at
            at += 1
    assert at <= 16
    t["table"] = table.cuda()
    ws = m.alloc_workspace(m.MODE_PAGED_APPEND, 3, n + T)
    for P, count, seed in (([0] * 3, 5, 1), ([e - n for e in ends], n + T, 2)):
        kv, pe = normal(seed, 3 * count, heads, 256), normal(seed + 5, 3 * count, 64)
        m.mla_paged_append(m.make_paged_cache(t), kv[..., :128], kv[..., 128:], pe, ints(P), count, ws)
        assert m.mla_device_status(ws) == 0
    theta = 10000.0 ** (-np.arange(32) / 32.0)
    x, keys = f64(pe).reshape(3, n + T, 64), f64(t["k_pe"])
    for b, e in enumerate(ends):                  # the last position of each: rotated by its angle
        pos = e + T - 1
        x1, x2, got = x[b, -1, :32], x[b, -1, 32:], keys[int(table[b, pos // page]), pos % page]
        want = np.concatenate([x1 * np.cos(pos * theta) - x2 * np.sin(pos * theta),
                               x2 * np.cos(pos * theta) + x1 * np.sin(pos * theta)])
        # 2^-8 of the value, 2^-20 of its parts, and the angle's own rounding, 2^-53 of up to 2^30, twice (here and there)
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -20 + 2.0 ** -21) * np.tile(np.abs(x1) + np.abs(x2), 2))
    q = normal(9, 3 * T, heads * 192)
    for window, sinks in ((200, 5), (64, 0), (1, 1)):
        got = attend(t, q, ends, T, window, sinks)
        # the same keys and values at small positions: pages in the order in which they are seen, the mask by hand
        for b, e in enumerate(ends):
            for i in range(T):
                pos = e + i
                j = np.concatenate([np.arange(sinks), np.arange(pos - window + 1, pos + 1)])
                pid, slot = t["table"][b][torch.from_numpy(j // page).cuda()].long(), torch.from_numpy(j % page).cuda()
                k = f64(t["k_codes"].view(torch.float8_e4m3fn)[pid, :, slot]) * f64(t["k_scales"][pid])[..., None]
                v = f64(t["v_codes"].view(torch.float8_e4m3fn)[pid, :, slot]) * f64(t["v_scales"][pid])[..., None]
                qn = f64(q).reshape(3, T, heads, 192)[b, i]
                s = np.einsum("hd,jhd->jh", qn[:, :128], k) + f64(t["k_pe"][pid, slot]) @ qn[:, 128:].T
                w = np.exp((s - s.max(0)) / math.sqrt(192))
                w /= w.sum(0)
                ref, A = np.einsum("jh,jhd->hd", w, v), np.einsum("jh,jhd->hd", w, np.abs(v))
                assert np.all(np.abs(got[b, i] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -14) * A), (b, i, window)


@gpu
def test_decode_step_at_positions_past_24_bits(gpu_available):
    """The sublayer's step depends on differences of positions only: the same tokens, under a window, from position 70
    and from 2^25 + 70 on."""
    import torch
    from mla_testlib import cuda_to_f64, cuda_weights, parity_out
    W, page, steps, outs = m.make_weights(cuda_weights(0)), 64, 6, []
    xs = normal(4, steps, 2, 7168)
    for base in (0, 2 ** 25):
        t = m.alloc_paged_cache(4, page)
        t["table"] = torch.full((2, base // page + 2), -1, dtype=torch.int32, device="cuda")
        t["table"][:, base // page:] = ints([[0, 1], [2, 3]])
        cache, ws = m.make_paged_cache(t), m.alloc_workspace(m.MODE_DECODE_PAGED, 2, base + 100)
        for i in range(steps):
            out = torch.empty_like(xs[i])
            m.mla_decode_paged(W, xs[i], ints([base + 70 + i] * 2), base + 100, cache, out, ws, window=3)
            assert m.mla_device_status(ws) == 0
            outs.append(cuda_to_f64(out))
    for i in range(steps):
        parity_out(outs[steps + i], outs[i], f"step {i}")


@gpu
def test_one_long_prompt_among_many_sequences(gpu_available):
    """600 sequences of which one brings 3,000 tokens and the others one each, with room for 32,768: more than 2^24
    tokens by their bound, 3,599 rows. The same pages as from two calls with close bounds."""
    import torch
    heads, page, B, n = 4, 64, 600, 3000
    counts = [1] * B
    counts[411] = n
    cu = np.cumsum([0] + counts)
    P = [(7 * b) % 100 for b in range(B)]
    P[411] = 5
    pages = [(p + c - 1) // page + 1 for p, c in zip(P, counts)]
    first = np.cumsum([0] + pages)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    for b in range(B):
        table[b, :pages[b]] = torch.arange(int(first[b]), int(first[b + 1]))
    N = int(cu[-1])
    kv, pe = normal(1, N, heads, 256), normal(2, N, 64)
    worlds = []
    for split in (False, True):
        t = m.alloc_paged_cache(int(first[-1]), page, heads)
        t["table"] = table.cuda()
        cache = m.make_paged_cache(t)
        for T, mine in (((32768, range(B)),) if not split else ((n, [411]), (1, [b for b in range(B) if b != 411]))):
            ws = m.alloc_workspace(m.MODE_PAGED_APPEND, B, T)
            now = [P[b] if b in set(mine) else -1 for b in range(B)]
            k = [counts[b] if b in set(mine) else 0 for b in range(B)]
            rows = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in mine])
            r = torch.from_numpy(rows).cuda()
            m.mla_paged_append(cache, kv[r][..., :128], kv[r][..., 128:], pe[r], ints(now), T, ws,
                               cu=ints(list(np.cumsum([0] + k))))
            assert m.mla_device_status(ws) == 0
        worlds.append(t)
    for name in m.PAGED_TENSORS:
        assert torch.equal(worlds[0][name], worlds[1][name]), name
