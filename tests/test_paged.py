"""The paged 8-bit cache: appending, attention over it, attention under a
sliding window, and the sublayer steps that use them.

References in 64 bits, written from the definitions in include/mla.h.
Tolerances count roundings (eps/2 relative to the rounded value):
- append: scales and codes are equal, bit for bit (power-of-two scaling is
  exact, so code = RNE(x / scale) has one answer; the reference rounds with
  torch's float64 -> float8 conversion of a value that float32 holds exactly).
  Rotary keys: two bf16 products and a sum in float32 of float32 cosines,
  rounded to bf16: 2^-8 |y| for the rounding and 2^-20 (|x1| + |x2|) for the
  float32 arithmetic.
- paged attention: out is rounded to bf16 (2^-8 |o|).  Each weight is rounded
  to float16, w (1 + d) with |d| <= 2^-11, and the output is sum w v / sum w
  with weights summing to one: off by at most 2^-11 max |v|.  The rest is
  float32: 2^-16 of the largest |v| seen by the row.  Together 2^-11 + 2^-16.
- window attention: as above, and the probabilities are rounded to bf16 while
  their sum is not: each product is off by 2^-9 p |v|, so the output by at
  most 2^-9 max |v| (the weights sum to one).
"""
import ctypes
import math

import numpy as np
import pytest

import mla_gb300 as m

FAKE = 1 << 40
gpu = pytest.mark.gpu
E4M3 = "float8_e4m3fn"


# ---- refusals (CPU: nothing is enqueued) --------------------------------------------------------------------
def fake_cache(**kw):
    v = dict(k_codes=FAKE, v_codes=FAKE + (1 << 20), k_pe=FAKE + (2 << 20), k_scales=FAKE + (3 << 20),
             v_scales=FAKE + (4 << 20), table=FAKE + (5 << 20), n_pages=8, max_pages=4, page=64, heads=64)
    v.update(kw)
    return m.MlaPagedCache(*[v[n] for n in ("k_codes", "v_codes", "k_pe", "k_scales", "v_scales", "table", "n_pages",
                                            "max_pages", "page", "heads")])


BAD_CACHES = [(dict(k_codes=None), -1), (dict(v_scales=None), -1), (dict(table=None), -1), (dict(n_pages=0), -1),
              (dict(max_pages=0), -1), (dict(v_codes=FAKE + 8), -2), (dict(k_scales=FAKE + 4), -2),
              (dict(table=FAKE + 2), -2), (dict(page=48), -4), (dict(page=8), -4), (dict(page=256), -4),
              (dict(heads=6), -4), (dict(heads=0), -4), (dict(heads=132), -4), (dict(n_pages=1 << 27), -4)]


def append(cache=None, **kw):
    a = dict(k=FAKE, kt=64 * 256, kh=256, v=FAKE + 256, vt=64 * 256, vh=256, pe=FAKE + 4096, pt=64, P=FAKE + 8192,
             cu=None, B=2, T=3, N=6, ws=FAKE + (9 << 20), wsb=None, params=None)
    a.update(kw)
    if a["wsb"] is None:
        a["wsb"] = max(m.lib().mla_workspace_size(m.MODE_PAGED_APPEND, max(a["B"], 1), max(a["T"], 1), 0), 1)
    c = cache or fake_cache()
    return m.lib().mla_paged_append(ctypes.byref(c), a["params"], a["k"], a["kt"], a["kh"], a["v"], a["vt"], a["vh"],
                                    a["pe"], a["pt"], a["P"], a["cu"], a["B"], a["T"], a["N"], a["ws"], a["wsb"],
                                    None)


def attend(cache=None, **kw):
    a = dict(q=FAKE, qr=64 * 192, B=2, T=1, P=FAKE + 8192, P_max=100, window=0, sinks=0, out=FAKE + (7 << 20),
             outr=64 * 128, ws=FAKE + (9 << 20), wsb=None, params=None)
    a.update(kw)
    if a["wsb"] is None:
        a["wsb"] = m.lib().mla_workspace_size(m.MODE_PAGED_ATTN, 2, 8, 0)
    c = cache or fake_cache()
    return m.lib().mla_paged_attention(ctypes.byref(c), a["params"], a["q"], a["qr"], a["B"], a["T"], a["P"],
                                       a["P_max"], a["window"], a["sinks"], a["out"], a["outr"], a["ws"], a["wsb"],
                                       None)


@pytest.mark.parametrize("over,rc", BAD_CACHES)
def test_bad_caches_are_refused(over, rc):
    assert append(fake_cache(**over)) == rc
    assert attend(fake_cache(**over)) == rc


def test_tables_that_pass_31_bits_are_refused():
    """positions (and a call's tokens behind the last one) are counted in 32-bit ints"""
    for over in (dict(max_pages=(1 << 24) + 1), dict(max_pages=(1 << 27) + 1, page=16), dict(max_pages=(1 << 31) - 1)):
        assert append(fake_cache(**over)) == -4
        assert attend(fake_cache(**over)) == -4
    assert append(fake_cache(max_pages=1 << 24), wsb=16) == -3  # 2^30 positions: the next check speaks


def test_append_refusals():
    L = m.lib()
    for kw in (dict(k=None), dict(v=None), dict(pe=None), dict(P=None), dict(B=0), dict(T=0), dict(N=0), dict(N=5),
               dict(N=(1 << 24) + 1), dict(kt=12), dict(vh=-256), dict(pt=4)):
        assert append(**kw) == -1, kw
    for kw in (dict(k=FAKE + 2), dict(v=FAKE + 8), dict(pe=FAKE + 2), dict(P=FAKE + 2), dict(cu=FAKE + 1),
               dict(ws=FAKE + 8)):
        assert append(**kw) == -2, kw
    assert append(ws=None) == -3 and append(wsb=16) == -3
    bad = m.MlaParams(1e-6, 0.5, 0.07, None, None)
    assert append(params=ctypes.byref(bad)) == -1
    assert L.mla_paged_append(None, None, FAKE, 0, 0, FAKE, 0, 0, FAKE, 0, FAKE, None, 1, 1, 1, FAKE, 4096, None) == -1


def test_attention_refusals():
    for kw in (dict(q=None), dict(out=None), dict(P=None), dict(B=0), dict(T=0), dict(P_max=-1), dict(P_max=256),
               dict(P_max=255, T=2), dict(window=-1), dict(sinks=-1, window=4), dict(qr=64 * 192 - 8),
               dict(qr=64 * 192 + 4), dict(outr=64 * 128 - 8)):
        assert attend(**kw) == -1, kw
    assert attend(T=9) == -4
    for kw in (dict(q=FAKE + 2), dict(out=FAKE + 8), dict(P=FAKE + 1), dict(ws=FAKE + 8)):
        assert attend(**kw) == -2, kw
    assert attend(ws=None) == -3 and attend(wsb=16) == -3


def test_window_attention_refusals():
    L = m.lib()

    def win(**kw):
        a = dict(q=FAKE, B=1, T=16, P0=8, k=FAKE + (1 << 20), v=FAKE + (2 << 20), cap=64, window=4, sinks=2,
                 out=FAKE + (3 << 20), ws=FAKE + (4 << 20), wsb=1 << 16)
        a.update(kw)
        return L.mla_window_attention(None, a["q"], a["B"], a["T"], a["P0"], a["k"], a["v"], a["cap"], a["window"],
                                      a["sinks"], a["out"], a["ws"], a["wsb"], None)

    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(B=0), dict(T=0), dict(P0=-1),
               dict(cap=23), dict(window=0), dict(sinks=-1)):
        assert win(**kw) == -1, kw
    for kw in (dict(q=FAKE + 2), dict(k=FAKE + 8), dict(v=FAKE + 8), dict(out=FAKE + 8), dict(ws=FAKE + 8)):
        assert win(**kw) == -2, kw
    assert win(ws=None) == -3 and win(wsb=16) == -3


def test_workspace_sizes():
    L = m.lib()
    assert 0 < m.workspace_size(m.MODE_PAGED_APPEND, 4, 100) <= m.workspace_size(m.MODE_PAGED_ATTN, 4, 1)
    assert m.workspace_size(m.MODE_PAGED_ATTN, 4, 8) > m.workspace_size(m.MODE_PAGED_ATTN, 4, 1)
    for mode, B, T in ((8, 0, 1), (8, 1, 0), (9, 1, 9), (9, 1, 0), (10, 1, 0)):
        assert L.mla_workspace_size(mode, B, T, 0) == 0


def test_binding_refuses_wrong_tensors():
    import torch
    t = {n: x for n, x in m.alloc_paged_cache(2, 16, 4, device="cpu").items()}
    t["table"] = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        m.make_paged_cache(t)  # not CUDA tensors
    m.make_params()
    x = torch.zeros((3, 4, 128), dtype=torch.bfloat16)
    c = fake_cache(heads=4, page=16)
    c._ref, c._device, c._batch = ctypes.byref(c), x.get_device(), 1
    for f in (lambda: m.mla_paged_append(c, x, x, x[:, 0, :64], x, 3, x),
              lambda: m.mla_paged_attention(c, x, x, 0, x, x),
              lambda: m.mla_window_attention(x, 0, x, x, x, x, 4)):
        with pytest.raises(ValueError):
            f()  # CPU tensors


@gpu
def test_binding_refuses_wrong_shapes_types_and_devices(gpu_available):
    import torch
    t = new_cache(4, 16, 4, [[0, 1], [2, 3]], 1, garbage=False)
    for n, bad in (("k_codes", t["k_codes"].to(torch.int8)), ("k_pe", t["k_pe"][:, :8]), ("table", t["table"][0]),
                   ("v_scales", t["v_scales"].cpu()), ("table", t["table"].long())):
        with pytest.raises(ValueError):
            m.make_paged_cache({**t, n: bad})
    c = m.make_paged_cache(t)
    k, pe, P, cu = normal(1, 6, 4, 128), normal(2, 6, 64), ints([0, 0]), ints([0, 2, 6])
    ws = m.alloc_workspace(m.MODE_PAGED_ATTN, 2, 4)
    good = dict(k=k, v=k, k_pe=pe, P=P, T=4, workspace=ws, cu=cu)
    m.mla_paged_append(c, **good)
    for over in (dict(k=k[:5]), dict(k=k.float()), dict(v=k[:, :3]), dict(v=k.cpu()), dict(k_pe=pe[:5]),
                 dict(k_pe=pe[:, :32]), dict(P=P.long()), dict(P=P[:1]), dict(cu=cu[:2]), dict(P=P.cpu()),
                 dict(workspace=ws.cpu()), dict(v=k.transpose(1, 2)), dict(P=ints([0, 0, 0, 0])[::2])):
        with pytest.raises(ValueError):
            m.mla_paged_append(c, **{**good, **over})
    q, out = normal(3, 2, 4 * 192), normal(4, 2, 4 * 128)
    good = dict(q=q, P=P, P_max=5, out=out, workspace=ws)
    m.mla_paged_attention(c, **good)
    for over in (dict(q=q[:1]), dict(q=q.half()), dict(q=q[:, :-8]), dict(out=out[:1]), dict(out=out.t()),
                 dict(out=out.cpu()), dict(P=P.float()), dict(workspace=ws[::2])):
        with pytest.raises(ValueError):
            m.mla_paged_attention(c, **{**good, **over})
    with pytest.raises(m.MlaError) as e:
        m.mla_paged_attention(c, q, P, 32, out, ws)
    assert e.value.status == -1


# ---- references -------------------------------------------------------------------------------------------
def new_cache(n_pages, page, heads, table, seed, garbage=True):
    """A cache whose unused slots hold anything, NaN codes among it (garbage), like memory that was never written."""
    import torch
    t = m.alloc_paged_cache(n_pages, page, heads)
    if garbage:
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        for n in ("k_codes", "v_codes"):
            t[n].random_(0, 256, generator=g)
            t[n][..., 5] = 0x7F
        t["k_pe"].fill_(float("nan"))
        t["k_scales"].fill_(float("nan"))
        t["v_scales"].fill_(float("nan"))
    t["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    return t


def shuffled_table(lengths, page, seed, extra=1):
    rng = np.random.RandomState(seed)
    n = [max(1, -(-x // page)) for x in lengths]
    ids = rng.permutation(sum(n) + extra)
    wide, at, table = max(n), 0, []
    for k in n:
        table.append(list(ids[at:at + k]) + [-1] * (wide - k))
        at += k
    return table, sum(n) + extra


def block_exp(top):
    if not top > 0:
        return -60
    return int(min(60, max(-60, math.ceil(math.log2(top / 448.0)))))


def to_code(x):
    """float64 numpy -> E4M3 values (saturating), as float64"""
    import torch
    y = torch.from_numpy(np.ascontiguousarray(np.clip(x, -448, 448))).to(torch.float32)
    return y.to(torch.float8_e4m3fn).to(torch.float64).numpy()


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def ref_append(state, k, v, pe, P, Ts, rows, page, base=10000.0):
    """state: {"k": values/scale f64 [pages, H, page, 128], "v", "ks", "vs": scale exponents, "pe"}; in place."""
    theta = base ** (-2.0 * np.arange(32) / 64)
    for b, (p, n) in enumerate(zip(P, Ts)):
        if p < 0:
            continue
        for pi in range(p // page, (p + n - 1) // page + 1 if n else p // page):
            lo, hi = max(p, pi * page), min(p + n, (pi + 1) * page)
            pid, slot = state["table"][b][pi], lo - pi * page
            r0 = rows[b] + lo - p
            for name, x in (("k", k), ("v", v)):
                new = x[r0:r0 + hi - lo]                       # [n, H, 128]
                for h in range(new.shape[1]):
                    e = block_exp(np.nanmax(np.abs(new[:, h]), initial=0.0))
                    if slot:
                        old = state[name + "s"][pid, h]
                        e = max(e, old)
                        state[name][pid, h, :slot] = to_code(state[name][pid, h, :slot] * 2.0 ** (old - e))
                    state[name + "s"][pid, h] = e
                    state[name][pid, h, slot:slot + hi - lo] = to_code(new[:, h] * 2.0 ** -e)
            ang = np.arange(lo, hi)[:, None] * theta
            x1, x2 = pe[r0:r0 + hi - lo, :32], pe[r0:r0 + hi - lo, 32:]
            c, s = np.cos(ang), np.sin(ang)
            state["pe"][pid, slot:slot + hi - lo] = np.concatenate([x1 * c - x2 * s, x2 * c + x1 * s], 1)
            state["mag"][pid, slot:slot + hi - lo] = np.tile(np.abs(x1) + np.abs(x2), (1, 2))


def state_of(t):
    import torch
    with np.errstate(all="ignore"):
        ex = {n: np.nan_to_num(np.round(np.log2(f64(t[n + "_scales"])))) for n in "kv"}
    pe = f64(t["k_pe"])
    return {"k": f64(t["k_codes"].view(torch.float8_e4m3fn)), "v": f64(t["v_codes"].view(torch.float8_e4m3fn)),
            "ks": ex["k"], "vs": ex["v"], "pe": pe, "mag": np.zeros_like(pe), "table": t["table"].cpu().tolist()}


def same(a, b):
    return bool(np.all((a == b) | (np.isnan(a) & np.isnan(b))))


def check_append(t, before, st, what):
    """t: the device's cache; before: its state before the call; st: the reference's after it."""
    now = state_of(t)
    for n in "kv":
        assert same(now[n], st[n]), f"{what}: {n} codes"
        assert same(now[n + "s"], st[n + "s"]), f"{what}: {n} scales"
    touched = st["mag"] > 0
    assert same(now["pe"][~touched], before["pe"][~touched]), f"{what}: rotary keys that nothing was appended to"
    d = np.abs(now["pe"] - st["pe"])[touched]
    assert np.all(d <= 2.0 ** -8 * np.abs(st["pe"][touched]) + 2.0 ** -20 * st["mag"][touched]), f"{what}: rotary keys"


def ref_attend(t, q, P, T, window, sinks, scale=1 / math.sqrt(192)):
    """[B*T, H, 128] in 64 bits, and the largest |v| that each row sees."""
    import torch
    heads, page = t["k_codes"].shape[1], t["k_codes"].shape[2]
    table, qn = t["table"].cpu().numpy(), f64(q).reshape(len(P), T, heads, 192)
    out, vmax = np.zeros((len(P), T, heads, 128)), np.zeros((len(P), T, 1, 1))
    for b, p in enumerate(P):
        for i in range(T):
            if p < 0:
                continue
            j = np.array([x for x in range(p + i + 1) if not window or p + i - x < window or x < sinks])
            pid = torch.from_numpy(table[b][j // page].astype(np.int64)).cuda()
            slot = torch.from_numpy(j % page).cuda()
            k = f64(t["k_codes"][pid, :, slot].view(torch.float8_e4m3fn)) * f64(t["k_scales"][pid])[..., None]
            v = f64(t["v_codes"][pid, :, slot].view(torch.float8_e4m3fn)) * f64(t["v_scales"][pid])[..., None]
            s = np.einsum("hd,jhd->jh", qn[b, i, :, :128], k) + f64(t["k_pe"][pid, slot]) @ qn[b, i, :, 128:].T
            w = np.exp((s - s.max(0)) * scale)
            out[b, i] = np.einsum("jh,jhd->hd", w / w.sum(0), v)
            vmax[b, i] = np.abs(v).max()
    return out.reshape(-1, heads, 128), np.broadcast_to(vmax, out.shape).reshape(-1, heads, 128)


def check_out(got, ref, vmax, what, slack=2.0 ** -11 + 2.0 ** -16):
    d, bound = np.abs(f64(got).reshape(ref.shape) - ref), 2.0 ** -8 * np.abs(ref) + slack * vmax
    assert np.all(np.isfinite(f64(got))), f"{what}: not finite"
    assert np.all(d <= bound), f"{what}: off by {np.max(d - bound):.3e} more than allowed at {np.argmax(d - bound)}"


def normal(seed, *shape, scale=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g) * scale).to(torch.bfloat16)


def ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- append ---------------------------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [4, 12, 64])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 150])
def test_append_matches_reference(gpu_available, page, heads, T):
    """Uniform batches that start on a page, inside one, and for an idle sequence; then a second append on top."""
    import torch
    if heads == 64 and T == 150 and page != 64:
        pytest.skip("the reference takes long; covered at fewer heads")
    P = [0, page, 5, -1, 2 * page - 1]
    table, n_pages = shuffled_table([p + 2 * T if p >= 0 else 1 for p in P], page, 3)
    t = new_cache(n_pages, page, heads, table, 5)
    # what sequences 1, 2 and 4 hold already: finite codes and scales
    for b, p in enumerate(P):
        for pi in range(-(-max(p, 0) // page)):
            pid = table[b][pi]
            for n in ("k", "v"):
                t[n + "_codes"][pid, :, :, 5] = 0x30
                t[n + "_codes"][pid] &= 0xF7          # no NaN
                t[n + "_scales"][pid] = 2.0 ** (-3 + (pid + b) % 4)
    cache = m.make_paged_cache(t)
    ws = m.alloc_workspace(m.MODE_PAGED_APPEND, len(P), T)
    for step in range(2):
        kv = normal(17 + step, len(P) * T, heads, 256, scale=3.0 ** step)
        pe = normal(19 + step, len(P) * T, 576)
        now = [p + step * T if p >= 0 else -1 for p in P]
        before, st = state_of(t), state_of(t)
        ref_append(st, f64(kv[..., :128]), f64(kv[..., 128:]), f64(pe[:, 512:]), now, [T] * len(P),
                   [b * T for b in range(len(P))], page)
        m.mla_paged_append(cache, kv[..., :128], kv[..., 128:], pe[:, 512:], ints(now), T, ws)
        assert m.mla_device_status(ws) == 0
        check_append(t, before, st, f"page {page} heads {heads} T {T} step {step}")


@gpu
@pytest.mark.parametrize("page,base", [(16, 10000.0), (64, 500000.0), (128, 10000.0)])
def test_append_ragged(gpu_available, page, base):
    """Rows of different counts, none among them, one that fills a page to its end, rows behind the last one."""
    import torch
    heads, P = 8, [3, 0, page - 1, 70001, -1, 40]
    Ts = [1, 0, page + 1, 33, 5, page - 40 % page]
    table, n_pages = shuffled_table([p + n for p, n in zip(P, Ts)], page, 4)
    t = new_cache(n_pages, page, heads, table, 6, garbage=False)
    cache = m.make_paged_cache(t)
    cu = np.cumsum([0] + Ts)
    N = int(cu[-1]) + 7
    k, v, pe = normal(1, N, heads, 128), normal(2, heads, N, 128).transpose(0, 1), normal(3, N, 64)
    before, st = state_of(t), state_of(t)
    ref_append(st, f64(k), f64(v), f64(pe), P, Ts, list(cu[:-1]), page, base)
    ws = m.alloc_workspace(m.MODE_PAGED_APPEND, len(P), max(Ts))
    m.mla_paged_append(cache, k, v, pe, ints(P), max(Ts), ws, cu=ints(list(cu)), params=m.make_params(rope_base=base))
    assert m.mla_device_status(ws) == 0
    check_append(t, before, st, f"ragged page {page}")


@gpu
def test_append_special_values(gpu_available):
    """Zeros take the smallest scale, tiny and huge values the ends of its range, NaN stays, infinity saturates."""
    import torch
    heads, page = 4, 16
    t = new_cache(3, page, heads, [[2, 0]], 1, garbage=False)
    cache, ws = m.make_paged_cache(t), m.alloc_workspace(m.MODE_PAGED_APPEND, 1, 4)
    k = torch.zeros((4, heads, 128), dtype=torch.bfloat16, device="cuda")
    k[:, 1] = 1e-30
    k[:, 2] = 3e38
    k[1, 3, 7], k[2, 3, 9] = float("nan"), 448.0
    v = k.clone()
    v[3, 0, 0], v[0, 1, 1] = float("inf"), 449.0     # 449 rounds to 448 in bf16: still 2^0
    m.mla_paged_append(cache, k, v, k[:, 0, :64], ints([0]), 4, ws)
    assert m.mla_device_status(ws) == 0
    ks, vs = f64(t["k_scales"][2]), f64(t["v_scales"][2])
    assert list(ks) == [2.0 ** -60, 2.0 ** -60, 2.0 ** 60, 1.0] and list(vs) == [2.0 ** 60, 1.0, 2.0 ** 60, 1.0]
    kc = f64(t["k_codes"].view(torch.float8_e4m3fn))[2]
    assert np.all(kc[0, :4] == 0) and np.all(kc[1, :4] == 0) and np.all(kc[2, :4] == 448)
    assert np.isnan(kc[3, 1, 7]) and kc[3, 2, 9] == 448 and np.isnan(kc).sum() == 1
    vc = f64(t["v_codes"].view(torch.float8_e4m3fn))[2]
    assert vc[0, 3, 0] == 448 and vc[1, 0, 1] == 448


@gpu
def test_append_skips_and_reports_bad_arguments_on_the_device(gpu_available):
    """Positions, row offsets and page numbers that only the kernel sees: the sequence or page is skipped and the
    call reports it; the others are appended."""
    import torch
    heads, page = 4, 16
    k, pe = normal(1, 8, heads, 128), normal(2, 8, 64)
    for P, cu, table in (([-2, 0], [0, 4, 8], [[0, 1], [2, 3]]), ([30, 0], [0, 4, 8], [[0, 1], [2, 3]]),
                         ([0, 0], [4, 4, 9], [[0, 1], [2, 3]]), ([0, 0], [5, 4, 8], [[0, 1], [2, 3]]),
                         ([0, 0], [0, 4, 8], [[7, 1], [2, 3]]), ([0, 0], [0, 4, 8], [[-1, 1], [2, 3]])):
        t = new_cache(4, page, heads, table, 1, garbage=False)
        cache, ws = m.make_paged_cache(t), m.alloc_workspace(m.MODE_PAGED_APPEND, 2, 4)
        before = state_of(t)
        m.mla_paged_append(cache, k, k, pe, ints(P), 4, ws, cu=ints(cu))
        assert m.mla_device_status(ws) == -1
        now = state_of(t)
        assert same(now["k"][[0, 1, 3]], before["k"][[0, 1, 3]])
        good = cu[2] <= 8 and cu[2] - cu[1] == 4
        assert same(now["k"][2], before["k"][2]) == (not good)


# ---- attention over the pages ------------------------------------------------------------------------------
def filled(P, T, page, heads, seed, table=None, spread=2):
    """A cache that holds positions 0 .. P + T - 1 of each sequence; everything else is garbage."""
    import torch
    lengths = [p + T if p >= 0 else 0 for p in P]
    tab, n_pages = shuffled_table(lengths, page, seed)
    t = new_cache(n_pages, page, heads, tab, seed)
    cache = m.make_paged_cache(t)
    n = sum(lengths)
    if n:
        size = torch.exp2(torch.randint(-spread, spread + 1, (n, 1, 1), device="cuda",
                                        generator=torch.Generator(device="cuda").manual_seed(seed)).float())
        kv = (normal(seed, n, heads, 256).float() * size).to(torch.bfloat16)
        cu = np.cumsum([0] + lengths)
        ws = m.alloc_workspace(m.MODE_PAGED_APPEND, len(P), max(max(lengths), 1))
        m.mla_paged_append(cache, kv[..., :128], kv[..., 128:], normal(seed + 1, n, 64), ints([0] * len(P)),
                           max(max(lengths), 1), ws, cu=ints(list(cu)))
        assert m.mla_device_status(ws) == 0
    return t, cache


ATTEND = [  # P, T, page, heads, window, sinks
    ([0], 1, 16, 4, 0, 0), ([0, -1, 1], 1, 128, 4, 0, 0), ([62, 63, 64, 65], 1, 64, 8, 0, 0),
    ([15, 16, 31, 127, 128, 500], 1, 16, 12, 0, 0), ([1000, 3, -1, 777], 1, 32, 64, 0, 0),
    ([4000], 1, 128, 4, 0, 0), ([9000, 2], 1, 64, 4, 0, 0), ([0, 5, 200], 8, 16, 4, 0, 0),
    ([61, 130, -1], 4, 64, 8, 0, 0), ([999], 5, 32, 64, 0, 0), ([7, 300, 4000], 1, 16, 4, 1, 0),
    ([7, 300, 1000], 1, 64, 8, 33, 0), ([7, 300, 1000], 1, 16, 8, 100, 3), ([50, 640, 1000], 3, 32, 4, 64, 70),
    ([500, 129], 8, 128, 4, 5, 1), ([2000], 2, 16, 4, 1500, 400), ([300], 1, 64, 4, 10000, 5),
    ([200], 1, 16, 4, 64, 300), ([255, 256, 257], 1, 64, 4, 64, 64), ([100] * 40, 1, 32, 8, 0, 0)]


@gpu
@pytest.mark.parametrize("P,T,page,heads,window,sinks", ATTEND)
def test_attention_matches_reference(gpu_available, P, T, page, heads, window, sinks):
    import torch
    t, cache = filled(P, T, page, heads, 11 + len(P))
    q = normal(23, len(P) * T, heads * 192, scale=1.5)
    out = torch.full((len(P) * T, heads * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = m.alloc_workspace(m.MODE_PAGED_ATTN, len(P), T)
    m.mla_paged_attention(cache, q, ints(P), max(max(P), 0), out, ws, window=window, sinks=sinks)
    assert m.mla_device_status(ws) == 0
    ref, vmax = ref_attend(t, q, P, T, window, sinks)
    check_out(out, ref, vmax, f"P {P} T {T} page {page} heads {heads} window {window} sinks {sinks}")
    assert torch.equal(out, _again(cache, q, P, window, sinks, T)), "the same call twice"


def _again(cache, q, P, window, sinks, T, **kw):
    import torch
    out = torch.empty((q.shape[0], q.shape[1] // 192 * 128), dtype=torch.bfloat16, device="cuda")
    ws = m.alloc_workspace(m.MODE_PAGED_ATTN, len(P), T)
    ws.random_(0, 256)                                  # a workspace is not expected to hold anything
    m.mla_paged_attention(cache, q, ints(P), max(max(P), 0), out, ws, window=window, sinks=sinks, **kw)
    assert m.mla_device_status(ws) == 0
    return out


@gpu
def test_attention_strides_scale_and_untouched_columns(gpu_available):
    """Rows inside wider buffers, a scale of its own, a P_max above every P; columns next to the rows stay."""
    import torch
    P, heads, page = [130, 0, 64], 8, 32
    t, cache = filled(P, 1, page, heads, 3)
    t["table"] = torch.cat([t["table"], torch.full((3, 4), -1, dtype=torch.int32, device="cuda")], 1)
    cache = m.make_paged_cache(t)
    wide = normal(5, 3, heads * 192 + 40)
    q = wide[:, 8:8 + heads * 192]
    buf = torch.full((3, heads * 128 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, 16:16 + heads * 128]
    ws = m.alloc_workspace(m.MODE_PAGED_ATTN, 3, 1)
    m.mla_paged_attention(cache, q, ints(P), 250, out, ws, params=m.make_params(softmax_scale=0.3))
    assert m.mla_device_status(ws) == 0
    ref, vmax = ref_attend(t, q, P, 1, 0, 0, scale=0.3)
    # float32 scores of up to 0.3 * |q||k| ~ 2^8 carry 2^-24 * 2^8 * sqrt(192): covered by the slack below
    check_out(out, ref, vmax, "strided", slack=2.0 ** -11 + 2.0 ** -12)
    assert bool((buf[:, :16] == 7).all()) and bool((buf[:, 16 + heads * 128:] == 7).all())


@gpu
def test_attention_large_scores_and_scales(gpu_available):
    """Pages whose scales lie far apart, and scores whose maximum moves by hundreds along the keys."""
    import torch
    P, heads, page = [700], 4, 16
    t, cache = filled(P, 1, page, heads, 9, spread=0)
    for i, pid in enumerate(t["table"][0].tolist()):
        if pid >= 0:
            t["v_scales"][pid] *= 2.0 ** ((i * 7) % 41 - 20)
            t["k_scales"][pid] *= 2.0 ** (i % 4)
    q = normal(8, 1, heads * 192, scale=8.0)
    ref, vmax = ref_attend(t, q, P, 1, 0, 0)
    # scores reach 2^12; in float32 they are off by up to 2^-24 * 2^12 * a few: weights by 2^-10
    check_out(_again(cache, q, P, 0, 0, 1), ref, vmax, "large", slack=2.0 ** -9 + 2.0 ** -11)


@gpu
def test_attention_reports_bad_arguments_on_the_device(gpu_available):
    """A position above P_max is idle, a bad page number of a visible page is reported; freed pages are not."""
    import torch
    P, heads, page = [100, 40], 4, 16
    t, cache = filled(P, 1, page, heads, 2)
    q = normal(1, 2, heads * 192)
    out = torch.empty((2, heads * 128), dtype=torch.bfloat16, device="cuda")
    ws = m.alloc_workspace(m.MODE_PAGED_ATTN, 2, 1)
    m.mla_paged_attention(cache, q, ints([100, 41]), 40, out, ws)
    assert m.mla_device_status(ws) == -1 and bool((out[0] == 0).all())
    m.mla_paged_attention(cache, q, ints([-7, 40]), 100, out, ws)
    assert m.mla_device_status(ws) == -1 and bool((out[0] == 0).all())
    ref, _ = ref_attend(t, q, P, 1, 20, 3)
    t["table"][0, 1:4] = torch.tensor([-1, 10 ** 6, -5], dtype=torch.int32)   # positions 16..63: passed by the window
    m.mla_paged_attention(cache, q, ints(P), 100, out, ws, window=20, sinks=3)
    assert m.mla_device_status(ws) == 0
    check_out(out, ref, np.full(ref.shape, 16.0), "freed pages")
    m.mla_paged_attention(cache, q, ints(P), 100, out, ws)
    assert m.mla_device_status(ws) == -1


@gpu
def test_append_then_attention_graph_and_streams(gpu_available):
    """Decode steps as a server runs them: append, then attend, captured once and replayed for the next positions
    and a changed table, on a stream of its own, against eager steps; two streams with workspaces of their own."""
    import torch
    heads, page, B, steps = 16, 16, 3, 20
    table, n_pages = shuffled_table([60, 40, 90], page, 1)
    start = [10, 31, 64]
    kv, pe = normal(3, steps, B, heads, 256), normal(4, steps, B, 64)
    q = normal(5, steps, B, heads * 192)

    def world():
        t = new_cache(n_pages, page, heads, table, 8, garbage=False)
        return t, m.make_paged_cache(t), m.alloc_workspace(m.MODE_PAGED_APPEND, B, 1), \
            m.alloc_workspace(m.MODE_PAGED_ATTN, B, 1)

    def step(w, kv, pe, q, P, out):
        m.mla_paged_append(w[1], kv[..., :128], kv[..., 128:], pe, P, 1, w[2])
        m.mla_paged_attention(w[1], q, P, 95, out, w[3])

    eager, outs = world(), []
    for i in range(steps):
        out = torch.empty((B, heads * 128), dtype=torch.bfloat16, device="cuda")
        step(eager, kv[i], pe[i], q[i], ints([s + i if (i + b) % 7 else -1 for b, s in enumerate(start)]), out)
        outs.append(out)
    torch.cuda.synchronize()

    w, x = world(), (kv[0].clone(), pe[0].clone(), q[0].clone(), ints([-1] * B),
                     torch.empty((B, heads * 128), dtype=torch.bfloat16, device="cuda"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(w, *x)
    for i in range(steps):
        with torch.cuda.stream(s):
            for dst, src in zip(x, (kv[i], pe[i], q[i], ints([s0 + i if (i + b) % 7 else -1
                                                              for b, s0 in enumerate(start)]))):
                dst.copy_(src)
            g.replay()
            got = x[4].clone()
        s.synchronize()
        assert torch.equal(got, outs[i]), f"step {i}"
    for n in m.PAGED_TENSORS:
        assert torch.equal(w[0][n], eager[0][n]), n

    # the same steps on two streams at once
    ws = [world(), world()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = [[], []]
    torch.cuda.synchronize()
    for i in range(steps):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                out = torch.empty((B, heads * 128), dtype=torch.bfloat16, device="cuda")
                step(ws[k], kv[i], pe[i], q[i], ints([s0 + i if (i + b) % 7 else -1 for b, s0 in enumerate(start)]),
                     out)
                res[k].append(out)
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(res[k], outs))


@gpu
def test_pages_past_32_bit_offsets(gpu_available):
    """A cache of more than 2^32 bytes of codes: its last pages against the same tokens in the first ones."""
    import torch
    heads, page, P, T = 64, 128, [299, 130], 1
    n_pages = 4400  # 1 MiB of key codes each
    ids = [[n_pages - 1, n_pages - 7, n_pages - 3], [n_pages - 4, n_pages - 2, -1]]
    tables = [ids, [[0, 3, 2], [4, 1, -1]]]
    t = new_cache(n_pages, page, heads, tables[0], 1, garbage=False)
    outs, pages = [], []
    lengths = [p + T for p in P]
    kv, pe, q = normal(1, sum(lengths), heads, 256), normal(2, sum(lengths), 64), normal(3, 2, heads * 192)
    for table in tables:
        t["table"] = ints(table)
        cache = m.make_paged_cache(t)
        ws = m.alloc_workspace(m.MODE_PAGED_APPEND, 2, max(lengths))
        m.mla_paged_append(cache, kv[..., :128], kv[..., 128:], pe, ints([0, 0]), max(lengths), ws,
                           cu=ints([0, lengths[0], sum(lengths)]))
        assert m.mla_device_status(ws) == 0
        outs.append(_again(cache, q, P, 0, 0, T))
        at = t["table"].flatten().clamp_min(0).long()[:5]
        pages.append([t[n][at].clone() for n in m.PAGED_TENSORS])
    assert torch.equal(outs[0], outs[1]) and bool(outs[0].abs().sum() > 0)
    assert all(torch.equal(a, b) for a, b in zip(*pages))
    assert bool((t["k_codes"][100:n_pages - 100] == 0).all()), "pages that belong to nobody"


@gpu
def test_many_short_sequences_and_few_tiles(gpu_available):
    """More sequences than threads of a block, one tile each; and fewer tiles than SMs, some of them cut."""
    import torch
    for P, heads, window in (([i % 7 - 1 for i in range(900)], 4, 0), ([70, -1, 3, 200], 4, 0), ([63] * 3, 8, 9)):
        t, cache = filled(P, 1, 16, heads, 5)
        q = normal(7, len(P), heads * 192)
        out = _again(cache, q, P, window, 0, 1)
        ref, vmax = ref_attend(t, q, P, 1, window, 0)
        check_out(out, ref, vmax, f"{len(P)} sequences")


# ---- window attention over the dense caches ----------------------------------------------------------------
@gpu
@pytest.mark.parametrize("B,T,P0,window,sinks", [
    (1, 1, 0, 1, 0), (1, 1, 200, 64, 3), (2, 17, 0, 5, 0), (1, 128, 0, 128, 0), (1, 129, 0, 1, 0),
    (2, 300, 77, 100, 4), (1, 257, 500, 129, 130), (1, 200, 1000, 1024, 7), (1, 400, 0, 10 ** 9, 0),
    (1, 300, 300, 2, 500), (1, 513, 0, 200, 128), (1, 260, 255, 256, 1)])
def test_window_attention_matches_reference(gpu_available, B, T, P0, window, sinks):
    """Keys that no query of the call sees, and slots behind the last key, hold NaN."""
    import torch
    L, cap = P0 + T, P0 + T + 3
    q, k, v = normal(1, B, T, 64 * 192, scale=1.5), normal(2, B, 64, cap, 192), normal(3, B, 64, cap, 128)
    kr, vr = f64(k), f64(v)
    hidden = [j for j in range(P0) if j < P0 - window + 1 and j >= sinks] + list(range(L, cap))
    if hidden:
        k[:, :, hidden], v[:, :, hidden] = float("nan"), float("nan")
    out = torch.full((B, T, 64 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = m.alloc_workspace(m.MODE_WINDOW_ATTN, B, T)
    m.mla_window_attention(q, P0, k, v, out, ws, window=window, sinks=sinks)
    assert m.mla_device_status(ws) == 0
    got, qn = f64(out).reshape(B, T, 64, 128), f64(q).reshape(B, T, 64, 192)
    i, j = np.arange(P0, L)[:, None], np.arange(L)[None, :]
    seen = (j <= i) & ((i - j < window) | (j < sinks))
    for b in range(B):
        for h in (0, 1, 31, 63):
            s = np.where(seen, qn[b, :, h] @ kr[b, h, :L].T / math.sqrt(192), -np.inf)
            w = np.exp(s - s.max(1, keepdims=True))
            ref = (w / w.sum(1, keepdims=True)) @ vr[b, h, :L]
            vmax = np.abs(vr[b, h, :L]).max()
            d = np.abs(got[b, :, h] - ref)
            # bf16 output, bf16 probabilities (2^-8 p |v| at most over the row), float32 in between
            assert np.all(d <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * vmax), (b, h, d.max())
            assert np.linalg.norm(d) <= 2.0 ** -8 * np.linalg.norm(ref)


@gpu
def test_window_that_holds_every_key_equals_the_causal_attention(gpu_available):
    """window >= P0 + T: the scores of mla_prefill_chunk's attention; here the same tiles in the same order."""
    import torch
    q, k, v = normal(1, 1, 300, 64 * 192), normal(2, 1, 64, 300, 192), normal(3, 1, 64, 300, 128)
    ws = m.alloc_workspace(m.MODE_WINDOW_ATTN, 1, 300)
    outs = []
    for window, sinks in ((300, 0), (2 ** 31 - 1, 0), (300, 2 ** 31 - 1)):
        out = torch.empty((1, 300, 64 * 128), dtype=torch.bfloat16, device="cuda")
        m.mla_window_attention(q, 0, k, v, out, ws, window=window, sinks=sinks)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.gpu
def test_single_rows_with_any_row_stride():
    """the stride of a tensor's only row says nothing: every view of it is taken, with the same results"""
    import torch

    heads, page = 4, 16
    torch.manual_seed(5)
    k, v = (torch.randn(1, heads, 128, device="cuda").bfloat16() for _ in range(2))
    pe, q = torch.randn(1, 64, device="cuda").bfloat16(), torch.randn(1, heads * 192, device="cuda").bfloat16()
    P = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for row in (None, 1, 3):
        def view(x):
            return x if row is None else x.as_strided(x.shape, (row,) + x.stride()[1:])
        t = m.alloc_paged_cache(1, page, heads)
        t["table"] = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        c = m.make_paged_cache(t)
        m.mla_paged_append(c, view(k), view(v), view(pe), P, 1, m.alloc_workspace(m.MODE_PAGED_APPEND, 1, 1))
        out = torch.empty(1, heads * 128, dtype=torch.bfloat16, device="cuda")
        m.mla_paged_attention(c, view(q), P, 0, view(out), m.alloc_workspace(m.MODE_PAGED_ATTN, 1, 1))
        got.append(torch.cat([out.view(-1).view(torch.int16).int(), t["k_codes"].view(-1).int(),
                              t["v_codes"].view(-1).int(), t["k_pe"].view(-1).view(torch.int16).int()]))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    assert got[0].any()


@gpu
@pytest.mark.parametrize("order", ["growing", "falling", "spikes"])
def test_window_attention_moving_maxima(gpu_available, order):
    """Scores whose maximum moves by far more than the rescale threshold from key tile to key tile, in the first or
    the second half of a tile; more items than SMs, so that every CTA takes several."""
    import torch
    B, T, P0, window, sinks, cap = 1, 700, 130, 300, 9, 830
    L = P0 + T
    q, k, v = normal(1, B, T, 64 * 192), normal(2, B, 64, cap, 192), normal(3, B, 64, cap, 128)
    u = normal(4, 192).sign()
    q = (q * 0.25 + u.repeat(64)).bfloat16()  # every query has a part along u
    j = torch.arange(cap, device="cuda")
    along = {"growing": j * 0.02, "falling": (cap - j) * 0.02,
             "spikes": ((j % 97 == 0) * 7.0 + (j % 64 == 63) * 4.0)}[order]
    k = (k * 0.25 + along[None, None, :, None] * u).bfloat16()
    out = torch.full((B, T, 64 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = m.alloc_workspace(m.MODE_WINDOW_ATTN, B, T)
    m.mla_window_attention(q, P0, k, v, out, ws, window=window, sinks=sinks)
    assert m.mla_device_status(ws) == 0
    got, qn, kr, vr = f64(out).reshape(T, 64, 128), f64(q).reshape(T, 64, 192), f64(k)[0], f64(v)[0]
    i, jj = np.arange(P0, L)[:, None], np.arange(L)[None, :]
    seen = (jj <= i) & ((i - jj < window) | (jj < sinks))
    for h in (0, 2, 40, 63):
        s = np.where(seen, qn[:, h] @ kr[h, :L].T / math.sqrt(192), -np.inf)
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        ref, mass = w @ vr[h, :L], w @ np.abs(vr[h, :L])
        # a score: 192 products summed in float32, then scaled and shifted by a maximum of the same size: at most
        # 200 roundings of 2^-24 of the sum of the products' magnitudes, for a key and for the row's sum
        ds = 2 * 200 * 2.0 ** -24 * (np.abs(qn[:, h]) @ np.abs(kr[h, :L]).T).max() / math.sqrt(192)
        d = np.abs(got[:, h] - ref)
        # output 2^-8 |ref|, probabilities 2^-8 of the weighted |v|, the scores' errors on all of it; 1 % for the
        # products of these and the exponential's own 2^-22
        assert np.all(d <= 1.01 * (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + math.expm1(ds)) * mass)), (h, d.max())


@gpu
def test_window_attention_captured_and_on_two_streams(gpu_available):
    """A captured call replayed with new inputs, and two streams at once with workspaces of their own, give the
    eager call's bits."""
    import torch
    B, T, P0, window, sinks = 2, 260, 100, 150, 5
    sets = [(normal(10 * i + 1, B, T, 64 * 192), normal(10 * i + 2, B, 64, P0 + T, 192),
             normal(10 * i + 3, B, 64, P0 + T, 128)) for i in range(4)]

    def run(x, out, ws):
        m.mla_window_attention(x[0], P0, x[1], x[2], out, ws, window=window, sinks=sinks)

    def fresh():
        return torch.empty((B, T, 64 * 128), dtype=torch.bfloat16, device="cuda"), \
            m.alloc_workspace(m.MODE_WINDOW_ATTN, B, T)

    want = []
    for x in sets:
        out, ws = fresh()
        run(x, out, ws)
        want.append(out)
    torch.cuda.synchronize()
    x, (out, ws) = [t.clone() for t in sets[0]], fresh()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run(x, out, ws)
    for i in range(4):
        with torch.cuda.stream(s):
            for dst, src in zip(x, sets[i]):
                dst.copy_(src)
            g.replay()
        s.synchronize()
        assert torch.equal(out, want[i]), i
    streams, res = [torch.cuda.Stream(), torch.cuda.Stream()], []
    own = [fresh() for _ in range(8)]
    torch.cuda.synchronize()
    for i in range(4):
        for n in range(2):
            with torch.cuda.stream(streams[n]):
                run(sets[i], *own[2 * i + n])
                res.append((i, own[2 * i + n][0]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in res)
