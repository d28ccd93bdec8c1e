"""The MLA sublayer over the paged 8-bit cache: prefill into pages, further
chunks, decode steps, against the oracle and against the dense entry points.

The pages' content is compared through the appended values; outputs are held
to the sublayer's parity bounds (max abs 2e-2, relative Frobenius 1e-2) against
the oracle's 64-bit attention over the keys and values that the pages hold.
E4M3 keeps 4 significant bits: a stored value is within 2^-4 of it (relative),
or 2^-10 of the page's scale near zero (half the smallest code, 2^-9).
"""
import ctypes

import numpy as np
import pytest

import synth
import mla_gb300 as m
from mla_testlib import bits_to_cuda, cuda_to_f64, cuda_weights, oracle_weights, parity, parity_out
from oracle import mla_oracle as om

FAKE = 1 << 40
gpu = pytest.mark.gpu


def fake_weights(**override):
    vals = {n: FAKE + 4096 * i for i, n in enumerate(m.WEIGHT_NAMES)}
    vals.update(override)
    return m.MlaWeights(*[vals[n] for n in m.WEIGHT_NAMES])


def fake_cache(**kw):
    v = dict(k_codes=FAKE, v_codes=FAKE + (1 << 20), k_pe=FAKE + (2 << 20), k_scales=FAKE + (3 << 20),
             v_scales=FAKE + (4 << 20), table=FAKE + (5 << 20), n_pages=8, max_pages=4, page=64, heads=64)
    v.update(kw)
    return m.MlaPagedCache(*v.values())


def test_decode_paged_refusals():
    L, w = m.lib(), fake_weights()

    def dec(c=None, weights=w, **kw):
        a = dict(x=FAKE + (1 << 30), B=3, P=FAKE, P_max=100, window=0, sinks=0, out=FAKE + (2 << 30),
                 ws=FAKE + (3 << 30), wsb=L.mla_workspace_size(m.MODE_DECODE_PAGED, 3, 255, 0))
        a.update(kw)
        return L.mla_decode_paged(ctypes.byref(weights), None, a["x"], a["B"], a["P"], a["P_max"],
                                  ctypes.byref(c or fake_cache()), a["window"], a["sinks"], a["out"], a["ws"],
                                  a["wsb"], None)

    assert dec(fake_cache(heads=16)) == -4 and dec(fake_cache(page=24)) == -4 and dec(fake_cache(k_pe=None)) == -1
    for kw in (dict(P=None), dict(B=0), dict(P_max=-1), dict(P_max=256), dict(window=-1), dict(sinks=-1),
               dict(x=None), dict(out=None), dict(out=FAKE + (1 << 30) + 64)):
        assert dec(**kw) == -1, kw
    assert dec(weights=fake_weights(w_o=None)) == -1
    for kw in (dict(P=FAKE + 2), dict(x=FAKE + 8), dict(ws=FAKE + 8)):
        assert dec(**kw) == -2, kw
    assert dec(ws=None) == -3 and dec(wsb=64) == -3


def test_prefill_paged_refusals():
    L, w = m.lib(), fake_weights()

    def pre(c=None, **kw):
        a = dict(x=FAKE + (1 << 30), B=2, T=20, P0=30, window=0, sinks=0, out=FAKE + (2 << 30), ws=FAKE + (3 << 30),
                 wsb=L.mla_workspace_size(m.MODE_PREFILL_PAGED, 2, 20, 300))
        a.update(kw)
        return L.mla_prefill_paged(ctypes.byref(w), None, a["x"], a["B"], a["T"], a["P0"],
                                   ctypes.byref(c or fake_cache()), a["window"], a["sinks"], a["out"], a["ws"],
                                   a["wsb"], None)

    assert pre(fake_cache(heads=32)) == -4 and pre(fake_cache(table=None)) == -1
    for kw in (dict(B=0), dict(T=0), dict(P0=-1), dict(P0=237), dict(window=-1), dict(sinks=-1), dict(x=None),
               dict(out=None), dict(out=FAKE + (1 << 30) + 64)):
        assert pre(**kw) == -1, kw
    assert pre(x=FAKE + 8) == -2 and pre(ws=None) == -3 and pre(wsb=64) == -3


# ---- GPU --------------------------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def W():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m.make_weights(cuda_weights(0)), oracle_weights(0)


def pages(B, positions, page, seed=0):
    """A cache for B sequences of that many positions, pages in random order, filled with NaN."""
    import torch
    n = -(-positions // page)
    rng = np.random.RandomState(seed)
    table = rng.permutation(B * n).reshape(B, n)
    t = m.alloc_paged_cache(B * n, page, 64)
    for x in t.values():
        x.fill_(0x7F if x.dtype == torch.uint8 else float("nan"))
    t["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    return t, m.make_paged_cache(t)


def dense(t, b, n):
    """Positions 0 .. n - 1 of sequence b as the pages hold them: K [64, n, 192], V [64, n, 128], and the scales."""
    import torch
    page = t["k_codes"].shape[2]
    j = torch.arange(n, device="cuda")
    pid, slot = t["table"][b][j // page].long(), j % page

    def get(name):
        s = t[name + "_scales"][pid].double()
        x = t[name + "_codes"][pid, :, slot].view(torch.float8_e4m3fn).double() * s[..., None]
        return x.transpose(0, 1).cpu().numpy(), s.T.cpu().numpy()

    (k, ks), (v, vs) = get("k"), get("v")
    pe = t["k_pe"][pid, slot].double().cpu().numpy()
    return np.concatenate([k, np.broadcast_to(pe, (64, n, 64))], 2), v, ks, vs


def run_prefill(W, t, cache, x, P0, window=0, sinks=0):
    import torch
    B, T = x.shape[:2]
    out = torch.empty_like(x)
    ws = m.alloc_workspace(m.MODE_PREFILL_PAGED, B, T, cap=P0 + T)
    ws.random_(0, 256)
    m.mla_prefill_paged(W[0], x, P0, cache, out, ws, window=window, sinks=sinks)
    assert m.mla_device_status(ws) == 0
    return out


@gpu
@pytest.mark.parametrize("B,T,page", [(1, 300, 64), (2, 150, 16), (1, 17, 128), (3, 129, 32)])
def test_prefill_paged_equals_prefill_and_append(W, B, T, page):
    """Same out as mla_prefill, bit for bit (the same kernels on the same values) where neither call splits K, and
    pages that hold the dense caches' rows as mla_paged_append writes them."""
    import torch
    x = synth.tensor_cuda(3, "x", (B, T, 7168), synth.X_DIST)
    t, cache = pages(B, T + 5, page)
    out = run_prefill(W, t, cache, x, 0)
    ref = torch.empty_like(x)
    kc = torch.empty((B, 64, T, 192), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((B, 64, T, 128), dtype=torch.bfloat16, device="cuda")
    m.mla_prefill(W[0], x, ref, m.alloc_workspace(m.MODE_PREFILL, B, T), kc, vc, cap=T)
    if B * T > 128:
        assert torch.equal(out, ref)
    parity(cuda_to_f64(out), cuda_to_f64(ref), "out against mla_prefill")
    # the dense caches' rows through the public append (rotary keys already rotated: position 0 leaves them)
    t2, cache2 = pages(B, T + 5, page)
    k = kc[..., :128].transpose(1, 2).reshape(B * T, 64, 128).contiguous()
    v = vc.transpose(1, 2).reshape(B * T, 64, 128).contiguous()
    pe = kc[:, 0, :, 128:].reshape(B * T, 64).contiguous()
    m.mla_paged_append(cache2, k, v, pe, torch.zeros(B, dtype=torch.int32, device="cuda"), T,
                       m.alloc_workspace(m.MODE_PAGED_APPEND, B, T))
    if B * T > 128:
        for n in ("k_codes", "v_codes"):
            assert torch.equal(t[n], t2[n]), n
        for n in ("k_scales", "v_scales"):
            assert torch.equal(torch.nan_to_num(t[n]), torch.nan_to_num(t2[n])), n
    for b in range(B):
        K = dense(t, b, T)[0]
        assert np.array_equal(K[0, :, 128:], cuda_to_f64(kc[b, 0, :, 128:].contiguous())), "rotary keys"


@gpu
@pytest.mark.parametrize("B,T,P0,window,sinks,page", [(2, 40, 100, 0, 0, 16), (1, 130, 77, 50, 3, 64),
                                                     (2, 5, 300, 128, 140, 32), (1, 64, 200, 30, 0, 128)])
def test_prefill_paged_chunk_parity(W, B, T, P0, window, sinks, page):
    """A chunk behind cached pages: attention over the quantized past and the chunk's own keys as computed."""
    import torch
    wo = W[1]
    xp = synth.tensor_cuda(5, "cache_x", (B, P0, 7168), synth.X_DIST)
    xb = synth.tensor_bits(6, "x", (B, T, 7168), synth.X_DIST)
    t, cache = pages(B, P0 + T + 3, page, 1)
    run_prefill(W, t, cache, xp, 0)
    past = [dense(t, b, P0) for b in range(B)]
    if window:  # pages that the window has passed are given back
        first = max(0, P0 - window + 1)
        for pi in range(-(-sinks // page), first // page):
            t["table"][:, pi] = -1
    out = run_prefill(W, t, cache, bits_to_cuda(xb), P0, window, sinks)
    x64 = synth.bf16_bits_to_f64(xb)
    pos = np.arange(P0, P0 + T)
    new = om.project_tokens(wo, x64, pos[None, :], om.KIMI_K2, om.DEFAULT_EPS, om.DEFAULT_ROPE_BASE)
    i, j = pos[:, None], np.arange(P0 + T)[None, :]
    seen = (j <= i) & ((i - j < window) | (j < sinks) if window else True)
    O = np.empty((B, T, 64, 128))
    for b in range(B):
        for h in range(64):
            K = np.concatenate([past[b][0][h], new["K"][b, :, h]])
            V = np.concatenate([past[b][1][h], new["V"][b, :, h]])
            s = np.where(seen, new["Q"][b, :, h] @ K.T / np.sqrt(192), -np.inf)
            e = np.exp(s - s.max(1, keepdims=True))
            O[b, :, h] = (e / e.sum(1, keepdims=True)) @ V
    delta = O.reshape(B, T, 8192) @ wo["w_o"].T
    parity_out(cuda_to_f64(out), x64 + delta, "out")


@gpu
@pytest.mark.parametrize("P,page,window,sinks", [([37, 0, -1], 16, 0, 0), ([130, 64, 63, 5], 64, 0, 0),
                                                 ([200, 199, -1, 17], 32, 60, 4)])
def test_decode_paged_parity(W, P, page, window, sinks):
    """One decode step of a ragged batch with idle rows: the new rows of the pages, out, and idle rows untouched."""
    import torch
    wo, B = W[1], len(P)
    top = max(P)
    t, cache = pages(B, top + 4, page, 2)
    past = synth.tensor_cuda(7, "cache_x", (B, max(top, 1), 7168), synth.X_DIST)
    run_prefill(W, t, cache, past, 0)  # positions from P[b] on are overwritten or hidden
    before = {n: t[n].clone() for n in m.PAGED_TENSORS}
    xb = synth.tensor_bits(8, "new_x", (B, 7168), synth.X_DIST)
    x = bits_to_cuda(xb)
    out, delta = torch.empty_like(x), torch.empty((B, 7168), dtype=torch.float32, device="cuda")
    ws = m.alloc_workspace(m.MODE_DECODE_PAGED, B, top + 2)
    ws.random_(0, 256)
    m.mla_decode_paged(W[0], x, torch.tensor(P, dtype=torch.int32, device="cuda"), top + 2, cache, out, ws,
                       window=window, sinks=sinks, params=m.make_params(delta_out=delta))
    assert m.mla_device_status(ws) == 0
    x64 = synth.bf16_bits_to_f64(xb)
    new = om.project_tokens(wo, x64, np.maximum(P, 0), om.KIMI_K2, om.DEFAULT_EPS, om.DEFAULT_ROPE_BASE)
    O = np.zeros((B, 64, 128))
    for b, p in enumerate(P):
        if p < 0:
            for pid in t["table"][b].tolist():
                for n in m.PAGED_TENSORS:
                    a, c = t[n][pid], before[n][pid]
                    assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(c.float())), "idle"
            continue
        K, V, ks, vs = dense(t, b, p + 1)
        for got, ref, s, what in ((K[:, p, :128], new["K"][b, :, :128], ks, "key"), (V[:, p], new["V"][b], vs, "value")):
            # 2^-4 |x| for the code; bf16 of the kv_b product and its float32 sums: 2^-8 |x| + 2e-2 (the cache bound)
            assert np.all(np.abs(got - ref) <= (2.0 ** -4 + 2.0 ** -8) * np.abs(ref) + 2e-2 + 2.0 ** -10 * s[:, p:p + 1]), what
        assert np.all(np.abs(K[0, p, 128:] - new["K"][b, 0, 128:]) <= 2e-2 + 2.0 ** -8 * np.abs(new["K"][b, 0, 128:]))
        j = np.arange(p + 1)
        hide = (p - j >= window) & (j >= sinks) if window else np.zeros(p + 1, bool)
        for h in range(64):
            s = np.where(hide, -np.inf, K[h] @ new["Q"][b, h] / np.sqrt(192))
            e = np.exp(s - s.max())
            O[b, h] = (e / e.sum()) @ V[h]
    ref = O.reshape(B, 8192) @ wo["w_o"].T
    parity(cuda_to_f64(delta), ref, "delta")
    parity_out(cuda_to_f64(out), x64 + ref, "out")
    for b, p in enumerate(P):
        if p < 0:
            assert torch.equal(out[b], x[b]), "idle rows keep x"


@gpu
@pytest.mark.parametrize("B", [65, 130, 300])
def test_decode_paged_larger_batches(W, B):
    """More rows than one tile of the small products: each row as in a batch of its own sequences alone."""
    import torch
    page = 16
    P = [(7 * i) % 33 - 1 for i in range(B)]
    past = synth.tensor_cuda(11, "cache_x", (B, 33, 7168), synth.X_DIST)
    x = synth.tensor_cuda(12, "new_x", (B, 7168), synth.X_DIST)
    t, cache = pages(B, 34, page, 4)
    run_prefill(W, t, cache, past, 0)
    first = {n: t[n].clone() for n in m.PAGED_TENSORS}
    out, delta = torch.empty_like(x), torch.empty((B, 7168), dtype=torch.float32, device="cuda")
    ws = m.alloc_workspace(m.MODE_DECODE_PAGED, B, 32)
    pos = torch.tensor(P, dtype=torch.int32, device="cuda")
    m.mla_decode_paged(W[0], x, pos, 32, cache, out, ws, params=m.make_params(delta_out=delta))
    assert m.mla_device_status(ws) == 0
    for n in m.PAGED_TENSORS:
        t[n].copy_(first[n])
    for lo in range(0, B, 50):
        n = min(50, B - lo)
        part = m.make_paged_cache({**{k: t[k] for k in m.PAGED_TENSORS}, "table": t["table"][lo:lo + n].contiguous()})
        o2, d2 = torch.empty_like(x[:n]), torch.empty((n, 7168), dtype=torch.float32, device="cuda")
        m.mla_decode_paged(W[0], x[lo:lo + n].contiguous(), pos[lo:lo + n].contiguous(), 32, part, o2,
                           m.alloc_workspace(m.MODE_DECODE_PAGED, n, 32), params=m.make_params(delta_out=d2))
        # other tile shapes and K splits: float32 sums in another order, bf16 roundings that may fall the other way
        parity(cuda_to_f64(delta[lo:lo + n]), cuda_to_f64(d2), f"rows from {lo}")


@gpu
def test_decode_paged_steps_equal_their_parts_and_capture(W):
    """Steps of mla_decode_paged, eager and replayed from one captured graph, give the same pages and outputs; a bad
    position is reported and changes nothing."""
    import torch
    B, page = 3, 16
    x = [synth.tensor_cuda(20 + i, "new_x", (B, 7168), synth.X_DIST) for i in range(4)]
    start = torch.tensor([14, 30, 5], dtype=torch.int32, device="cuda")
    past = synth.tensor_cuda(9, "cache_x", (B, 31, 7168), synth.X_DIST)

    def world():
        t, cache = pages(B, 48, page, 3)
        run_prefill(W, t, cache, past, 0)
        return t, cache, m.alloc_workspace(m.MODE_DECODE_PAGED, B, 40)

    t1, c1, w1 = world()
    outs = []
    for i in range(4):
        out = torch.empty_like(x[0])
        m.mla_decode_paged(W[0], x[i], start + i, 40, c1, out, w1)
        outs.append(out)
    torch.cuda.synchronize()
    t2, c2, w2 = world()
    xs, ps, out = x[0].clone(), torch.full_like(start, -1), torch.empty_like(x[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.mla_decode_paged(W[0], xs, ps, 40, c2, out, w2)
    for i in range(4):
        xs.copy_(x[i])
        ps.copy_(start + i)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, outs[i]), i
    for n in m.PAGED_TENSORS:
        assert torch.equal(torch.nan_to_num(t1[n].float()), torch.nan_to_num(t2[n].float())), n
    m.mla_decode_paged(W[0], x[0], torch.tensor([-2, 41, -1], dtype=torch.int32, device="cuda"), 40, c2, out, w2)
    assert m.mla_device_status(w2) == -1
    for n in ("k_codes", "v_codes"):
        assert torch.equal(t1[n], t2[n]), n
