"""Attention under a sliding window at scores of -infinity, and against the causal attention.

Tolerances count roundings: the output's to bf16 is off by at most 2^-8 of it, each probability's by 2^-8 p, i.e. the
output by 2^-8 sum p |v| more; float32 scores, exponentials and sums by 2^-14 of that sum."""
import math

import numpy as np
import pytest

import mla_gb300 as m
from test_paged import f64, normal

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("T,P0,window,sinks,keys", [
    (256, 0, 2, 0, [254]), (300, 40, 3, 1, [0]), (200, 300, 130, 2, [0, 1]), (140, 260, 64, 0, list(range(250, 330))),
    (130, 0, 200, 0, [0, 1, 2])])
def test_scores_of_minus_infinity(gpu_available, T, P0, window, sinks, keys):
    """Visible keys that score -infinity have weight zero, also where a row sees nothing else of its first key tile
    (or, further on, of any but its last)."""
    import torch
    L = P0 + T
    q, k, v = normal(1, 1, T, 64 * 192), normal(2, 1, 64, L, 192), normal(3, 1, 64, L, 128)
    q[0].view(T, 64, 192)[..., 7] = 1.0
    k[0, :, keys, 7] = -math.inf
    out = torch.full((1, T, 64 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = m.alloc_workspace(m.MODE_WINDOW_ATTN, 1, T)
    m.mla_window_attention(q, P0, k, v, out, ws, window=window, sinks=sinks)
    assert m.mla_device_status(ws) == 0
    got, qn = f64(out).reshape(T, 64, 128), f64(q).reshape(T, 64, 192)
    i, j = np.arange(P0, L)[:, None], np.arange(L)[None, :]
    seen = (j <= i) & ((i - j < window) | (j < sinks))
    seen[:, keys] = False
    some = seen.any(1)                  # a row that sees only such keys has no answer
    assert some.sum() > T // 2
    kf = f64(k[0])
    kf[:, keys, 7] = 0
    for h in (0, 13, 63):
        s = np.where(seen, qn[:, h] @ kf[h].T / math.sqrt(192), -np.inf)[some]
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        vh = f64(v[0, h])
        ref, A = w @ vh, w @ np.abs(vh)
        d = np.abs(got[some, h] - ref)
        assert np.all(d <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -14) * A), (h, np.nanmax(d))


@gpu
@pytest.mark.parametrize("B,T,P0,page", [(2, 300, 0, 64), (1, 200, 150, 16)])
def test_window_that_holds_every_key_against_the_causal_kernel(gpu_available, B, T, P0, page):
    """mla_prefill_paged without a window runs the causal kernel; under a window of every key it runs the windowed one,
    which sums a row in two halves: the same output within the sublayer's bounds, and the same pages."""
    import torch
    from mla_testlib import cuda_to_f64, cuda_weights, parity, parity_out
    W, outs, deltas, pages = m.make_weights(cuda_weights(0)), [], [], []
    x0, x = normal(1, B, max(P0, 1), 7168), normal(2, B, T, 7168)
    n = -(-(P0 + T) // page)
    for window, sinks in ((0, 0), (P0 + T, 0), (3, P0 + T)):
        t = m.alloc_paged_cache(B * n, page)
        t["table"] = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n)
        cache = m.make_paged_cache(t)
        ws = m.alloc_workspace(m.MODE_PREFILL_PAGED, B, max(T, P0), cap=P0 + T)
        if P0:
            m.mla_prefill_paged(W, x0, 0, cache, torch.empty_like(x0), ws)
        out, delta = torch.empty_like(x), torch.empty((B * T, 7168), dtype=torch.float32, device="cuda")
        m.mla_prefill_paged(W, x, P0, cache, out, ws, window=window, sinks=sinks, params=m.make_params(delta_out=delta))
        assert m.mla_device_status(ws) == 0
        outs.append(out)
        deltas.append(delta)
        pages.append([t[name].clone() for name in m.PAGED_TENSORS])
    for i, what in ((1, "by the window"), (2, "by the sinks")):
        parity_out(cuda_to_f64(outs[i]), cuda_to_f64(outs[0]), f"out, every key seen {what}")
        parity(cuda_to_f64(deltas[i]), cuda_to_f64(deltas[0]), f"Delta, every key seen {what}")
    for other in pages[1:]:
        assert all(torch.equal(a, b) for a, b in zip(other, pages[0]))


@gpu
@pytest.mark.parametrize("T,P0,window,sinks,page", [(130, 600, 90, 5, 64), (40, 333, 20, 150, 16), (300, 200, 7, 0, 128),
                                                    (5, 700, 1, 1, 32)])
def test_prefill_over_pages_needs_nothing_of_its_workspace(gpu_available, T, P0, window, sinks, page):
    """The cached positions that no query sees are not expanded: whatever the workspace holds in their place (NaN here)
    does not reach the output."""
    import torch
    from mla_testlib import cuda_weights
    W, B = m.make_weights(cuda_weights(0)), 2
    x0, x = normal(1, B, P0, 7168), normal(2, B, T, 7168)
    n = -(-(P0 + T) // page)
    outs = []
    for fill in (0, 255):
        t = m.alloc_paged_cache(B * n, page)
        t["table"] = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n)
        cache = m.make_paged_cache(t)
        m.mla_prefill_paged(W, x0, 0, cache, torch.empty_like(x0),
                            m.alloc_workspace(m.MODE_PREFILL_PAGED, B, P0, cap=P0))
        ws = m.alloc_workspace(m.MODE_PREFILL_PAGED, B, T, cap=P0 + T).fill_(fill)
        out = torch.empty_like(x)
        m.mla_prefill_paged(W, x, P0, cache, out, ws, window=window, sinks=sinks)
        assert m.mla_device_status(ws) == 0
        outs.append(out)
    assert bool(torch.isfinite(outs[0]).all()) and torch.equal(outs[0], outs[1])
