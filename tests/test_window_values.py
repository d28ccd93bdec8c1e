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
