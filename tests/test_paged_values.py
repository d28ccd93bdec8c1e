"""The paged 8-bit cache at values that its own append does not make, or makes seldom: scales of other quantizers,
pages whose scale no visible key needs, long contexts of small weights, far positions.

References in 64 bits, from the definitions in include/mla.h.  Tolerances count roundings: a value rounded to nearest
in bf16 is off by at most 2^-8 of it, in float16 by 2^-11 (eps/2 of the type)."""

import numpy as np
import pytest

import mla_gb300 as m
from test_paged import f64, ints, normal

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
