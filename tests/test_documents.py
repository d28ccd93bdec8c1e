"""Attention over packed documents.

The reference is the definition in include/mla.h in 64 bits, document by document.  Tolerances count roundings, as for
the attention under a window: the output's to bf16 is off by at most 2^-8 of it, each probability's (relative to the
row's sum, which is not rounded) by 2^-8 p, i.e. the output by 2^-8 sum p |v| more; float32 scores, exponentials and
sums by 2^-14 of that sum."""
import ctypes
import math

import numpy as np
import pytest

import mla_gb300 as m
from test_paged import FAKE, f64, normal

gpu = pytest.mark.gpu


# ---- refusals (CPU: nothing is enqueued) --------------------------------------------------------------------
def attend_c(**kw):
    a = dict(params=None, q=FAKE, qr=64 * 192, N=100, cq=FAKE + 4096, k=FAKE + (1 << 20), v=FAKE + (2 << 20), cap=200,
             ck=FAKE + 8192, pre=FAKE + 12288, n=3, window=0, sinks=0, out=FAKE + (3 << 20), outr=64 * 128,
             ws=FAKE + (4 << 20), wsb=1 << 16)
    a.update(kw)
    return m.lib().mla_document_attention(a["params"], a["q"], a["qr"], a["N"], a["cq"], a["k"], a["v"], a["cap"], a["ck"],
                                          a["pre"], a["n"], a["window"], a["sinks"], a["out"], a["outr"], a["ws"],
                                          a["wsb"], None)


def test_refusals():
    for kw in (dict(q=None), dict(cq=None), dict(k=None), dict(v=None), dict(out=None), dict(N=0), dict(N=(1 << 24) + 1),
               dict(cap=0), dict(cap=(1 << 24) + 1), dict(n=0), dict(n=(1 << 20) + 1), dict(window=-1), dict(sinks=-1),
               dict(qr=64 * 192 - 8), dict(qr=64 * 192 + 4), dict(outr=64 * 128 - 8), dict(outr=64 * 128 + 2),
               dict(qr=(1 << 30) + 8), dict(outr=-8)):
        assert attend_c(**kw) == -1, kw
    for kw in (dict(q=FAKE + 2), dict(k=FAKE + 8), dict(v=FAKE + 8), dict(out=FAKE + 8), dict(cq=FAKE + 2),
               dict(ck=FAKE + 1), dict(pre=FAKE + 3), dict(ws=FAKE + 8)):
        assert attend_c(**kw) == -2, kw
    assert attend_c(ws=None) == -3 and attend_c(wsb=256) == -3
    bad = m.MlaParams(1e-6, 10000.0, -1.0, None, None)
    assert attend_c(params=ctypes.byref(bad)) == -1


def test_workspace_sizes():
    assert m.workspace_size(m.MODE_DOCUMENTS, 4, 10000) > m.workspace_size(m.MODE_DOCUMENTS, 4, 100)
    assert m.workspace_size(m.MODE_DOCUMENTS, 400, 10000) > m.workspace_size(m.MODE_DOCUMENTS, 4, 10000)
    for n, N in ((0, 1), (1, 0), ((1 << 20) + 1, 5), (1, (1 << 24) + 1)):
        assert m.lib().mla_workspace_size(m.MODE_DOCUMENTS, n, N, 0) == 0


# ---- on the GPU ---------------------------------------------------------------------------------------------
def ints(x):
    import torch
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device="cuda")


def starts(lengths, first=0):
    return [first] + list(first + np.cumsum(lengths))


def visible(n, L, prefix, window, sinks):
    i, j = np.arange(L - n, L)[:, None], np.arange(L)[None, :]
    seen = j <= i
    if window:
        seen &= (i - j < window) | (j < sinks)
    return seen | (j < prefix)


def reference(q, k, v, n, L, prefix, window, sinks, scale=1 / math.sqrt(192)):
    """One document and head in 64 bits: the output and sum p |v|; rows that see nothing are zeros."""
    seen = visible(n, L, prefix, window, sinks)
    s = np.where(seen, q @ k.T * scale, -np.inf)
    top = s.max(1, keepdims=True, initial=-np.inf)
    w = np.exp(s - np.where(np.isfinite(top), top, 0))
    w /= np.maximum(w.sum(1, keepdims=True), 1e-300)
    return w @ v, w @ np.abs(v)


def check(got, q, k, v, cu_q, cu_k, prefix, window, sinks, heads=(0, 17, 63), scale=1 / math.sqrt(192)):
    """got [N, 64 * 128], q [N, 64 * 192] and the caches in 64 bits."""
    assert np.isfinite(got[cu_q[0]:cu_q[-1]]).all()
    for d in range(len(cu_q) - 1):
        a, b, e, f = cu_q[d], cu_q[d + 1], cu_k[d], cu_k[d + 1]
        p = min(max(prefix[d], 0), f - e) if prefix is not None else 0
        for h in heads:
            ref, mag = reference(q[a:b, h * 192:h * 192 + 192], k[h, e:f], v[h, e:f], b - a, f - e, p, window, sinks,
                                 scale)
            diff = np.abs(got[a:b, h * 128:h * 128 + 128] - ref)
            assert (diff <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -14) * mag).all(), (d, h, diff.max())


def run(q, k, v, cu_q, cu_k, prefix=None, window=0, sinks=0, status=0, params=None, fill=float("nan")):
    import torch
    out = torch.full((q.shape[0], 64 * 128), fill, dtype=torch.bfloat16, device="cuda")
    ws = m.alloc_workspace(m.MODE_DOCUMENTS, len(cu_q) - 1, q.shape[0]).fill_(0xa5)
    m.mla_document_attention(q, ints(cu_q), k, v, out, ws, cu_k=None if cu_k is None else ints(cu_k),
                             prefix=None if prefix is None else ints(prefix), window=window, sinks=sinks, params=params)
    assert m.mla_device_status(ws) == status
    return out


CASES = [
    # new tokens, cached ones before them, prefix, window, sinks
    ([1], [0], None, 0, 0),
    ([128], [0], None, 0, 0),
    ([129], [0], None, 0, 0),
    ([300, 1, 17, 128, 64], [0] * 5, None, 0, 0),
    ([5, 0, 33, 0, 0, 70], [0, 7, 0, 0, 200, 1], None, 0, 0),
    ([1, 1, 1, 1, 1], [0, 500, 127, 128, 129], None, 0, 0),
    ([100, 260, 31], [333, 1, 128], None, 0, 0),
    ([200, 40, 128, 9], [0, 300, 5, 0], [77, 310, 0, 9], 0, 0),
    ([150, 150], [0, 0], [150, 999], 0, 0),
    ([300, 90, 400], [0, 222, 50], None, 64, 0),
    ([300, 90, 400], [0, 222, 50], None, 1, 0),
    ([300, 90, 400], [0, 222, 50], None, 100, 4),
    ([300, 90, 400, 513], [100, 222, 50, 0], [10, 20, 130, 200], 33, 150),
    ([260, 700], [900, 10], [140, 0], 50, 3),
    ([40] * 30, list(range(0, 300, 10)), [i % 41 for i in range(30)], 0, 0),
    ([513], [1000], [1513], 0, 0),
    ([64, 64], [0, 0], [0, 0], 1 << 30, 1 << 30),
]


@gpu
@pytest.mark.parametrize("new,past,prefix,window,sinks", CASES)
def test_values(gpu_available, new, past, prefix, window, sinks):
    keys = [a + b for a, b in zip(new, past)]
    cu_q, cu_k = starts(new), starts(keys)
    q, k, v = normal(1, cu_q[-1], 64 * 192), normal(2, 64, cu_k[-1], 192), normal(3, 64, cu_k[-1], 128)
    out = run(q, k, v, cu_q, cu_k, prefix, window, sinks)
    check(f64(out), f64(q), f64(k), f64(v), cu_q, cu_k, prefix, window, sinks)


@gpu
@pytest.mark.parametrize("new,keys,prefix", [([10, 200, 5], [3, 100, 0], None), ([10, 200, 300], [3, 100, 130], [2, 0, 130]),
                                             ([130], [1], None), ([3, 3], [0, 0], [4, 4])])
def test_more_queries_than_keys(gpu_available, new, keys, prefix):
    """Rows before the document's first key see nothing (but a prefix): zeros."""
    cu_q, cu_k = starts(new), starts(keys)
    q, k, v = normal(1, cu_q[-1], 64 * 192), normal(2, 64, max(cu_k[-1], 1), 192), normal(3, 64, max(cu_k[-1], 1), 128)
    out = run(q, k, v, cu_q, cu_k, prefix)
    check(f64(out), f64(q), f64(k), f64(v), cu_q, cu_k, prefix, 0, 0)
    if prefix is None:
        assert bool((out[:new[0] - keys[0]] == 0).all())


@gpu
def test_without_keys_of_their_own(gpu_available):
    """cu_k left out: queries and keys share their rows; offsets that begin behind the first row, rows behind the last
    document, rows with strides."""
    import torch
    new = [200, 3, 140]
    cu = starts(new, 7)
    wide_q, wide_o = normal(1, cu[-1] + 30, 64 * 192 + 16), torch.full((cu[-1] + 30, 64 * 128 + 8), 3.0,
                                                                       dtype=torch.bfloat16, device="cuda")
    q, out = wide_q[:, :64 * 192], wide_o[:, :64 * 128]
    k, v = normal(2, 64, cu[-1] + 50, 192), normal(3, 64, cu[-1] + 50, 128)
    ws = m.alloc_workspace(m.MODE_DOCUMENTS, 3, q.shape[0])
    m.mla_document_attention(q, ints(cu), k, v, out, ws)
    assert m.mla_device_status(ws) == 0
    check(f64(out.contiguous()), f64(q.contiguous()), f64(k), f64(v), cu, cu, None, 0, 0)
    assert bool((wide_o[:7] == 3).all()) and bool((wide_o[cu[-1]:] == 3).all()) and bool((wide_o[:, 64 * 128:] == 3).all())


@gpu
def test_neighbours_do_not_matter(gpu_available):
    """NaN and infinities in the other documents, in front of the first and behind the last: the same bits."""
    import torch
    new, past = [37, 130, 260, 5], [11, 0, 77, 300]
    keys = [a + b for a, b in zip(new, past)]
    cu_q, cu_k = starts(new, 3), starts(keys, 9)
    q, k, v = normal(1, cu_q[-1] + 20, 64 * 192), normal(2, 64, cu_k[-1] + 20, 192), normal(3, 64, cu_k[-1] + 20, 128)
    for kw in (dict(), dict(prefix=[5, 0, 300, 305]), dict(window=40, sinks=3)):
        clean = run(q, k, v, cu_q, cu_k, **kw)
        for d in range(4):
            q2, k2, v2 = q.clone(), k.clone(), v.clone()
            for value in (float("nan"), float("inf"), -float("inf")):
                for x, cu, axis in ((q2, cu_q, 0), (k2, cu_k, 1), (v2, cu_k, 1)):
                    rows = torch.ones(x.shape[axis], dtype=torch.bool, device="cuda")
                    rows[cu[d]:cu[d + 1]] = False
                    if axis == 0:
                        x[rows] = value
                    else:
                        x[:, rows] = value
                got = run(q2, k2, v2, cu_q, cu_k, **kw)
                assert torch.equal(got[cu_q[d]:cu_q[d + 1]], clean[cu_q[d]:cu_q[d + 1]]), (kw, d, value)


@gpu
def test_keys_behind_the_last_query(gpu_available):
    """Keys that no query of a tile sees (behind a short prefix's end): whatever they hold, the rows before them keep
    their bits."""
    import torch
    q, k, v = normal(1, 256, 64 * 192), normal(2, 64, 256, 192), normal(3, 64, 256, 128)
    clean = run(q, k, v, [0, 256], None, [20])
    k[:, 128:], v[:, 128:] = float("nan"), float("inf")
    assert torch.equal(run(q, k, v, [0, 256], None, [20])[:128], clean[:128])


@gpu
@pytest.mark.parametrize("cu_q,cu_k", [([0, 50, 40, 100], None), ([-1, 50, 60, 100], None), ([0, 50, 60, 101], None),
                                       ([0, 50, 60, 100], [0, 30, 90, 121]), ([0, 50, 60, 100], [0, 90, 30, 120]),
                                       ([0, 50, 60, 100], [-5, 0, 30, 120]),
                                       ([0, 1 << 30, -(1 << 30), 100], None)])
def test_offsets_out_of_range_write_nothing(gpu_available, cu_q, cu_k):
    q, k, v = normal(1, 100, 64 * 192), normal(2, 64, 120, 192), normal(3, 64, 120, 128)
    out = run(q, k, v, cu_q, cu_k, status=-1, fill=5.0)
    assert bool((out == 5).all())


@gpu
def test_against_the_causal_and_the_windowed_kernel(gpu_available):
    """Documents of equal lengths give what mla_window_attention gives, sequence by sequence."""
    import torch
    B, T, P0 = 3, 300, 41
    L = P0 + T
    q, k, v = normal(1, B, T, 64 * 192), normal(2, B, 64, L, 192), normal(3, B, 64, L, 128)
    pk, pv = (x.transpose(0, 1).reshape(64, B * L, -1).contiguous() for x in (k, v))
    for window, sinks in ((90, 7), (1 << 20, 0)):
        a = torch.empty((B, T, 64 * 128), dtype=torch.bfloat16, device="cuda")
        m.mla_window_attention(q, P0, k, v, a, m.alloc_workspace(m.MODE_WINDOW_ATTN, B, T), window=window, sinks=sinks)
        b = run(q.view(B * T, -1), pk, pv, [T * i for i in range(B + 1)], [L * i for i in range(B + 1)], None, window, sinks)
        x, y = f64(a).reshape(B * T, -1), f64(b)
        mag = np.abs(y).max()
        assert np.abs(x - y).max() <= 2.0 ** -6 * mag


@gpu
def test_many_documents(gpu_available):
    """More documents than the plan keeps in shared memory, most of them of a token or none."""
    rng = np.random.default_rng(1)
    new = np.where(rng.random(6000) < 0.3, 0, 1)
    new[[5, 700, 5999]] = [140, 3, 33]
    past = rng.integers(0, 3, 6000)
    past[700] = 400
    cu_q, cu_k = starts(new), starts(new + past)
    q, k, v = normal(1, cu_q[-1], 64 * 192), normal(2, 64, cu_k[-1], 192), normal(3, 64, cu_k[-1], 128)
    out = run(q, k, v, cu_q, cu_k)
    check(f64(out), f64(q), f64(k), f64(v), cu_q, cu_k, None, 0, 0, heads=(5,))


@gpu
def test_moving_maxima_and_scale(gpu_available):
    """Scores that grow along the keys (the running maximum moves in every tile), and another scale."""
    new, past = [200, 150], [500, 300]
    cu_q, cu_k = starts(new), starts([700, 450])
    q, k, v = normal(1, 350, 64 * 192), normal(2, 64, 1150, 192), normal(3, 64, 1150, 128)
    q.view(350, 64, 192)[..., 5] = 3.0
    for d in range(2):
        n = cu_k[d + 1] - cu_k[d]
        import torch
        k[:, cu_k[d]:cu_k[d + 1], 5] = torch.linspace(-60, 60, n, device="cuda").to(torch.bfloat16)
    for scale in (1 / math.sqrt(192), 0.3):
        out = run(q, k, v, cu_q, cu_k, params=m.make_params(softmax_scale=scale))
        check(f64(out), f64(q), f64(k), f64(v), cu_q, cu_k, None, 0, 0, scale=scale)


@gpu
def test_captured_and_on_two_streams(gpu_available):
    """A captured call replayed with other offsets, and two calls at once on streams of their own."""
    import torch
    q, k, v = normal(1, 400, 64 * 192), normal(2, 64, 400, 192), normal(3, 64, 400, 128)
    plans = [[0, 400, 400, 400], [0, 100, 101, 380], [5, 5, 205, 399]]
    want = [run(q, k, v, cu, None, fill=1.0) for cu in plans]
    cu, out = ints(plans[0]), torch.empty((400, 64 * 128), dtype=torch.bfloat16, device="cuda")
    ws = m.alloc_workspace(m.MODE_DOCUMENTS, 3, 400)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.mla_document_attention(q, cu, k, v, out, ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        m.mla_document_attention(q, cu, k, v, out, ws)
    for i in (1, 2, 0, 1):
        cu.copy_(ints(plans[i]))
        out.fill_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.full_like(out, 1.0) for _ in range(2)]
    cus, wss = [ints(p) for p in plans[:2]], [m.alloc_workspace(m.MODE_DOCUMENTS, 3, 400) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            m.mla_document_attention(q, cus[i], k, v, outs[i], wss[i], stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@gpu
def test_rows_past_32_bit_offsets(gpu_available):
    """Caches of more than 2^32 numbers and rows of q and out that lie as far apart: the same bits as packed ones."""
    import torch
    new, past, at, cap = [130, 1, 33], [50, 200, 0], 399000, 400000
    cu_q, cu_k = starts(new), starts([a + b for a, b in zip(new, past)])
    q, k, v = normal(1, cu_q[-1], 64 * 192), normal(2, 64, cu_k[-1], 192), normal(3, 64, cu_k[-1], 128)
    want = run(q, k, v, cu_q, cu_k, [100, 0, 33])
    far_k, far_v = (torch.empty((64, cap, n), dtype=torch.bfloat16, device="cuda") for n in (192, 128))
    far_k[:, at:at + cu_k[-1]], far_v[:, at:at + cu_k[-1]] = k, v
    far_q, far_o = (torch.empty((cu_q[-1], 1 << 25), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    far_q[:, :64 * 192] = q
    ws = m.alloc_workspace(m.MODE_DOCUMENTS, 3, cu_q[-1])
    m.mla_document_attention(far_q[:, :64 * 192], ints(cu_q), far_k, far_v, far_o[:, :64 * 128], ws,
                             cu_k=ints([c + at for c in cu_k]), prefix=ints([100, 0, 33]))
    assert m.mla_device_status(ws) == 0
    assert torch.equal(far_o[:, :64 * 128], want)


@gpu
def test_binding_refuses_wrong_shapes_types_and_devices(gpu_available):
    import torch
    q, k, v = normal(1, 30, 64 * 192), normal(2, 64, 40, 192), normal(3, 64, 40, 128)
    good = dict(q=q, cu_q=ints([0, 10, 30]), k_cache=k, v_cache=v, out=torch.empty_like(q[:, :64 * 128].contiguous()),
                workspace=m.alloc_workspace(m.MODE_DOCUMENTS, 2, 30), cu_k=ints([0, 20, 40]), prefix=ints([3, 4]))
    m.mla_document_attention(**good)
    for over in (dict(q=q[:29]), dict(q=q.float()), dict(q=q[:, :-8]), dict(q=q.cpu()), dict(q=q.t()),
                 dict(out=good["out"][:29]), dict(out=good["out"].half()), dict(out=good["out"].cpu()),
                 dict(k_cache=k[:63]), dict(k_cache=k[:, :39]), dict(k_cache=k.float()), dict(k_cache=k.transpose(0, 1)),
                 dict(v_cache=v[..., :64]), dict(v_cache=v.cpu()), dict(cu_q=good["cu_q"].long()),
                 dict(cu_q=ints([0, 1, 10, 30])), dict(cu_k=ints([0, 40])), dict(cu_k=good["cu_k"].cpu()),
                 dict(prefix=ints([1, 2, 3])), dict(prefix=ints([1, 0, 2, 0])[::2]), dict(workspace=good["workspace"].cpu())):
        with pytest.raises(ValueError):
            m.mla_document_attention(**{**good, **over})
    for over, status in ((dict(workspace=good["workspace"][:256]), -3), (dict(window=-1), -1)):
        with pytest.raises(m.MlaError) as e:
            m.mla_document_attention(**{**good, **over})
        assert e.value.status == status


LONG = [
    # many key tiles an item, query tiles of 128
    ([1536], [0], None, 0, 0),
    ([1663], [0], None, 0, 0),
    ([1537], [100], [900], 0, 0),
    ([3000, 1400, 300], [0, 77, 500], [10, 1477, 0], 0, 0),
    ([4700, 0, 5], [0, 40, 300], None, 0, 0),
    ([2000, 1100], [100, 50], [10, 300], 300, 20),
    ([1700], [30], None, 1, 0),
    ([1900], [600], None, 1024, 100),
    ([2600], [0], None, 2000, 4),
    ([3200], [500], None, 1600, 130),
    ([3500, 100], [0, 900], [200, 1000], 1700, 0),
]


@gpu
@pytest.mark.parametrize("new,past,prefix,window,sinks", LONG)
def test_long_documents(gpu_available, new, past, prefix, window, sinks):
    keys = [a + b for a, b in zip(new, past)]
    cu_q, cu_k = starts(new), starts(keys)
    q, k, v = normal(1, cu_q[-1], 64 * 192), normal(2, 64, cu_k[-1], 192), normal(3, 64, cu_k[-1], 128)
    out = run(q, k, v, cu_q, cu_k, prefix, window, sinks)
    check(f64(out), f64(q), f64(k), f64(v), cu_q, cu_k, prefix, window, sinks, heads=(0, 37, 63))


@gpu
def test_long_documents_and_their_neighbours(gpu_available):
    """Long documents with more queries than keys, offsets, rows behind the last; NaN and infinities in the others, in
    front and behind: the same bits; scores that grow along the keys; the same again from a graph, on two streams."""
    import torch
    new, keys = [1700, 1433, 1600], [1700, 1333, 2000]
    cu_q, cu_k = starts(new, 3), starts(keys, 9)
    N = cu_q[-1] + 20
    q, k, v = normal(1, N, 64 * 192), normal(2, 64, cu_k[-1] + 20, 192), normal(3, 64, cu_k[-1] + 20, 128)
    q.view(N, 64, 192)[..., 5] = 3.0
    for d in range(3):
        k[:, cu_k[d]:cu_k[d + 1], 5] = torch.linspace(-60, 60, keys[d], device="cuda").to(torch.bfloat16)
    clean = run(q, k, v, cu_q, cu_k, fill=7.0)
    check(f64(clean), f64(q), f64(k), f64(v), cu_q, cu_k, None, 0, 0, heads=(5, 60))
    assert bool((clean[:3] == 7).all()) and bool((clean[cu_q[-1]:] == 7).all())
    assert bool((clean[cu_q[1]:cu_q[1] + 100] == 0).all()), "rows before the document's first key"
    for d in range(3):
        for value in (float("nan"), float("inf")):
            q2, k2, v2 = torch.full_like(q, value), torch.full_like(k, value), torch.full_like(v, value)
            q2[cu_q[d]:cu_q[d + 1]] = q[cu_q[d]:cu_q[d + 1]]
            for x2, x in ((k2, k), (v2, v)):
                x2[:, cu_k[d]:cu_k[d + 1]] = x[:, cu_k[d]:cu_k[d + 1]]
            got = run(q2, k2, v2, cu_q, cu_k)
            assert torch.equal(got[cu_q[d]:cu_q[d + 1]], clean[cu_q[d]:cu_q[d + 1]]), (d, value)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.full_like(clean, 7.0) for _ in range(2)]
    cq, ck, wss = ints(cu_q), ints(cu_k), [m.alloc_workspace(m.MODE_DOCUMENTS, 3, N) for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for s, out, ws in zip(streams, outs, wss):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            for _ in range(3):
                m.mla_document_attention(q, cq, k, v, out, ws, cu_k=ck)
    torch.cuda.synchronize()
    for _ in range(2):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert [m.mla_device_status(ws) for ws in wss] == [0, 0]
    assert torch.equal(outs[0], clean) and torch.equal(outs[1], clean)


PAIRS = [
    # 2,048 rows a document on average and more (in pairs of thread blocks: test_in_pairs_by_room)
    ([2048], [0], None, 0, 0),
    ([2175], [0], None, 0, 0),
    ([2177], [100], [900], 0, 0),
    ([4100, 2100, 300], [0, 77, 500], [10, 2177, 0], 0, 0),
    ([6200, 0, 5], [0, 40, 300], None, 0, 0),
    ([2900], [500], None, 2048, 130),
    ([2500, 2000], [0, 1500], [200, 3500], 2400, 7),
]


@gpu
@pytest.mark.parametrize("new,past,prefix,window,sinks", PAIRS)
def test_documents_in_pairs(gpu_available, new, past, prefix, window, sinks):
    test_long_documents(gpu_available, new, past, prefix, window, sinks)


@gpu
def test_pairs_and_their_neighbours(gpu_available):
    """As the test of long documents and their neighbours, with more queries than keys."""
    import torch
    new, keys = [2300, 2033, 2200], [2300, 333, 2600]
    cu_q, cu_k = starts(new, 3), starts(keys, 9)
    N = cu_q[-1] + 20
    q, k, v = normal(1, N, 64 * 192), normal(2, 64, cu_k[-1] + 20, 192), normal(3, 64, cu_k[-1] + 20, 128)
    q.view(N, 64, 192)[..., 5] = 3.0
    for d in range(3):
        k[:, cu_k[d]:cu_k[d + 1], 5] = torch.linspace(-60, 60, keys[d], device="cuda").to(torch.bfloat16)
    clean = run(q, k, v, cu_q, cu_k, fill=7.0)
    check(f64(clean), f64(q), f64(k), f64(v), cu_q, cu_k, None, 0, 0, heads=(5, 60))
    assert bool((clean[:3] == 7).all()) and bool((clean[cu_q[-1]:] == 7).all())
    assert bool((clean[cu_q[1]:cu_q[1] + 1700] == 0).all()), "rows before the document's first key"
    for d in range(3):
        for value in (float("nan"), float("inf")):
            q2, k2, v2 = torch.full_like(q, value), torch.full_like(k, value), torch.full_like(v, value)
            q2[cu_q[d]:cu_q[d + 1]] = q[cu_q[d]:cu_q[d + 1]]
            for x2, x in ((k2, k), (v2, v)):
                x2[:, cu_k[d]:cu_k[d + 1]] = x[:, cu_k[d]:cu_k[d + 1]]
            got = run(q2, k2, v2, cu_q, cu_k)
            assert torch.equal(got[cu_q[d]:cu_q[d + 1]], clean[cu_q[d]:cu_q[d + 1]]), (d, value)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.full_like(clean, 7.0) for _ in range(2)]
    cq, ck, wss = ints(cu_q), ints(cu_k), [m.alloc_workspace(m.MODE_DOCUMENTS, 3, N) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, out, ws in zip(streams, outs, wss):
            m.mla_document_attention(q, cq, k, v, out, ws, cu_k=ck, stream=s)
    torch.cuda.synchronize()
    assert [m.mla_device_status(ws) for ws in wss] == [0, 0]
    assert torch.equal(outs[0], clean) and torch.equal(outs[1], clean)


@gpu
@pytest.mark.parametrize("cu,status", [([5, 5], 0), ([2100, 2100], 0), ([7, 8], 0), ([0, 2101], -1), ([-1, 2000], -1),
                                       ([50, 40], -1)])
def test_room_for_many_rows_that_are_not_there(gpu_available, cu, status):
    """Room for many rows, offsets that use hardly any or none of it, or that are refused."""
    q, k, v = normal(1, 2100, 64 * 192), normal(2, 64, 2100, 192), normal(3, 64, 2100, 128)
    out = run(q, k, v, cu, None, status=status, fill=5.0)
    if status == 0:
        check(f64(out), f64(q), f64(k), f64(v), cu, cu, None, 0, 0)
    rest = out.clone()
    if status == 0:
        rest[cu[0]:cu[1]] = 5
    assert bool((rest == 5).all())


@gpu
@pytest.mark.parametrize("n,rows", [(32, 16), (33, 16), (32, 17), (17, 16), (5, 1400), (5, 1500)])
def test_few_tiles_and_more(gpu_available, n, rows):
    """Around the numbers of documents and rows up to which the thread blocks plan by themselves; many documents empty."""
    rng = np.random.default_rng(n + rows)
    cut = np.sort(rng.integers(0, rows + 1, n - 1))
    cu_q = [int(c) for c in [0, *cut, rows]]
    past = rng.integers(0, 300, n)
    cu_k = starts([b - a + int(p) for a, b, p in zip(cu_q, cu_q[1:], past)])
    prefix = [int(x) for x in rng.integers(-3, 200, n)]
    q, k, v = normal(1, rows, 64 * 192), normal(2, 64, cu_k[-1], 192), normal(3, 64, cu_k[-1], 128)
    for kw in (dict(prefix=prefix, window=0, sinks=0), dict(prefix=None, window=50, sinks=3)):
        out = run(q, k, v, cu_q, cu_k, **kw)
        check(f64(out), f64(q), f64(k), f64(v), cu_q, cu_k, heads=(0, 63), **kw)


@gpu
@pytest.mark.parametrize("cu", [[0, 500, 400, 2000], [0, 500, 600, 2001], [-1, 500, 600, 2000]])
def test_offsets_out_of_range_of_more_tiles(gpu_available, cu):
    q, k, v = normal(1, 2000, 64 * 192), normal(2, 64, 2000, 192), normal(3, 64, 2000, 128)
    assert bool((run(q, k, v, cu, None, status=-1, fill=5.0) == 5).all())


@gpu
def test_a_document_of_millions_of_keys(gpu_available):
    """An item that takes tens of milliseconds, by itself, in pairs and among short ones; every key alike, so that each
    row's answer is the mean of the values it sees."""
    import torch
    keys, short = 3_000_000, 40
    k = torch.zeros((64, keys + short, 192), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((64, keys + short, 128), dtype=torch.bfloat16, device="cuda")
    value = (torch.arange(64, device="cuda") % 3).to(torch.bfloat16)  # (its sums stay below 2^24)
    v[:] = value[:, None, None]
    want = value.repeat_interleave(128)
    for cu_q in ([0, 1, 6], [0, 130, 2500]):  # (a few rows; many)
        q = normal(1, 6 if cu_q[2] == 6 else 4100, 64 * 192)
        out = run(q, k, v, cu_q, [0, keys, keys + short], window=0)
        seen = out[cu_q[1]:cu_q[2]][-short:]
        for got in (out[:cu_q[1]], seen):
            assert bool((got == want).all())


@gpu
def test_pairs_captured_and_replayed(gpu_available):
    """Room enough for pairs: three calls of one graph after one another, two of them on one workspace, replayed with
    other offsets (short documents in the room of long ones, none, such as are refused) on two streams at once."""
    import torch
    N, cap = 12000, 7000  # (room for 4,000 rows a document)
    q, k, v = normal(1, N, 64 * 192), normal(2, 64, cap, 192), normal(3, 64, cap, 128)
    plans = [([0, 2300, 4100, 6300], [0, 2900, 4700, 7000], 0), ([5, 5, 6200, 6291], [3, 40, 6700, 6791], 0),
             ([0, 300, 301, 429], [0, 300, 3000, 3128], 0), ([0, 2000, 1000, 6300], [0, 2000, 4000, 7000], -1),
             ([70, 70, 70, 70], [0, 0, 0, 0], 0), ([0, 2300, 4100, 6300], [0, 2900, 4700, 7001], -1)]
    kw = [dict(), dict(window=2100, sinks=33), dict(prefix=[100, 3000, 0])]
    want = [[run(q, k, v, cq, ck, status=status, fill=1.0, **w) for w in kw] for cq, ck, status in plans]
    for cq, ck, status in plans[:3]:
        check(f64(want[plans.index((cq, ck, status))][0]), f64(q), f64(k), f64(v), cq, ck, None, 0, 0, heads=(11,))
    streams, sides = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        cu_q, cu_k, prefix = ints(plans[0][0]), ints(plans[0][1]), ints(kw[2]["prefix"])
        outs = [torch.empty((N, 64 * 128), dtype=torch.bfloat16, device="cuda") for _ in kw]
        wss = [m.alloc_workspace(m.MODE_DOCUMENTS, 3, N) for _ in range(2)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for i in range(3):
                m.mla_document_attention(q, cu_q, k, v, outs[i], wss[i // 2], cu_k=cu_k, window=kw[i].get("window", 0),
                                         sinks=kw[i].get("sinks", 0), prefix=prefix if i == 2 else None)
        sides.append((graph, cu_q, cu_k, outs, wss, prefix))  # (what the graph reads is kept)
    for turn in ((0, 1), (1, 2), (3, 0), (2, 4), (5, 5), (0, 0)):
        for i, (_, cu_q, cu_k, outs, *_) in zip(turn, sides):
            cu_q.copy_(ints(plans[i][0]))
            cu_k.copy_(ints(plans[i][1]))
            for out in outs:
                out.fill_(1.0)
        torch.cuda.synchronize()
        for s, side in zip(streams, sides):
            with torch.cuda.stream(s):
                side[0].replay()
        torch.cuda.synchronize()
        for i, (_, _, _, outs, wss, _) in zip(turn, sides):
            assert [m.mla_device_status(ws) for ws in wss] == [plans[i][2]] * 2
            for j, out in enumerate(outs):
                assert torch.equal(out, want[i][j]), (i, j)


@gpu
@pytest.mark.parametrize("cu_q,N", [([0, 1, 6], 6), ([0, 200, 2500], 2500), ([0, 130, 4100], 8000)])
def test_each_key_tile_of_a_long_document_counts_once(gpu_available, cu_q, N):
    """Keys alike, so that a row's answer is the mean of its values; a value is 1 in one dimension of 128 and 0 in the
    others, the next dimension every 96 keys (another first one in each head).  A tile left out, taken twice or from
    elsewhere moves a dimension by 4%; what is rounded is the answer, and the quotient by 2^-20 before."""
    import torch
    keys, short = 300_007, 40
    total = keys + short
    if torch.cuda.mem_get_info()[0] < 2 * 64 * total * (192 + 128) * 2:
        pytest.skip("too little free memory")
    j, h = torch.arange(total, device="cuda"), torch.arange(64, device="cuda")
    k = torch.zeros((64, total, 192), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((64, total, 128), dtype=torch.bfloat16, device="cuda")
    at = (j[None] // 96 + 5 * h[:, None]) % 128
    v.scatter_(2, at[..., None], 1.0)
    q = normal(1, N, 64 * 192)
    out = run(q, k, v, cu_q, [0, keys, total])
    for d, row in ((0, 0), (0, cu_q[1] - 1), (1, cu_q[2] - 1)):
        first = 0 if d == 0 else keys
        last = (keys if d == 0 else total) - (cu_q[d + 1] - 1 - row)  # behind the row's own key
        seen = torch.zeros((64, 128), dtype=torch.float64, device="cuda")
        seen.scatter_add_(1, at[:, first:last], torch.ones_like(at[:, first:last], dtype=torch.float64))
        ref = seen / (last - first)
        got = out[row].double().view(64, 128)
        assert bool(((got - ref).abs() <= (2.0 ** -8 + 2.0 ** -20) * ref).all()), (d, row)


PAIRED = [c for c in CASES + LONG + PAIRS if c[3] == 0 or c[3] >= 2048] + [
    ([2900], [500], None, 2049, 130),
    ([2500, 2000, 3], [0, 1500, 6000], [200, 3500, 0], 2400, 7),
    ([300, 256, 1], [4000, 2100, 9000], None, 2048, 100),
    ([300, 0, 255, 257], [4000, 7, 2100, 1], [4300, 1, 500, 2], 3000, 40),
]


@gpu
@pytest.mark.parametrize("new,past,prefix,window,sinks", PAIRED)
def test_in_pairs_by_room(gpu_available, new, past, prefix, window, sinks):
    """Room for 4,000 rows a document, so that pairs of thread blocks take 256 queries at a time, whatever lies in it."""
    import torch
    keys = [a + b for a, b in zip(new, past)]
    cu_q, cu_k = starts(new, 5), starts(keys, 3)
    k, v = normal(2, 64, cu_k[-1] + 7, 192), normal(3, 64, cu_k[-1] + 7, 128)
    q = torch.full((4000 * len(new), 64 * 192), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[5:cu_q[-1]] = normal(1, cu_q[-1] - 5, 64 * 192)
    out = run(q, k, v, cu_q, cu_k, prefix, window, sinks, fill=9.0)
    assert bool((out[:5] == 9).all()) and bool((out[cu_q[-1]:] == 9).all())
    rows = slice(0, cu_q[-1])
    check(f64(out[rows]), f64(q[rows]), f64(k), f64(v), cu_q, cu_k, prefix, window, sinks, heads=(0, 37, 63))


@gpu
def test_neighbours_in_pairs_by_room(gpu_available):
    """NaN and infinities in the other documents, in front of the first and behind the last: the same bits, with rows
    that have strides."""
    import torch
    new, past = [37, 530, 260, 5, 1], [11, 0, 77, 300, 2000]
    cu_q, cu_k = starts(new, 3), starts([a + b for a, b in zip(new, past)], 9)
    N = 5 * 4000
    q = torch.zeros((N, 64 * 192 + 8), dtype=torch.bfloat16, device="cuda")
    q[:cu_q[-1] + 20] = normal(1, cu_q[-1] + 20, 64 * 192 + 8)
    k, v = normal(2, 64, cu_k[-1] + 20, 192), normal(3, 64, cu_k[-1] + 20, 128)

    def strided(q, k, v, prefix=None, window=0, sinks=0):
        wide = torch.full((N, 64 * 128 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = m.alloc_workspace(m.MODE_DOCUMENTS, 5, N)
        m.mla_document_attention(q[:, :64 * 192], ints(cu_q), k, v, wide[:, :64 * 128], ws, cu_k=ints(cu_k),
                                 prefix=None if prefix is None else ints(prefix), window=window, sinks=sinks)
        assert m.mla_device_status(ws) == 0
        assert bool((wide[:, 64 * 128:] == 7).all()) and bool((wide[:3] == 7).all()) and bool((wide[cu_q[-1]:] == 7).all())
        return wide[:cu_q[-1], :64 * 128].contiguous()

    for kw in (dict(), dict(prefix=[5, 0, 300, 305, 1000]), dict(window=2050, sinks=3)):
        clean = strided(q, k, v, **kw)
        full = dict(dict(prefix=None, window=0, sinks=0), **kw)
        check(f64(clean), f64(q[:cu_q[-1], :64 * 192].contiguous()), f64(k), f64(v), cu_q, cu_k, heads=(2, 61), **full)
        for d in range(5):
            for value in (float("nan"), float("inf"), -float("inf")):
                q2, k2, v2 = torch.full_like(q, value), torch.full_like(k, value), torch.full_like(v, value)
                q2[cu_q[d]:cu_q[d + 1]] = q[cu_q[d]:cu_q[d + 1]]
                for x2, x in ((k2, k), (v2, v)):
                    x2[:, cu_k[d]:cu_k[d + 1]] = x[:, cu_k[d]:cu_k[d + 1]]
                got = strided(q2, k2, v2, **kw)
                assert torch.equal(got[cu_q[d]:cu_q[d + 1]], clean[cu_q[d]:cu_q[d + 1]]), (kw, d, value)


@gpu
@pytest.mark.parametrize("cu,status", [([5, 5], 0), ([4000, 4000], 0), ([7, 8], 0), ([0, 4001], -1), ([-1, 2000], -1),
                                       ([50, 40], -1)])
def test_room_for_a_long_document_that_is_not_there(gpu_available, cu, status):
    """As test_room_for_many_rows_that_are_not_there, in pairs of thread blocks."""
    q, k, v = normal(1, 4000, 64 * 192), normal(2, 64, 4000, 192), normal(3, 64, 4000, 128)
    out = run(q, k, v, cu, None, status=status, fill=5.0)
    if status == 0:
        check(f64(out), f64(q), f64(k), f64(v), cu, cu, None, 0, 0)
        out[cu[0]:cu[1]] = 5
    assert bool((out == 5).all())
