"""The steps of serving ragged prompts, as a user strings them together: pages reserved, the prompts' keys and values
appended, attention over the packed prompts, beams forked off them, captured decode steps that take their pages
themselves, drafts that are given back, a compaction.

The numbers are multiples of 1/8 below 2: E4M3 holds them exactly at every scale that a page gets, so the paged cache
and the packed bf16 caches hold the same keys and values (the rotary keys are read back from the cache), and each
kernel is held to the tolerance of its own file against one reference in 64 bits."""
import numpy as np
import pytest

import mla_gb300 as m
from test_documents import reference, starts
from test_paged import f64, normal

gpu = pytest.mark.gpu
HEADS, PAGE, ROWS, LEN, BEAMS = 64, 64, 8, [70, 1, 200, 128], [(2, 4, 200), (2, 5, 200), (0, 6, 70)]
SEEN_HEADS = (0, 17, 63)


def ints(x):
    import torch
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device="cuda")


def eighths(seed, *shape):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randint(-14, 15, shape, generator=g, device="cuda").float() / 8).to(torch.bfloat16)


class Server:
    def __init__(self, n_pages=40, max_pages=6):
        import torch
        self.t = m.alloc_paged_cache(n_pages, PAGE, HEADS)
        self.t["table"] = torch.full((ROWS, max_pages), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.cache, self.pool = m.make_paged_cache(self.t), m.make_page_pool(self.t["table"], self.refs, PAGE)
        self.seq = {}  # row -> keys and values of its tokens, [n, 64, 256]

    def pages(self, name, *lists):
        ws = m.alloc_workspace(m.MODE_PAGES, len(lists[0]), self.refs.numel(), cap=ROWS)
        f = getattr(m, "mla_pages_" + name)
        f(*([self.cache] if name == "fork" else []), self.pool, *[ints(x) for x in lists], ws)
        assert m.mla_device_status(ws) == 0, name

    def row(self, r):
        """Row r's keys [n, 64, 192] and values [n, 64, 128] in bf16."""
        import torch
        kv = self.seq[r]
        j = torch.arange(kv.shape[0], device="cuda")
        pe = self.t["k_pe"][self.t["table"][r][j // PAGE].long(), j % PAGE]
        return torch.cat([kv[..., :128], pe[:, None].expand(-1, HEADS, -1)], 2), kv[..., 128:]

    def packed(self, rows):
        """Their keys and values one after the other, as mla_document_attention takes them, and the offsets."""
        import torch
        k, v = zip(*[self.row(r) for r in rows])
        return (torch.cat(k).transpose(0, 1).contiguous(), torch.cat(v).transpose(0, 1).contiguous(),
                starts([x.shape[0] for x in k]))

    def attend(self, q, last):
        import torch
        out = torch.empty((ROWS, HEADS * 128), dtype=torch.bfloat16, device="cuda")
        ws = m.alloc_workspace(m.MODE_PAGED_ATTN, ROWS, 1)
        m.mla_paged_attention(self.cache, q, ints(last), max(last), out, ws)
        assert m.mla_device_status(ws) == 0
        return out


def documents(server, rows, q, new):
    import torch
    k, v, cu_k = server.packed(rows)
    out = torch.empty((q.shape[0], HEADS * 128), dtype=torch.bfloat16, device="cuda")
    ws = m.alloc_workspace(m.MODE_DOCUMENTS, len(rows), q.shape[0])
    m.mla_document_attention(q, ints(starts(new)), k, v, out, ws, cu_k=ints(cu_k))
    assert m.mla_device_status(ws) == 0
    return out


def close(server, row, n, q, packed=None, paged=None):
    """The last n tokens of a row against the reference: from the packed caches, from the pages."""
    k, v = (f64(x) for x in server.row(row))
    q = f64(q).reshape(n, HEADS, 192)
    for h in SEEN_HEADS:
        ref, mag = reference(q[:, h], k[:, h], v[:, h], n, k.shape[0], 0, 0, 0)
        at = slice(h * 128, h * 128 + 128)
        if packed is not None:
            assert (np.abs(f64(packed)[:, at] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -14) * mag).all(), (row, h)
        if paged is not None:
            bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -16) * np.abs(v[:, h]).max()
            assert (np.abs(f64(paged)[:, at] - ref) <= bound).all(), (row, h)


@gpu
def test_ragged_prompts_beams_and_drafts(gpu_available):
    import torch
    s, N, cu = Server(), sum(LEN), starts(LEN)
    kv, pe, q = eighths(1, N, HEADS, 256), normal(2, N, 64), normal(3, N, HEADS * 192)
    for b in range(4):
        s.seq[b] = kv[cu[b]:cu[b + 1]]

    # the prompts: pages, keys and values, attention over the pack
    s.pages("reserve", range(4), LEN)
    ws = m.alloc_workspace(m.MODE_PAGED_APPEND, ROWS, max(LEN))
    m.mla_paged_append(s.cache, kv[..., :128], kv[..., 128:], pe, ints([0] * 4 + [-1] * 4), max(LEN), ws,
                       cu=ints(list(cu) + [N] * 4))
    assert m.mla_device_status(ws) == 0
    packed = documents(s, range(4), q, LEN)
    q_last = torch.zeros((ROWS, HEADS * 192), dtype=torch.bfloat16, device="cuda")
    q_last[:4] = q[[c - 1 for c in cu[1:]]]
    paged = s.attend(q_last, [n - 1 for n in LEN] + [-1] * 4)
    for b in range(4):
        close(s, b, LEN[b], q[cu[b]:cu[b + 1]], packed=packed[cu[b]:cu[b + 1]])
        close(s, b, 1, q_last[b], paged=paged[b:b + 1])

    # beams: two of the third prompt, which ends, one of the first
    parents, children, P = zip(*BEAMS)
    s.pages("fork", parents, children, P)
    for a, b, n in BEAMS:
        s.seq[b] = s.seq[a][:n]
    s.pages("free", [2], [0])
    del s.seq[2]
    rows = sorted(s.seq)

    # three tokens each, by one captured step that takes their pages itself
    at = {r: s.seq[r].shape[0] for r in rows}
    lists = [ints(rows), ints([0] * len(rows)), ints([-1] * ROWS)]  # reserve's rows and positions, the step's positions
    x = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for shape in ((ROWS, HEADS, 256), (ROWS, 64),
                                                                             (ROWS, HEADS * 192), (ROWS, HEADS * 128))]
    spaces = [m.alloc_workspace(m.MODE_PAGES, len(rows), s.refs.numel(), cap=ROWS),
              m.alloc_workspace(m.MODE_PAGED_APPEND, ROWS, 1), m.alloc_workspace(m.MODE_PAGED_ATTN, ROWS, 1)]

    def step():
        m.mla_pages_reserve(s.pool, lists[0], lists[1], spaces[0])
        m.mla_paged_append(s.cache, x[0][..., :128], x[0][..., 128:], x[1], lists[2], 1, spaces[1])
        m.mla_paged_attention(s.cache, x[2], lists[2], 256, x[3], spaces[2])

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()  # (nothing yet: no positions to reserve, all sequences idle)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    queries, answers = [], []
    for i in range(3):
        new = (eighths(10 + i, ROWS, HEADS, 256), normal(20 + i, ROWS, 64), normal(30 + i, ROWS, HEADS * 192))
        for d, y in zip(x, new):
            d.copy_(y)
        lists[1].copy_(ints([at[r] + i + 1 for r in rows]))
        lists[2].copy_(ints([at[r] + i if r in at else -1 for r in range(ROWS)]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert [m.mla_device_status(w) for w in spaces] == [0, 0, 0]
        for r in rows:
            s.seq[r] = torch.cat([s.seq[r], new[0][r:r + 1]])
            close(s, r, 1, new[2][r], paged=x[3][r:r + 1])
        queries.append(new[2])
        answers.append(x[3].clone())
    assert int(s.refs.sum()) == sum(-(-(at[r] + 3) // PAGE) for r in rows)
    assert bool((answers[-1][[2, 7]] == 0).all())

    # the same three tokens of every sequence in one call over the packed caches
    q3 = torch.stack(queries)[:, rows].transpose(0, 1).reshape(3 * len(rows), -1).contiguous()
    packed = documents(s, rows, q3, [3] * len(rows))
    for i, r in enumerate(rows):
        close(s, r, 3, q3[3 * i:3 * i + 3], packed=packed[3 * i:3 * i + 3])

    # the fourth prompt's tokens are rejected: their page comes back; the rest moves together and answers as before
    held = int((s.refs > 0).sum())
    s.pages("free", [3], [at[3]])
    s.seq[3] = s.seq[3][:at[3]]
    assert int((s.refs > 0).sum()) == held - 1
    last = [s.seq[r].shape[0] - 1 if r in s.seq else -1 for r in range(ROWS)]
    before = s.attend(queries[-1], last)
    ws = m.alloc_workspace(m.MODE_PAGES, 1, s.refs.numel(), cap=ROWS)
    moved, n_live = ints([0] * s.refs.numel()), ints([0])
    m.mla_pages_compact(s.cache, s.pool, moved, n_live, ws)
    assert m.mla_device_status(ws) == 0 and n_live.item() == held - 1
    assert int(s.t["table"].max()) == held - 2
    assert torch.equal(s.attend(queries[-1], last), before)
    for r in rows:
        close(s, r, 1, queries[-1][r], paged=before[r:r + 1])
