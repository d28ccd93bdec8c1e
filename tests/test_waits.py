"""The bounded waits of the kernels whose roles are watched by a warp of their own (attention over packed documents)."""
import pytest

import mla_hooks as m

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [20_000_000, 50_000_000])
def test_roles_that_stand_still_give_up_together(gpu_available, limit):
    """Nothing ends while one role gets on; then the limit counts, every wait ends with it, and a drain of what never
    comes takes the limit once more."""
    import torch
    out = torch.zeros((4, 4), dtype=torch.int64, device="cuda")
    m.mla_debug_watched_waits(out, limit, True)
    torch.cuda.synchronize()
    (a, da, ra, fa), (b, db, rb, fb), (c, _, _, _), (w, _, _, fw) = out.tolist()
    assert (ra, rb) == (1, 1), "what was there is seen, what never comes is not"
    assert fa == fb == fw == 7
    for t in (a, b):  # ten steps of half the limit, then the limit; a try and a step of the clock are microseconds
        assert c + limit - 10_000_000 <= t <= c + limit + 100_000_000
        assert abs(a - b) <= 10_000_000
    for t in (da, db):
        assert limit <= t <= limit + 100_000_000
    assert w >= a
    assert float(torch.ones(1024, device="cuda").sum().item()) == 1024.0  # the context is still usable


def test_roles_that_end_are_not_reported(gpu_available):
    import torch
    out = torch.zeros((4, 4), dtype=torch.int64, device="cuda")
    m.mla_debug_watched_waits(out, 500_000_000, False)
    torch.cuda.synchronize()
    rows = out.tolist()
    assert [r[3] for r in rows] == [0, 0, 0, 0]
    assert [r[2] for r in rows[:2]] == [5, 5]
    assert all(r[0] + r[1] < 100_000_000 for r in rows)


@pytest.mark.parametrize("cu,N", [([0, 300], 300), ([0, 700, 1400, 1401, 2600], 2600), ([0, 3100], 3100),
                                  ([0, 5800, 5801], 6000)])
def test_attention_that_gives_up(gpu_available, cu, N):
    """A limit that no tile can keep: the call reports it and leaves; a call behind it, without a wait in between, has
    the bits that it always has.  A few tiles planned by each thread block, a plan of its own, pairs."""
    import torch
    from test_paged import normal
    q, k, v = normal(1, N, 64 * 192), normal(2, 64, N, 192), normal(3, 64, N, 128)
    at = torch.tensor(cu, dtype=torch.int32, device="cuda")
    n = len(cu) - 1

    def call(limit_ns):
        out = torch.zeros((N, 64 * 128), dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(4096, dtype=torch.int32, device="cuda")
        plan = torch.zeros(48 * (N // 128 + n + 1), dtype=torch.uint8, device="cuda")
        m.mla_debug_document_attention(q, at, k, v, out, status, plan, torch.zeros(n, dtype=torch.int32, device="cuda"),
                                       limit_ns)
        return out, status

    want, status = call(2_000_000_000)
    assert int(status[0]) == 0
    for _ in range(2):
        stopped, got = call(0), call(2_000_000_000)
        torch.cuda.synchronize()
        assert int(stopped[1][0]) & 1 == 1 and int(got[1][0]) == 0
        assert torch.equal(got[0], want)
        # what it stored before it gave up is right, the rest is as it was
        rows = stopped[0].view(N, 64, 128)
        assert bool(((rows == want.view(N, 64, 128)) | (rows == 0)).all())
