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
