"""The packed attention's bounded wait: it gives up after its limit, says so in the plan's status word, and the context
and the plan stay usable."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_packed_wait_gives_up_and_context_stays_usable():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as vsa

    plan = vsa.vsa_packed_plan((100, 30), 4, 2, 64)
    q, k, v = (torch.randn(130, n, 64, device="cuda").to(torch.bfloat16) for n in (4, 2, 2))
    want = vsa.vsa_packed_attn(plan, q, k, v)
    for limit in (50_000_000, 5_000_000):
        t0 = time.monotonic()
        code, where = plan.wait_selftest(timeout_ns=limit)
        assert code == 6 and where in (240, 241)
        assert limit * 1e-9 <= time.monotonic() - t0 < 1.0
        assert plan.status() == (0, 0)
        assert torch.equal(vsa.vsa_packed_attn(plan, q, k, v), want)
        assert plan.status() == (0, 0)
    for limit in (0, 999, 10_000_000_001):
        with pytest.raises(vsa.VsaError):
            plan.wait_selftest(timeout_ns=limit)
    plan.destroy()
