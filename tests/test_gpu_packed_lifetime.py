"""A packed plan that is collected while a graph is captured leaves the capture alone."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_plan_collected_during_a_capture():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as vsa

    q, k, v = (torch.randn(130, n, 64, device="cuda").to(torch.bfloat16) for n in (4, 2, 2))
    plan, other = vsa.vsa_packed_plan((100, 30), 4, 2, 64), vsa.vsa_packed_plan((130,), 4, 2, 64)
    want = vsa.vsa_packed_attn(plan, q, k, v)
    vsa.vsa_packed_attn(other, q, k, v)  # still running, perhaps, when its plan is collected
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        del other
        gc.collect()
        vsa.vsa_packed_attn(plan, q, k, v, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and plan.status() == (0, 0)
    fresh = vsa.vsa_packed_plan((130,), 4, 2, 64)  # frees the collected one
    assert not vsa._collected_plans
    vsa.vsa_packed_attn(fresh, q, k, v)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
