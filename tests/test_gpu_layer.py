"""The token operators as a transformer block uses them, one after another on one stream: norm (with the residual's
addition) -> projection -> head norm and rotary positions on slices of the projection, in place -> attention
(packed prompts, or the video forward) -> projection -> norm.  Every call is held to its own formula in 64 bits on
the inputs it really got (the tolerances are those of test_gpu_token_ops.py and test_gpu_packed.py, and the oracle's
for the video forward); the whole run is also captured and replayed with other inputs."""
import numpy as np
import pytest
import torch

import synth
from test_gpu_packed import check as check_attn
from test_gpu_token_ops import check_norm, check_rope

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-6


@pytest.fixture(scope="module")
def vsa():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as m

    m.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    return m


def weights(g, C, H, Hk, D):
    def r(*s, scale=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * scale).to(BF16)

    return dict(norm1=1 + 0.1 * r(C), norm2=1 + 0.1 * r(C), q=1 + 0.1 * r(D), k=1 + 0.1 * r(D),
                qkv=r(C, (H + 2 * Hk) * D, scale=C ** -0.5), out=r(H * D, C, scale=(H * D) ** -0.5))


@pytest.mark.parametrize("D,out_dtype", [(128, E4M3), (96, BF16), (64, E4M3)])
def test_text_block(vsa, D, out_dtype):
    lengths, H, Hk, C = (77, 1, 0, 300, 129), 10, 2, 640
    T = sum(lengths)
    g = torch.Generator(device="cuda").manual_seed(D)
    w = weights(g, C, H, Hk, D)
    rope = vsa.vsa_rope_create(D, (D // 4, D // 8, D // 8), shared_ladder=True)
    plan = vsa.vsa_packed_plan(lengths, H, Hk, D)
    pos = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in lengths])[:, None].expand(-1, 3).contiguous()

    def block(x, res):
        """x: the block before's output; res: the residual stream, updated in place."""
        y, scale, _ = vsa.vsa_rms_norm(x, w["norm1"], EPS, residual=res, residual_out=res, out_dtype=out_dtype)
        h = y if scale is None else (y.float() * scale[:, None]).to(BF16)
        qkv = (h @ w["qkv"]).view(T, H + 2 * Hk, D)
        raw = qkv.clone()
        q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        vsa.vsa_qk_rope(rope, q, k, pos, q_weight=w["q"], k_weight=w["k"], eps=EPS, q_out=q, k_out=k)
        o = vsa.vsa_packed_attn(plan, q, k, v)
        a = o.view(T, H * D) @ w["out"]
        z, _, res2 = vsa.vsa_rms_norm(a, w["norm2"], EPS, residual=res)
        return dict(y=y, scale=scale, raw=raw, qkv=qkv, o=o, a=a, z=z, res2=res2)

    xs = [(torch.randn(T, C, generator=g, device="cuda").to(BF16), torch.randn(T, C, generator=g, device="cuda") * 3)
          for _ in range(2)]
    for x, res0 in xs:
        res = res0.clone()
        s = block(x, res)
        torch.cuda.synchronize()
        check_norm((s["y"], s["scale"], res), x, w["norm1"], EPS, res0)
        check_rope(s["qkv"][:, :H], rope, s["raw"][:, :H], pos, w["q"])
        check_rope(s["qkv"][:, H:H + Hk], rope, s["raw"][:, H:H + Hk], pos, w["k"])
        assert torch.equal(s["qkv"][:, H + Hk:], s["raw"][:, H + Hk:])
        check_attn(s["o"], s["qkv"][:, :H], s["qkv"][:, H:H + Hk], s["qkv"][:, H + Hk:], lengths, True)
        check_norm((s["z"], None, s["res2"]), s["a"], w["norm2"], EPS, res)
    # captured: the projections' library calls warm up on the capture's stream first
    x, res = xs[0][0].clone(), xs[0][1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, res.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(x, res)
    for i in (1, 0):
        x.copy_(xs[i][0])
        res.copy_(xs[i][1])
        graph.replay()
        torch.cuda.synchronize()
        # a product's library kernel may differ between eager and captured runs, so each stage by its own inputs
        check_norm((got["y"], got["scale"], res), xs[i][0], w["norm1"], EPS, xs[i][1])
        check_attn(got["o"], got["qkv"][:, :H], got["qkv"][:, H:H + Hk], got["qkv"][:, H + Hk:], lengths, True)
        check_norm((got["z"], None, got["res2"]), got["a"], w["norm2"], EPS, res)
    assert plan.status() == (0, 0)


@pytest.mark.parametrize("name", ["tiny", "small"])
def test_video_block(vsa, oracle_mod, name):
    """Head norm and rotary positions (time, height, width behind the prefix) in place on the projection's Q and K,
    then the video forward on them, against the oracle on the same bits."""
    w = synth.workload(name)
    L, H, D, C = w.seq_len, w.heads, w.head_dim, 512
    g = torch.Generator(device="cuda").manual_seed(3)
    wt = weights(g, C, H, H, D)
    x = (torch.randn(w.batch, L, C, generator=g, device="cuda")).to(BF16)
    gate = (0.1 * torch.randn(w.batch, L, H, generator=g, device="cuda")).to(BF16)
    prefix = sum(w.segments)
    t, h, ww = w.grid
    grid = torch.stack(torch.meshgrid(*(torch.arange(n, device="cuda", dtype=torch.int32) for n in (t, h, ww)), indexing="ij"), -1)
    pos = torch.cat((torch.arange(prefix, device="cuda", dtype=torch.int32)[:, None].expand(-1, 3), grid.reshape(-1, 3) + prefix)).contiguous()
    y, _, _ = vsa.vsa_rms_norm(x, wt["norm1"], EPS)
    check_norm((y, None, None), x, wt["norm1"], EPS)
    qkv = (y @ wt["qkv"]).view(w.batch, L, 3 * H, D)
    raw = qkv.clone()
    q, k = qkv[:, :, :H], qkv[:, :, H:2 * H]
    rope = vsa.vsa_rope_create(D, (D // 8, 3 * D // 16, 3 * D // 16))
    vsa.vsa_qk_rope(rope, q, k, pos, q_weight=wt["q"], k_weight=wt["k"], q_out=q, k_out=k)
    every = pos.repeat(w.batch, 1)
    check_rope(q.flatten(0, 1), rope, raw[:, :, :H].flatten(0, 1), every, wt["q"])
    check_rope(k.flatten(0, 1), rope, raw[:, :, H:2 * H].flatten(0, 1), every, wt["k"])
    q, k, v = (s.contiguous() for s in (q, k, qkv[:, :, 2 * H:]))
    plan = vsa.vsa_plan_tiles(batch=w.batch, heads=H, head_dim=D, segments=w.segments, grid=w.grid, sparsity=w.sparsity)
    ws = vsa.alloc_workspace(plan)
    out = vsa.vsa_forward(plan, q, k, v, gate, workspace=ws)
    torch.cuda.synchronize()
    assert vsa.device_status(plan) == (0, 0)
    bits = [synth.as_bits(s) for s in (q, k, v, gate)]
    ref = oracle_mod.forward(*bits, w.segments, w.grid, w.sparsity)
    assert np.array_equal(vsa.workspace_views(plan, ws)["idx"].cpu().numpy(), ref.idx)
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - ref.out)
    assert err.max() <= 2e-2 and err.mean() <= 2e-3
    plan.destroy()


def test_packed_matches_the_dense_forward(vsa):
    """One sequence without a mask is the video forward's dense case (no video tiles: every query attends to every
    key; the gate zero, so no compression term): two kernels, one formula."""
    for D, L in ((128, 700), (64, 129), (96, 1000)):
        g = torch.Generator(device="cuda").manual_seed(L)
        q, k, v = (torch.randn(1, L, 4, D, generator=g, device="cuda").to(BF16) for _ in range(3))
        gate = torch.zeros(1, L, 4, dtype=BF16, device="cuda")
        plan = vsa.vsa_plan_tiles(batch=1, heads=4, head_dim=D, segments=(L,))
        want = vsa.vsa_forward(plan, q, k, v, gate)
        packed = vsa.vsa_packed_plan((L,), 4, 4, D, causal=False)
        got = vsa.vsa_packed_attn(packed, q, k, v)
        check_attn(got[0], q[0], k[0], v[0], (L,), False)
        check_attn(want[0], q[0], k[0], v[0], (L,), False)
        plan.destroy()
        packed.destroy()
