"""Calls with `stream=`: what a call allocates and fills belongs to that stream, as under torch.cuda.stream(stream)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
BUSY = 200_000_000  # cycles for which a stream is kept busy, about a tenth of a second


@pytest.fixture(scope="module")
def vsa():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as m

    m.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    return m


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)


@pytest.mark.parametrize("raw", [False, True])
def test_packed_rows_behind_are_zeroed_on_the_calls_stream(vsa, raw):
    """The current stream is busy; a reader on the call's stream sees the zeros all the same."""
    lengths, T, D = (60, 41), 165, 64
    n = sum(lengths)
    q, k, v = randn(1, T, 4, D), randn(2, T, 2, D), randn(3, T, 2, D)
    plan = vsa.vsa_packed_plan(lengths, 4, 2, D)
    want = vsa.vsa_packed_attn(plan, q, k, v)
    s = torch.cuda.Stream()
    used = [torch.full_like(q, 7.0) for _ in range(4)]  # what memory the allocator may hand out holds sevens
    with torch.cuda.stream(s):
        used += [torch.full_like(q, 7.0) for _ in range(4)]
    torch.cuda.synchronize()
    del used
    torch.cuda._sleep(BUSY)
    out = vsa.vsa_packed_attn(plan, q, k, v, stream=s.cuda_stream if raw else s)
    with torch.cuda.stream(s):
        seen = out.clone()
    s.synchronize()
    assert torch.equal(seen[:n], want[:n])
    assert (seen[n:] == 0).all()


def reused_by_the_current_stream(call, s):
    """Whether memory that `call` allocated goes to the current stream while the call's stream is still busy with it."""
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    outs = [t for t in call(s) if t is not None]
    like = [(t.shape, t.dtype, t.data_ptr()) for t in outs]
    del outs
    fresh = {torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype, _ in like}
    hit = {t.data_ptr() for t in fresh} & {p for _, _, p in like}
    s.synchronize()
    return hit


def test_outputs_are_not_reused_while_the_calls_stream_writes_them(vsa):
    x, w = randn(4, 300, 5120), randn(5, 5120)
    q, k, v = randn(6, 700, 8, 128), randn(7, 700, 2, 128), randn(8, 700, 2, 128)
    rope = vsa.vsa_rope_create(128, (64,))
    pos = torch.arange(700, dtype=torch.int32, device="cuda")[:, None]
    plan = vsa.vsa_packed_plan((700,), 8, 2, 128)
    s = torch.cuda.Stream()
    for call in (lambda s: vsa.vsa_rms_norm(x, w, residual=x, out_dtype=E4M3, stream=s),
                 lambda s: vsa.vsa_qk_rope(rope, q, k, pos, stream=s),
                 lambda s: (vsa.vsa_packed_attn(plan, q, k, v, stream=s),)):
        call(None)
        torch.cuda.synchronize()
        assert not reused_by_the_current_stream(call, s)


def test_forward_allocates_on_the_calls_stream(vsa, monkeypatch):
    plan = vsa.vsa_plan_tiles(1, 2, 64, segments=(70,), grid=(4, 8, 8), sparsity=0.5)
    q, k, v = (randn(9 + i, 1, 70 + 256, 2, 64) for i in range(3))
    gate = randn(12, 1, 70 + 256, 2)
    want = vsa.vsa_forward(plan, q, k, v, gate)
    s, at = torch.cuda.Stream(), []
    alloc = vsa.alloc_workspace
    monkeypatch.setattr(vsa, "alloc_workspace", lambda *a: (at.append(torch.cuda.current_stream()), alloc(*a))[1])
    assert not reused_by_the_current_stream(lambda s: (vsa.vsa_forward(plan, q, k, v, gate, stream=s),), s)
    torch.cuda.synchronize()
    out = torch.zeros_like(q)
    vsa.vsa_forward_parts(plan, [q], [k], [v], [gate], [out], 0, stream=s)
    s.synchronize()
    assert at == [s, s] and torch.equal(out, want)


@pytest.mark.parametrize("raw", [0, 1, 2])
def test_raw_handles_of_the_default_streams(vsa, raw):
    """0 and 1 name the legacy default stream, 2 the calling thread's own."""
    x, w = randn(20, 30, 512), randn(21, 512)
    q, k, v = randn(22, 40, 4, 64), randn(23, 40, 2, 64), randn(24, 40, 2, 64)
    plan = vsa.vsa_packed_plan((30,), 4, 2, 64)
    want = vsa.vsa_rms_norm(x, w, residual=x, out_dtype=E4M3)
    attn = vsa.vsa_packed_attn(plan, q, k, v)
    torch.cuda.synchronize()
    got = vsa.vsa_rms_norm(x, w, residual=x, out_dtype=E4M3, stream=raw)
    out = vsa.vsa_packed_attn(plan, q, k, v, stream=raw)
    torch.cuda.synchronize()
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
    assert torch.equal(got[2], want[2]) and torch.equal(out, attn)
