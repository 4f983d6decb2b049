"""Outputs over memory that a call still reads, through the binding: refused; slices that lie beside one another work."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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


def refused(call, *args, **kw):
    with pytest.raises(RuntimeError, match="VSA_ERR_INVALID_ARG"):
        call(*args, **kw)


@pytest.mark.parametrize("D", [64, 96, 128])
def test_packed_output_beside_and_over_the_inputs(vsa, D):
    T, H, Hk = 200, 4, 2
    plan = vsa.vsa_packed_plan((150, 50), H, Hk, D)
    buf = randn(D, T, 2 * H + 2 * Hk, D)
    q, k, v, rest = buf.split((H, Hk, Hk, H), 1)
    keep = buf.clone()
    for out in (buf[:, 1:1 + H], buf[:, H - 1:2 * H - 1], buf[:, H + Hk:2 * H + Hk], buf[:, H + 2 * Hk - 1:-1]):
        refused(vsa.vsa_packed_attn, plan, q, k, v, out=out)
    flat = buf.view(-1, D)
    refused(vsa.vsa_packed_attn, plan, q, k, v, out=flat[:T * H].view(T, H, D))  # other strides over all of them
    refused(vsa.vsa_packed_attn, plan, q.contiguous(), k, v, out=buf[:, H:2 * H])  # over k and v, and no more
    assert torch.equal(buf, keep)
    want = vsa.vsa_packed_attn(plan, q, k, v)
    got = vsa.vsa_packed_attn(plan, q, k, v, out=rest)
    assert got.data_ptr() == rest.data_ptr() and torch.equal(rest, want) and torch.equal(buf[:, :-H], keep[:, :-H])
    vsa.vsa_packed_attn(plan, q, k, v, out=q)
    assert torch.equal(q, want) and torch.equal(buf[:, H:-H], keep[:, H:-H])


def test_rope_output_beside_and_over_the_inputs(vsa):
    T, H, Hk, D = 90, 4, 2, 64
    rope = vsa.vsa_rope_create(D, (32,))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[:, None]
    buf = randn(1, T, 2 * H + Hk, D)
    q, k, rest = buf.split((H, Hk, H), 1)
    keep = buf.clone()
    refused(vsa.vsa_qk_rope, rope, q, k, pos, q_out=buf[:, 1:1 + H])
    refused(vsa.vsa_qk_rope, rope, q, k, pos, k_out=q[:, :Hk])
    refused(vsa.vsa_qk_rope, rope, q, q, pos, q_out=q)  # k is read from the rows that q_out replaces
    refused(vsa.vsa_qk_rope, rope, q, k, pos, q_out=rest, k_out=rest[:, 2:])
    assert torch.equal(buf, keep)
    want = vsa.vsa_qk_rope(rope, q, k, pos)
    vsa.vsa_qk_rope(rope, q, k, pos, q_out=rest, k_out=k)
    assert torch.equal(rest, want[0]) and torch.equal(k, want[1]) and torch.equal(q, keep[:, :H])
    pairs = torch.empty(T, Hk, 2, D, dtype=BF16, device="cuda")  # two outputs interleaved head by head
    vsa.vsa_qk_rope(rope, q[:, :Hk], keep[:, H:H + Hk], pos, q_out=pairs[:, :, 0], k_out=pairs[:, :, 1])
    assert torch.equal(pairs[:, :, 0], want[0][:, :Hk]) and torch.equal(pairs[:, :, 1], want[1])


def test_norm_output_beside_and_over_the_inputs(vsa):
    rows, C = 70, 256
    buf = randn(2, rows + 1, 3 * C)
    x, r = buf[:rows, :C], buf[:rows, C:2 * C]
    keep = buf.clone()
    refused(vsa.vsa_rms_norm, x, residual=r, out=buf[1:, :C])
    refused(vsa.vsa_rms_norm, x, residual=r, out=buf[:rows, C - 8:2 * C - 8])
    refused(vsa.vsa_rms_norm, x, residual=r, residual_out=buf[1:, C:2 * C])
    refused(vsa.vsa_rms_norm, x, residual=r, out=x, residual_out=x)
    assert torch.equal(buf, keep)
    want = vsa.vsa_rms_norm(x, residual=r)
    vsa.vsa_rms_norm(x, residual=r, out=buf[:rows, 2 * C:], residual_out=x)  # the stream moves from r to x
    assert torch.equal(buf[:rows, 2 * C:], want[0]) and torch.equal(x, want[2])


def test_chunks_of_positions_and_scales(vsa):
    """A chunk of the positions, and of a buffer of scales, from any row on."""
    T, D = 61, 64
    rope = vsa.vsa_rope_create(D, (10, 12, 10))
    pos = torch.randint(0, 99, (T, 3), dtype=torch.int32, device="cuda")
    q, x = randn(3, T, 2, D), randn(4, T, 128)
    every, _ = vsa.vsa_qk_rope(rope, q, None, pos)
    codes, scales, _ = vsa.vsa_rms_norm(x, out_dtype=torch.float8_e4m3fn)
    chunked = torch.full((T + 3,), 7.0, device="cuda")
    for a, b in ((0, 5), (5, 6), (6, 61)):
        part, _ = vsa.vsa_qk_rope(rope, q[a:b], None, pos[a:b])
        assert torch.equal(part, every[a:b])
        out, _, _ = vsa.vsa_rms_norm(x[a:b], out_dtype=torch.float8_e4m3fn, scale=chunked[1 + a:1 + b])
        assert torch.equal(out.view(torch.uint8), codes[a:b].view(torch.uint8))
    assert torch.equal(chunked[1:T + 1], scales) and (chunked[[0, T + 1, T + 2]] == 7).all()
