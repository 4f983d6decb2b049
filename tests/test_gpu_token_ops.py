"""vsa_rms_norm and vsa_qk_rope on the GPU against their formulas in 64 bits.

Tolerances.  Every output is one rounding of a binary32 value: a bf16 rounding is off by at most 2^-8 of the
value, an E4M3 rounding by 2^-4 of it (2^-10 of the scale below the normal range).  F32 bounds the binary32
arithmetic before it, relative to the magnitudes added: a row sum of up to 16384 squares is added in chains of
at most 64 and then 14 levels of a tree (78 roundings of 2^-24, halved by the square root), and a handful of
products, a sine and a cosine of at most 2 ulp each; 1e-5 covers the sum of them, 78/2 * 2^-24 + 16 * 2^-24
= 3.3e-6, three times over."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
B_HALF, E_HALF, ARITH = 2.0 ** -8, 2.0 ** -4, 1e-5
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, scale=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# ---------------------------------------------------------------------------------------------- norm


def norm_ref(x, weight, eps, residual=None):
    t = x.double() if residual is None else x.double() + residual.double()
    y = t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)
    return t, y if weight is None else y * weight.double()


def check_norm(got, x, weight, eps, residual=None):
    out, scale, res = got
    t, y = norm_ref(x, weight, eps, residual)
    if residual is not None:
        half = B_HALF if res.dtype == BF16 else 2.0 ** -24
        assert ((res.double() - t).abs() <= half * t.abs() + 2.0 ** -24 * t.abs()).all()
    else:
        assert res is None
    if out.dtype == BF16:
        assert ((out.double() - y).abs() <= (B_HALF + 2 * ARITH) * y.abs()).all()
        return
    want = y.abs().amax(-1) / 448.0
    assert ((scale.double() - want).abs() <= ARITH * want).all()
    err = (out.double() * scale.double()[..., None] - y).abs()
    assert (err <= (E_HALF + 4 * ARITH) * y.abs() + 2.0 ** -10 * (1 + ARITH) * scale.double()[..., None]).all()
    # the codes use the whole range: the largest of a row is 448
    live = want > 0
    assert (out.double().abs().amax(-1)[live] == 448.0).all()
    assert (out.double().abs().amax(-1)[~live] == 0.0).all()


@pytest.mark.parametrize("residual", [None, BF16, F32])
@pytest.mark.parametrize("rows,width", [(300, 1016), (1537, 5120), (700, 8200)])
def test_norm_codes_are_the_nearest(vsa, rows, width, residual):
    """A code is E4M3(448 y / max|y|), off only where that value lies within the binary32 roundings of a tie:
    of t, of the largest product and its t, and of the value itself, 2^-24 of it each."""
    g = gen(rows + width)
    x, w = randn(g, rows, width), 1.0 + randn(g, width, scale=0.2)
    r = None if residual is None else randn(g, rows, width, scale=3.0, dtype=residual)
    out = torch.empty(rows, width, dtype=E4M3, device="cuda")
    scale = torch.empty(rows, dtype=F32, device="cuda")
    vsa.vsa_rms_norm(x, w, EPS, residual=r, out=out, scale=scale)
    _, y = norm_ref(x, w, EPS, r)
    value = 448.0 * y / y.abs().amax(-1, keepdim=True)
    nearest = value.float().to(E4M3)
    off = out.double() != nearest.double()
    tie = (out.double() + nearest.double())[off] / 2
    # (2^-25 more: the oracle's own rounding to binary32 before the conversion)
    assert ((tie - value[off]).abs() <= 4.5 * 2.0 ** -24 * value[off].abs()).all()


@pytest.mark.parametrize("out_dtype", [BF16, E4M3])
@pytest.mark.parametrize("residual", [None, BF16, F32])
@pytest.mark.parametrize("rows,width", [(1, 8), (3, 64), (5, 136), (33, 768), (257, 1032), (1, 5120), (64, 5376),
                                        (7, 8192), (600, 5120), (2, 16384)])
def test_norm(vsa, rows, width, residual, out_dtype):
    g = gen(rows * 1000 + width)
    x = randn(g, rows, width)
    r = None if residual is None else randn(g, rows, width, scale=3.0, dtype=residual)
    for w in (randn(g, width), randn(g, width, dtype=F32), None):
        check_norm(vsa.vsa_rms_norm(x, w, EPS, residual=r, out_dtype=out_dtype), x, w, EPS, r)


def test_norm_strided_rows_and_shapes(vsa):
    g = gen(1)
    wide = randn(g, 37, 3 * 256)
    x, r = wide[:, 256:512], wide[:, 512:]
    w = randn(g, 256)
    keep = wide.clone()
    buf = torch.full((37, 512), 7.0, dtype=BF16, device="cuda")
    got = vsa.vsa_rms_norm(x, w, EPS, residual=r, out=buf[:, 128:384])
    check_norm(got, x, w, EPS, r)
    assert torch.equal(wide, keep)
    assert (buf[:, :128] == 7).all() and (buf[:, 384:] == 7).all()  # nothing beside the rows
    x4 = randn(g, 2, 3, 5, 64)
    out, scale, _ = vsa.vsa_rms_norm(x4, None, EPS, out_dtype=E4M3)
    assert out.shape == x4.shape and scale.shape == (2, 3, 5)
    check_norm((out, scale, None), x4, None, EPS)
    one = randn(g, 1, 64).expand(9, 64)  # one row for all
    check_norm(vsa.vsa_rms_norm(one, w[:64].contiguous(), EPS), one, w[:64], EPS)
    empty = torch.empty(0, 64, dtype=BF16, device="cuda")
    out, scale, res = vsa.vsa_rms_norm(empty, None, EPS, residual=empty, out_dtype=E4M3)
    assert out.shape == (0, 64) and scale.shape == (0,) and res.shape == (0, 64)


@pytest.mark.parametrize("residual", [BF16, F32])
def test_norm_in_place(vsa, residual):
    g = gen(2)
    x, r, w = randn(g, 130, 5376), randn(g, 130, 5376, dtype=residual), randn(g, 5376)
    want = vsa.vsa_rms_norm(x, w, EPS, residual=r)
    x1, r1 = x.clone(), r.clone()
    out, _, res = vsa.vsa_rms_norm(x1, w, EPS, residual=r1, out=x1, residual_out=r1)
    assert out.data_ptr() == x1.data_ptr() and res.data_ptr() == r1.data_ptr()
    assert torch.equal(out, want[0]) and torch.equal(res, want[2])


def test_norm_magnitudes_and_zeros(vsa):
    """Rows of zeros, rows so small that 448 / max overflows, rows near the largest square: each its own row."""
    g = gen(3)
    base = torch.randn(6, 512, generator=g, device="cuda")
    r = base * torch.tensor([0.0, 1e-38, 1e-36, 1e-20, 1.0, 1e18], device="cuda")[:, None]
    x = torch.zeros(6, 512, dtype=BF16, device="cuda")
    w = 1.0 + 0.1 * torch.randn(512, generator=g, device="cuda")
    for eps in (1e-6, 1e-12):
        check_norm(vsa.vsa_rms_norm(x, w, eps, residual=r), x, w, eps, r)
        check_norm(vsa.vsa_rms_norm(x, w, eps, residual=r, out_dtype=E4M3), x, w, eps, r)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_norm_not_finite_stays_in_its_row(vsa, bad):
    g = gen(4)
    x = randn(g, 40, 1024)
    x[17, 1000] = bad
    w = randn(g, 1024)
    ok = torch.arange(40, device="cuda") != 17
    out, _, _ = vsa.vsa_rms_norm(x, w, EPS)
    assert out[17].isnan().any()
    check_norm((out[ok], None, None), x[ok], w, EPS)
    codes, scale, _ = vsa.vsa_rms_norm(x, w, EPS, out_dtype=E4M3)
    assert scale[17].isnan()
    check_norm((codes[ok], scale[ok], None), x[ok], w, EPS)


def test_norm_other_stream_capture_and_two_at_once(vsa):
    g = gen(5)
    xs = [randn(g, 300, 5120) for _ in range(2)]
    w = randn(g, 5120)
    want = [vsa.vsa_rms_norm(x, w, EPS, residual=x, out_dtype=E4M3) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            got.append(vsa.vsa_rms_norm(x, w, EPS, residual=x, out_dtype=E4M3))
    for s in streams:
        s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
        assert torch.equal(a[2], b[2])
    x, out, scale, res = xs[0].clone(), torch.empty(300, 5120, dtype=E4M3, device="cuda"), None, torch.empty_like(xs[0])
    scale = torch.empty(300, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsa.vsa_rms_norm(x, w, EPS, residual=x, out=out, scale=scale, residual_out=res)
    for i in (1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.uint8), want[i][0].view(torch.uint8)) and torch.equal(scale, want[i][1])


def test_norm_binding_refusals(vsa):
    g = gen(6)
    x = randn(g, 4, 64)
    for kw, err in [(dict(residual=x.half()), TypeError), (dict(out=torch.empty_like(x, dtype=F32)), TypeError),
                    (dict(weight=x[0].half()), TypeError), (dict(weight=x[0, :32]), ValueError),
                    (dict(residual=x[:2]), ValueError), (dict(out=x[:, :32]), ValueError),
                    (dict(scale=torch.empty(4, device="cuda")), ValueError), (dict(residual_out=x), ValueError),
                    (dict(out_dtype=E4M3, scale=torch.empty(3, device="cuda")), ValueError),
                    (dict(residual=x.cpu()), ValueError)]:
        with pytest.raises(err):
            vsa.vsa_rms_norm(x, eps=EPS, **kw)
    with pytest.raises(TypeError):
        vsa.vsa_rms_norm(x.float())
    with pytest.raises(ValueError):
        vsa.vsa_rms_norm(randn(g, 64, 4).t())  # rows are not contiguous
    with pytest.raises(vsa.VsaError):
        vsa.vsa_rms_norm(randn(g, 4, 60))
    with pytest.raises(vsa.VsaError):
        vsa.vsa_rms_norm(randn(g, 4, 72)[:, 1:65])  # rows that do not start on 16 bytes


# ---------------------------------------------------------------------------------------------- rope


def rope_ref(rope, x, positions, weight=None, eps=EPS):
    """(value, magnitude of the terms added) in 64 bits; x [T, H, D], positions [T, axes]."""
    f, axis = rope.table()
    f, axis = torch.from_numpy(f).cuda(), torch.from_numpy(axis).long().cuda()
    angle = (positions.double()[:, axis] * f)[:, None]
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    half = y.shape[-1] // 2
    a, b = (y[..., 0::2], y[..., 1::2]) if rope.interleaved else (y[..., :half], y[..., half:])
    lo, hi = a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()
    mag = a.abs() + b.abs()
    if rope.interleaved:
        return torch.stack((lo, hi), -1).flatten(-2), torch.stack((mag, mag), -1).flatten(-2)
    return torch.cat((lo, hi), -1), torch.cat((mag, mag), -1)


def check_rope(got, rope, x, positions, weight=None, eps=EPS):
    want, mag = rope_ref(rope, x, positions, weight, eps)
    assert ((got.double() - want).abs() <= B_HALF * want.abs() + 2 * ARITH * mag).all()


def positions_for(g, tokens, axes, dtype=torch.int32, most=3000):
    p = torch.randint(-most // 8, most, (tokens, axes), generator=g, device="cuda", dtype=torch.int32)
    return p if dtype == torch.int32 else p.float() * 0.375


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,H,Hk", [(1, 1, 1), (3, 56, 56), (77, 40, 8), (130, 2, 1), (65, 7, 1), (5, 300, 3),
                                         (1, 64, 8), (33, 1, 0)])
def test_rope(vsa, D, interleaved, tokens, H, Hk):
    g = gen(D + tokens * 7 + H)
    sections = {64: (8, 12, 12), 96: (16, 16, 16), 128: (16, 22, 22)}[D]
    q = randn(g, tokens, H, D, scale=2.0)
    k = randn(g, tokens, Hk, D, scale=2.0) if Hk else None
    for shared, dtype, weighted in ((False, torch.int32, True), (True, torch.float32, False)):
        rope = vsa.vsa_rope_create(D, sections, interleaved=interleaved, shared_ladder=shared)
        pos = positions_for(g, tokens, 3, dtype)
        qw = 1 + 0.2 * randn(g, D) if weighted else None
        kw = 1 + 0.2 * randn(g, D) if weighted and Hk else None
        qo, ko = vsa.vsa_qk_rope(rope, q, k, pos, q_weight=qw, k_weight=kw, eps=EPS)
        check_rope(qo, rope, q, pos, qw)
        if Hk:
            check_rope(ko, rope, k, pos, kw)
        else:
            assert ko is None


def test_rope_norm_on_one_side_only(vsa):
    g = gen(11)
    q, k, w = randn(g, 50, 5, 96), randn(g, 50, 2, 96), randn(g, 96)
    rope = vsa.vsa_rope_create(96, (10, 20, 5))
    pos = positions_for(g, 50, 3)
    for qw, kw in ((w, None), (None, w)):
        qo, ko = vsa.vsa_qk_rope(rope, q, k, pos, q_weight=qw, k_weight=kw)
        check_rope(qo, rope, q, pos, qw)
        check_rope(ko, rope, k, pos, kw)
    # pairs behind the sections do not turn: without a norm they come back as they were
    qo, _ = vsa.vsa_qk_rope(rope, q, k, pos)
    still = torch.cat((torch.arange(35, 48), torch.arange(83, 96))).cuda()
    assert torch.equal(qo[..., still], q[..., still])


@pytest.mark.parametrize("D", [64, 96, 128])
def test_rope_many_tokens_of_one_head(vsa, D):
    """One head, no keys: the most tokens a CTA takes at a time, over more tokens than the GPU holds CTAs for, so that
    each takes several in turn; the last CTA's run past the end."""
    g = gen(D)
    T = 4 * 8 * 148 * 64 + 37
    q = randn(g, T, 1, D)
    rope = vsa.vsa_rope_create(D, (D // 4, D // 4))
    pos = positions_for(g, T, 2)
    w = randn(g, D)
    buf = torch.full((T + 64, 1, D), 5.0, dtype=BF16, device="cuda")
    out, _ = vsa.vsa_qk_rope(rope, q, None, pos, q_weight=w, q_out=buf[:T])
    check_rope(out, rope, q, pos, w)
    assert (buf[T:] == 5).all()


def test_norm_many_rows(vsa):
    """More rows than CTAs, uneven, at widths of every chunk count per thread and of the warp rows."""
    g = gen(20)
    for width in (200, 520, 1000, 1024, 1048, 2048, 4104, 5376, 8200, 12296):
        rows = 5003 if width <= 5376 else 1301
        x, w = randn(g, rows, width), randn(g, width)
        check_norm(vsa.vsa_rms_norm(x, w, EPS), x, w, EPS)
        r = randn(g, rows, width, dtype=F32)
        check_norm(vsa.vsa_rms_norm(x, w, EPS, residual=r, out_dtype=E4M3), x, w, EPS, r)
        check_norm(vsa.vsa_rms_norm(x, w, EPS, residual=x), x, w, EPS, x)


def test_rope_norm_of_extreme_rows(vsa):
    """Head rows whose squares leave binary32's range on either side, each its own row."""
    g = gen(18)
    scale = torch.tensor([1e-38, 1e-25, 1e-12, 1.0, 1e12, 1e19, 1e37, 0.0], device="cuda")
    for D in (64, 96, 128):
        q = (torch.randn(13, 8, D, generator=g, device="cuda").clamp(-4, 4) * scale[:, None]).to(BF16)
        rope = vsa.vsa_rope_create(D, (D // 2,))
        pos, w = positions_for(g, 13, 1), randn(g, D)
        for eps in (1e-6, 1e-36):
            qo, _ = vsa.vsa_qk_rope(rope, q, None, pos, q_weight=w, eps=eps)
            check_rope(qo, rope, q, pos, w, eps)


def test_rope_far_positions(vsa):
    """Positions up to the largest int32: the angle's error stays that of the 64-bit reference's own product
    (2^31 * 2^-53 = 2.4e-7 rad) plus binary32's."""
    g = gen(12)
    q = randn(g, 64, 2, 128)
    rope = vsa.vsa_rope_create(128, (64,), theta=1e6)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (64, 1), generator=g, device="cuda", dtype=torch.int64).int()
    pos[0], pos[1] = 2 ** 31 - 1, -2 ** 31
    qo, _ = vsa.vsa_qk_rope(rope, q, None, pos)
    check_rope(qo, rope, q, pos)
    posf = torch.full((64, 1), 16777215.0, device="cuda")
    qo, _ = vsa.vsa_qk_rope(rope, q, None, posf)
    check_rope(qo, rope, q, posf)


def test_rope_own_table(vsa):
    g = gen(13)
    freq = [0.5 ** (i / 8) * (-1) ** i for i in range(32)]
    axis = [(0, 1, 2, 3)[i % 4] for i in range(32)]
    rope = vsa.vsa_rope_create(64, inv_freq=freq, axis=axis)
    q, pos = randn(g, 9, 3, 64), positions_for(g, 9, 4)
    check_rope(vsa.vsa_qk_rope(rope, q, None, pos)[0], rope, q, pos)


def test_rope_strides_in_place_and_batches(vsa):
    g = gen(14)
    H, Hk, D, B, L = 5, 2, 128, 3, 41
    rope = vsa.vsa_rope_create(D, (16, 24, 24), interleaved=True)
    qkv = randn(g, B, L, H + 2 * Hk, D)
    keep = qkv.clone()
    pos = positions_for(g, L, 3)
    w = randn(g, D)
    q, k = qkv[:, :, :H], qkv[:, :, H:H + Hk]
    qo, ko = vsa.vsa_qk_rope(rope, q, k, pos, q_weight=w, k_weight=w)  # [L, 3] serves every sequence
    assert qo.shape == q.shape and torch.equal(qkv, keep)
    every = pos.repeat(B, 1)
    check_rope(qo.flatten(0, 1), rope, q.flatten(0, 1), every, w)
    check_rope(ko.flatten(0, 1), rope, k.flatten(0, 1), every, w)
    vsa.vsa_qk_rope(rope, q, k, every.view(B, L, 3), q_weight=w, k_weight=w, q_out=q, k_out=k)  # in place, both slices
    assert torch.equal(qkv[:, :, :H], qo) and torch.equal(qkv[:, :, H:H + Hk], ko)
    assert torch.equal(qkv[:, :, H + Hk:], keep[:, :, H + Hk:])  # V untouched
    # head-major storage
    heads_first = randn(g, H, L, D)
    q2 = heads_first.transpose(0, 1)
    out2 = torch.empty(H, L, D, dtype=BF16, device="cuda").transpose(0, 1)
    vsa.vsa_qk_rope(rope, q2, None, pos, q_out=out2)
    check_rope(out2, rope, q2, pos)


def test_rope_not_finite_stays_in_its_head(vsa):
    g = gen(15)
    q, w = randn(g, 20, 6, 64), randn(g, 64)
    q[7, 3, 9] = float("nan")
    q[8, 2, 40] = float("inf")
    rope = vsa.vsa_rope_create(64, (32,))
    pos = positions_for(g, 20, 1)
    qo, _ = vsa.vsa_qk_rope(rope, q, None, pos, q_weight=w)
    bad = torch.zeros(20, 6, dtype=torch.bool, device="cuda")
    bad[7, 3] = bad[8, 2] = True
    want, mag = rope_ref(rope, q, pos, w)
    assert qo[7, 3].isnan().all() and qo[8, 2].isnan().any()
    assert ((qo.double() - want).abs() <= B_HALF * want.abs() + 2 * ARITH * mag)[~bad].all()


def test_rope_capture_and_other_stream(vsa):
    g = gen(16)
    rope = vsa.vsa_rope_create(96, (16, 16, 16))
    qs = [randn(g, 100, 8, 96) for _ in range(2)]
    pos = positions_for(g, 100, 3)
    want = [vsa.vsa_qk_rope(rope, q, q, pos) for q in qs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(qs[0])
    vsa.vsa_qk_rope(rope, qs[1], None, pos, q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want[1][0])
    q, ko = qs[0].clone(), torch.empty_like(qs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsa.vsa_qk_rope(rope, q, q, pos, q_out=out, k_out=ko)
    for i in (1, 0):
        q.copy_(qs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(ko, want[i][1])


def test_rope_binding_refusals(vsa):
    g = gen(17)
    rope = vsa.vsa_rope_create(64, (16, 16))
    q, pos = randn(g, 4, 2, 64), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for args, kw, err in [((q.float(), None, pos), {}, TypeError), ((q, None, pos.long()), {}, TypeError),
                          ((q, None, pos[:, :1]), {}, ValueError), ((q, q[:3], pos), {}, ValueError),
                          ((q, None, pos), dict(k_weight=q[0, 0]), ValueError),
                          ((q, None, pos), dict(q_weight=q[0, 0].float()), TypeError),
                          ((q, None, pos), dict(q_weight=q[0, 0, :32]), ValueError),
                          ((q, None, pos), dict(q_out=q[:2]), ValueError),
                          ((q[..., :32], None, pos), {}, ValueError),
                          ((q, None, pos.cpu()), {}, ValueError)]:
        with pytest.raises(err):
            vsa.vsa_qk_rope(rope, *args, **kw)
    with pytest.raises(vsa.VsaError):
        vsa.vsa_qk_rope(rope, q, None, torch.zeros(3, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):  # unevenly spaced tokens
        vsa.vsa_qk_rope(rope, randn(g, 2, 9, 2, 64)[:, :5], None, pos)
