"""vsa_packed_attn on the GPU against softmax(scale q k^T) v in 64 bits, sequence by sequence.

Tolerances.  The kernel rounds twice: every weight p to bf16 for the P.V product and the output to bf16, each by
at most H = 2^-8 of its value.  So |error| <= H (sum_j p_ij |v_j| + |o|) in the worst case; and the roundings
being independent and each uniform within its step (a root mean square of at most H / sqrt 3), the error's root
mean square over an output stays below H / sqrt 3 * rms(sqrt(sum_j p_ij^2 v_j^2 + o^2)).  The binary32 arithmetic
between them: scores of up to about 2^6 log2 units held to 2^-24 of themselves give weights within 2^-17, the
exponential 2^-22, sums of up to 8192 terms in chains of 64 per partial product 2^-17: ARITH = 2^-14 of
sum_j p_ij |v_j| covers them.  A key dropped, doubled or taken from a neighbour moves an output row by a weight
times a value, which the root-mean-square bound sees at the lengths tested."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, H, ARITH = torch.bfloat16, 2.0 ** -8, 2.0 ** -14


@pytest.fixture(scope="module")
def vsa():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as m

    m.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    return m


def inputs(seed, tokens, heads, kv_heads, D, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(n):
        return (torch.randn(tokens, n, D, generator=g, device="cuda") * scale).to(BF16)

    return r(heads), r(kv_heads), r(kv_heads)


def reference(q, k, v, lengths, causal, scale=None):
    """(output, sum p |v|, sum p^2 v^2) in 64 bits, [T, H, D]."""
    T, Hq, D = q.shape
    g = Hq // k.shape[1]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = [torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device) for _ in range(3)]
    at = 0
    for n in lengths:
        s = slice(at, at + n)
        at += n
        if n == 0:
            continue
        kk, vv = (x[s].double().transpose(0, 1).repeat_interleave(g, 0) for x in (k, v))
        x = q[s].double().transpose(0, 1) @ kk.transpose(1, 2) * scale
        if causal:
            x.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1), -math.inf)
        p = torch.softmax(x, -1)
        for o, (a, b) in zip(out, ((p, vv), (p, vv.abs()), (p * p, vv * vv))):
            o[s] = (a @ b).transpose(0, 1)
    return out


def check(got, q, k, v, lengths, causal, scale=None):
    n = sum(lengths)
    want, mag, sq = (x[:n] for x in reference(q, k, v, lengths, causal, scale))
    err = (got[:n].double() - want).abs()
    assert torch.isfinite(got[:n]).all()
    assert (err <= (H + ARITH) * mag + H * (1 + H) * want.abs()).all(), (err / (mag + want.abs())).max().item()
    if n:
        rms = err.square().mean().sqrt()
        most = H / math.sqrt(3) * (sq + want.square()).mean().sqrt() + ARITH * mag.square().mean().sqrt()
        assert rms <= 1.05 * most, (rms.item(), most.item())


def run(vsa, q, k, v, lengths, causal, **kw):
    plan = vsa.vsa_packed_plan(lengths, q.shape[1], k.shape[1], q.shape[2], causal=causal, **kw)
    out = vsa.vsa_packed_attn(plan, q, k, v)
    torch.cuda.synchronize()
    assert plan.status() == (0, 0)
    plan.destroy()
    return out


LENGTHS = [(1,), (17,), (128,), (129,), (1, 0, 1, 33, 5), (255, 256, 257), (64, 500, 3, 127, 16, 900), (1537,)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (5, 1), (40, 8), (9, 3)])
def test_packed(vsa, heads, kv_heads, D, causal):
    for i, lengths in enumerate(LENGTHS):
        q, k, v = inputs(100 * i + D + heads, sum(lengths), heads, kv_heads, D)
        check(run(vsa, q, k, v, lengths, causal), q, k, v, lengths, causal)


@pytest.mark.parametrize("heads,kv_heads", [(128, 1), (66, 1), (120, 2), (56, 56), (3, 1)])
def test_packed_groups(vsa, heads, kv_heads):
    """Tiles of one token, of tokens that do not fill 128 rows, of 128 tokens."""
    for causal in (True, False):
        lengths = (70, 1, 200, 13)
        q, k, v = inputs(heads, sum(lengths), heads, kv_heads, 64)
        check(run(vsa, q, k, v, lengths, causal), q, k, v, lengths, causal)


def test_packed_every_short_length(vsa):
    """All lengths 0..145 in one batch: every position of a sequence's end inside a 16-key step and a block."""
    lengths = list(range(146))
    for D, causal in ((128, True), (64, False)):
        q, k, v = inputs(D, sum(lengths), 2, 1, D)
        check(run(vsa, q, k, v, lengths, causal), q, k, v, lengths, causal)


def test_packed_long(vsa):
    lengths = (5000, 1, 3333)
    for D, heads, kv_heads, causal in ((128, 4, 2, True), (96, 2, 2, False), (64, 6, 1, True)):
        q, k, v = inputs(D, sum(lengths), heads, kv_heads, D)
        check(run(vsa, q, k, v, lengths, causal), q, k, v, lengths, causal)


def test_packed_growing_scores(vsa):
    """Keys whose scores grow along the sequence, so the running maximum is raised again and again, by small
    steps and by jumps of hundreds; then scores that fall."""
    lengths = (1000, 700)
    q, k, v = inputs(5, 1700, 4, 2, 64)
    ramp = torch.linspace(0.1, 6.0, 1700, device="cuda")
    steps = torch.where(torch.arange(1700, device="cuda") % 300 == 299, 30.0, 1.0)
    for f in (ramp, ramp.flip(0), steps):
        kf = (k.float() * f[:, None, None]).to(BF16)
        for causal in (True, False):
            check(run(vsa, q, kf, v, lengths, causal), q, kf, v, lengths, causal)


def test_packed_scale(vsa):
    lengths = (300, 20)
    q, k, v = inputs(6, 320, 4, 4, 128)
    for scale in (0.01, 0.3):
        check(run(vsa, q, k, v, lengths, True, softmax_scale=scale), q, k, v, lengths, True, scale)


def test_packed_strides_and_rows_behind(vsa):
    """q, k, v as slices of one projection with rows behind the last sequence that hold NaN; the output's rows
    there, and everything beside the output's slice, stay as they were."""
    lengths, Hq, Hk, D = (77, 5, 130), 6, 2, 96
    n, T = sum(lengths), sum(lengths) + 50
    g = torch.Generator(device="cuda").manual_seed(7)
    qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g, device="cuda").to(BF16)
    qkv[n:] = float("nan")
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    buf = torch.full((T, Hq + 3, D), 9.0, dtype=BF16, device="cuda")
    for causal in (True, False):
        plan = vsa.vsa_packed_plan(lengths, Hq, Hk, D, causal=causal)
        out = vsa.vsa_packed_attn(plan, q, k, v, out=buf[:, 1:1 + Hq])
        check(out, q, k, v, lengths, causal)
        assert (buf[n:] == 9).all() and (buf[:, 0] == 9).all() and (buf[:, 1 + Hq:] == 9).all()
        fresh = vsa.vsa_packed_attn(plan, q, k, v)
        assert torch.equal(fresh[:n], out[:n]) and (fresh[n:] == 0).all()
    # head-major storage, inputs and output
    qh, kh, vh = (x[:n].transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    oh = torch.empty(Hq, n, D, dtype=BF16, device="cuda").transpose(0, 1)
    vsa.vsa_packed_attn(plan, qh, kh, vh, out=oh)
    assert torch.equal(oh, fresh[:n])
    # one key head and one value row for all, by stride 0
    ke, ve = k[:n, :1].expand(-1, Hk, -1), v[:1, :1].expand(n, Hk, -1)
    check(vsa.vsa_packed_attn(plan, qh, ke, ve), qh, ke, ve, lengths, False)


def test_packed_output_over_the_queries(vsa):
    """out = q: every query row is read by one item only, before that item stores."""
    lengths = (513, 40, 1, 300)
    for heads, kv_heads, D in ((5, 1, 128), (4, 4, 64), (6, 2, 96)):
        q, k, v = inputs(heads, sum(lengths), heads, kv_heads, D)
        want = run(vsa, q, k, v, lengths, True)
        plan = vsa.vsa_packed_plan(lengths, heads, kv_heads, D)
        assert vsa.vsa_packed_attn(plan, q, k, v, out=q) is q
        assert torch.equal(q, want)


def test_packed_batch_of_equal_lengths(vsa):
    """[B, L, H, D] as B sequences of L."""
    q, k, v = inputs(8, 3 * 150, 4, 2, 64)
    plan = vsa.vsa_packed_plan([150] * 3, 4, 2, 64)
    out = vsa.vsa_packed_attn(plan, *(x.view(3, 150, -1, 64) for x in (q, k, v)))
    assert out.shape == (3, 150, 4, 64)
    check(out.view(450, 4, 64), q, k, v, [150] * 3, True)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_packed_neighbours_do_not_leak(vsa, D, bad):
    """Whole neighbouring sequences of NaN or infinity before, between and behind: the others' outputs are the
    same bits as with finite neighbours."""
    lengths = [40, 133, 1, 250, 17, 128, 16, 9]
    for causal in (True, False):
        q, k, v = inputs(9, sum(lengths), 5, 1, D)
        want = run(vsa, q, k, v, lengths, causal)
        starts = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
        for ill in range(len(lengths)):
            s = slice(starts[ill], starts[ill + 1])
            q2, k2, v2 = q.clone(), k.clone(), v.clone()
            for x in (q2, k2, v2):
                x[s] = bad
            got = run(vsa, q2, k2, v2, lengths, causal)
            ok = torch.ones(sum(lengths), dtype=torch.bool, device="cuda")
            ok[s] = False
            assert torch.equal(got[ok], want[ok])
            assert got[s].isnan().all()


def test_packed_bad_keys_stay_where_they_are_seen(vsa):
    lengths = (400,)
    q, k, v = inputs(10, 400, 4, 2, 128)
    want = run(vsa, q, k, v, lengths, True)
    k2 = k.clone()
    k2[250, 0] = float("nan")
    got = run(vsa, q, k2, v, lengths, True)
    assert torch.equal(got[:250], want[:250]) and torch.equal(got[:, 2:], want[:, 2:])
    assert got[250:, :2].isnan().all()
    for at in range(248, 256):  # whichever pipe takes a key's exponential
        k2 = k.clone()
        k2[at, 1, 5] = float("nan")
        got = run(vsa, q, k2, v, lengths, True)
        assert got[at:, 2:].isnan().all() and torch.equal(got[:at], want[:at])
    q2 = q.clone()
    q2[100, 1, 3] = float("nan")  # a query row harms itself only
    got = run(vsa, q2, k, v, lengths, True)
    same = torch.ones(400, 4, dtype=torch.bool, device="cuda")
    same[100, 1] = False
    assert torch.equal(got[same], want[same]) and got[100, 1].isnan().all()


def test_packed_one_plan_on_two_streams_and_captured(vsa):
    lengths = (300, 77, 513)
    n = sum(lengths)
    plan = vsa.vsa_packed_plan(lengths, 8, 2, 128)
    sets = [inputs(20 + i, n, 8, 2, 128) for i in range(2)]
    want = [vsa.vsa_packed_attn(plan, *x) for x in sets]
    for w, x in zip(want, sets):
        check(w, *x, lengths, True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [torch.empty_like(want[0]) for _ in range(2)]
    for _ in range(10):
        for s, x, o in zip(streams, sets, outs):
            vsa.vsa_packed_attn(plan, *x, out=o, stream=s)
    for s in streams:
        s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    static = [x.clone() for x in sets[0]]
    out = torch.empty_like(want[0])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr in graphs:
        with torch.cuda.graph(gr):
            vsa.vsa_packed_attn(plan, *static, out=out)
    for i, gr in ((1, graphs[0]), (0, graphs[1]), (1, graphs[1])):
        for a, b in zip(static, sets[i]):
            a.copy_(b)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    assert plan.status() == (0, 0)


def test_packed_binding_refusals(vsa):
    q, k, v = inputs(30, 20, 4, 2, 64)
    plan = vsa.vsa_packed_plan((12, 8), 4, 2, 64)
    for args, kw, err in [((q.float(), k, v), {}, TypeError), ((q, k.cpu(), v), {}, ValueError),
                          ((q[:, :2], k, v), {}, ValueError), ((q, k[:, :1], v), {}, ValueError),
                          ((q, k[:19], v), {}, ValueError), ((q, k, v), dict(out=q[:19]), ValueError),
                          ((q[..., :32], k, v), {}, ValueError)]:
        with pytest.raises(err):
            vsa.vsa_packed_attn(plan, *args, **kw)
    with pytest.raises(vsa.VsaError):  # fewer rows than the plan's sequences hold
        vsa.vsa_packed_attn(plan, q[:19], k[:19], v[:19])
    with pytest.raises(vsa.VsaError):  # the output's rows overlap
        vsa.vsa_packed_attn(plan, q, k, v, out=torch.empty(64 * 30, dtype=BF16, device="cuda").as_strided((20, 4, 64), (64, 64, 1)))
    wide = torch.zeros(20, 4, 68, dtype=BF16, device="cuda")
    with pytest.raises(vsa.VsaError):  # strides that are not multiples of 8
        vsa.vsa_packed_attn(plan, wide[..., :64], k, v)
    empty = vsa.vsa_packed_plan((0, 0), 4, 2, 64)
    out = vsa.vsa_packed_attn(empty, q, k, v)
    assert (out == 0).all()
    empty.destroy()
    with pytest.raises(ValueError):
        vsa.vsa_packed_attn(empty, q, k, v)


def test_packed_refuses_an_output_over_its_inputs(vsa):
    """The output may replace q in place, row for row; over k or v, or over q in another layout, items would
    overwrite what others still read."""
    q, k, v = inputs(12, 256, 2, 2, 64)
    plan = vsa.vsa_packed_plan([200, 56], 2, 2, 64)
    for other in (k, v):
        with pytest.raises(vsa.VsaError):
            vsa.vsa_packed_attn(plan, q, k, v, out=other)
    turned = q.view(2, 256, 64).transpose(0, 1)  # q's memory, heads apart
    with pytest.raises(vsa.VsaError):
        vsa.vsa_packed_attn(plan, q, k, v, out=turned)
    want = vsa.vsa_packed_attn(plan, q, k, v)
    assert torch.equal(vsa.vsa_packed_attn(plan, q, k, v, out=q), want)
