"""vsa_rms_norm at the ends of binary32's range and on values that are not finite, against its formula.
Bounds as in test_gpu_token_ops.py: half a step of the output's type, and 1e-5 for the binary32 arithmetic before it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
B_HALF, E_HALF, ARITH, EPS = 2.0 ** -8, 2.0 ** -4, 1e-5, 1e-6
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def vsa():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as m

    m.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    return m


def randn(seed, *shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("width", [64, 1024, 5120, 8200])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_8bit_scale_of_a_row_that_is_not_finite(vsa, width, bad):
    """max|y| of a row with a NaN in y is NaN, whatever the weight there: infinity times a weight of 0 is NaN too."""
    x, w = randn(1, 9, width), randn(2, width)
    for weight in (0.0, -0.0, 1.5):
        for at in (0, width // 2 + 3, width - 1):
            wt, xt = w.clone(), x.clone()
            wt[at], xt[4, at] = weight, bad
            for weights in (wt, wt.float()):
                _, scale, _ = vsa.vsa_rms_norm(xt, weights, EPS, out_dtype=E4M3)
                ok = torch.arange(9, device="cuda") != 4
                assert scale[4].isnan() and torch.isfinite(scale[ok]).all() and (scale[ok] > 0).all()


@pytest.mark.parametrize("width", [64, 5120])
def test_8bit_scale_under_a_weight_that_is_not_a_number(vsa, width):
    x, w = randn(3, 5, width), randn(4, width)
    w[width - 7] = NAN
    _, scale, _ = vsa.vsa_rms_norm(x, w, EPS, out_dtype=E4M3)
    assert scale.isnan().all()


@pytest.mark.parametrize("width", [64, 1024, 5120])
@pytest.mark.parametrize("bad", [INF, -INF])
def test_bf16_row_with_an_infinity(vsa, width, bad):
    """The formula's values: 1 / sqrt(inf) = 0 at the finite elements, infinity times 0 at the others; a row with a NaN
    is NaN throughout."""
    x, w = randn(5, 6, width), randn(6, width)
    x[2, width // 3] = bad
    x[4, width // 3] = NAN
    out, _, _ = vsa.vsa_rms_norm(x, w, EPS)
    there = torch.arange(width, device="cuda") == width // 3
    assert out[2, there].isnan().all() and (out[2, ~there] == 0).all()
    assert out[4].isnan().all()
    assert torch.isfinite(out[[0, 1, 3, 5]]).all()


@pytest.mark.parametrize("width", [64, 1024, 5120, 8200, 16384])
@pytest.mark.parametrize("lo,hi", [(2.0e38, 3.3e38), (1.0e19, 4.0e19), (1.2e17, 1.6e17)])
def test_wide_rows_near_the_largest_number(vsa, width, lo, hi):
    """Rows that are finite, however large and wide, and however far the sum of their squares is out of range."""
    g = torch.Generator(device="cuda").manual_seed(width)
    size = torch.empty(5, width, device="cuda").uniform_(lo, hi, generator=g)
    r = torch.where(torch.rand(5, width, generator=g, device="cuda") < 0.5, size, -size)
    x, w = torch.zeros(5, width, dtype=BF16, device="cuda"), randn(7, width)
    t = r.double()
    y = t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS) * w.double()
    out, _, res = vsa.vsa_rms_norm(x, w, EPS, residual=r)
    assert torch.equal(res, r)
    assert ((out.double() - y).abs() <= (B_HALF + 2 * ARITH) * y.abs()).all()
    codes, scale, _ = vsa.vsa_rms_norm(x, w, EPS, residual=r, out_dtype=E4M3)
    want = y.abs().amax(-1) / 448.0
    s = scale.double()[:, None]
    assert ((scale.double() - want).abs() <= ARITH * want).all()
    assert ((codes.double() * s - y).abs() <= (E_HALF + 4 * ARITH) * y.abs() + 2.0 ** -10 * (1 + ARITH) * s).all()
