"""vsa_rms_norm on values that are not finite, against what its formula gives."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-6
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
