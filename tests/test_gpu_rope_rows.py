"""The head norm of D = 96, whose row is six lanes: their sum must not depend on the lane that takes it.

The sum is three binary32 values v0 + v1 + v2.  For rows whose squares add up to the border of binary32's range the order
of the additions decides whether it overflows; all lanes of a row have to answer alike."""
import numpy as np
import pytest
import torch

F32 = np.float32


def partials(x):
    """v0, v1, v2 of rows x [n, 96] (halves layout): per lane the squares of elements 8 l .. 8 l + 7 and 48 + 8 l ..,
    even and odd ones apart, in order; then lane l with lane l + 3.  (A bf16 square is exact in binary32.)"""
    with np.errstate(over="ignore"):
        n = len(x)
        words = np.stack((x[:, :48].reshape(n, 6, 4, 2), x[:, 48:].reshape(n, 6, 4, 2)), 2).reshape(n, 6, 8, 2)
        s = np.zeros((n, 6, 2), F32)
        for j in range(8):
            s = s + words[:, :, j] * words[:, :, j]
        lane = s[..., 0] + s[..., 1]
        return lane[:, :3] + lane[:, 3:]


def sums(v):
    with np.errstate(over="ignore"):
        return np.stack([(v[:, i] + v[:, (i + 1) % 3]) + v[:, (i + 2) % 3] for i in range(3)], 1)


def border_rows(count):
    """Rows of bf16 values whose three orders of addition disagree about infinity."""
    rng, found = np.random.default_rng(1), []
    while len(found) < count:
        n = 4096
        x = np.zeros((n, 96), F32)
        # 93 large elements, the sum of squares a little below 2^128, and three that fill it up to about a step
        x[:, :93] = torch.from_numpy(rng.uniform(0.8, 1.2, (n, 93)) * 2.0 ** 64 / 93 ** 0.5).to(torch.bfloat16).float().numpy()
        total = (x.astype(np.float64) ** 2).sum(1)
        keep = total < 2.0 ** 128 * (1 - 1e-6)
        x, total = x[keep], total[keep]
        for at in (93, 94, 95):
            left = np.maximum(2.0 ** 128 * (1 - 2.0 ** -25) - total, 0.0)
            fit = torch.from_numpy(np.sqrt(left) * (rng.uniform(0.6, 1.0, len(left)) if at < 95 else 1.0))
            x[:, at] = fit.to(torch.bfloat16).float().numpy()
            total = (x.astype(np.float64) ** 2).sum(1)
        x = x[np.isfinite(x).all(1)]
        for r in range(len(x)):
            x[r] = x[r][rng.permutation(96)]
        s = np.isinf(sums(partials(x)))
        found += list(x[s.any(1) & ~s.all(1)])
    return np.stack(found[:count])


def test_the_order_of_addition_matters_at_the_border():
    s = np.isinf(sums(partials(border_rows(4))))
    assert (s.any(1) & ~s.all(1)).all()


@pytest.mark.gpu
def test_border_rows_are_scaled_alike_in_every_lane():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as vsa

    rows = border_rows(40)
    q = torch.from_numpy(rows).cuda().to(torch.bfloat16).view(8, 5, 96)
    assert torch.equal(q.float().cpu().view(40, 96), torch.from_numpy(rows))
    rope = vsa.vsa_rope_create(96, (48,))
    pos = torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    w = torch.linspace(0.5, 1.5, 96, device="cuda").to(torch.bfloat16)
    out, _ = vsa.vsa_qk_rope(rope, q, None, pos, q_weight=w)
    y = q.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.double()
    # position 0 turns nothing: one rounding to bf16 and 1e-5 of binary32 arithmetic
    assert ((out.double() - y).abs() <= (2.0 ** -8 + 2e-5) * y.abs()).all()
