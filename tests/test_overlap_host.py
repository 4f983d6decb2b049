"""Outputs over memory that a call still reads or writes: refused on the host.  The rule (csrc/rows.h) is held to sets
of bytes; the calls name addresses that nothing reads."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20


@pytest.fixture(scope="module")
def vsa():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as m

    m.load_library()
    return m


HARNESS = r"""
#include <cstdio>
#include <random>
#include <set>
#include "rows.h"
using vsa::Rows;
static std::set<long> bytes(const Rows& r) {
  std::set<long> s;
  for (long i = 0; i < r.n; ++i)
    for (long h = 0; h < r.heads; ++h)
      for (long b = 0; b < r.row; ++b) s.insert((long)(size_t)r.base + i * r.ld + h * r.hd + b);
  return s;
}
static bool truly_meet(const Rows& a, const Rows& b) {
  const auto x = bytes(a), y = bytes(b);
  for (long v : x) if (y.count(v)) return true;
  return false;
}
int main() {
  std::mt19937 g(7);
  const auto in = [&](int lo, int hi) { return (long)(lo + g() % (hi - lo + 1)); };
  long apart = 0, wrong = 0, refused = 0;
  for (int t = 0; t < 60000; ++t) {  // any two layouts: said to be apart only if they are
    const long n = in(1, 4);
    const auto any = [&]() { return Rows{(void*)(size_t)in(100, 160), n, in(0, 24), in(1, 3), in(0, 12), in(1, 6)}; };
    const Rows a = any();
    Rows b = any();
    if (g() & 1) b.ld = a.ld;
    if (g() & 1) b.hd = a.hd;
    const bool meet = vsa::rows_meet(a, b);
    apart += !meet;
    wrong += !meet && truly_meet(a, b);
    if (bytes(a).size() != (size_t)(a.n * a.heads * a.row) && vsa::rows_disjoint(a)) ++wrong;
    if (vsa::same_rows(a, b) && bytes(a) != bytes(b)) ++wrong;
  }
  // slices of one projection, token-major, head-major, K and V interleaved by head: apart, and meeting where they meet
  for (int t = 0; t < 4000; ++t) {
    const long n = in(1, 4), row = in(1, 4), h1 = in(1, 3), h2 = in(1, 3), gap = in(0, 3), all = h1 + h2 + gap;
    const long one = 1000;
    const auto at = [&](long o) { return (void*)(size_t)(one + o); };
    const Rows tm1{at(0), n, all * row, h1, row, row}, tm2{at((h1 + gap) * row), n, all * row, h2, row, row};
    const Rows hm1{at(0), n, row, h1, n * row, row}, hm2{at((h1 + gap) * n * row), n, row, h2, n * row, row};
    const Rows il1{at(0), n, 2 * h1 * row, h1, 2 * row, row}, il2{at(row), n, 2 * h1 * row, h1, 2 * row, row};
    refused += vsa::rows_meet(tm1, tm2) + vsa::rows_meet(tm2, tm1) + vsa::rows_meet(hm1, hm2) + vsa::rows_meet(hm2, hm1) +
               vsa::rows_meet(il1, il2) + vsa::rows_meet(il2, il1);
    const Rows over{at(h1 * row - 1), n, all * row, h2, row, row};
    wrong += !vsa::rows_meet(tm1, over) || !vsa::rows_meet(over, tm1) || !vsa::rows_meet(tm1, tm1);
  }
  std::printf("%ld %ld %ld\n", apart, wrong, refused);
}
"""


def test_rows_meet_against_sets_of_bytes(tmp_path):
    (tmp_path / "h.cpp").write_text(HARNESS)
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", f"-I{ROOT}/block_sparse_tiled_b200/csrc",
                           str(tmp_path / "h.cpp"), "-o", str(tmp_path / "h")])
    apart, wrong, refused = (int(x) for x in subprocess.check_output([str(tmp_path / "h")]).split())
    assert apart > 5000 and wrong == 0 and refused == 0


def status(vsa, call, *args):
    return vsa.STATUS_NAMES[getattr(vsa.load_library(), call)(*args, None)]


# four rows of 64 bf16 values, 128 bytes each
NORM = dict(rows=4, width=64, eps=1e-6, x=A, out=8 * A, x_stride=64, out_stride=64)
RES = dict(residual=2 * A, residual_stride=64, residual_out=3 * A, residual_out_stride=64)


@pytest.mark.parametrize("over", [
    dict(out=A + 128),  # one row further on
    dict(out=A + 128, out_stride=128),
    dict(RES, out=2 * A + 128), dict(RES, residual_out=A + 256), dict(RES, residual_out=8 * A + 128),
    dict(RES, out=2 * A, residual_f32=1),  # bf16 over binary32 rows
    dict(weight=8 * A + 128), dict(RES, weight=3 * A + 128),
    dict(out_e4m3=1, scale=A + 16), dict(out_e4m3=1, scale=8 * A), dict(RES, out_e4m3=1, scale=3 * A + 48),
    dict(RES, out_e4m3=1, scale=2 * A), dict(weight=9 * A, out_e4m3=1, scale=9 * A + 32),
    dict(out=A + 64, out_e4m3=1, scale=9 * A),
])
def test_norm_outputs_over_operands(vsa, over):
    a = vsa.RmsNormArgs(**dict(NORM, **over))
    assert status(vsa, "vsa_rms_norm", ctypes.byref(a)) == "VSA_ERR_INVALID_ARG"
    assert "over" in vsa.load_library().vsa_last_error().decode()


# q [4, 2, 64], k [4, 1, 64]
ROPE = dict(tokens=4, pos_rows=4, heads=2, eps=1e-6, positions=A, q=2 * A, q_out=3 * A, q_stride=128, q_head_stride=64,
            q_out_stride=128, q_out_head_stride=64, kv_heads=1, k=4 * A, k_out=5 * A, k_stride=64, k_head_stride=64,
            k_out_stride=64, k_out_head_stride=64)


@pytest.mark.parametrize("over", [
    dict(q_out=4 * A), dict(k_out=2 * A), dict(k_out=2 * A, k_out_stride=128),  # over the other input
    dict(k=2 * A, k_stride=128, q_out=2 * A),  # in place over q, which k is a part of
    dict(q_out=2 * A + 256), dict(k_out=4 * A + 128),  # over its own input, one token on
    dict(k_out=3 * A + 256), dict(q_out=5 * A + 128),  # over one another
    dict(q_out=A), dict(q_out=A - 1024 + 16), dict(k_out=A - 512 + 16),  # over the positions
    dict(q_weight=3 * A + 128), dict(k_weight=3 * A), dict(k_weight=5 * A + 256),
])
def test_rope_outputs_over_operands(vsa, over):
    r = vsa.vsa_rope_create(64, (32,))
    a = vsa.QkRopeArgs(**dict(ROPE, **over))
    assert status(vsa, "vsa_qk_rope", r.handle, ctypes.byref(a)) == "VSA_ERR_INVALID_ARG"
    assert "over" in vsa.load_library().vsa_last_error().decode()


def launched(vsa, call, *args):
    """Past every check: without a usable GPU, what is left is the CUDA error of the launch."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    return status(vsa, call, *args) == "VSA_ERR_CUDA"


@pytest.mark.parametrize("over", [
    dict(), dict(out=A), dict(RES), dict(RES, out=A, residual_out=2 * A), dict(RES, out=2 * A, residual_out=A),
    dict(RES, x_stride=256, residual=A + 128, residual_stride=256, out=A + 256, out_stride=256),  # slices of one buffer
    dict(x_stride=0), dict(rows=1, x_stride=0, out=A + 128),
    dict(out_e4m3=1, scale=8 * A + 256),  # right behind the codes
])
def test_norm_layouts_that_stay(vsa, over):
    assert launched(vsa, "vsa_rms_norm", ctypes.byref(vsa.RmsNormArgs(**dict(NORM, **over))))


QKV = dict(q=2 * A, k=2 * A + 256, q_stride=256, k_stride=256)  # [4, 2 + 1 + 1, 64]


@pytest.mark.parametrize("over", [
    dict(), dict(q_out=2 * A, k_out=4 * A), dict(QKV), dict(QKV, q_out=2 * A, k_out=2 * A + 256, q_out_stride=256, k_out_stride=256),
    dict(QKV, q_out=2 * A, q_out_stride=256), dict(q=2 * A, k=2 * A, k_stride=128),  # k is q's first head
    dict(tokens=1, pos_rows=1, q_out=2 * A, k=2 * A + 256, k_out=2 * A + 256),
    # head-major storage: [2 + 1, 4, 64]
    dict(q_stride=64, q_head_stride=256, k=2 * A + 1024, q_out=2 * A, q_out_stride=64, q_out_head_stride=256, k_out=2 * A + 1024),
])
def test_rope_layouts_that_stay(vsa, over):
    r = vsa.vsa_rope_create(64, (32,))
    assert launched(vsa, "vsa_qk_rope", r.handle, ctypes.byref(vsa.QkRopeArgs(**dict(ROPE, **over))))


def test_positions_and_scales_may_start_anywhere(vsa):
    """Both are read and written a number at a time: a chunk of a longer table starts at any row of it."""
    r = vsa.vsa_rope_create(64, (32,))
    assert launched(vsa, "vsa_qk_rope", r.handle, ctypes.byref(vsa.QkRopeArgs(**dict(ROPE, positions=A + 12))))
    assert launched(vsa, "vsa_rms_norm", ctypes.byref(vsa.RmsNormArgs(**dict(NORM, out_e4m3=1, scale=4 * A + 20))))
    for size in (1, 2):
        a = vsa.QkRopeArgs(**dict(ROPE, positions=A + size))
        assert status(vsa, "vsa_qk_rope", r.handle, ctypes.byref(a)) == "VSA_ERR_INVALID_ARG"
        n = vsa.RmsNormArgs(**dict(NORM, out_e4m3=1, scale=4 * A + size))
        assert status(vsa, "vsa_rms_norm", ctypes.byref(n)) == "VSA_ERR_INVALID_ARG"
