"""The row operators without a GPU: every refusal of vsa_rms_norm, vsa_rope_create and vsa_qk_rope happens on
the host before anything is launched (so these calls name addresses that nothing reads), the rope table's
frequencies, and the ctypes mirrors of their structs."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # a 16-byte aligned address


@pytest.fixture(scope="module")
def vsa():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as m

    m.load_library()
    return m


@pytest.mark.parametrize("cname,pyname", [("vsa_rms_norm_args", "RmsNormArgs"), ("vsa_rope_desc", "RopeDesc"),
                                          ("vsa_qk_rope_args", "QkRopeArgs")])
def test_struct_layout(vsa, tmp_path, cname, pyname):
    cls = getattr(vsa, pyname)
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "vsa.h"', "int main(void) {",
           f'printf("%zu\\n", sizeof({cname}));']
    src += [f'printf("%zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(src) + "return 0; }\n")
    subprocess.check_call(["gcc", "-std=c11", f"-I{ROOT}/include", str(tmp_path / "l.c"), "-o", str(tmp_path / "l")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "l")], text=True).split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]


NORM = dict(rows=4, width=64, eps=1e-6, x=A, out=2 * A, x_stride=64, out_stride=64)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), "VSA_ERR_INVALID_ARG"),
    (dict(rows=1 << 31), "VSA_ERR_INVALID_ARG"),
    (dict(width=60), "VSA_ERR_UNSUPPORTED"),
    (dict(width=0), "VSA_ERR_UNSUPPORTED"),
    (dict(width=16392), "VSA_ERR_UNSUPPORTED"),
    (dict(eps=-1.0), "VSA_ERR_INVALID_ARG"),
    (dict(eps=float("nan")), "VSA_ERR_INVALID_ARG"),
    (dict(eps=float("inf")), "VSA_ERR_INVALID_ARG"),
    (dict(out_e4m3=2), "VSA_ERR_INVALID_ARG"),
    (dict(x=0), "VSA_ERR_INVALID_ARG"),
    (dict(x=A + 8), "VSA_ERR_INVALID_ARG"),
    (dict(out=0), "VSA_ERR_INVALID_ARG"),
    (dict(weight=A + 2), "VSA_ERR_INVALID_ARG"),
    (dict(x_stride=65), "VSA_ERR_INVALID_ARG"),
    (dict(x_stride=-64), "VSA_ERR_INVALID_ARG"),
    (dict(out_stride=56), "VSA_ERR_SHAPE"),
    (dict(out_e4m3=1), "VSA_ERR_INVALID_ARG"),  # no scale
    (dict(residual_out=3 * A, residual_out_stride=64), "VSA_ERR_INVALID_ARG"),  # without a residual
    (dict(residual=3 * A, residual_stride=64, residual_out=2 * A, residual_out_stride=64), "VSA_ERR_INVALID_ARG"),
    (dict(out=A, out_stride=128), "VSA_ERR_INVALID_ARG"),  # in place with another stride
    (dict(out=A, out_e4m3=1, scale=4 * A), "VSA_ERR_INVALID_ARG"),  # codes over the bf16 rows
    (dict(residual=3 * A, residual_f32=1, residual_stride=64, residual_out=A, residual_out_stride=64),
     "VSA_ERR_INVALID_ARG"),
    # a single row has no stride to compare, but types still differ: its writes would run ahead of its reads
    (dict(rows=1, residual=3 * A, residual_f32=1, residual_stride=64, residual_out=A, residual_out_stride=64),
     "VSA_ERR_INVALID_ARG"),
    (dict(rows=1, out=A, out_e4m3=1, scale=4 * A), "VSA_ERR_INVALID_ARG"),
])
def test_rms_norm_refusals(vsa, over, status):
    a = vsa.RmsNormArgs(**dict(NORM, **over))
    rc = vsa.load_library().vsa_rms_norm(ctypes.byref(a), None)
    assert vsa.STATUS_NAMES[rc] == status
    assert vsa.load_library().vsa_last_error().decode()


def test_no_rows_is_nothing_to_do(vsa):
    a = vsa.RmsNormArgs(**dict(NORM, rows=0, x=0, out=0))
    assert vsa.load_library().vsa_rms_norm(ctypes.byref(a), None) == 0
    assert vsa.load_library().vsa_rms_norm(None, None) == 1
    r = vsa.vsa_rope_create(64, (32,))
    q = vsa.QkRopeArgs(**dict(ROPE, tokens=0, q=0))
    assert vsa.load_library().vsa_qk_rope(r.handle, ctypes.byref(q), None) == 0


@pytest.mark.parametrize("kw", [
    dict(head_dim=80, sections=(8,)), dict(head_dim=64, sections=(16, 17)), dict(head_dim=64, sections=(-1, 4)),
    dict(head_dim=64, sections=()), dict(head_dim=64, sections=(1, 1, 1, 1, 1)),
    dict(head_dim=64, sections=(8,), theta=0.0), dict(head_dim=64, sections=(8,), theta=float("inf")),
    dict(head_dim=64, inv_freq=[1.0] * 32, axis=[0] * 31 + [3], n_axes=3),
    dict(head_dim=64, inv_freq=[float("nan")] * 32, axis=[0] * 32),
])
def test_rope_create_refusals(vsa, kw):
    with pytest.raises(vsa.VsaError):
        vsa.vsa_rope_create(**kw)


def test_rope_create_binding_refusals(vsa):
    for kw in (dict(sections=(8,), inv_freq=[1.0] * 32, axis=[0] * 32), dict(), dict(inv_freq=[1.0] * 32),
               dict(inv_freq=[1.0] * 31, axis=[0] * 31), dict(sections=(8, 8), n_axes=3)):
        with pytest.raises(ValueError):
            vsa.vsa_rope_create(64, **kw)
    r = vsa.vsa_rope_create(64, (32,))
    r.destroy()
    with pytest.raises(ValueError):
        r.table()


def test_rope_table(vsa):
    f, x = vsa.vsa_rope_create(128, (16, 24, 20), theta=10000.0).table()
    assert list(x[:60]) == [0] * 16 + [1] * 24 + [2] * 20
    want = [10000.0 ** (-i / n) for n in (16, 24, 20) for i in range(n)] + [0.0] * 4
    assert np.allclose(f, want, rtol=1e-14, atol=0)
    f, _ = vsa.vsa_rope_create(96, (16, 0, 32), theta=500.0, shared_ladder=True).table()
    assert np.allclose(f, [500.0 ** (-p / 48) for p in range(48)], rtol=1e-14, atol=0)
    mine = [math.sin(i) for i in range(32)]
    f, x = vsa.vsa_rope_create(64, inv_freq=mine, axis=[i % 4 for i in range(32)]).table()
    assert list(f) == mine and list(x) == [i % 4 for i in range(32)]


ROPE = dict(tokens=4, pos_rows=4, heads=2, eps=1e-6, positions=A, q=A, q_out=2 * A, q_stride=128, q_head_stride=64,
            q_out_stride=128, q_out_head_stride=64)
K = dict(kv_heads=1, k=3 * A, k_out=4 * A, k_stride=64, k_head_stride=64, k_out_stride=64, k_out_head_stride=64)


@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), "VSA_ERR_INVALID_ARG"),
    (dict(tokens=1 << 31), "VSA_ERR_INVALID_ARG"),
    (dict(heads=0), "VSA_ERR_INVALID_ARG"),
    (dict(kv_heads=-1), "VSA_ERR_INVALID_ARG"),
    (dict(pos_rows=3), "VSA_ERR_SHAPE"),
    (dict(pos_rows=0), "VSA_ERR_SHAPE"),
    (dict(positions=0), "VSA_ERR_INVALID_ARG"),
    (dict(positions_f32=2), "VSA_ERR_INVALID_ARG"),
    (dict(eps=-1.0), "VSA_ERR_INVALID_ARG"),
    (dict(q=0), "VSA_ERR_INVALID_ARG"),
    (dict(q_out=A + 4), "VSA_ERR_INVALID_ARG"),
    (dict(q_weight=A + 4), "VSA_ERR_INVALID_ARG"),
    (dict(q_stride=132), "VSA_ERR_INVALID_ARG"),
    (dict(q_head_stride=-64), "VSA_ERR_INVALID_ARG"),
    (dict(q_out_stride=64), "VSA_ERR_SHAPE"),
    (dict(q_out_head_stride=32), "VSA_ERR_SHAPE"),
    (dict(q_out=A, q_out_stride=256), "VSA_ERR_INVALID_ARG"),
    (dict(K, k_out=0), "VSA_ERR_INVALID_ARG"),
    (dict(K, k_stride=60), "VSA_ERR_INVALID_ARG"),
    (dict(K, k_out=2 * A), "VSA_ERR_INVALID_ARG"),  # both outputs in one place
])
def test_qk_rope_refusals(vsa, over, status):
    r = vsa.vsa_rope_create(64, (32,))
    a = vsa.QkRopeArgs(**dict(ROPE, **over))
    assert vsa.STATUS_NAMES[vsa.load_library().vsa_qk_rope(r.handle, ctypes.byref(a), None)] == status
    assert vsa.load_library().vsa_last_error().decode()


def test_cpu_tensors_are_refused(vsa):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        vsa.vsa_rms_norm(x)
    with pytest.raises(ValueError):
        vsa.vsa_qk_rope(vsa.vsa_rope_create(64, (32,)), x.view(2, 1, 64), None, torch.zeros(2, 1, dtype=torch.int32))
