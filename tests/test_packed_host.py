"""vsa_packed_attn without a GPU: the schedule (every query row of every head in exactly one item, longest items
first, balanced CTAs, the walk of key blocks that the kernel's index arithmetic makes stays inside the tensors
and rings), the refusals, and the ctypes mirrors."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def vsa():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as m

    m.load_library()
    return m


@pytest.mark.parametrize("cname,pyname", [("vsa_packed_desc", "PackedDesc"), ("vsa_packed_dims", "PackedDims"),
                                          ("vsa_packed_args", "PackedArgs")])
def test_struct_layout(vsa, tmp_path, cname, pyname):
    cls = getattr(vsa, pyname)
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "vsa.h"', "int main(void) {",
           f'printf("%zu\\n", sizeof({cname}));']
    src += [f'printf("%zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(src) + "return 0; }\n")
    subprocess.check_call(["gcc", "-std=c11", f"-I{ROOT}/include", str(tmp_path / "l.c"), "-o", str(tmp_path / "l")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "l")], text=True).split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]


def span(item, tb, causal):
    """Keys and key blocks of an item, as the kernel derives them."""
    _, n, t0, _ = (int(x) for x in item)
    keys = min(n, t0 + tb) if causal else n
    return keys, -(-keys // 128)


def lengths_of(seed):
    rng = random.Random(seed)
    return [rng.choice((0, 1, rng.randint(1, 40), rng.randint(1, 700))) for _ in range(rng.randint(1, 30))]


@pytest.mark.parametrize("lengths,heads,kv_heads,causal,sms", [
    ((1,), 1, 1, True, 148), ((0, 0), 4, 2, True, 148), ((), 4, 2, True, 148), ((129, 0, 1, 300), 40, 8, True, 148),
    ((513, 64), 128, 1, False, 148), ((200, 57), 7, 1, True, 3), ((2048,), 56, 56, False, 148),
    *[(tuple(lengths_of(s)), h, k, s % 2 == 0, sms)
      for s, (h, k, sms) in enumerate([(8, 2, 148), (6, 6, 5), (12, 4, 148), (9, 3, 1), (66, 1, 148), (100, 1, 20)])],
])
def test_schedule_covers_every_row_once(vsa, lengths, heads, kv_heads, causal, sms):
    d = vsa.vsa_packed_query(lengths, heads, kv_heads, 64, causal=causal, sms=sms)
    g = heads // kv_heads
    tb = 128 // g
    assert d["tile_tokens"] == tb and d["tokens"] == sum(lengths)
    assert d["pairs"] == sum(n * (n + 1) // 2 if causal else n * n for n in lengths)
    items, first = d["items"], d["first"]
    assert first[0] == 0 and first[-1] == len(items) == d["items"].shape[0] and (np.diff(first) >= 1).all()
    assert d["ctas"] == min(sms, len(items))
    seen = np.zeros((sum(lengths), kv_heads), np.int32)
    starts = np.cumsum([0, *lengths])
    length_at = {int(s): n for s, n in zip(starts, lengths) if n > 0}
    cost = []
    for row0, n, t0, h in items:
        assert n > 0 and length_at[row0] == n
        assert 0 <= t0 < n and 0 <= h < kv_heads
        seen[row0 + t0:row0 + min(n, t0 + tb), h] += 1
        keys, blocks = span((row0, n, t0, h), tb, causal)
        assert 1 <= keys <= n and 128 * (blocks - 1) < n
        assert keys >= min(n, t0 + tb)  # every token of the item sees itself
        cost.append(1 + blocks)
    assert (seen == 1).all()
    cost = np.array(cost)
    for c in range(d["ctas"]):
        mine = cost[first[c]:first[c + 1]]
        assert (np.diff(mine) <= 0).all()  # longest first
    if len(items):
        loads = [cost[first[c]:first[c + 1]].sum() for c in range(d["ctas"])]
        assert max(loads) <= cost.sum() / d["ctas"] + cost.max()


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), "VSA_ERR_INVALID_ARG"), (dict(heads=3, kv_heads=2), "VSA_ERR_SHAPE"),
    (dict(kv_heads=0), "VSA_ERR_INVALID_ARG"), (dict(heads=129, kv_heads=1), "VSA_ERR_UNSUPPORTED"),
    (dict(heads=70000, kv_heads=70000), "VSA_ERR_INVALID_ARG"),
    (dict(head_dim=80), "VSA_ERR_UNSUPPORTED"), (dict(lengths=(3, -1)), "VSA_ERR_INVALID_ARG"),
    (dict(lengths=(0x7fffffff, 5)), "VSA_ERR_UNSUPPORTED"), (dict(softmax_scale=-1.0), "VSA_ERR_INVALID_ARG"),
    (dict(softmax_scale=float("nan")), "VSA_ERR_INVALID_ARG"), (dict(sms=0), "VSA_ERR_INVALID_ARG"),
    (dict(lengths=(1,) * 70000, heads=256, kv_heads=256), "VSA_ERR_UNSUPPORTED"),  # 2^24 items and more
])
def test_refusals(vsa, kw, status):
    with pytest.raises(vsa.VsaError) as e:
        vsa.vsa_packed_query(**dict(dict(lengths=(5, 7), heads=4, kv_heads=2, head_dim=64), **kw))
    assert vsa.STATUS_NAMES[e.value.status] == status


def test_null_arguments(vsa):
    lib = vsa.load_library()
    d, keep = vsa.make_packed_desc((5,), 1, 1, 64)
    dims = vsa.PackedDims()
    assert lib.vsa_packed_query(None, 148, ctypes.byref(dims), None, None) == 1
    assert lib.vsa_packed_query(ctypes.byref(d), 148, None, None, None) == 1
    assert lib.vsa_packed_query(ctypes.byref(d), 148, ctypes.byref(dims), None, (ctypes.c_int32 * 9)()) == 1
    d.lengths = None
    assert lib.vsa_packed_query(ctypes.byref(d), 148, ctypes.byref(dims), None, None) == 1
    d, keep = vsa.make_packed_desc((5,), 1, 1, 64)
    d.causal = 2
    assert lib.vsa_packed_query(ctypes.byref(d), 148, ctypes.byref(dims), None, None) == 1
    assert lib.vsa_packed_attn(None, None, None) == 1 and lib.vsa_packed_info(None, ctypes.byref(dims)) == 1
    assert lib.vsa_packed_status(None, None, None, None) == 1 and lib.vsa_packed_destroy(None) == 0
    with pytest.raises(ValueError):
        vsa.vsa_packed_query((1 << 31,), 1)
