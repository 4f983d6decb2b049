"""Refusals of the token operators' Python binding that need no GPU: the checks that come before anything is launched,
with CPU tensors standing in for CUDA ones where the device check is replaced."""
import pytest
import torch


@pytest.fixture(scope="module")
def vsa():
    from block_sparse_tiled_b200 import build

    build.build()
    import block_sparse_tiled_b200 as m

    m.load_library()
    return m


class Launched(Exception):
    """Every check of the binding has passed."""


@pytest.fixture
def no_device(vsa, monkeypatch):
    def launch(*_):
        raise Launched

    monkeypatch.setattr(vsa, "_launch_index", lambda *_: 0)
    monkeypatch.setattr(vsa, "_stream_on", launch)
    return vsa


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("q,rows", [
    ((100, 2, 64), 50), ((100, 2, 64), 1), ((100, 2, 64), 25),  # [T, H, D] takes a row for every token
    ((2, 30, 2, 64), 2), ((2, 30, 2, 64), 15), ((2, 30, 2, 64), 1), ((4, 1, 2, 64), 2),  # [B, L, H, D]: L or B * L
])
def test_positions_that_would_be_used_for_other_tokens(no_device, q, rows):
    rope = no_device.vsa_rope_create(64, (16, 16))
    for k in (None, bf16(*q)):
        with pytest.raises(ValueError, match="positions"):
            no_device.vsa_qk_rope(rope, bf16(*q), k, torch.zeros(rows, 2, dtype=torch.int32))


@pytest.mark.parametrize("q,pos", [((100, 2, 64), (100, 2)), ((2, 30, 2, 64), (30, 2)), ((2, 30, 2, 64), (60, 2)),
                                   ((2, 30, 2, 64), (2, 30, 2)), ((2, 30, 2, 64), (1, 30, 2)), ((1, 2, 64), (1, 2)),
                                   ((4, 1, 2, 64), (1, 2)), ((0, 2, 64), (0, 2))])
def test_positions_that_fit(no_device, q, pos):
    rope = no_device.vsa_rope_create(64, (16, 16))
    with pytest.raises(Launched):
        no_device.vsa_qk_rope(rope, bf16(*q), None, torch.zeros(*pos, dtype=torch.int32))


class FakeLibrary:
    """Handles without a device; the calls made, in order."""

    def __init__(self, vsa):
        self.calls, self.next = [], 100

    def vsa_packed_plan(self, desc, stream, out):
        out._obj.value = self.next
        self.next += 1
        self.calls.append(("plan", out._obj.value))
        return 0

    def vsa_packed_info(self, handle, dims):
        return 0

    def vsa_packed_destroy(self, handle):
        self.calls.append(("destroy", handle.value))
        return 0


def test_a_collected_plan_is_freed_by_the_next_call_that_may(vsa, monkeypatch):
    """The garbage collector may run while another stream is captured, and freeing a plan synchronises the device, which
    would end the capture: a plan that is collected waits for the next plan (made outside of captures) or destroy()."""
    import gc

    lib = FakeLibrary(vsa)
    monkeypatch.setattr(vsa, "load_library", lambda *_: lib)
    monkeypatch.setattr(vsa, "_stream", lambda *_: None)
    a = vsa.vsa_packed_plan((5,), 1)
    b = vsa.vsa_packed_plan((6,), 1)
    c = vsa.vsa_packed_plan((7,), 1)
    del a
    gc.collect()
    assert lib.calls == [("plan", 100), ("plan", 101), ("plan", 102)]
    d = vsa.vsa_packed_plan((8,), 1)
    assert sorted(lib.calls[3:]) == [("destroy", 100), ("plan", 103)]
    del b, d
    gc.collect()
    assert len(lib.calls) == 5
    c.destroy()  # at once, and what waits with it
    assert sorted(lib.calls[5:]) == [("destroy", 101), ("destroy", 102), ("destroy", 103)]
    c.destroy()
    del c
    gc.collect()
    vsa.vsa_packed_plan((9,), 1).destroy()
    assert lib.calls[8:] == [("plan", 104), ("destroy", 104)]


WRAPS = 1 << 32  # a multiple of 2^32 added to a 32-bit field would vanish


@pytest.mark.parametrize("kw", [dict(lengths=(5 - WRAPS,)), dict(lengths=(5 + WRAPS,)), dict(heads=4 + WRAPS, kv_heads=4),
                                dict(kv_heads=1 + WRAPS), dict(head_dim=64 + WRAPS), dict(sms=148 + WRAPS)])
def test_packed_numbers_past_32_bits(vsa, kw):
    with pytest.raises(ValueError):
        vsa.vsa_packed_query(**dict(dict(lengths=(5, 7), heads=4, kv_heads=2, head_dim=64), **kw))


@pytest.mark.parametrize("kw", [dict(head_dim=64 + WRAPS, sections=(8,)), dict(head_dim=64, sections=(8 + WRAPS,)),
                                dict(head_dim=64, sections=(8 - WRAPS,)),
                                dict(head_dim=64, inv_freq=[1.0] * 32, axis=[0] * 31 + [WRAPS]),
                                dict(head_dim=64, inv_freq=[1.0] * 32, axis=[0] * 32, n_axes=1 + WRAPS)])
def test_rope_numbers_past_32_bits(vsa, kw):
    with pytest.raises(ValueError):
        vsa.vsa_rope_create(**kw)


def test_norm_width_past_32_bits(no_device):
    """A row of 2^32 + 8 elements is not a row of 8."""
    wide = torch.empty(1, WRAPS + 8, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError):
        no_device.vsa_rms_norm(wide, out=wide)


def test_a_plan_alive_at_exit_says_nothing():
    """At the interpreter's end a module's names may be gone before its plans."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import block_sparse_tiled_b200 as vsa, test_token_ops_binding as t\n"
            "lib = t.FakeLibrary(vsa); vsa.load_library = lambda *_: lib; vsa._stream = lambda *_: None\n"
            "plan = vsa.vsa_packed_plan((5,), 1)\n"
            "calls = {'attn': lambda: plan}\n" % (root, os.path.join(root, "tests")))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stderr == ""
