"""Python binding of libvsa, the VSA-H3 block-sparse attention forward for B200.

Argument marshalling only: every step of the forward runs in the CUDA kernels
of ``libvsa.so`` (built from ``csrc/`` for sm_100a).  PyTorch supplies device
memory and streams.  There is no fallback: if the library is missing or the
device is not sm_100, the calls raise.

The functions mirror the C ABI in ``include/vsa.h``:

    vsa_plan_tiles      S1  tile plan (host) + upload of the tile tables
    vsa_gather_tiles    S2  sequence order -> tile order (optionally pooled)
    vsa_pool_and_score  S3  pooled tiles and fp32 pooled tile scores
    vsa_topk_select     S4  top-k key tiles per video query tile + compression
    vsa_sparse_attn_fwd S5  block-sparse attention + gated epilogue
    vsa_forward             S2..S5 in one call

and the operators of a transformer block on either side of it:

    vsa_rms_norm        RMS norm with the residual's addition, bf16 or 8-bit output
    vsa_qk_rope         head norm and multi-axis rotary positions of Q and K
    vsa_packed_attn     attention over packed whole prompts (vsa_packed_plan)

Work runs on `stream` (a torch.cuda.Stream or a raw handle; by default the current stream).  What a call allocates on
the device belongs to that stream, as if it were made under torch.cuda.stream(stream): its inputs have to be ready on
it, and another stream that reads its outputs has to wait for it.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvsa.so")

VSA_OK = 0
STATUS_NAMES = {
    0: "VSA_OK", 1: "VSA_ERR_INVALID_ARG", 2: "VSA_ERR_SHAPE", 3: "VSA_ERR_UNSUPPORTED",
    4: "VSA_ERR_WORKSPACE", 5: "VSA_ERR_CUDA", 6: "VSA_ERR_TIMEOUT", 7: "VSA_ERR_DEVICE",
}

# every symbol include/vsa.h declares
EXPORTED = (
    "vsa_plan_tiles", "vsa_plan_info", "vsa_plan_tables", "vsa_plan_query", "vsa_plan_tables_host",
    "vsa_plan_destroy",
    "vsa_gather_tiles", "vsa_pool_and_score", "vsa_topk_select", "vsa_sparse_attn_fwd", "vsa_forward",
    "vsa_forward_noalloc", "vsa_forward_host", "vsa_forward_host_workspace", "vsa_forward_parts", "vsa_wait_selftest",
    "vsa_plan_workspace", "vsa_device_status", "vsa_last_error", "vsa_version",
    "vsa_rms_norm", "vsa_rope_create", "vsa_rope_table", "vsa_rope_destroy", "vsa_qk_rope",
    "vsa_packed_plan", "vsa_packed_query", "vsa_packed_info", "vsa_packed_destroy", "vsa_packed_attn",
    "vsa_packed_status", "vsa_packed_wait_selftest",
)


class VsaError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {message}")


class Geometry(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("n_segments", ctypes.c_int32), ("segment_len", ctypes.POINTER(ctypes.c_int32)),
        ("token_tags", ctypes.POINTER(ctypes.c_int32)), ("seq_len", ctypes.c_int64),
        ("video_tag", ctypes.c_int32),
        ("grid_t", ctypes.c_int32), ("grid_h", ctypes.c_int32), ("grid_w", ctypes.c_int32),
        ("tile_size", ctypes.c_int32), ("sparsity", ctypes.c_double), ("softmax_scale", ctypes.c_float),
        ("gate_per_channel", ctypes.c_int32), ("seq_tiles", ctypes.c_int32), ("qk_fp8", ctypes.c_int32),
        ("cube_t", ctypes.c_int32), ("cube_h", ctypes.c_int32), ("cube_w", ctypes.c_int32),
        ("segment_reference", ctypes.POINTER(ctypes.c_int32)), ("reference_keep", ctypes.c_double),
    ]


class SeqParts(ctypes.Structure):
    _fields_ = [
        ("nparts", ctypes.c_int32), ("tokens_per_part", ctypes.c_int64), ("heads_total", ctypes.c_int32),
        ("head_offset", ctypes.c_int32),
        ("q", ctypes.POINTER(ctypes.c_void_p)), ("k", ctypes.POINTER(ctypes.c_void_p)),
        ("v", ctypes.POINTER(ctypes.c_void_p)), ("gate", ctypes.POINTER(ctypes.c_void_p)),
        ("out", ctypes.POINTER(ctypes.c_void_p)),
    ]


class PlanDims(ctypes.Structure):
    _fields_ = [
        ("n_tiles", ctypes.c_int32), ("n_prefix_tiles", ctypes.c_int32), ("n_video_tiles", ctypes.c_int32),
        ("topk", ctypes.c_int32), ("seq_len", ctypes.c_int64), ("softmax_scale", ctypes.c_float),
        ("workspace_bytes", ctypes.c_size_t), ("selected_pairs", ctypes.c_int64), ("tile_size", ctypes.c_int32),
        ("n_ref_tiles", ctypes.c_int32), ("ref_topk", ctypes.c_int32),
    ]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t)
                for n in ("q_t", "k_t", "v_t", "q_s", "k_s", "q_n", "kv_max", "pq", "pk", "pv", "scores", "idx", "o_c",
                          "q_c", "k_c", "q_n8", "kv_max8", "k_sum", "k_mu", "total")]


class RmsNormArgs(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("width", ctypes.c_int32), ("residual_f32", ctypes.c_int32),
        ("weight_f32", ctypes.c_int32), ("out_e4m3", ctypes.c_int32), ("eps", ctypes.c_float),
        ("x", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("weight", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("residual_out", ctypes.c_void_p), ("scale", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
        ("residual_out_stride", ctypes.c_int64),
    ]


class RopeDesc(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("shared_ladder", ctypes.c_int32), ("sections", ctypes.POINTER(ctypes.c_int32)), ("theta", ctypes.c_double),
        ("inv_freq", ctypes.POINTER(ctypes.c_double)), ("axis", ctypes.POINTER(ctypes.c_int32)),
    ]


class QkRopeArgs(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64), ("pos_rows", ctypes.c_int64), ("heads", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32), ("positions_f32", ctypes.c_int32), ("eps", ctypes.c_float),
        ("positions", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
        ("k_out", ctypes.c_void_p), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
        *[(n, ctypes.c_int64) for n in ("q_stride", "q_head_stride", "k_stride", "k_head_stride", "q_out_stride",
                                        "q_out_head_stride", "k_out_stride", "k_out_head_stride")],
    ]


class PackedDesc(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("causal", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
        ("lengths", ctypes.POINTER(ctypes.c_int32)),
    ]


class PackedDims(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64), ("pairs", ctypes.c_int64), ("items", ctypes.c_int64), ("ctas", ctypes.c_int32),
        ("tile_tokens", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
    ]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class PackedArgs(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        *[(n, ctypes.c_int64) for n in ("q_stride", "q_head_stride", "k_stride", "k_head_stride", "v_stride",
                                        "v_head_stride", "out_stride", "out_head_stride")],
    ]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libvsa.so; raise if it is missing (no fallback path exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libvsa.so not found at {path}; build it with `python -m block_sparse_tiled_b200.build`")
    lib = ctypes.CDLL(path)
    P, st = ctypes.c_void_p, ctypes.c_int
    lib.vsa_last_error.restype = ctypes.c_char_p
    lib.vsa_version.restype = ctypes.c_char_p
    lib.vsa_plan_query.argtypes = [ctypes.POINTER(Geometry), ctypes.POINTER(PlanDims)]
    lib.vsa_plan_tables_host.argtypes = [ctypes.POINTER(Geometry), P, P]
    lib.vsa_plan_tiles.argtypes = [ctypes.POINTER(Geometry), P, ctypes.POINTER(P)]
    lib.vsa_plan_info.argtypes = [P, ctypes.POINTER(PlanDims)]
    lib.vsa_plan_tables.argtypes = [P, P, P]
    lib.vsa_plan_workspace.argtypes = [P, ctypes.POINTER(WorkspaceLayout)]
    lib.vsa_plan_destroy.argtypes = [P]
    lib.vsa_gather_tiles.argtypes = [P] * 13
    lib.vsa_pool_and_score.argtypes = [P] * 9
    lib.vsa_topk_select.argtypes = [P] * 6
    lib.vsa_sparse_attn_fwd.argtypes = [P] * 11
    lib.vsa_forward.argtypes = [P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.vsa_forward_noalloc.argtypes = [P] * 7
    lib.vsa_forward_host_workspace.argtypes = [P, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
    lib.vsa_forward_host.argtypes = [P, P, P, P, P, P, ctypes.c_int32, P, ctypes.c_size_t, P]
    lib.vsa_forward_parts.argtypes = [P, ctypes.POINTER(SeqParts), P, ctypes.c_size_t, P]
    lib.vsa_wait_selftest.argtypes = [P, ctypes.c_int64, P, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
    lib.vsa_device_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
    lib.vsa_rms_norm.argtypes = [ctypes.POINTER(RmsNormArgs), P]
    lib.vsa_rope_create.argtypes = [ctypes.POINTER(RopeDesc), ctypes.POINTER(P)]
    lib.vsa_rope_table.argtypes = [P, P, P]
    lib.vsa_rope_destroy.argtypes = [P]
    lib.vsa_qk_rope.argtypes = [P, ctypes.POINTER(QkRopeArgs), P]
    lib.vsa_packed_plan.argtypes = [ctypes.POINTER(PackedDesc), P, ctypes.POINTER(P)]
    lib.vsa_packed_query.argtypes = [ctypes.POINTER(PackedDesc), ctypes.c_int32, ctypes.POINTER(PackedDims), P, P]
    lib.vsa_packed_info.argtypes = [P, ctypes.POINTER(PackedDims)]
    lib.vsa_packed_destroy.argtypes = [P]
    lib.vsa_packed_attn.argtypes = [P, ctypes.POINTER(PackedArgs), P]
    lib.vsa_packed_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
    lib.vsa_packed_wait_selftest.argtypes = [P, ctypes.c_int64, P, ctypes.POINTER(ctypes.c_int32),
                                             ctypes.POINTER(ctypes.c_int32)]
    for name in EXPORTED:
        if name not in ("vsa_last_error", "vsa_version"):
            getattr(lib, name).restype = st
    _lib = lib
    return lib


def _check(rc: int, where: str):
    if rc != VSA_OK:
        raise VsaError(rc, where, load_library().vsa_last_error().decode())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _allocating_on(stream, device):
    """The context in which torch allocates and fills memory for a call on `stream` of `device`: memory of that
    stream's pool, whose earlier and later uses the stream orders (None: the current stream's, as anywhere)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        # torch knows the legacy default stream as 0 only, not by its other name, cudaStreamLegacy = 1
        stream = torch.cuda.ExternalStream(0 if handle == 1 else handle, device=device)
    return torch.cuda.stream(stream)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _qk_mode(qk_fp8) -> int:
    """qk_fp8: False / True (8-bit Q/K logits for every query tile) / "prefix" (for the dense prefix query
    tiles only, the pages' split) / "fp4" (the split, and FP4 Q and smoothed FP4 K for the video query
    tiles) -> the geometry's 0 / 1 / 2 / 3."""
    if isinstance(qk_fp8, str):
        modes = {"prefix": 2, "fp4": 3}
        if qk_fp8 not in modes:
            raise ValueError(f"qk_fp8 must be a bool, 'prefix' or 'fp4', got {qk_fp8!r}")
        return modes[qk_fp8]
    return int(bool(qk_fp8))


def make_geometry(batch, heads, head_dim, segments=(), grid=(0, 0, 0), sparsity=0.0, softmax_scale=0.0,
                  token_tags=None, video_tag=0, tile_size=64, gate_per_channel=False, seq_tiles=False, qk_fp8=False,
                  cube=None, ref_segments=None, ref_keep=0.0):
    """Build the ``vsa_geometry`` struct; returns (struct, keep-alive buffers).  cube: (t, h, w) of a
    video tile, None for the default (4x4x4 for 64-token tiles, 4x4x8 for 128).  ref_segments: one
    flag per prefix segment marking reference segments, with their keep ratio ref_keep."""
    g = Geometry()
    g.batch, g.heads, g.head_dim = int(batch), int(heads), int(head_dim)
    keep = []
    if token_tags is not None:
        tags = (ctypes.c_int32 * len(token_tags))(*[int(t) for t in token_tags])
        keep.append(tags)
        g.token_tags = ctypes.cast(tags, ctypes.POINTER(ctypes.c_int32))
        g.seq_len = len(token_tags)
        g.video_tag = int(video_tag)
        g.n_segments = 0
    else:
        seg = (ctypes.c_int32 * max(1, len(segments)))(*[int(s) for s in segments])
        keep.append(seg)
        g.segment_len = ctypes.cast(seg, ctypes.POINTER(ctypes.c_int32))
        g.n_segments = len(segments)
        g.seq_len = 0
    g.grid_t, g.grid_h, g.grid_w = (int(x) for x in grid)
    g.tile_size = int(tile_size)
    g.sparsity = float(sparsity)
    g.softmax_scale = float(softmax_scale)
    g.gate_per_channel = int(bool(gate_per_channel))
    g.seq_tiles = int(bool(seq_tiles))
    g.qk_fp8 = _qk_mode(qk_fp8)
    g.cube_t, g.cube_h, g.cube_w = (int(c) for c in (cube or (0, 0, 0)))
    if ref_segments is not None:
        flags = (ctypes.c_int32 * max(1, len(ref_segments)))(*[int(f) for f in ref_segments])
        keep.append(flags)
        g.segment_reference = ctypes.cast(flags, ctypes.POINTER(ctypes.c_int32))
        g.reference_keep = float(ref_keep)
    return g, keep


def vsa_plan_query(**kw) -> dict:
    """Resolve sizes without touching a device."""
    g, keep = make_geometry(**kw)
    d = PlanDims()
    _check(load_library().vsa_plan_query(ctypes.byref(g), ctypes.byref(d)), "vsa_plan_query")
    return d.as_dict()


def vsa_plan_tables_host(**kw):
    """Host-only token table of a geometry: (tile_token [n_tiles, tile_size], tile_valid [n_tiles])."""
    import numpy as np

    d = vsa_plan_query(**kw)
    g, keep = make_geometry(**kw)
    n = d["n_tiles"]
    tok = np.empty((max(n, 1), d["tile_size"]), np.int32)
    val = np.empty((max(n, 1),), np.int32)
    _check(load_library().vsa_plan_tables_host(ctypes.byref(g), tok.ctypes.data_as(ctypes.c_void_p),
                                               val.ctypes.data_as(ctypes.c_void_p)), "vsa_plan_tables_host")
    return tok[:n], val[:n]


class Plan:
    """Owns a ``vsa_plan`` handle (the device tile tables of one geometry)."""

    def __init__(self, handle, geometry_kwargs):
        self._h = handle
        self.geometry = dict(geometry_kwargs)
        d = PlanDims()
        _check(load_library().vsa_plan_info(self._h, ctypes.byref(d)), "vsa_plan_info")
        self.dims = d.as_dict()
        ws = WorkspaceLayout()
        _check(load_library().vsa_plan_workspace(self._h, ctypes.byref(ws)), "vsa_plan_workspace")
        self.workspace_layout = {f: getattr(ws, f) for f, _ in WorkspaceLayout._fields_}

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("plan destroyed")
        return self._h

    def tables(self):
        import numpy as np

        n = self.dims["n_tiles"]
        tok = np.empty((max(n, 1), self.dims["tile_size"]), np.int32)
        val = np.empty((max(n, 1),), np.int32)
        _check(load_library().vsa_plan_tables(self.handle, tok.ctypes.data_as(ctypes.c_void_p),
                                              val.ctypes.data_as(ctypes.c_void_p)), "vsa_plan_tables")
        return tok[:n], val[:n]

    def destroy(self):
        if self._h is not None:
            load_library().vsa_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def vsa_plan_tiles(batch, heads, head_dim, segments=(), grid=(0, 0, 0), sparsity=0.0, softmax_scale=0.0,
                   token_tags=None, video_tag=0, tile_size=64, gate_per_channel=False, seq_tiles=False,
                   qk_fp8=False, cube=None, ref_segments=None, ref_keep=0.0, stream=None) -> Plan:
    kw = dict(batch=batch, heads=heads, head_dim=head_dim, segments=tuple(segments), grid=tuple(grid),
              sparsity=sparsity, softmax_scale=softmax_scale, token_tags=token_tags, video_tag=video_tag,
              tile_size=tile_size, gate_per_channel=bool(gate_per_channel), seq_tiles=bool(seq_tiles),
              qk_fp8=qk_fp8 if isinstance(qk_fp8, str) else bool(qk_fp8), cube=None if cube is None else tuple(cube),
              ref_segments=None if ref_segments is None else tuple(ref_segments), ref_keep=float(ref_keep))
    g, keep = make_geometry(**kw)
    h = ctypes.c_void_p()
    _check(load_library().vsa_plan_tiles(ctypes.byref(g), _stream(stream), ctypes.byref(h)), "vsa_plan_tiles")
    return Plan(h, kw)


def vsa_gather_tiles(plan, q, k, v, q_t, k_t, v_t, pq=None, pk=None, pv=None, q_norm=None, kv_max=None,
                     stream=None):
    bf, f32 = torch.bfloat16, torch.float32
    _check(load_library().vsa_gather_tiles(
        plan.handle, _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"), _ptr(q_t, bf, "q_t"),
        _ptr(k_t, bf, "k_t"), _ptr(v_t, bf, "v_t"), _ptr(pq, f32, "pq"), _ptr(pk, f32, "pk"), _ptr(pv, f32, "pv"),
        _ptr(q_norm, f32, "q_norm"), _ptr(kv_max, f32, "kv_max"), _stream(stream)), "vsa_gather_tiles")


def vsa_pool_and_score(plan, q_t, k_t, v_t, pq, pk, pv, scores, stream=None):
    bf, f32 = torch.bfloat16, torch.float32
    _check(load_library().vsa_pool_and_score(
        plan.handle, _ptr(q_t, bf, "q_t"), _ptr(k_t, bf, "k_t"), _ptr(v_t, bf, "v_t"), _ptr(pq, f32, "pq"),
        _ptr(pk, f32, "pk"), _ptr(pv, f32, "pv"), _ptr(scores, f32, "scores"), _stream(stream)),
        "vsa_pool_and_score")


def vsa_topk_select(plan, scores, pv, idx, o_c, stream=None):
    f32 = torch.float32
    _check(load_library().vsa_topk_select(
        plan.handle, _ptr(scores, f32, "scores"), _ptr(pv, f32, "pv"), _ptr(idx, torch.int32, "idx"),
        _ptr(o_c, f32, "o_c"), _stream(stream)), "vsa_topk_select")


def vsa_sparse_attn_fwd(plan, q_t, k_t, v_t, idx, o_c, gate, out, q_norm=None, kv_max=None, stream=None):
    bf, f32 = torch.bfloat16, torch.float32
    _check(load_library().vsa_sparse_attn_fwd(
        plan.handle, _ptr(q_t, bf, "q_t"), _ptr(k_t, bf, "k_t"), _ptr(v_t, bf, "v_t"),
        _ptr(idx, torch.int32, "idx"), _ptr(o_c, f32, "o_c"), _ptr(gate, bf, "gate"),
        _ptr(out, bf, "out"), _ptr(q_norm, f32, "q_norm"), _ptr(kv_max, f32, "kv_max"), _stream(stream)),
        "vsa_sparse_attn_fwd")


def alloc_workspace(plan, device=None) -> torch.Tensor:
    """A uint8 device buffer of ``workspace_bytes`` (torch's allocator aligns to >= 256 bytes)."""
    n = max(256, plan.dims["workspace_bytes"])
    return torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda", torch.cuda.current_device()))


def default_head_chunk(heads: int, head_dim: int = 128) -> int:
    """Heads per chunk of the host pipeline.  Small chunks keep the forward and copy-back of the last
    chunk, which nothing overlaps, short; but each chunk's copies are strided rows of chunk*head_dim
    bf16 values, and rows under 512 bytes copy slowly (measured at 1344x768, 56 heads, D = 128:
    1 head per chunk 104.7 ms, 2: 62.7 ms, 4: 64.2 ms, 8: 67.5 ms, 14: 76.2 ms).  So: the smallest
    chunk with rows of at least 512 bytes, and at most 32 chunks."""
    rows = -(-512 // (2 * head_dim))
    return max(1, min(heads, max(rows, -(-heads // 32))))


def host_workspace_bytes(plan, head_chunk=None) -> int:
    g = plan.geometry
    hc = default_head_chunk(g["heads"], g["head_dim"]) if head_chunk is None else int(head_chunk)
    n = ctypes.c_size_t()
    _check(load_library().vsa_forward_host_workspace(plan.handle, hc, ctypes.byref(n)), "vsa_forward_host_workspace")
    return n.value


def _host_ptr(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.is_cuda:
        raise ValueError(f"{name} must be a CPU tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def vsa_forward_host(plan, q, k, v, gate, out=None, workspace=None, head_chunk=None, stream=None):
    """The whole forward for CPU (ideally pinned) q, k, v, gate; returns the CPU
    output.  The heads run in chunks whose copies overlap the compute of the
    neighbouring chunks (vsa_forward_host).  Without a workspace, one is
    allocated on first use and kept on the plan.  Returns once the stream has
    drained."""
    g = plan.geometry
    hc = default_head_chunk(g["heads"], g["head_dim"]) if head_chunk is None else int(head_chunk)
    need = host_workspace_bytes(plan, hc)
    if workspace is None:
        cached = getattr(plan, "_host_ws", None)
        if cached is None or cached.numel() < need:
            device = torch.device("cuda", torch.cuda.current_device())
            with _allocating_on(stream, device):
                cached = torch.empty(need, dtype=torch.uint8, device=device)
            plan._host_ws = cached
        workspace = cached
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    _check(load_library().vsa_forward_host(
        plan.handle, _host_ptr(q, "q"), _host_ptr(k, "k"), _host_ptr(v, "v"), _host_ptr(gate, "gate"),
        _host_ptr(out, "out"), hc, _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)),
        "vsa_forward_host")
    if stream is None:
        torch.cuda.current_stream().synchronize()
    elif isinstance(stream, torch.cuda.Stream):
        stream.synchronize()
    else:
        torch.cuda.synchronize()
    return out


def vsa_forward(plan, q, k, v, gate, out=None, workspace=None, stream=None):
    """The whole forward.  CUDA inputs: runs in place on the stream.  CPU
    inputs (ideally pinned): the head-chunked host pipeline (vsa_forward_host),
    with `workspace` sized by host_workspace_bytes when given."""
    if not q.is_cuda:
        return vsa_forward_host(plan, q, k, v, gate, out=out, workspace=workspace, stream=stream)
    with _allocating_on(stream, q.device):
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            workspace = alloc_workspace(plan, q.device)
    bf = torch.bfloat16
    _check(load_library().vsa_forward(
        plan.handle, _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"), _ptr(gate, bf, "gate"),
        _ptr(out, bf, "out"), _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)),
        "vsa_forward")
    return out


MAX_PARTS = 64


def ulysses_partition(seq_len: int, heads: int, world: int, rank: int):
    """Sequence-parallel layout of one rank: (tokens per part, heads of this rank, first head).  Rank r
    holds tokens [r*Ls, (r+1)*Ls) of q/k/v/gate/out and runs the forward for heads [r*Hn, (r+1)*Hn)."""
    if world < 1 or not 0 <= rank < world:
        raise ValueError(f"rank {rank} outside a world of {world}")
    if seq_len % world or heads % world:
        raise ValueError(f"the world size {world} must divide the sequence length {seq_len} and the heads {heads}")
    hn = heads // world
    return seq_len // world, hn, rank * hn


def vsa_forward_parts(plan, q_parts, k_parts, v_parts, gate_parts, out_parts, head_offset, workspace=None, stream=None):
    """The forward for this plan's heads over a sequence split into parts (lists of CUDA tensors
    [B, Ls, Htot, D], gate [B, Ls, Htot] or [B, Ls, Htot*D]); parts may be peer mappings of other
    GPUs' buffers.  Writes heads [head_offset, head_offset + H) of every out part."""
    n = len(q_parts)
    if not (len(k_parts) == len(v_parts) == len(gate_parts) == len(out_parts) == n) or not 1 <= n <= MAX_PARTS:
        raise ValueError("q, k, v, gate and out need the same number of parts, at most MAX_PARTS")
    B, Ls, Htot, D = q_parts[0].shape
    if workspace is None:
        with _allocating_on(stream, q_parts[0].device):
            workspace = alloc_workspace(plan, q_parts[0].device)
    bf = torch.bfloat16

    def arr(ts, name):
        return (ctypes.c_void_p * n)(*[_ptr(t, bf, f"{name}[{i}]") for i, t in enumerate(ts)])

    keep = [arr(q_parts, "q"), arr(k_parts, "k"), arr(v_parts, "v"), arr(gate_parts, "gate"), arr(out_parts, "out")]
    cast = lambda a: ctypes.cast(a, ctypes.POINTER(ctypes.c_void_p))  # noqa: E731
    sp = SeqParts(n, Ls, Htot, int(head_offset), *[cast(a) for a in keep])
    _check(load_library().vsa_forward_parts(plan.handle, ctypes.byref(sp), _ptr(workspace, torch.uint8, "workspace"),
                                            workspace.numel(), _stream(stream)), "vsa_forward_parts")
    return out_parts


NOALLOC_SCRATCH_BYTES = 64 << 20


def vsa_forward_noalloc(plan, q, k, v, gate, out, stream=None):
    """The whole forward with the library's static device scratch instead of a
    caller workspace (for callers that cannot allocate device memory).  Calls
    on one device share that scratch: do not let them overlap on the GPU."""
    bf = torch.bfloat16
    _check(load_library().vsa_forward_noalloc(
        plan.handle, _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"), _ptr(gate, bf, "gate"),
        _ptr(out, bf, "out"), _stream(stream)), "vsa_forward_noalloc")
    return out


def wait_selftest(plan, timeout_ns=50_000_000, stream=None):
    """Run the bounded-wait self-test; returns the (code, site) it recorded."""
    code, where = ctypes.c_int32(), ctypes.c_int32()
    _check(load_library().vsa_wait_selftest(plan.handle, int(timeout_ns), _stream(stream), ctypes.byref(code),
                                            ctypes.byref(where)), "vsa_wait_selftest")
    return code.value, where.value


def device_status(plan, stream=None):
    code, where = ctypes.c_int32(), ctypes.c_int32()
    _check(load_library().vsa_device_status(plan.handle, _stream(stream), ctypes.byref(code), ctypes.byref(where)),
           "vsa_device_status")
    return code.value, where.value


def workspace_views(plan, workspace):
    """Typed views of vsa_forward's intermediates inside ``workspace`` (no tile-order views for a plan
    with seq_tiles, whose workspace holds none).  With qk_fp8, q_t and k_t are the E4M3 codes
    [B, H, n_t, tile, 128] (uint8) and q_s, k_s their row scales [B, H, n_t, tile].  q_n holds the
    query row norms [B, H, n_t, tile] (with qk_fp8 of the dequantised rows) and kv_max the (b, h)
    maxima of key norm and |v| [B, H, 2] (the attention's overflow bound).  With qk_fp8="prefix" q_t and
    k_t are the bf16 copies, q_c and k_c the codes, q_s and k_s their scales, and q_n8, kv_max8 the
    statistics of the dequantised rows.  With qk_fp8="fp4" the same, except that q_t's video query tiles
    and k_t's valid rows hold their FP4 roundings (bf16 numbers; keys after smoothing), k_sum the binary64
    key column sums [B, H, D] and k_mu the key means [B, H, D]; q_n and kv_max describe the rounded copies."""
    d, g = plan.dims, plan.geometry
    B, H, D, n_t, V, k = g["batch"], g["heads"], g["head_dim"], d["n_tiles"], d["n_video_tiles"], d["topk"]
    lay = plan.workspace_layout
    seq = bool(g.get("seq_tiles", False))
    mode = _qk_mode(g.get("qk_fp8", False))
    f8, split = mode == 1, mode >= 2
    T = d["tile_size"]  # rows per tile

    def view(off, n, dtype, shape):
        nbytes = n * torch.tensor([], dtype=dtype).element_size()
        return workspace[off:off + nbytes].view(dtype).view(*shape)

    def tiles(name):
        return None if seq else view(lay[name], B * H * n_t * T * D, torch.bfloat16, (B, H, n_t, T, D))

    def codes(name):
        return view(lay[name], B * H * n_t * T * 128, torch.uint8, (B, H, n_t, T, 128))

    def row_scales(name):
        return view(lay[name], B * H * n_t * T, torch.float32, (B, H, n_t, T)) if (f8 or split) else None

    extra = {} if not split else {
        "q_c": codes("q_c"), "k_c": codes("k_c"),
        "q_n8": view(lay["q_n8"], B * H * n_t * T, torch.float32, (B, H, n_t, T)),
        "kv_max8": view(lay["kv_max8"], B * H * 2, torch.float32, (B, H, 2)),
    }
    if mode == 3:
        extra["k_sum"] = view(lay["k_sum"], B * H * D, torch.float64, (B, H, D))
        extra["k_mu"] = view(lay["k_mu"], B * H * D, torch.float32, (B, H, D))
    return {
        **extra,
        "q_t": codes("q_t") if f8 else tiles("q_t"),
        "k_t": codes("k_t") if f8 else tiles("k_t"),
        "v_t": tiles("v_t"),
        "q_s": row_scales("q_s"),
        "k_s": row_scales("k_s"),
        "q_n": view(lay["q_n"], B * H * n_t * T, torch.float32, (B, H, n_t, T)),
        "kv_max": view(lay["kv_max"], B * H * 2, torch.float32, (B, H, 2)),
        "pq": view(lay["pq"], B * H * n_t * D, torch.float32, (B, H, n_t, D)),
        "pk": view(lay["pk"], B * H * n_t * D, torch.float32, (B, H, n_t, D)),
        "pv": view(lay["pv"], B * H * n_t * D, torch.float32, (B, H, n_t, D)),
        "scores": view(lay["scores"], B * H * n_t * n_t, torch.float32, (B, H, n_t, n_t)),
        "idx": view(lay["idx"], B * H * V * (k + d["ref_topk"]), torch.int32, (B, H, V, k + d["ref_topk"])),
        "o_c": view(lay["o_c"], B * H * n_t * D, torch.float32, (B, H, n_t, D)),
    }


# ---------------------------------------------------------------------------
# Row operators around the attention
# ---------------------------------------------------------------------------


_BF16, _F32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _int32(x, name):
    """x as the library's 32-bit field takes it (ctypes would drop the bits above)."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def _launch_index(names, *tensors):
    """The index of the one CUDA device that holds every given tensor, which must be the current device (the
    library launches there).  These calls are a few microseconds of GPU work at their smallest, so the checks
    go by index and build nothing."""
    index = None
    for t in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            name = next(n for n, x in zip(names, tensors) if x is t)
            raise TypeError(f"{name} must be a torch.Tensor")
        i = t.get_device()
        if index is None:
            index = i
        if i < 0 or i != index:
            name = next(n for n, x in zip(names, tensors) if x is t)
            raise ValueError(f"{name} is on {t.device}: every tensor must be on one CUDA device")
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on cuda:{index}, the current device is cuda:{torch.cuda.current_device()}")
    return index


def _stream_on(stream, index):
    """The raw handle of `stream`, by default the current stream of device `index`."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if not isinstance(stream, torch.cuda.Stream):
        return int(stream)
    if stream.device_index != index:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors on cuda:{index}")
    return stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """An output that a call on `stream` allocates."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _allocating_on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _row_stride(t, shape, name):
    """Elements between rows of a tensor of this shape: two-dimensional with unit stride inside its rows, or
    contiguous."""
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if len(shape) == 2:
        s = t.stride()
        if s[1] == 1:
            return s[0] if shape[0] > 1 else shape[1]
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, or two-dimensional with contiguous rows")
    return shape[-1]


def vsa_rms_norm(x, weight=None, eps=1e-6, residual=None, out=None, residual_out=None, scale=None, out_dtype=None,
                 stream=None):
    """Root-mean-square norm over the last dimension of x + residual, times weight, in one pass.

    x: [..., C] bf16 (contiguous, or [rows, C] with any row stride that is a multiple of 8), C a multiple of 8
    up to 16384; weight: [C] bf16 or float32, None for ones; residual: like x, bf16 or float32.
    out_dtype (or the type of `out`): torch.bfloat16, or torch.float8_e4m3fn for 8-bit codes with one
    float32 scale per row, scale = max|y| / 448 (out.float() * scale[..., None] is y, rounded).
    residual_out receives x + residual in the residual's type (allocated when there is a residual; the residual
    itself may be passed, and out may be x).  Returns (out, scale or None, residual_out or None)."""
    index = _launch_index(("x", "weight", "residual", "out", "residual_out", "scale"), x, weight, residual, out,
                          residual_out, scale)
    if x.dtype != _BF16:
        raise TypeError(f"x must be torch.bfloat16, got {x.dtype}")
    shape = x.shape
    if not shape or shape[-1] == 0:
        raise ValueError(f"x must end in a dimension that is not empty, got {tuple(shape)}")
    C = shape[-1]
    if C > 0x7fffffff:
        raise ValueError(f"the width must fit 32 bits, got {C}")
    rows = x.numel() // C
    if out is None:
        out = _empty(shape, out_dtype or _BF16, x.device, stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype is {out_dtype}")
    f8 = out.dtype == _E4M3
    if not f8 and out.dtype != _BF16:
        raise TypeError(f"the output type must be torch.bfloat16 or torch.float8_e4m3fn, got {out.dtype}")
    w_ptr = w_f32 = s_ptr = r_ptr = ro_ptr = r_f32 = r_ld = ro_ld = 0
    if weight is not None:
        w_f32 = weight.dtype == _F32
        if not w_f32 and weight.dtype != _BF16:
            raise TypeError(f"weight must be torch.bfloat16 or torch.float32, got {weight.dtype}")
        if weight.shape != (C,) or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous [{C}], got {tuple(weight.shape)}")
        w_ptr = weight.data_ptr()
    if f8:
        if scale is None:
            scale = _empty(shape[:-1], _F32, x.device, stream)
        elif scale.dtype != _F32:
            raise TypeError(f"scale must be torch.float32, got {scale.dtype}")
        elif scale.numel() != rows or not scale.is_contiguous():
            raise ValueError(f"scale must be contiguous with one value for each of the {rows} rows")
        s_ptr = scale.data_ptr()
    elif scale is not None:
        raise ValueError("scale belongs to an 8-bit output")
    if residual is not None:
        r_f32 = residual.dtype == _F32
        if not r_f32 and residual.dtype != _BF16:
            raise TypeError(f"residual must be torch.bfloat16 or torch.float32, got {residual.dtype}")
        if residual_out is None:
            residual_out = _empty(shape, residual.dtype, x.device, stream)
        elif residual_out.dtype != residual.dtype:
            raise TypeError(f"residual_out must be {residual.dtype}, got {residual_out.dtype}")
        r_ptr, r_ld = residual.data_ptr(), _row_stride(residual, shape, "residual")
        ro_ptr, ro_ld = residual_out.data_ptr(), _row_stride(residual_out, shape, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    a = RmsNormArgs(rows, C, r_f32, w_f32, f8, eps, x.data_ptr(), r_ptr, w_ptr, out.data_ptr(), ro_ptr, s_ptr,
                    _row_stride(x, shape, "x"), r_ld, _row_stride(out, shape, "out"), ro_ld)
    rc = (_lib or load_library()).vsa_rms_norm(ctypes.byref(a), _stream_on(stream, index))
    if rc:
        _check(rc, "vsa_rms_norm")
    return out, scale, residual_out


class Rope:
    """Owns a ``vsa_rope`` handle: the frequency and axis of every pair of a head row (host only)."""

    def __init__(self, handle, head_dim, n_axes, interleaved):
        self._h, self.head_dim, self.n_axes, self.interleaved = handle, head_dim, n_axes, interleaved

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("rope destroyed")
        return self._h

    def table(self):
        """(inv_freq float64 [head_dim / 2], axis int32 [head_dim / 2])."""
        import numpy as np

        freq, axis = np.empty(self.head_dim // 2), np.empty(self.head_dim // 2, np.int32)
        _check(load_library().vsa_rope_table(self.handle, freq.ctypes.data, axis.ctypes.data), "vsa_rope_table")
        return freq, axis

    def destroy(self):
        if self._h is not None:
            load_library().vsa_rope_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def vsa_rope_create(head_dim, sections=None, theta=10000.0, interleaved=False, shared_ladder=False, inv_freq=None,
                    axis=None, n_axes=None) -> Rope:
    """Rotary positions of a head row of head_dim (64, 96 or 128): sections = rotated pairs per axis, e.g.
    (16, 24, 24) for (time, height, width); pairs behind them do not turn.  The i-th of an axis's n pairs turns
    theta^(-i / n) radians per step, with shared_ladder pair p of the head theta^(-p / (head_dim / 2)).  Or
    inv_freq and axis, head_dim / 2 values each, give any other table (n_axes: 1 + the largest axis).
    interleaved: pair p is elements (2p, 2p + 1), else (p, p + head_dim / 2)."""
    d = RopeDesc(head_dim=_int32(head_dim, "head_dim"), interleaved=int(bool(interleaved)), shared_ladder=int(bool(shared_ladder)),
                 theta=float(theta))
    if (inv_freq is None) != (axis is None):
        raise ValueError("inv_freq and axis go together")
    if inv_freq is not None:
        if sections is not None:
            raise ValueError("give sections, or inv_freq and axis")
        freq, ax = [float(f) for f in inv_freq], [_int32(x, "an axis") for x in axis]
        if len(freq) != d.head_dim // 2 or len(ax) != d.head_dim // 2:
            raise ValueError(f"inv_freq and axis need head_dim / 2 = {d.head_dim // 2} values each")
        d.n_axes = _int32(1 + max(ax) if n_axes is None else n_axes, "n_axes")
        keep = [(ctypes.c_double * len(freq))(*freq), (ctypes.c_int32 * len(ax))(*ax)]
        d.inv_freq = ctypes.cast(keep[0], ctypes.POINTER(ctypes.c_double))
        d.axis = ctypes.cast(keep[1], ctypes.POINTER(ctypes.c_int32))
    else:
        if sections is None:
            raise ValueError("give sections, or inv_freq and axis")
        sec = [_int32(s, "a section") for s in sections]
        if n_axes is not None and n_axes != len(sec):
            raise ValueError("n_axes must be the number of sections")
        d.n_axes = len(sec)
        keep = [(ctypes.c_int32 * max(1, len(sec)))(*sec)]
        d.sections = ctypes.cast(keep[0], ctypes.POINTER(ctypes.c_int32))
    h = ctypes.c_void_p()
    _check(load_library().vsa_rope_create(ctypes.byref(d), ctypes.byref(h)), "vsa_rope_create")
    return Rope(h, d.head_dim, d.n_axes, bool(interleaved))


def _head_rows(t, D, name):
    """(tokens, heads, elements between tokens, between heads) of [T, H, D], or of [B, L, H, D] whose tokens are
    evenly spaced."""
    if t.dtype != _BF16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    sh, st = t.shape, t.stride()
    if len(sh) not in (3, 4) or sh[-1] != D:
        raise ValueError(f"{name} must be [T, H, {D}] or [B, L, H, {D}], got {tuple(sh)}")
    if st[-1] != 1:
        raise ValueError(f"{name} must have contiguous head rows")
    H = sh[-2]
    tokens, ld, hd = sh[-3], st[-3], (st[-2] if H > 1 else D)
    if len(sh) == 4:
        if sh[0] > 1 and sh[1] > 1 and st[0] != sh[1] * st[1]:
            raise ValueError(f"{name}: the tokens of [B, L, H, D] must be evenly spaced")
        tokens, ld = sh[0] * sh[1], (st[1] if sh[1] > 1 else st[0])
    return tokens, H, (ld if tokens > 1 else H * D), hd


def _head_weight(w, D, name):
    if w.dtype != _BF16:
        raise TypeError(f"{name} must be torch.bfloat16, got {w.dtype}")
    if w.shape != (D,) or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{D}], got {tuple(w.shape)}")
    return w.data_ptr()


def vsa_qk_rope(rope, q, k, positions, q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None, stream=None):
    """Head norm (with q_weight / k_weight [D]) and rotary positions of q [T, H, D] and k [T, Hk, D] (or
    [B, L, H, D]; any token and head strides that are multiples of 8, e.g. slices of one projection; k may be
    None), bf16.  positions: [T, n_axes] int32 or float32 (any leading dimensions of T rows in all), or for q
    [B, L, H, D] the [L, n_axes] that every sequence uses.  In place with q_out = q, k_out = k.  Returns (q_out, k_out)."""
    D, axes = rope.head_dim, rope.n_axes
    index = _launch_index(("q", "k", "positions", "q_weight", "k_weight", "q_out", "k_out"), q, k, positions, q_weight,
                          k_weight, q_out, k_out)
    tokens, H, q_ld, q_hd = _head_rows(q, D, "q")
    pos_f32 = positions.dtype == _F32
    if not pos_f32 and positions.dtype != torch.int32:
        raise TypeError(f"positions must be torch.int32 or torch.float32, got {positions.dtype}")
    if positions.dim() < 2 or positions.shape[-1] != axes or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous [tokens, {axes}], got {tuple(positions.shape)}")
    rows = positions.numel() // axes
    # the library repeats any number of rows that divides the tokens (and refuses others); here only a batch's sequences do
    if rows != tokens and rows > 0 and tokens % rows == 0 and not (q.dim() == 4 and rows == q.shape[1]):
        fits = f"{tokens}" if q.dim() == 3 else f"{q.shape[1]} or {tokens}"
        raise ValueError(f"positions must have {fits} rows for q {tuple(q.shape)}, got {rows}")
    if q_out is None:
        q_out = _empty(q.shape, _BF16, q.device, stream)
    elif q_out.shape != q.shape:
        raise ValueError(f"q_out must have q's shape {tuple(q.shape)}, got {tuple(q_out.shape)}")
    _, _, qo_ld, qo_hd = _head_rows(q_out, D, "q_out")
    Hk = k_ptr = ko_ptr = k_ld = k_hd = ko_ld = ko_hd = 0
    if k is not None:
        tk, Hk, k_ld, k_hd = _head_rows(k, D, "k")
        if tk != tokens:
            raise ValueError(f"k has {tk} tokens, q {tokens}")
        if k_out is None:
            k_out = _empty(k.shape, _BF16, k.device, stream)
        elif k_out.shape != k.shape:
            raise ValueError(f"k_out must have k's shape {tuple(k.shape)}, got {tuple(k_out.shape)}")
        _, _, ko_ld, ko_hd = _head_rows(k_out, D, "k_out")
        k_ptr, ko_ptr = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    a = QkRopeArgs(tokens, rows, H, Hk, pos_f32, eps, positions.data_ptr(), q.data_ptr(), k_ptr,
                   q_out.data_ptr(), ko_ptr, 0 if q_weight is None else _head_weight(q_weight, D, "q_weight"),
                   0 if k_weight is None else _head_weight(k_weight, D, "k_weight"), q_ld, q_hd, k_ld, k_hd, qo_ld,
                   qo_hd, ko_ld, ko_hd)
    rc = (_lib or load_library()).vsa_qk_rope(rope.handle, ctypes.byref(a), _stream_on(stream, index))
    if rc:
        _check(rc, "vsa_qk_rope")
    return q_out, k_out


# ---------------------------------------------------------------------------
# Attention over packed whole prompts
# ---------------------------------------------------------------------------


def make_packed_desc(lengths, heads, kv_heads=None, head_dim=128, causal=True, softmax_scale=0.0):
    """Build the ``vsa_packed_desc`` struct; returns (struct, keep-alive buffer)."""
    n = [_int32(x, "a length") for x in lengths]
    buf = (ctypes.c_int32 * max(1, len(n)))(*n)
    d = PackedDesc(len(n), _int32(heads, "heads"), _int32(heads if kv_heads is None else kv_heads, "kv_heads"),
                   _int32(head_dim, "head_dim"), int(bool(causal)), float(softmax_scale),
                   ctypes.cast(buf, ctypes.POINTER(ctypes.c_int32)))
    return d, buf


def vsa_packed_query(lengths, heads, kv_heads=None, head_dim=128, causal=True, softmax_scale=0.0, sms=148) -> dict:
    """Resolve the sizes of a packed plan without touching a device, with its schedule for a GPU of `sms` SMs:
    "items" [n, 4] (sequence's first row, its length, the item's first token inside it, key head) and
    "first" [ctas + 1]."""
    import numpy as np

    desc, keep = make_packed_desc(lengths, heads, kv_heads, head_dim, causal, softmax_scale)
    d, lib, sms = PackedDims(), load_library(), _int32(sms, "sms")
    _check(lib.vsa_packed_query(ctypes.byref(desc), sms, ctypes.byref(d), None, None), "vsa_packed_query")
    items, first = np.zeros((max(1, d.items), 4), np.int32), np.zeros(d.ctas + 1, np.int32)
    _check(lib.vsa_packed_query(ctypes.byref(desc), sms, ctypes.byref(d), items.ctypes.data, first.ctypes.data),
           "vsa_packed_query")
    return dict(d.as_dict(), items=items[:d.items], first=first)


# Handles of packed plans that were collected.  The garbage collector may run while some stream is captured, and
# vsa_packed_destroy synchronises the device, which would end that capture: they wait here for a call that may.
_collected_plans = []


def _free_collected_plans():
    while True:
        try:
            handle = _collected_plans.pop()
        except IndexError:  # empty, here or by another thread
            return
        load_library().vsa_packed_destroy(handle)


class PackedPlan:
    """Owns a ``vsa_packed_plan_t`` handle: the lengths of packed sequences and the schedule made from them.  destroy()
    frees it at once, after the device's work (so not during a capture); a plan that is collected is freed by the next
    vsa_packed_plan or destroy()."""

    def __init__(self, handle, heads, kv_heads, head_dim, causal):
        self._h = handle
        self.heads, self.kv_heads, self.head_dim, self.causal = heads, kv_heads, head_dim, causal
        d = PackedDims()
        _check(load_library().vsa_packed_info(self._h, ctypes.byref(d)), "vsa_packed_info")
        self.dims = d.as_dict()

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("plan destroyed")
        return self._h

    def status(self, stream=None):
        """(code, site) of the plan's device status word, (0, 0) unless a device-side wait ran out."""
        code, where = ctypes.c_int32(), ctypes.c_int32()
        _check(load_library().vsa_packed_status(self.handle, _stream(stream), ctypes.byref(code), ctypes.byref(where)),
               "vsa_packed_status")
        return code.value, where.value

    def wait_selftest(self, timeout_ns=50_000_000, stream=None):
        """Run the packed attention's bounded-wait self-test; returns the (code, site) it recorded."""
        code, where = ctypes.c_int32(), ctypes.c_int32()
        _check(load_library().vsa_packed_wait_selftest(self.handle, int(timeout_ns), _stream(stream),
                                                       ctypes.byref(code), ctypes.byref(where)),
               "vsa_packed_wait_selftest")
        return code.value, where.value

    def destroy(self):
        _free_collected_plans()
        if self._h is not None:
            load_library().vsa_packed_destroy(self._h)
            self._h = None

    def __del__(self, collected=_collected_plans):  # (the module's names may be gone at the interpreter's end)
        if getattr(self, "_h", None) is not None:
            collected.append(self._h)


def vsa_packed_plan(lengths, heads, kv_heads=None, head_dim=128, causal=True, softmax_scale=0.0, stream=None) -> PackedPlan:
    """A plan for attention over sequences of these lengths packed end to end (0 allowed), for heads query heads
    and kv_heads key heads (heads / kv_heads query heads share one, in order)."""
    _free_collected_plans()
    desc, keep = make_packed_desc(lengths, heads, kv_heads, head_dim, causal, softmax_scale)
    h = ctypes.c_void_p()
    _check(load_library().vsa_packed_plan(ctypes.byref(desc), _stream(stream), ctypes.byref(h)), "vsa_packed_plan")
    return PackedPlan(h, desc.heads, desc.kv_heads, desc.head_dim, bool(causal))


def vsa_packed_attn(plan, q, k, v, out=None, stream=None):
    """softmax(scale q k^T) v of every packed sequence: q [T, H, D], k and v [T, Hk, D] bf16 (any token and head
    strides that are multiples of 8), T at least the lengths' sum; rows behind the last sequence are left as they
    are in `out` (zero in an output allocated here)."""
    index = _launch_index(("q", "k", "v", "out"), q, k, v, out)
    D, n = plan.head_dim, plan.dims["tokens"]
    T, H, q_ld, q_hd = _head_rows(q, D, "q")
    Tk, Hk, k_ld, k_hd = _head_rows(k, D, "k")
    Tv, Hv, v_ld, v_hd = _head_rows(v, D, "v")
    if H != plan.heads or Hk != plan.kv_heads or Hv != Hk:
        raise ValueError(f"the plan has {plan.heads} query and {plan.kv_heads} key heads, got {H}, {Hk} and {Hv}")
    if Tk != T or Tv != T:
        raise ValueError(f"q has {T} rows, k {Tk}, v {Tv}")
    if out is None:
        out = _empty(q.shape, _BF16, q.device, stream)
        if T > n:
            with _allocating_on(stream, q.device):
                out.view(T, H, D)[n:].zero_()
    elif out.shape != q.shape:
        raise ValueError(f"out must have q's shape {tuple(q.shape)}, got {tuple(out.shape)}")
    _, _, o_ld, o_hd = _head_rows(out, D, "out")
    a = PackedArgs(T, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), q_ld, q_hd, k_ld, k_hd, v_ld, v_hd,
                   o_ld, o_hd)
    rc = (_lib or load_library()).vsa_packed_attn(plan.handle, ctypes.byref(a), _stream_on(stream, index))
    if rc:
        _check(rc, "vsa_packed_attn")
    return out
