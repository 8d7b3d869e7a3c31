"""Thin ctypes binding of liblca_attn.so (include/lca_attn.h).

Argument marshalling only: it builds the C structs, allocates outputs and the
workspace with PyTorch when the caller does not pass them, and calls the
library on the current CUDA stream.  Every step of the attention path runs in
the library's kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass, field

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblca_attn.so")

MASK_KINDS = (
    "FULL", "CAUSAL", "SLIDING", "CAUSAL_SLIDING", "DOC", "CAUSAL_DOC", "SHARED_QUESTION", "GLOBAL_SLIDING",
    "CAUSAL_BLOCKWISE", "PREFIX_LM_CAUSAL", "PREFIX_LM_DOC", "BLOCK_CAUSAL_DOC", "BLOCK_SPARSE_UNIFORM",
    "BLOCK_SPARSE_VARIABLE", "FLASHMASK",
)
STATUS = {0: "LCA_OK", 1: "LCA_ERR_INVALID_ARG", 2: "LCA_ERR_UNSUPPORTED", 3: "LCA_ERR_WORKSPACE",
          4: "LCA_ERR_CUDA", 5: "LCA_ERR_TIMEOUT", 6: "LCA_ERR_DEVICE_ARG"}
EXPORTED = ("lca_workspace_size", "lca_attn_fwd", "lca_attn_bwd", "lca_mask_materialize", "lca_mask_tile_classes",
            "lca_mask_nnz", "lca_read_status", "lca_probe_wait_timeout", "lca_set_kernel_events", "lca_launch_count",
            "lca_last_error_detail", "lca_attn_fwd_static_workspace", "lca_status_string", "lca_version",
            "lca_attn_merge", "lca_cad_plan", "lca_attn_fwd_dropout", "lca_attn_bwd_dropout", "lca_set_cta_profile",
            "lca_paged_plan", "lca_paged_write", "lca_attn_paged", "lca_attn_paged_workspace_size")
PHASES = ("fwd_plan", "fwd", "d_prepass", "dkv_plan", "dkv", "dq_plan", "dq")


class LcaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)}")
        self.code = code


class Segment_t(C.Structure):
    _fields_ = [("q_off", C.c_int32), ("q_len", C.c_int32), ("k_off", C.c_int32), ("k_len", C.c_int32)]


class MaskDesc_t(C.Structure):
    _fields_ = [
        ("kind", C.c_int32),
        ("window_left", C.c_int32), ("window_right", C.c_int32),
        ("num_global", C.c_int32),
        ("prefix_len", C.c_int32),
        ("seg_prefix", C.POINTER(C.c_int32)),
        ("block", C.c_int32),
        ("part_bounds", C.POINTER(C.c_int32)),
        ("n_part_bounds", C.c_int32),
        ("q_block", C.c_int32), ("kv_block", C.c_int32),
        ("qb_bounds", C.POINTER(C.c_int32)), ("kb_bounds", C.POINTER(C.c_int32)),
        ("n_qb", C.c_int32), ("n_kb", C.c_int32),
        ("heads_in_map", C.c_int32),
        ("blk_row_ptr", C.c_void_p), ("blk_col_idx", C.c_void_p),
        ("blk_nnz", C.c_int64),
        ("col_bounds", C.c_void_p),
    ]


class Shape_t(C.Structure):
    _fields_ = [("Tq", C.c_int32), ("Tk", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32), ("d", C.c_int32),
                ("n_seg", C.c_int32), ("segs", C.POINTER(Segment_t)), ("scale", C.c_float)]


class Dropout_t(C.Structure):
    _fields_ = [("p", C.c_float), ("seed", C.c_uint64)]


class PagedCache_t(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("n_pages", C.c_int32), ("page_size", C.c_int32),
                ("Hkv", C.c_int32), ("d", C.c_int32), ("dtype", C.c_int32), ("page_stride", C.c_int64),
                ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


class PagedShape_t(C.Structure):
    _fields_ = [("Tq", C.c_int32), ("Hq", C.c_int32), ("n_seq", C.c_int32), ("max_pages", C.c_int32),
                ("table_stride", C.c_int64), ("q_stride", C.c_int64), ("max_q_len", C.c_int32), ("scale", C.c_float),
                ("ctx_len", C.c_void_p)]


_lib = None


def load(path: str = LIB_PATH):
    """Loads the library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with long_context_masked_attention_gb300._build.build()")
    lib = C.CDLL(path)
    st = C.c_int
    vp = C.c_void_p
    lib.lca_workspace_size.argtypes = [C.POINTER(Shape_t), C.POINTER(MaskDesc_t), C.c_int, C.POINTER(C.c_size_t)]
    lib.lca_attn_fwd.argtypes = [vp, vp, vp, vp, vp, C.POINTER(Shape_t), C.POINTER(MaskDesc_t), vp, C.c_size_t, vp]
    lib.lca_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, C.POINTER(Shape_t), C.POINTER(MaskDesc_t), vp,
                                 C.c_size_t, vp]
    lib.lca_attn_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, C.POINTER(Shape_t), C.POINTER(MaskDesc_t),
                                         C.POINTER(Dropout_t), vp, C.c_size_t, vp]
    lib.lca_attn_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, C.POINTER(Shape_t),
                                         C.POINTER(MaskDesc_t), C.POINTER(Dropout_t), vp, C.c_size_t, vp]
    lib.lca_mask_materialize.argtypes = [C.POINTER(Shape_t), C.POINTER(MaskDesc_t), C.c_int32, C.c_int32, vp, vp,
                                         C.c_size_t, vp]
    lib.lca_mask_tile_classes.argtypes = lib.lca_mask_materialize.argtypes
    lib.lca_mask_nnz.argtypes = [C.POINTER(Shape_t), C.POINTER(MaskDesc_t), vp, vp, C.c_size_t, vp]
    lib.lca_read_status.argtypes = [vp, C.POINTER(C.c_int32), vp]
    lib.lca_probe_wait_timeout.argtypes = [vp, C.c_size_t, C.c_int32, vp]
    lib.lca_set_kernel_events.argtypes = [C.POINTER(C.c_void_p), C.c_int32, C.POINTER(C.c_int32)]
    lib.lca_set_cta_profile.argtypes = [vp, C.c_size_t]
    i32, i64 = C.c_int32, C.c_int64
    lib.lca_paged_plan.argtypes = [vp, vp, i32, vp, i32, vp, vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    lib.lca_paged_write.argtypes = [vp, vp, i64, i64, vp, i32, C.POINTER(PagedCache_t), vp]
    lib.lca_attn_paged.argtypes = [vp, C.POINTER(PagedCache_t), vp, vp, vp, vp, vp, C.POINTER(PagedShape_t),
                                   C.POINTER(MaskDesc_t), vp, C.c_size_t, vp]
    lib.lca_attn_paged_workspace_size.argtypes = [C.POINTER(PagedShape_t), C.POINTER(PagedCache_t),
                                                  C.POINTER(MaskDesc_t), C.POINTER(C.c_size_t)]
    lib.lca_launch_count.restype = C.c_uint64
    lib.lca_launch_count.argtypes = []
    lib.lca_attn_fwd_static_workspace.argtypes = [vp, vp, vp, vp, vp, C.POINTER(Shape_t), C.POINTER(MaskDesc_t), vp]
    lib.lca_last_error_detail.restype = C.c_char_p
    lib.lca_last_error_detail.argtypes = []
    lib.lca_status_string.argtypes = [st]
    lib.lca_status_string.restype = C.c_char_p
    lib.lca_version.restype = C.c_int32
    for name in EXPORTED:
        if name not in ("lca_status_string", "lca_version", "lca_launch_count", "lca_last_error_detail"):
            getattr(lib, name).restype = st
    _lib = lib
    return lib


# ------------------------------------------------------------------ descriptors
@dataclass
class Mask:
    """Mask descriptor; attribute names match lca_mask_desc (any object with
    these attributes is accepted too)."""
    kind: str
    window_left: int = 0
    window_right: int = 0
    num_global: int = 0
    prefix_len: int = 0
    seg_prefix: list | None = None
    block: int = 0
    part_bounds: list | None = None
    q_block: int = 0
    kv_block: int = 0
    qb_bounds: np.ndarray | None = None
    kb_bounds: np.ndarray | None = None
    heads_in_map: int = 1
    blk_row_ptr: object = None
    blk_col_idx: object = None
    col_bounds: object = None  # FLASHMASK: int32 [Tk, 4] {lts, lte, uts, ute}


@dataclass
class Call:
    """Marshalled C arguments plus the Python objects they point into."""
    shape: Shape_t
    mask: MaskDesc_t
    keep: list = field(default_factory=list)


def _i32(seq):
    arr = np.ascontiguousarray(np.asarray(seq, dtype=np.int32))
    return arr, arr.ctypes.data_as(C.POINTER(C.c_int32))


def _int32(x, name):
    """x as a C int32 field takes it; ctypes would keep the low 32 bits."""
    x = int(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name}: {x} does not fit 32 bits")
    return x


def marshal(Tq, Tk, Hq, Hkv, d, segments, mask, scale=0.0, device=None) -> Call:
    """segments: iterable of objects with q_off/q_len/k_off/k_len or 4-tuples."""
    import torch

    segs = list(segments)
    seg_arr = (Segment_t * max(1, len(segs)))()
    for i, s in enumerate(segs):
        if isinstance(s, (tuple, list)):
            seg_arr[i] = Segment_t(*[_int32(x, f"segment {i}") for x in s])
        else:
            seg_arr[i] = Segment_t(*[_int32(x, f"segment {i}") for x in (s.q_off, s.q_len, s.k_off, s.k_len)])
    dims = [_int32(x, name) for x, name in ((Tq, "Tq"), (Tk, "Tk"), (Hq, "Hq"), (Hkv, "Hkv"), (d, "d"))]
    shape = Shape_t(*dims, len(segs), seg_arr, float(scale))
    md = MaskDesc_t()
    keep = [seg_arr]
    kind = mask.kind if isinstance(mask.kind, int) else MASK_KINDS.index(mask.kind)
    md.kind = _int32(kind, "kind")
    for name in ("window_left", "window_right", "num_global", "prefix_len", "block", "q_block", "kv_block"):
        setattr(md, name, _int32(getattr(mask, name, 0) or 0, name))
    if getattr(mask, "seg_prefix", None) is not None:
        arr, ptr = _i32(mask.seg_prefix)
        keep.append(arr)
        md.seg_prefix = ptr
    if getattr(mask, "part_bounds", None) is not None:
        arr, ptr = _i32(mask.part_bounds)
        keep.append(arr)
        md.part_bounds = ptr
        md.n_part_bounds = len(arr)
    md.heads_in_map = _int32(getattr(mask, "heads_in_map", 1) or 1, "heads_in_map")
    for name, cnt in (("qb_bounds", "n_qb"), ("kb_bounds", "n_kb")):
        b = getattr(mask, name, None)
        if b is not None:
            arr, ptr = _i32(b)
            keep.append(arr)
            setattr(md, name, ptr)
            setattr(md, cnt, len(arr) - 1)
    rp = getattr(mask, "blk_row_ptr", None)
    ci = getattr(mask, "blk_col_idx", None)
    if rp is not None:
        dev = device if device is not None else torch.device("cuda")

        def to_dev(x):
            if isinstance(x, torch.Tensor):
                return x.to(device=dev, dtype=torch.int32).contiguous()
            return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).to(dev)

        trp, tci = to_dev(rp), to_dev(ci)
        keep += [trp, tci]
        md.blk_row_ptr = trp.data_ptr()
        md.blk_col_idx = tci.data_ptr() if tci.numel() else None
        md.blk_nnz = int(tci.numel())
    cb = getattr(mask, "col_bounds", None)
    if cb is not None:
        dev = device if device is not None else torch.device("cuda")
        tcb = (cb.to(device=dev, dtype=torch.int32) if isinstance(cb, torch.Tensor)
               else torch.from_numpy(np.ascontiguousarray(np.asarray(cb, dtype=np.int32))).to(dev)).contiguous()
        keep.append(tcb)
        md.col_bounds = tcb.data_ptr()
    return Call(shape, md, keep)


def _check(code, what):
    if code != 0:
        if code == 4:
            what += " (" + load().lca_last_error_detail().decode() + ")"
        raise LcaError(code, what)


def _stream(stream, device=None):
    """The stream handle for a call: the given one, else the current stream
    of `device` (the device the call's tensors live on)."""
    import torch

    if stream is None:
        stream = torch.cuda.current_stream(device)
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _on_device(device):
    """Context that makes `device` the current CUDA device for a library call:
    the library launches on the current device and refuses pointers into
    another device's memory, so every call runs with its tensors' device
    current, whichever device the caller had selected."""
    import contextlib

    import torch

    if device is None or torch.device(device).type != "cuda":
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def workspace_size(call: Call, for_bwd: bool) -> int:
    n = C.c_size_t(0)
    _check(load().lca_workspace_size(C.byref(call.shape), C.byref(call.mask), int(for_bwd), C.byref(n)),
           "lca_workspace_size")
    return n.value


def _workspace(call, for_bwd, workspace, device):
    import torch

    need = workspace_size(call, for_bwd)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    return workspace


# ------------------------------------------------------------------ entry points
def _require(t, name, shape, dtype, device=None, host_ok=False):
    """The library reads and writes raw device pointers, so every tensor is
    checked here: a CUDA tensor of the given dtype, shape and device, laid out
    densely (a host or strided tensor would be read as garbage).  With
    host_ok (outputs the kernels only store to), a pinned host tensor is
    accepted too: the kernels write it through its device mapping."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if host_ok and t.device.type == "cpu":
        if not t.is_pinned():
            raise ValueError(f"{name}: must be a CUDA tensor or a pinned host tensor (got unpinned {t.device})")
    elif t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor (got {t.device})")
    elif device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t


def _dropout(dropout):
    """(seed, p) -> lca_dropout, or None."""
    if dropout is None:
        return None
    seed, p = dropout
    return Dropout_t(float(p), int(seed) & 0xFFFFFFFFFFFFFFFF)


def attn_fwd(q, k, v, segments, mask, scale=0.0, out=None, lse=None, workspace=None, stream=None, call=None,
             dropout=None):
    """q [Tq,Hq,128], k/v [Tk,Hkv,128] bf16 CUDA tensors -> (o, lse[Hq,Tq]).
    out / lse may be given as CUDA or pinned host tensors.
    dropout: (seed, p) for attention dropout with drop probability p."""
    import torch

    Tq, Hq, d = q.shape
    Tk, Hkv, _ = k.shape
    bf = torch.bfloat16
    _require(q, "q", (Tq, Hq, d), bf)
    _require(k, "k", (Tk, Hkv, d), bf, q.device)
    _require(v, "v", (Tk, Hkv, d), bf, q.device)
    call = call or marshal(Tq, Tk, Hq, Hkv, d, segments, mask, scale, q.device)
    out = torch.empty_like(q) if out is None else _require(out, "out", (Tq, Hq, d), bf, q.device, host_ok=True)
    lse = (torch.empty((Hq, Tq), dtype=torch.float32, device=q.device) if lse is None
           else _require(lse, "lse", (Hq, Tq), torch.float32, q.device, host_ok=True))
    workspace = _workspace(call, False, workspace, q.device)
    drop = _dropout(dropout)
    with _on_device(q.device):
        if drop is None:
            _check(load().lca_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                       C.byref(call.shape), C.byref(call.mask), workspace.data_ptr(),
                                       workspace.numel(), _stream(stream, q.device)), "lca_attn_fwd")
        else:
            _check(load().lca_attn_fwd_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                               lse.data_ptr(), C.byref(call.shape), C.byref(call.mask),
                                               C.byref(drop), workspace.data_ptr(), workspace.numel(),
                                               _stream(stream, q.device)), "lca_attn_fwd_dropout")
    return out, lse


class CadShard_t(C.Structure):
    _fields_ = [("doc", C.c_int32), ("start", C.c_int32), ("len", C.c_int32), ("server", C.c_int32)]


@dataclass
class CadPlan:
    """Shards (doc, start, len, server) ordered by server then document, and
    each server's causal attention cells per head."""
    shards: list
    server_cells: list

    def server_batch(self, server: int, doc_lengths):
        """The server's packed query batch: CAUSAL segments (q_off, q_len,
        k_off, k_len) over keys packed in document order, and for each packed
        query row its row in the document-ordered token buffer."""
        starts = np.concatenate([[0], np.cumsum(np.asarray(doc_lengths, dtype=np.int64))])
        segs, rows, q = [], [], 0
        for doc, start, n, srv in self.shards:
            if srv != server:
                continue
            segs.append((q, n, int(starts[doc]), start + n))
            rows.append(np.arange(starts[doc] + start, starts[doc] + start + n))
            q += n
        return segs, (np.concatenate(rows) if rows else np.zeros(0, dtype=np.int64))


def cad_plan(doc_lengths, n_servers, min_shard=1024, max_shard=32768, tolerance=0.05) -> CadPlan:
    """Core-attention disaggregation plan (host only, lca_cad_plan)."""
    arr, ptr = _i32(doc_lengths)
    n = C.c_int32(0)
    cells = (C.c_int64 * max(1, int(n_servers)))()
    cap = max(16, 4 * len(arr) + 4 * int(n_servers))
    while True:
        buf = (CadShard_t * cap)()
        code = load().lca_cad_plan(ptr, len(arr), int(n_servers), int(min_shard), int(max_shard),
                                   C.c_double(float(tolerance)), buf, cap, C.byref(n), cells)
        if code == 3 and n.value > cap:  # LCA_ERR_WORKSPACE: more shards than room
            cap = n.value
            continue
        _check(code, "lca_cad_plan")
        break
    shards = [(buf[i].doc, buf[i].start, buf[i].len, buf[i].server) for i in range(n.value)]
    return CadPlan(shards, [int(cells[i]) for i in range(int(n_servers))])


def attn_merge(o_parts, lse_parts, out=None, lse=None, stream=None):
    """Merges forward results of the same queries over disjoint key sets:
    o_parts [Tq,Hq,128] bf16 and lse_parts [Hq,Tq] f32 CUDA tensors ->
    (o, lse).  `out`/`lse` may be part 0's tensors."""
    import torch

    n = len(o_parts)
    if n != len(lse_parts):
        raise ValueError("o_parts and lse_parts differ in length")
    Tq, Hq, d = o_parts[0].shape
    dev = o_parts[0].device
    for p, (o_p, l_p) in enumerate(zip(o_parts, lse_parts)):
        _require(o_p, f"o_parts[{p}]", (Tq, Hq, d), torch.bfloat16, dev if p else None)
        _require(l_p, f"lse_parts[{p}]", (Hq, Tq), torch.float32, dev)
    out = torch.empty_like(o_parts[0]) if out is None else _require(out, "out", (Tq, Hq, d), torch.bfloat16, dev)
    lse = torch.empty_like(lse_parts[0]) if lse is None else _require(lse, "lse", (Hq, Tq), torch.float32, dev)
    optrs = (C.c_void_p * n)(*[t.data_ptr() for t in o_parts])
    lptrs = (C.c_void_p * n)(*[t.data_ptr() for t in lse_parts])
    with _on_device(dev):
        _check(load().lca_attn_merge(optrs, lptrs, n, C.c_void_p(out.data_ptr()), C.c_void_p(lse.data_ptr()), Tq, Hq,
                                     d, _stream(stream, dev)), "lca_attn_merge")
    return out, lse


def attn_bwd(do, q, k, v, o, lse, segments, mask, scale=0.0, dq=None, dk=None, dv=None, workspace=None, stream=None,
             call=None, dropout=None):
    """Returns (dq, dk, dv) bf16; given dq / dk / dv may be CUDA or pinned host
    tensors.  dropout: the (seed, p) the forward used."""
    import torch

    Tq, Hq, d = q.shape
    Tk, Hkv, _ = k.shape
    bf = torch.bfloat16
    _require(q, "q", (Tq, Hq, d), bf)
    for name, t in (("do", do), ("o", o)):
        _require(t, name, (Tq, Hq, d), bf, q.device)
    _require(k, "k", (Tk, Hkv, d), bf, q.device)
    _require(v, "v", (Tk, Hkv, d), bf, q.device)
    _require(lse, "lse", (Hq, Tq), torch.float32, q.device)
    call = call or marshal(Tq, Tk, Hq, Hkv, d, segments, mask, scale, q.device)
    dq = torch.empty_like(q) if dq is None else _require(dq, "dq", (Tq, Hq, d), bf, q.device, host_ok=True)
    dk = torch.empty_like(k) if dk is None else _require(dk, "dk", (Tk, Hkv, d), bf, q.device, host_ok=True)
    dv = torch.empty_like(v) if dv is None else _require(dv, "dv", (Tk, Hkv, d), bf, q.device, host_ok=True)
    workspace = _workspace(call, True, workspace, q.device)
    drop = _dropout(dropout)
    args = (do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), C.byref(call.shape), C.byref(call.mask))
    with _on_device(q.device):
        tail = (workspace.data_ptr(), workspace.numel(), _stream(stream, q.device))
        if drop is None:
            _check(load().lca_attn_bwd(*args, *tail), "lca_attn_bwd")
        else:
            _check(load().lca_attn_bwd_dropout(*args, C.byref(drop), *tail), "lca_attn_bwd_dropout")
    return dq, dk, dv


# ------------------------------------------------------------------ paged cache
@dataclass
class PagedPlan:
    """A batch's rows: first row of each request, its keys, and for each row
    its slot in the cache and its position (see lca_paged_plan)."""
    q_start: object
    k_len: object
    slots: object
    positions: object
    state: object


def _side_stream(stream, device):
    """The torch stream of a call given another stream than the current one,
    else None."""
    import torch

    if stream is None:
        return None
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(
        int(getattr(stream, "cuda_stream", stream)), device)
    return None if s == torch.cuda.current_stream(device) else s


def _empty(shape, dtype, device, side):
    """A tensor that belongs to the call's stream, so that its memory is not
    handed on while that stream uses it."""
    import torch

    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(side):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _call(fn, name, device, side, *args):
    """fn(*args, stream) on the tensors' device: the current stream of that
    device, or the side stream.  What these calls cost is mostly this side of
    them, so the common case, that device being current, takes no context."""
    from torch import _C

    index = device.index
    raw = _C._cuda_getCurrentRawStream(index) if side is None else side.cuda_stream
    if _C._cuda_getDevice() == index:
        code = fn(*args, raw)
    else:
        import torch

        with torch.cuda.device(device):
            code = fn(*args, raw)
    if code:
        _check(code, name)


def _refuse(t, name, dtype, shape, device):
    """Why tensor t is not what an entry point reads."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name}: shape {tuple(t.shape)}, strides {t.stride()}, expected a contiguous {tuple(shape)}")


def _ptr(t, name, dtype, shape, device):
    """Address of a dense CUDA tensor of this dtype, shape and device."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, device)


def _paged_cache(k, v):
    """lca_paged_cache of two [n_pages, page_size, Hkv, d] tensors."""
    import torch

    for name, t in (("k_cache", k), ("v_cache", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if not t.is_cuda:
            raise ValueError(f"{name}: must be a CUDA tensor (got {t.device})")
    shape, dt = k.shape, k.dtype
    if len(shape) != 4:
        raise ValueError(f"k_cache: shape {tuple(shape)}, expected [n_pages, page_size, Hkv, d]")
    if v.shape != shape or v.dtype is not dt or v.device != k.device:
        raise ValueError(f"v_cache: {tuple(v.shape)} {v.dtype} on {v.device}, expected {tuple(shape)} {dt} on {k.device} "
                         "as k_cache")
    if dt is torch.bfloat16:
        code = 0
    elif dt is torch.float16:
        code = 1
    else:
        raise ValueError(f"k_cache: dtype {dt}, expected torch.bfloat16 or torch.float16")
    n, page, Hkv, d = shape
    ks, vs = k.stride(), v.stride()
    if n <= 1 or page == 1 or Hkv == 1 or d == 1:
        # the stride of an axis of length one (or of an empty cache) moves nothing
        def moves(st):
            return (st[0] if n > 1 else d, st[1] if n and page > 1 else d, st[2] if n and Hkv > 1 else d,
                    st[3] if n and d > 1 else 1)

        ks, vs = moves(ks), moves(vs)
    if ks != vs:
        raise ValueError(f"v_cache: strides {vs}, expected {ks} as k_cache")
    if ks[3] != 1:
        raise ValueError("k_cache, v_cache: the last dimension must be contiguous")
    return PagedCache_t(k.data_ptr(), v.data_ptr(), n, page, Hkv, d, code, ks[0], ks[1], ks[2])


def _rows(t, name, heads, d, dtype, device):
    """[T, heads, d] CUDA tensor whose rows are dense; returns its row stride."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != d or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [T, {'H' if heads is None else heads}, {d}]")
    T, H, _ = shape
    a, b, c = t.stride()
    if T and ((c != 1 and d > 1) or (H > 1 and b != d)):
        raise ValueError(f"{name}: each row's heads must be contiguous")
    return a if T > 1 else H * d


def _table(t, n_seq, device):
    """Block table [n_seq, max_pages] with dense rows -> (pointer, entries per row, row stride)."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"block_table: expected a torch.Tensor, got {type(t).__name__}")
    if t.device != device:
        raise ValueError(f"block_table: on {t.device}, expected {device}")
    if t.dtype is not torch.int32:
        raise ValueError(f"block_table: dtype {t.dtype}, expected torch.int32")
    shape = t.shape
    if len(shape) != 2 or (n_seq is not None and shape[0] != n_seq):
        raise ValueError(f"block_table: shape {tuple(shape)}, expected [{'n_seq' if n_seq is None else n_seq}, max_pages]")
    n_seq, width = shape
    a, b = t.stride()
    if (n_seq and b != 1 and width > 1) or (n_seq > 1 and a < width):
        raise ValueError("block_table: each row must be contiguous, and rows must not overlap")
    return t.data_ptr(), _int32(width, "block_table: entries per row"), a if n_seq > 1 else width


def paged_plan(ctx_len, new_len, free_pages, taken, block_table, page_size, n_pages, n_rows, q_start=None, k_len=None,
               slots=None, positions=None, state=None, stream=None) -> PagedPlan:
    """The bookkeeping of a batch over a paged cache, on the GPU: gives the new
    tokens' pages from free_pages[taken:] to the requests' rows of block_table
    (in place) and returns where every row goes.  ctx_len, new_len [n_seq],
    free_pages [n], taken [1]: int32 CUDA tensors; block_table [n_seq,
    max_pages] int32; n_rows: rows of the packed batch, those behind the last
    request get slot -1.  state holds {free pages used so far, pages missing,
    requests with unusable lengths, new tokens}; state[:1] is the next call's
    `taken`."""
    import torch

    for name, t in (("ctx_len", ctx_len), ("free_pages", free_pages)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    n_seq, n_free = _int32(ctx_len.numel(), "ctx_len: entries"), _int32(free_pages.numel(), "free_pages: entries")
    dev, i32, n_rows = ctx_len.device, torch.int32, int(n_rows)
    if not 0 <= n_rows < 1 << 31:  # a C int32 would keep the low bits
        raise ValueError(f"n_rows: {n_rows}, expected 0 to 2^31 - 1")
    if not 0 < page_size < 1 << 31:
        raise ValueError(f"page_size: {page_size}, expected 1 to 2^31 - 1")
    if not 0 <= n_pages < 1 << 31:
        raise ValueError(f"n_pages: {n_pages}, expected 0 to 2^31 - 1")
    ins = (_ptr(ctx_len, "ctx_len", i32, (n_seq,), dev), _ptr(new_len, "new_len", i32, (n_seq,), dev), n_seq,
           _ptr(free_pages, "free_pages", i32, (n_free,), dev), n_free, _ptr(taken, "taken", i32, (1,), dev))
    tp, width, tstride = _table(block_table, n_seq, dev)
    side = _side_stream(stream, dev)
    # an allocation each: parts of one would cost more than they save
    outs, ptrs = [], []
    for t, name, n in ((q_start, "q_start", n_seq + 1), (k_len, "k_len", n_seq), (slots, "slots", n_rows),
                       (positions, "positions", n_rows), (state, "state", 4)):
        if t is None:
            t = _empty(n, i32, dev, side)
            ptrs.append(t.data_ptr())
        else:
            ptrs.append(_ptr(t, name, i32, (n,), dev))
        outs.append(t)
    if side is not None:
        for t in (ctx_len, new_len, free_pages, taken, block_table, *outs):
            t.record_stream(side)
    _call(load().lca_paged_plan, "lca_paged_plan", dev, side, *ins, tp, tstride, width, int(page_size), int(n_pages),
          n_rows, *ptrs)
    return PagedPlan(*outs)


def paged_write(k, v, k_cache, v_cache, slots, stream=None):
    """Stores rows k, v [T, Hkv, 128] (row stride free) at slots [T] int32 of
    the cache [n_pages, page_size, Hkv, 128] (strides free, bf16 or fp16), in
    place; rows whose slot is outside the cache (-1) are skipped."""
    import torch

    cache = _paged_cache(k_cache, v_cache)
    dev, dt = k_cache.device, k_cache.dtype
    ks = _rows(k, "k", cache.Hkv, cache.d, dt, dev)
    vs = _rows(v, "v", cache.Hkv, cache.d, dt, dev)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError(f"v: {v.shape[0]} rows, expected {T} as k")
    sp = _ptr(slots, "slots", torch.int32, (T,), dev)
    side = _side_stream(stream, dev)
    if side is not None:
        for t in (k, v, k_cache, v_cache, slots):
            t.record_stream(side)
    _call(load().lca_paged_write, "lca_paged_write", dev, side, k.data_ptr(), v.data_ptr(), ks, vs, sp, T,
          C.byref(cache))


def _paged_mask(mask):
    kind = mask.kind
    if not isinstance(kind, int):
        kind = MASK_KINDS.index(kind)
    md = MaskDesc_t(_int32(kind, "kind"))
    if kind not in _PLAIN_KINDS:
        for name in ("window_left", "window_right", "num_global", "prefix_len", "block"):
            setattr(md, name, _int32(getattr(mask, name, 0) or 0, name))
    return md


_SIZES: dict = {}  # workspace bytes of attn_paged by shape
_PLAIN_KINDS = tuple(MASK_KINDS.index(k) for k in ("FULL", "CAUSAL", "DOC", "CAUSAL_DOC"))  # no parameters


def _paged_shape(q, cache, k_cache, block_table, scale, max_q_len):
    dev = k_cache.device
    qs = _rows(q, "q", None, cache.d, k_cache.dtype, dev)
    tp, width, tstride = _table(block_table, None, dev)
    shape = q.shape
    return PagedShape_t(shape[0], shape[1], block_table.shape[0], width, tstride, qs, _int32(max_q_len, "max_q_len"),
                        scale), tp


def _paged_size(shape, cache, md):
    n = C.c_size_t(0)
    _check(load().lca_attn_paged_workspace_size(C.byref(shape), C.byref(cache), C.byref(md), C.byref(n)),
           "lca_attn_paged_workspace_size")
    return n.value


def attn_paged_workspace_size(q, k_cache, v_cache, block_table, mask, scale=0.0, max_q_len=0) -> int:
    """Bytes of workspace that attn_paged needs for these tensors."""
    cache = _paged_cache(k_cache, v_cache)
    return _paged_size(_paged_shape(q, cache, k_cache, block_table, scale, max_q_len)[0], cache, _paged_mask(mask))


def attn_paged(q, k_cache, v_cache, block_table, q_start, k_len, mask, scale=0.0, max_q_len=0, out=None, lse=None,
               workspace=None, stream=None, ctx_len=None):
    """Attention of packed new tokens q [T, Hq, 128] (row stride free) over a
    paged cache [n_pages, page_size, Hkv, 128] (strides free), bf16 or fp16 ->
    (o [T, Hq, 128], lse [Hq, T]).  Request i owns rows q_start[i] to
    q_start[i + 1] and the first k_len[i] tokens of the pages in
    block_table[i]; its new tokens are the last of them.  q_start, k_len and
    block_table are int32 CUDA tensors read when the kernels run.  mask: any
    interval family (see lca_attn_paged).  max_q_len: no request has more new
    tokens (0: unknown, which costs a decode step workspace and launches).  A
    cache whose pages are not its outermost axis is slow with prompts.  ctx_len [n_seq]: the cached tokens that paged_plan was
    given; with it the new tokens are those that follow them, also in a request
    that the plan had no room for all of (plan.state[2] counts those).  After
    a synchronize, read_status(workspace) tells whether a table entry or a
    length was out of range."""
    import torch

    cache = _paged_cache(k_cache, v_cache)
    dev, dt = k_cache.device, q.dtype
    shape, tp = _paged_shape(q, cache, k_cache, block_table, scale, max_q_len)
    md = _paged_mask(mask)
    n_seq = shape.n_seq
    qsp = _ptr(q_start, "q_start", torch.int32, (n_seq + 1,), dev)
    klp = _ptr(k_len, "k_len", torch.int32, (n_seq,), dev)
    if ctx_len is not None and n_seq:
        shape.ctx_len = _ptr(ctx_len, "ctx_len", torch.int32, (n_seq,), dev)
    side = _side_stream(stream, dev)
    size, lsize = q.shape, (shape.Hq, shape.Tq)
    if out is None:
        out = _empty(size, dt, dev, side)
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", dt, size, dev)
    if lse is None:
        lse = _empty(lsize, torch.float32, dev, side)
        lp = lse.data_ptr()
    else:
        lp = _ptr(lse, "lse", torch.float32, lsize, dev)
    if workspace is None:
        # the size depends on these alone
        key = (shape.Tq, shape.Hq, n_seq, shape.max_q_len, cache.Hkv, min(cache.n_pages, 2), cache.page_stride,
               cache.token_stride, cache.head_stride)
        need = _SIZES.get(key)
        if need is None:
            if len(_SIZES) >= 4096:
                _SIZES.clear()
            need = _SIZES[key] = _paged_size(shape, cache, md)
        workspace = _empty((need,), torch.uint8, dev, side)
    else:
        _ptr(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
    if side is not None:
        for t in (q, k_cache, v_cache, block_table, q_start, k_len, out, lse, workspace):
            t.record_stream(side)
        if ctx_len is not None:
            ctx_len.record_stream(side)
    _call(load().lca_attn_paged, "lca_attn_paged", dev, side, q.data_ptr(), C.byref(cache), tp, qsp, klp, op, lp,
          C.byref(shape), C.byref(md), workspace.data_ptr(), workspace.numel())
    return out, lse


def mask_materialize(call: Call, head: int, seg: int, q_len: int, k_len: int, device="cuda", stream=None):
    import torch

    out = torch.empty((q_len, k_len), dtype=torch.uint8, device=device)
    ws = _workspace(call, False, None, device)
    with _on_device(out.device):
        _check(load().lca_mask_materialize(C.byref(call.shape), C.byref(call.mask), head, seg, out.data_ptr(),
                                           ws.data_ptr(), ws.numel(), _stream(stream, out.device)),
               "lca_mask_materialize")
    return out


def mask_tile_classes(call: Call, head: int, seg: int, q_len: int, k_len: int, device="cuda", stream=None):
    import torch

    nq, nk = -(-q_len // 128), -(-k_len // 128)
    out = torch.empty((max(nq, 0), max(nk, 0)), dtype=torch.uint8, device=device)
    ws = _workspace(call, False, None, device)
    with _on_device(out.device):
        _check(load().lca_mask_tile_classes(C.byref(call.shape), C.byref(call.mask), head, seg, out.data_ptr(),
                                            ws.data_ptr(), ws.numel(), _stream(stream, out.device)),
               "lca_mask_tile_classes")
    return out


def mask_nnz(call: Call, device="cuda", stream=None):
    import torch

    out = torch.zeros(call.shape.Hq, dtype=torch.int64, device=device)
    ws = _workspace(call, False, None, device)
    with _on_device(out.device):
        _check(load().lca_mask_nnz(C.byref(call.shape), C.byref(call.mask), out.data_ptr(), ws.data_ptr(),
                                   ws.numel(), _stream(stream, out.device)), "lca_mask_nnz")
    return out


def read_status(workspace, stream=None):
    buf = (C.c_int32 * 2)()
    with _on_device(workspace.device):
        _check(load().lca_read_status(workspace.data_ptr(), buf, _stream(stream, workspace.device)),
               "lca_read_status")
    return int(buf[0]), int(buf[1])


def probe_wait_timeout(workspace, limit_ms: int, stream=None):
    with _on_device(workspace.device):
        _check(load().lca_probe_wait_timeout(workspace.data_ptr(), workspace.numel(), int(limit_ms),
                                             _stream(stream, workspace.device)), "lca_probe_wait_timeout")


class KernelEvents:
    """Ring of CUDA event pairs the library records around each phase of its
    fwd/bwd calls (lca_set_kernel_events)."""

    def __init__(self, n_pairs: int):
        import torch

        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * n_pairs)]
        for e in self.events:  # torch creates the CUDA event lazily, on first record
            e.record()
        torch.cuda.synchronize()
        self._arr = (C.c_void_p * (2 * n_pairs))(*[e.cuda_event for e in self.events])
        self._ph = (C.c_int32 * n_pairs)(*([-1] * n_pairs))
        self.n_pairs = n_pairs

    def start(self):
        for i in range(self.n_pairs):
            self._ph[i] = -1
        _check(load().lca_set_kernel_events(self._arr, 2 * self.n_pairs, self._ph), "lca_set_kernel_events")

    def stop(self):
        _check(load().lca_set_kernel_events(None, 0, None), "lca_set_kernel_events")

    def durations(self):
        """{phase name: [ms, ...]} for every recorded pair (call after a sync)."""
        out = {}
        for i in range(self.n_pairs):
            ph = self._ph[i]
            if ph < 0:
                continue
            out.setdefault(PHASES[ph], []).append(self.events[2 * i].elapsed_time(self.events[2 * i + 1]))
        return out


def launch_count() -> int:
    return int(load().lca_launch_count())


CTA_PROFILE_BYTES = 3 * 1024 * 64
PROFILE_KERNELS = ("fwd", "dkv", "dq")


class CtaProfile:
    """Per-CTA records of the attention kernels (lca_set_cta_profile): after a
    call, records() gives for each kernel the rows (start_ns, end_ns, items,
    full, partial, grid, sm) of the CTAs it launched."""

    def __init__(self, device="cuda"):
        import torch

        self.buf = torch.zeros(CTA_PROFILE_BYTES // 8, dtype=torch.int64, device=device)

    def start(self):
        with _on_device(self.buf.device):
            _check(load().lca_set_cta_profile(self.buf.data_ptr(), CTA_PROFILE_BYTES), "lca_set_cta_profile")

    def stop(self):
        _check(load().lca_set_cta_profile(None, 0), "lca_set_cta_profile")

    def records(self):
        """{kernel: int64 array [grid, 7]} for every kernel slot the last call
        filled (call after a synchronize)."""
        r = self.buf.view(3, 1024, 8).cpu().numpy()
        out = {}
        for k, name in enumerate(PROFILE_KERNELS):
            grid = int(r[k, 0, 5])
            if grid > 0:
                out[name] = r[k, :grid, :7].copy()
        return out

