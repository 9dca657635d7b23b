"""ctypes binding of libsketchssm.so: the C entry points under the same names.

Argument marshalling only: tensors become device pointers, the stream defaults
to torch's current stream, and a non-OK status raises ``SketchSSMError``.  Every
step of the decode path runs in the HIP library; if the library is not built
this module raises instead of falling back to anything.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsketchssm.so")

KIND = {"mamba2": 0, "gdn": 1, "kda": 2}
DTYPE = {"bf16": 0, "f32": 1}
CACHE = {"i8": 0, "e4m3": 1}
GATE = {"none": 0, "silu_first": 1, "silu": 2, "sigmoid": 3}
STATUS = {0: "SKSSM_OK", 1: "SKSSM_EINVAL", 2: "SKSSM_ESHAPE", 3: "SKSSM_EALIGN",
          4: "SKSSM_ENOMEM", 5: "SKSSM_EDEVICE", 6: "SKSSM_ELAUNCH"}

c_i32 = ctypes.c_int32
c_vp = ctypes.c_void_p
c_i32p = ctypes.POINTER(ctypes.c_int32)


class SketchSSMError(RuntimeError):
    def __init__(self, where: str, status: int):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


class Shape(ctypes.Structure):
    _fields_ = [("B", c_i32), ("H", c_i32), ("K", c_i32), ("V", c_i32), ("W", c_i32),
                ("G", c_i32), ("basis_rows", c_i32), ("rank_cap", c_i32), ("kind", c_i32),
                ("qkv", c_i32), ("kq_heads", c_i32)]


_lib = None

_PROTOS = {
    "sketchssm_plan_create": (c_i32, [ctypes.POINTER(Shape), c_i32p, c_i32p, ctypes.POINTER(c_vp)]),
    "sketchssm_plan_create_ordered": (c_i32, [ctypes.POINTER(Shape), c_i32p, c_i32p, c_i32p,
                                              ctypes.POINTER(c_vp)]),
    "sketchssm_plan_export": (c_i32, [c_vp] + [c_i32p] * 8),
    "sketchssm_plan_destroy": (None, [c_vp]),
    "sketchssm_z_elems": (ctypes.c_size_t, [c_vp]),
    "sketchssm_frame_elems": (ctypes.c_size_t, [c_vp]),
    "sketchssm_flush": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_vp]),
    "sketchssm_decode_read": (c_i32, [c_vp] * 13 + [c_i32, c_vp, c_vp]),
    "sketchssm_dense_read": (c_i32, [ctypes.POINTER(Shape)] + [c_vp] * 10 + [c_i32, c_vp, c_vp]),
    "sketchssm_rmw_step": (c_i32, [ctypes.POINTER(Shape)] + [c_vp] * 8),
    "sketchssm_decode_read_seq": (c_i32, [c_vp] * 16),
    "sketchssm_flush_seq": (c_i32, [c_vp] * 10 + [c_i32, c_vp]),
    "sketchssm_decode_read_flush": (c_i32, [c_vp] * 16),
    "sketchssm_rmw_seq": (c_i32, [ctypes.POINTER(Shape), c_vp, c_i32] + [c_vp] * 4 + [c_i32] * 3 + [c_vp] * 7),
    "sketchssm_prefill": (c_i32, [ctypes.POINTER(Shape), c_vp, c_i32] + [c_vp] * 4 + [c_i32] * 3 + [c_vp] * 7
                          + [ctypes.c_size_t, c_vp]),
    "sketchssm_prefill_workspace": (ctypes.c_size_t, [ctypes.POINTER(Shape)] + [c_i32] * 3),
    "sketchssm_gated_norm": (c_i32, [ctypes.POINTER(Shape)] + [c_vp] * 5 + [c_i32] * 3 + [ctypes.c_float, c_i32]
                             + [c_vp] * 2),
    "sketchssm_tree_read": (c_i32, [c_vp] * 11 + [c_i32] * 3 + [c_vp] * 8),
    "sketchssm_tree_accept": (c_i32, [ctypes.POINTER(Shape)] + [c_vp] * 8 + [c_i32] * 2 + [c_vp] * 7),
    "sketchssm_cache_store": (c_i32, [ctypes.POINTER(Shape)] + [c_vp] * 5 + [c_i32] * 3 + [c_vp]),
    "sketchssm_cache_load": (c_i32, [ctypes.POINTER(Shape)] + [c_vp] * 3 + [c_i32] + [c_vp] * 2 + [c_i32] * 2 + [c_vp]),
    "sketchssm_status_string": (ctypes.c_char_p, [c_i32]),
    "sketchssm_stream_probe": (c_i32, [c_vp, ctypes.c_size_t, c_vp, ctypes.c_size_t, c_i32, c_i32, c_i32, c_vp]),
}


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m rank_state_read_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _PROTOS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().sketchssm_status_string(int(status)).decode()


def _check(where: str, st: int):
    if st != 0:
        raise SketchSSMError(where, st)


def make_shape(B, H, K, V, W, G, basis_rows, rank_cap, kind, qkv, kq_heads=0) -> Shape:
    return Shape(int(B), int(H), int(K), int(V), int(W), int(G), int(basis_rows), int(rank_cap),
                 KIND[kind] if isinstance(kind, str) else int(kind),
                 DTYPE[qkv] if isinstance(qkv, str) else int(qkv), int(kq_heads or 0))


def _ptr(x) -> Optional[int]:
    """Device address of a tensor (None -> NULL).  Integers pass through."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("expected a device tensor")
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        # the handle alone: a Stream object around it costs 2.5 us of a call's 14
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Plan:
    """Owner of a ``sketchssm_plan`` (host only)."""

    def __init__(self, shape: Shape, rank, group, order=None):
        self.shape = shape
        r = np.ascontiguousarray(rank, dtype=np.int32)
        g = np.ascontiguousarray(group, dtype=np.int32)
        if shape.H >= 1 and (r.shape != (shape.H,) or g.shape != (shape.H,)):
            raise ValueError("rank and group must have H entries")
        h = c_vp()
        if order is None:
            _check("sketchssm_plan_create",
                   lib().sketchssm_plan_create(ctypes.byref(shape), r.ctypes.data_as(c_i32p),
                                               g.ctypes.data_as(c_i32p), ctypes.byref(h)))
        else:
            o = np.ascontiguousarray(order, dtype=np.int32)
            if o.shape != (shape.H,):
                raise ValueError("order must have H entries")
            _check("sketchssm_plan_create_ordered",
                   lib().sketchssm_plan_create_ordered(ctypes.byref(shape), r.ctypes.data_as(c_i32p),
                                                       g.ctypes.data_as(c_i32p), o.ctypes.data_as(c_i32p),
                                                       ctypes.byref(h)))
        self.handle = h.value
        self.rank = r.copy()
        self.group = g.copy()
        self._elems = int(lib().sketchssm_z_elems(self.handle)), int(lib().sketchssm_frame_elems(self.handle))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:
            _lib.sketchssm_plan_destroy(h)
            self.handle = None

    @property
    def z_elems(self) -> int:
        return self._elems[0]

    @property
    def frame_elems(self) -> int:
        return self._elems[1]

    def export(self) -> dict:
        H = self.shape.H
        n = c_i32()
        fi = np.zeros(H, np.int32)
        zo = np.zeros(H + 1, np.int32)
        bk = np.zeros(H, np.int32)
        od = np.zeros(H, np.int32)
        fg = np.zeros(H, np.int32)
        fr = np.zeros(H, np.int32)
        fo = np.zeros(H + 1, np.int32)
        P = lambda a: a.ctypes.data_as(c_i32p)  # noqa: E731
        _check("sketchssm_plan_export",
               lib().sketchssm_plan_export(self.handle, P(fi), P(fo), P(zo), P(bk), P(od), P(fg), P(fr),
                                           ctypes.byref(n)))
        F = n.value
        return {"frame_index": fi, "frame_row_off": fo[:F + 1], "z_row_off": zo, "bucket": bk,
                "order": od, "frames": list(zip(fg[:F].tolist(), fr[:F].tolist())), "n_frames": F}


def sketchssm_flush(plan: Plan, S, Z, basis, kbuf, vbuf, abuf, bbuf, n_tokens: int, stream=None):
    _check("sketchssm_flush",
           lib().sketchssm_flush(plan.handle, _ptr(S), _ptr(Z), _ptr(basis), _ptr(kbuf), _ptr(vbuf),
                                 _ptr(abuf), _ptr(bbuf), int(n_tokens), _stream(stream)))


def sketchssm_decode_read(plan: Plan, S, Z, frames, q, k, v, a, beta, kbuf, vbuf, abuf, bbuf,
                          pos: int, y, stream=None):
    _check("sketchssm_decode_read",
           lib().sketchssm_decode_read(plan.handle, _ptr(S), _ptr(Z), _ptr(frames), _ptr(q), _ptr(k),
                                       _ptr(v), _ptr(a), _ptr(beta), _ptr(kbuf), _ptr(vbuf),
                                       _ptr(abuf), _ptr(bbuf), int(pos), _ptr(y), _stream(stream)))


def sketchssm_dense_read(shape: Shape, S, q, k, v, a, beta, kbuf, vbuf, abuf, bbuf, pos: int, y,
                         stream=None):
    _check("sketchssm_dense_read",
           lib().sketchssm_dense_read(ctypes.byref(shape), _ptr(S), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                      _ptr(beta), _ptr(kbuf), _ptr(vbuf), _ptr(abuf), _ptr(bbuf),
                                      int(pos), _ptr(y), _stream(stream)))


def sketchssm_rmw_step(shape: Shape, S, q, k, v, a, beta, y, stream=None):
    _check("sketchssm_rmw_step",
           lib().sketchssm_rmw_step(ctypes.byref(shape), _ptr(S), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                    _ptr(beta), _ptr(y), _stream(stream)))


def sketchssm_decode_read_seq(plan: Plan, S, Z, frames, q, k, v, a, beta, kbuf, vbuf, abuf, bbuf, pos,
                              y, stream=None):
    _check("sketchssm_decode_read_seq",
           lib().sketchssm_decode_read_seq(plan.handle, _ptr(S), _ptr(Z), _ptr(frames), _ptr(q), _ptr(k),
                                           _ptr(v), _ptr(a), _ptr(beta), _ptr(kbuf), _ptr(vbuf),
                                           _ptr(abuf), _ptr(bbuf), _ptr(pos), _ptr(y), _stream(stream)))


def sketchssm_flush_seq(plan: Plan, S, Z, basis, kbuf, vbuf, abuf, bbuf, seqs, n_tokens, n_seqs: int,
                        stream=None):
    with _AS_IS if S is None or isinstance(S, int) else _on_device(S.device, stream):
        _check("sketchssm_flush_seq",
               lib().sketchssm_flush_seq(plan.handle, _ptr(S), _ptr(Z), _ptr(basis), _ptr(kbuf), _ptr(vbuf),
                                         _ptr(abuf), _ptr(bbuf), _ptr(seqs), _ptr(n_tokens), int(n_seqs),
                                         _stream(stream)))


def sketchssm_decode_read_flush(plan: Plan, S, Z, frames, basis, q, k, v, a, beta, kbuf, vbuf, abuf, bbuf, y,
                                stream=None):
    _check("sketchssm_decode_read_flush",
           lib().sketchssm_decode_read_flush(plan.handle, _ptr(S), _ptr(Z), _ptr(frames), _ptr(basis), _ptr(q),
                                             _ptr(k), _ptr(v), _ptr(a), _ptr(beta), _ptr(kbuf), _ptr(vbuf),
                                             _ptr(abuf), _ptr(bbuf), _ptr(y), _stream(stream)))


def _arg(name, x, dtype, shape, device):
    """Device address of a tensor, refused where its type, shape or device is not what the call takes (None and
    addresses pass through)."""
    if x is None or isinstance(x, int):
        return x
    if x.dtype is not dtype or x.shape != shape or x.device != device:
        raise ValueError(f"{name}: expected {dtype} {list(shape)} on {device}, "
                         f"got {x.dtype} {list(x.shape)} on {x.device}")
    if not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return x.data_ptr()


def _int32(name, x):
    """A number as a C call takes it (ctypes would cut it to 32 bits without a word)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}: {x} does not fit 32 bits")
    return x


_AS_IS = contextlib.nullcontext()


def _on_device(device, stream):
    """The context in which a call on tensors of `device` is made: that device current, if it is not."""
    import torch
    if device.type != "cuda":
        raise ValueError("expected a device tensor")
    if stream is not None and not isinstance(stream, int) and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    if device.index == torch.cuda.current_device():
        return _AS_IS
    return torch.cuda.device(device)


def owned_by(stream, device):
    """The context in which a tensor for calls on `stream` is allocated: it belongs to that stream, so torch's
    allocator gives its memory to nothing else before the work queued there is done."""
    import torch
    if stream is None:
        return _AS_IS
    if isinstance(stream, int):  # (with 0, the null stream's handle, ExternalStream takes a stream of torch's pool)
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _ragged(shape, S0, rows0, S, rows, offsets, max_len, q, k, v, a, beta, y):
    """Checks of the ragged calls' tensors; the arguments both entry points begin with."""
    import torch
    dev, i32, f32 = S.device, torch.int32, torch.float32
    H, K, V, Hk, T = shape.H, shape.K, shape.V, shape.kq_heads or shape.H, v.shape[0]
    qkv = torch.bfloat16 if shape.qkv == 0 else f32
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets: expected n_seqs + 1 entries")
    n = offsets.numel() - 1
    if rows is None and n > shape.B:
        raise ValueError(f"rows: {n} sequences and {shape.B} state rows")
    n0 = 0 if S0 is None else S0.shape[0]
    if rows0 is not None and n0 == 0:
        raise ValueError("rows0: first rows of no states (S0 is None or empty)")
    return [ctypes.byref(shape), _arg("S0", S0, f32, (n0, H, K, V), dev), n0,
            _arg("rows0", rows0, i32, (n,), dev), _arg("S", S, f32, (shape.B, H, K, V), dev),
            _arg("rows", rows, i32, (n,), dev), _arg("offsets", offsets, i32, (n + 1,), dev), n, T,
            _int32("max_len", max_len), _arg("q", q, qkv, (T, Hk, K), dev), _arg("k", k, qkv, (T, Hk, K), dev),
            _arg("v", v, qkv, (T, H, V), dev),
            _arg("a", a, f32, (T, H, K) if shape.kind == KIND["kda"] else (T, H), dev),
            _arg("beta", beta, f32, (T, H), dev), _arg("y", y, f32, (T, H, V), dev)]


def sketchssm_rmw_seq(shape: Shape, S0, rows0, S, rows, offsets, max_len: int, q, k, v, a, beta, y, stream=None):
    """The recurrent form for a few tokens of each listed sequence."""
    args = _ragged(shape, S0, rows0, S, rows, offsets, max_len, q, k, v, a, beta, y)
    with _on_device(S.device, stream):
        _check("sketchssm_rmw_seq", lib().sketchssm_rmw_seq(*args, _stream(stream)))


def sketchssm_prefill(shape: Shape, S0, rows0, S, rows, offsets, max_len: int, q, k, v, a, beta, y, workspace=None,
                      stream=None):
    """The chunked form for ragged prompts.  `workspace`: a uint8 tensor of at least
    ``sketchssm_prefill_workspace`` bytes; None takes one from torch's allocator for this call."""
    import torch
    args = _ragged(shape, S0, rows0, S, rows, offsets, max_len, q, k, v, a, beta, y)
    with _on_device(S.device, stream):
        st = _stream(stream)
        if workspace is None:
            need = sketchssm_prefill_workspace(shape, args[7], args[8], max_len)
            if need:
                with owned_by(stream, S.device):
                    workspace = torch.empty(need, dtype=torch.uint8, device=S.device)
        elif workspace.device != S.device:
            raise ValueError(f"workspace: expected a tensor on {S.device}, got one on {workspace.device}")
        size = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check("sketchssm_prefill", lib().sketchssm_prefill(*args, _ptr(workspace), size, st))


def sketchssm_prefill_workspace(shape: Shape, n_seqs: int, total_tokens: int, max_len: int) -> int:
    return int(lib().sketchssm_prefill_workspace(ctypes.byref(shape), _int32("n_seqs", n_seqs),
                                                 _int32("total_tokens", total_tokens), _int32("max_len", max_len)))


def sketchssm_gated_norm(shape: Shape, y, skip, D, z, weight, norm_heads: int, gate, eps: float, out, stream=None):
    """The gated norm behind a layer's output (``gate``: a key of ``GATE`` or its value)."""
    import torch
    dev, f32 = y.device, torch.float32
    qkv = torch.bfloat16 if shape.qkv == 0 else f32
    full = (y.shape[0], shape.H, shape.V)
    w_heads = 1 if weight.dim() == 1 else weight.shape[0]
    args = [_arg("y", y, f32, full, dev), _arg("skip", skip, qkv, full, dev), _arg("D", D, f32, (shape.H,), dev),
            _arg("z", z, qkv, full, dev),
            _arg("weight", weight, f32, (shape.V,) if weight.dim() == 1 else (w_heads, shape.V), dev)]
    with _on_device(dev, stream):
        _check("sketchssm_gated_norm",
               lib().sketchssm_gated_norm(ctypes.byref(shape), *args, w_heads, int(norm_heads),
                                          GATE[gate] if isinstance(gate, str) else int(gate), float(eps), full[0],
                                          _arg("out", out, qkv, full, dev), _stream(stream)))


def _tree(shape, rows, offsets, parents, k, v, a, beta, kbuf, vbuf, abuf, bbuf, pos, dev):
    """Checks of what both tree calls take: (window, lists, n_seqs, n_nodes, tokens)."""
    import torch
    i32, f32 = torch.int32, torch.float32
    B, H, K, V, W, Hk = shape.B, shape.H, shape.K, shape.V, shape.W, shape.kq_heads or shape.H
    T, kda = v.shape[0], shape.kind == KIND["kda"]
    qkv = torch.bfloat16 if shape.qkv == 0 else f32
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets: expected n_seqs + 1 entries")
    n = offsets.numel() - 1
    if rows is None and n > B:
        raise ValueError(f"rows: {n} sequences and {B} state rows")
    window = [_arg("kbuf", kbuf, qkv, (W, Hk, B, K), dev), _arg("vbuf", vbuf, qkv, (W, H, B, V), dev),
              _arg("abuf", abuf, f32, (W, H, B, K) if kda else (W, H, B), dev), _arg("bbuf", bbuf, f32, (W, H, B), dev)]
    lists = [_arg("pos", pos, i32, (B,), dev), _arg("rows", rows, i32, (n,), dev),
             _arg("offsets", offsets, i32, (n + 1,), dev), _arg("parents", parents, i32, (T,), dev)]
    tokens = [_arg("k", k, qkv, (T, Hk, K), dev), _arg("v", v, qkv, (T, H, V), dev),
              _arg("a", a, f32, (T, H, K) if kda else (T, H), dev), _arg("beta", beta, f32, (T, H), dev)]
    return window, lists, n, T, tokens


def sketchssm_tree_read(plan: Plan, S, Z, frames, kbuf, vbuf, abuf, bbuf, pos, rows, offsets, max_nodes: int, parents, q, k,
                        v, a, beta, y, stream=None):
    """Trees of drafted tokens over listed rows' sketch (or state) and window; only y is written."""
    import torch
    sh, dev, f32 = plan.shape, v.device, torch.float32
    window, lists, n, T, tokens = _tree(sh, rows, offsets, parents, k, v, a, beta, kbuf, vbuf, abuf, bbuf, pos, dev)
    cache = [_arg("S", S, f32, (sh.B, sh.H, sh.K, sh.V), dev), _flat("Z", Z, plan.z_elems, dev),
             _flat("frames", frames, plan.frame_elems, dev)]
    qq = _arg("q", q, torch.bfloat16 if sh.qkv == 0 else f32, (T, sh.kq_heads or sh.H, sh.K), dev)
    yy = _arg("y", y, f32, (T, sh.H, sh.V), dev)
    with _on_device(dev, stream):
        _check("sketchssm_tree_read",
               lib().sketchssm_tree_read(plan.handle, *cache, *window, *lists[:3], n, T, _int32("max_nodes", max_nodes),
                                         lists[3], qq, *tokens, yy, _stream(stream)))


def sketchssm_tree_accept(shape: Shape, kbuf, vbuf, abuf, bbuf, pos, new_pos, rows, offsets, parents, accepted, k, v, a,
                          beta, stream=None):
    """The accepted path of each tree, appended to its row's window; new_pos: every row's held-back tokens then."""
    import torch
    dev, i32 = v.device, torch.int32
    window, lists, n, T, tokens = _tree(shape, rows, offsets, parents, k, v, a, beta, kbuf, vbuf, abuf, bbuf, pos, dev)
    new = _arg("new_pos", new_pos, i32, (shape.B,), dev)
    acc = _arg("accepted", accepted, i32, (n,), dev)
    with _on_device(dev, stream):
        _check("sketchssm_tree_accept",
               lib().sketchssm_tree_accept(ctypes.byref(shape), *window, lists[0], new, *lists[1:3], n, T, lists[3], acc,
                                           *tokens, _stream(stream)))


def _flat(name, x, elems, device):
    """Device address of a float32 array of at least so many elements, whatever its shape."""
    import torch
    if x is None or isinstance(x, int):
        return x
    if x.dtype is not torch.float32 or x.numel() < elems or x.device != device or not x.is_contiguous():
        raise ValueError(f"{name}: expected at least {elems} contiguous {torch.float32} on {device}, "
                         f"got {x.dtype} {list(x.shape)} on {x.device}")
    return x.data_ptr()


def _cache(shape, S, rows, codes, scales, slots, fmt):
    """Checks of the cache calls: (state, rows, codes, scales, slots, n_slots, pairs, format)."""
    import torch
    dev, i32 = S.device, torch.int32
    f = CACHE[fmt] if isinstance(fmt, str) else _int32("format", fmt)
    n_slots, H, K, V = codes.shape[0], shape.H, shape.K, shape.V
    lists = [x for x in (rows, slots) if x is not None]
    sized = [x for x in lists if not isinstance(x, int)]
    if lists and not sized:
        raise ValueError("rows, slots: the number of pairs is that of a tensor, got addresses")
    n = sized[0].numel() if sized else n_slots
    for name, x, most in (("rows", rows, shape.B), ("slots", slots, n_slots)):
        if x is None and n > most:
            raise ValueError(f"{name}: {n} pairs and {most} {name}")
    kind = torch.float8_e4m3fn if f == CACHE["e4m3"] else torch.int8
    return [_arg("S", S, torch.float32, (shape.B, H, K, V), dev), _arg("rows", rows, i32, (n,), dev),
            _arg("codes", codes, kind, (n_slots, H, K, V), dev),
            _arg("scales", scales, torch.bfloat16, (n_slots, H, K), dev), _arg("slots", slots, i32, (n,), dev),
            _int32("n_slots", n_slots), _int32("n", n), f]


def sketchssm_cache_store(shape: Shape, S, rows, codes, scales, slots, format, stream=None):
    """States of listed rows to slots of an 8-bit cache (``format``: a key of ``CACHE`` or its value)."""
    args = _cache(shape, S, rows, codes, scales, slots, format)
    with _on_device(S.device, stream):
        _check("sketchssm_cache_store", lib().sketchssm_cache_store(ctypes.byref(shape), *args, _stream(stream)))


def sketchssm_cache_load(shape: Shape, codes, scales, slots, S, rows, format, stream=None):
    """Slots of an 8-bit cache back to listed state rows (a negative slot: the zero state)."""
    st, rw, cd, sc, sl, n_slots, n, f = _cache(shape, S, rows, codes, scales, slots, format)
    with _on_device(S.device, stream):
        _check("sketchssm_cache_load",
               lib().sketchssm_cache_load(ctypes.byref(shape), cd, sc, sl, n_slots, st, rw, n, f, _stream(stream)))


def sketchssm_stream_probe(src, read_bytes: int, dst, write_bytes: int, unroll: int = 8, blocks: int = 0,
                           nontemporal: bool = False, stream=None):
    """Measurement aid (include/sketchssm_measure.h): stream read_bytes of src,
    writing write_bytes of sums to dst."""
    _check("sketchssm_stream_probe",
           lib().sketchssm_stream_probe(_ptr(src), int(read_bytes), _ptr(dst), int(write_bytes), int(unroll),
                                        int(blocks), 1 if nontemporal else 0, _stream(stream)))
