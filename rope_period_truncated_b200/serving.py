"""Rotary, cache-append, tree-attention, compaction and page calls (the second
half of ``include/waveprune.h``), bound like the calls of the package module:
arguments are checked and marshalled here, all arithmetic runs in the library.

A K/V cache is given by its two tensors and, when paged, a block table:
contiguous V [B,Hkv,Lmax,d] with K the same (rows) or [B,Hkv,d/16,Lmax,16]
(group-major); paged V [n_pages,Hkv,P,d] with K the same or
[n_pages,Hkv,d/16,P,16] and ``block_table`` int32 [B,max_pages] (device).

Calls run on ``stream``, or on the current stream of the tensors' device.
"""
from __future__ import annotations

import contextlib
import ctypes

import numpy as np
import torch

P, I, L, D, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_float, ctypes.c_size_t

PAGES_OK, PAGES_SHORT, PAGES_BAD_ARGUMENT = range(3)
TREE_MAX_NODES = 64


class _Rows(ctypes.Structure):
    _fields_ = [("data", P), ("stride_b", L), ("stride_n", L), ("stride_h", L)]


_RP = ctypes.POINTER(_Rows)
SIGNATURES = {
    "wp_cutoffs_partial": (I, [I, I, D, P, D, D, I, P, P]),
    "wp_rope_scaling": (I, [I, D, D, I, D, D, P, P]),
    "wp_rope_qk": (I, [_RP, _RP, I, _RP, _RP, I, I, I, I, I, P, I, D, P, D, D, I, I, P]),
    "wp_rope_append": (I, [_RP, _RP, I, _RP, _RP, I, I, I, I, P, P, P, P, I, P, I, I, P, I, I, I, D, P, D, D, I, P]),
    "wp_decode_tree_workspace_bytes": (S, [I, I, I, I, I, I]),
    "wp_decode_tree": (I, [P, P, I, P, P, P, P, I, I, P, I, I, I, I, I, I, I, P, F, P, P, P, S, P]),
    "wp_kv_compact": (I, [P, I, P, P, P, I, P, P, I, P, I, I, I, I, I, I, P]),
    "wp_pages_update_workspace_bytes": (S, [I, I]),
    "wp_pages_update": (I, [P] * 11 + [I, I, I, I, P, S, P]),
    "wp_pages_copy": (I, [P, I, P, P, I, I, I, I, I, P]),
}


def declare(lib):
    """Result and argument types of this module's C calls."""
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args


def _base():
    import rope_period_truncated_b200 as base
    return base


def _call(name, *args):
    base = _base()
    code = getattr(base.load_library(), name)(*args)
    if code:
        raise base.WavePruneError(name, code)


def _tensor(t, name, dtype, ndim, device=None, contiguous=True):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _ptr(t):
    return None if t is None else t.data_ptr()


class _On:
    """The launch's device and stream: the given stream, or the current one of the tensors' device. Buffers that a call
    allocates are marked as used on a stream that is not the current one."""

    def __init__(self, device, stream):
        current = torch.cuda.current_stream(device)
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        self.stream = current if stream is None else stream
        self.elsewhere = self.stream != current
        self.guard = contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)
        self.device = device

    @property
    def handle(self):
        return self.stream.cuda_stream

    def empty(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device=self.device)
        if self.elsewhere:
            t.record_stream(self.stream)
        return t


def _freqs(scale, n):
    if scale is None:
        return None, None
    a = np.ascontiguousarray(scale, dtype=np.float64)
    if a.shape != (n,):
        raise ValueError(f"freq_scale must have {n} entries (rot_dim/2)")
    return a, a.ctypes.data


def _cuts(group_cut, n):
    if group_cut is None:
        return None, None
    a = np.ascontiguousarray(group_cut, dtype=np.int32)
    if a.shape != (n,):
        raise ValueError(f"group_cut must have {n} entries (d/16)")
    return a, a.ctypes.data


def _rows(t):
    """wp_rows of a [B,N,H,d] or [T,H,d] tensor whose dims are contiguous."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError("the head dims must be contiguous")
    return _Rows(t.data_ptr(), st[0] if t.dim() == 4 else 0, st[-3], st[-2])


def _cache(kcache, vcache, block_table, device, B=None, Hkv=None, d=None):
    """(k_layout, B, Lmax, max_pages, page_size, n_pages, Hkv, d) of a cache, its shapes checked."""
    _tensor(vcache, "vcache", torch.bfloat16, 4, device)
    n, H, rows, dd = vcache.shape
    if kcache.dim() == 5:
        _tensor(kcache, "kcache", torch.bfloat16, 5, device)
        if tuple(kcache.shape) != (n, H, dd // 16, rows, 16):
            raise ValueError("group-major K cache shape mismatch")
        layout = 1
    else:
        _tensor(kcache, "kcache", torch.bfloat16, 4, device)
        if kcache.shape != vcache.shape:
            raise ValueError("K cache shape mismatch")
        layout = 0
    if (Hkv is not None and H != Hkv) or (d is not None and dd != d):
        raise ValueError("the cache's heads or head dim do not match")
    if block_table is None:
        if B is not None and n != B:
            raise ValueError(f"the cache holds {n} sequences, expected {B}")
        return layout, n, rows, 0, 0, 0, H, dd
    _tensor(block_table, "block_table", torch.int32, 2, device)
    if B is not None and block_table.shape[0] != B:
        raise ValueError(f"the block table has {block_table.shape[0]} rows, expected {B}")
    return layout, block_table.shape[0], 0, block_table.shape[1], rows, n, H, dd


# --------------------------------------------------------------------- host

def wp_cutoffs_partial(d_h: int, rot_dim: int, theta: float, layout: int, alpha: float = 2.0, freq_scale=None,
                       scale_all: float = 1.0):
    """Integer cutoffs (chan_cut [rot_dim/2], group_cut [d_h/16]) of a model that rotates the first rot_dim dims."""
    fs, fs_p = _freqs(freq_scale, rot_dim // 2)
    wc = np.zeros(max(rot_dim // 2, 1), dtype=np.int32)
    wg = np.zeros(max(d_h // 16, 1), dtype=np.int32)
    _call("wp_cutoffs_partial", d_h, rot_dim, theta, fs_p, scale_all, alpha, layout, wc.ctypes.data, wg.ctypes.data)
    return wc, wg


def wp_rope_scaling(rot_dim: int, theta: float, factor: float, original_len: int, turns_slow: float = 1.0,
                    turns_fast: float = 32.0):
    """(freq_scale [rot_dim/2] float64, amplitude) for a context ``factor`` times ``original_len``."""
    fs = np.zeros(max(rot_dim // 2, 1), dtype=np.float64)
    amp = D(0.0)
    _call("wp_rope_scaling", rot_dim, theta, factor, original_len, turns_slow, turns_fast, fs.ctypes.data,
          ctypes.addressof(amp))
    return fs, amp.value


# ------------------------------------------------------------------- device

def wp_rope_qk(q: torch.Tensor | None, k: torch.Tensor | None, theta: float, layout: int, pos: torch.Tensor | None = None,
               pos0: int = 0, rot_dim: int | None = None, freq_scale=None, scale_all: float = 1.0,
               amplitude: float = 1.0, inverse: bool = False, out_q: torch.Tensor | None = None,
               out_k: torch.Tensor | None = None, stream=None):
    """Rotate q [B,N,Hq,d] and k [B,N,Hk,d] (bf16; strided views of a fused
    projection are fine; either may be None) by pos [B,N] (int32, device;
    None: pos0 + n) in one launch. The first ``rot_dim`` dims (None: all)
    rotate, times ``amplitude``. ``inverse``: the transposed rotation, i.e.
    the gradient with respect to the inputs of the same forward call. Returns
    (out_q, out_k); out_q is q rotates in place (not with
    ROPE_HALF_SPLIT_PAIRED)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    _tensor(x, "q" if q is not None else "k", torch.bfloat16, 4, None, False)
    device = x.device
    B, N, _, d = x.shape
    if k is not None:
        _tensor(k, "k", torch.bfloat16, 4, device, False)
        if (k.shape[0], k.shape[1], k.shape[3]) != (B, N, d):
            raise ValueError("q/k shape mismatch")
    if pos is not None:
        _tensor(pos, "pos", torch.int32, 2, device)
        if tuple(pos.shape) != (B, N):
            raise ValueError("pos must be [B, N]")
    rot = d if rot_dim is None else int(rot_dim)
    on = _On(device, stream)
    args = []
    outs = []
    for t, out, name in ((q, out_q, "out_q"), (k, out_k, "out_k")):
        if t is None:
            if out is not None:
                raise ValueError(f"{name} without its input")
            args += [None, None, 0]
            outs.append(None)
            continue
        if out is None:
            out = on.empty(t.shape, torch.bfloat16)
        else:
            _tensor(out, name, torch.bfloat16, 4, device, False)
            if out.shape != t.shape:
                raise ValueError(f"{name} shape mismatch")
        args += [_rows(t), _rows(out), t.shape[2]]
        outs.append(out)
    if x.numel() == 0:
        raise ValueError("empty tensors")
    fs, fs_p = _freqs(freq_scale, rot // 2)
    with on.guard:
        _call("wp_rope_qk", *args, B, N, d, rot, _ptr(pos), int(pos0), theta, fs_p, scale_all, amplitude, int(layout),
              1 if inverse else 0, on.handle)
    return outs[0], outs[1]


def wp_rope_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                   pos: torch.Tensor, seq: torch.Tensor, slot: torch.Tensor, theta: float, layout: int,
                   block_table: torch.Tensor | None = None, rot_dim: int | None = None, freq_scale=None,
                   scale_all: float = 1.0, amplitude: float = 1.0, out_q: torch.Tensor | None = None, stream=None):
    """Rotate the new tokens' q [T,Hq,d] (or None) and k [T,Hkv,d] by pos [T]
    and write k and v [T,Hkv,d] into key slot[i] of sequence seq[i] of the
    cache (int32 [T], device; seq -1 = padding). Returns the rotated q."""
    _tensor(k, "k", torch.bfloat16, 3, None, False)
    device = k.device
    T, Hkv, d = k.shape
    _tensor(v, "v", torch.bfloat16, 3, device, False)
    if v.shape != k.shape:
        raise ValueError("k/v shape mismatch")
    for t, name in ((pos, "pos"), (seq, "seq"), (slot, "slot")):
        _tensor(t, name, torch.int32, 1, device)
        if t.shape[0] != T:
            raise ValueError(f"{name} must be [T]")
    klay, B, Lmax, max_pages, page, n_pages, _, _ = _cache(kcache, vcache, block_table, device, None, Hkv, d)
    rot = d if rot_dim is None else int(rot_dim)
    on = _On(device, stream)
    args = [None, None, 0]
    if q is not None:
        _tensor(q, "q", torch.bfloat16, 3, device, False)
        if (q.shape[0], q.shape[2]) != (T, d):
            raise ValueError("q shape mismatch")
        if out_q is None:
            out_q = on.empty(q.shape, torch.bfloat16)
        else:
            _tensor(out_q, "out_q", torch.bfloat16, 3, device, False)
            if out_q.shape != q.shape:
                raise ValueError("out_q shape mismatch")
        args = [_rows(q), _rows(out_q), q.shape[1]]
    elif out_q is not None:
        raise ValueError("out_q without q")
    fs, fs_p = _freqs(freq_scale, rot // 2)
    with on.guard:
        _call("wp_rope_append", *args, _rows(k), _rows(v), Hkv, T, d, rot, _ptr(pos), _ptr(seq), _ptr(slot), _ptr(kcache),
              klay, _ptr(vcache), B, Lmax, _ptr(block_table), max_pages, page, n_pages, theta, fs_p, scale_all, amplitude,
              int(layout), on.handle)
    return out_q


def wp_decode_tree_workspace_bytes(B: int, T: int, Hq: int, Hkv: int, d_h: int, Lmax: int) -> int:
    """Scratch bytes of wp_decode_tree; Lmax: capacity per sequence (paged: max_pages * page size)."""
    return int(_base().load_library().wp_decode_tree_workspace_bytes(B, T, Hq, Hkv, d_h, Lmax))


def wp_decode_tree(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
                   n_nodes: torch.Tensor | None = None, block_table: torch.Tensor | None = None, group_cut=None,
                   softmax_scale: float = 0.0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, want_lse: bool = True, stream=None):
    """Attention of a tree of drafted tokens over a cache: q [B,T,Hq,d]
    (rotated at position lens + depth), node t's K/V at key lens[b] + t,
    parents int32 [B,T] (-1 = follows the context), n_nodes int32 [B] or None
    (= T), lens int32 [B]; all on the device. ``group_cut``: group cutoffs
    [d/16] or None (dense). Returns (o [B,T,Hq,d] bf16, lse [B,Hq,T] fp32);
    rows t >= n_nodes[b] are 0 and -inf."""
    _tensor(q, "q", torch.bfloat16, 4)
    device = q.device
    B, T, Hq, d = q.shape
    _tensor(lens, "lens", torch.int32, 1, device)
    _tensor(parents, "parents", torch.int32, 2, device)
    if lens.shape[0] != B or tuple(parents.shape) != (B, T):
        raise ValueError("lens must be [B] and parents [B, T]")
    if n_nodes is not None:
        _tensor(n_nodes, "n_nodes", torch.int32, 1, device)
        if n_nodes.shape[0] != B:
            raise ValueError("n_nodes must be [B]")
    klay, _, Lmax, max_pages, page, n_pages, Hkv, _ = _cache(kcache, vcache, block_table, device, B, None, d)
    on = _On(device, stream)
    if out is None:
        out = on.empty(q.shape, torch.bfloat16)
    else:
        _tensor(out, "out", torch.bfloat16, 4, device)
        if out.shape != q.shape:
            raise ValueError("out shape mismatch")
    if lse is not None:
        _tensor(lse, "lse", torch.float32, 3, device)
        if tuple(lse.shape) != (B, Hq, T):
            raise ValueError("lse must be [B, Hq, T]")
    elif want_lse:
        lse = on.empty((B, Hq, T), torch.float32)
    if workspace is None:
        need = wp_decode_tree_workspace_bytes(B, T, Hq, Hkv, d, Lmax if block_table is None else max_pages * page)
        workspace = on.empty(max(need, 1), torch.uint8)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    cut, cut_p = _cuts(group_cut, d // 16)
    with on.guard:
        _call("wp_decode_tree", _ptr(q), _ptr(kcache), klay, _ptr(vcache), _ptr(lens), _ptr(parents), _ptr(n_nodes), T, Lmax,
              _ptr(block_table), max_pages, page, n_pages, B, Hq, Hkv, d, cut_p, softmax_scale, _ptr(out), _ptr(lse),
              _ptr(workspace), workspace.numel() * workspace.element_size(), on.handle)
    return out, lse


def wp_kv_compact(kcache: torch.Tensor, vcache: torch.Tensor, lens: torch.Tensor, path: torch.Tensor, n_keep: torch.Tensor,
                  block_table: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """Move the rows of key lens[b] + path[b,i] to key lens[b] + i, i <
    n_keep[b] (int32 [B,A] increasing, int32 [B]; device), in place. Returns
    the new lengths int32 [B] (``out``, which may be lens; -1 where a path,
    length or page is out of range)."""
    _tensor(lens, "lens", torch.int32, 1)
    device = lens.device
    B = lens.shape[0]
    _tensor(path, "path", torch.int32, 2, device)
    _tensor(n_keep, "n_keep", torch.int32, 1, device)
    if path.shape[0] != B or n_keep.shape[0] != B:
        raise ValueError("path must be [B, A] and n_keep [B]")
    klay, _, Lmax, max_pages, page, n_pages, Hkv, d = _cache(kcache, vcache, block_table, device, B)
    on = _On(device, stream)
    if out is None:
        out = on.empty((B,), torch.int32)
    else:
        _tensor(out, "out", torch.int32, 1, device)
        if out.shape[0] != B:
            raise ValueError("out must be [B]")
    with on.guard:
        _call("wp_kv_compact", _ptr(kcache), klay, _ptr(vcache), _ptr(lens), _ptr(path), path.shape[1], _ptr(n_keep), _ptr(out),
              Lmax, _ptr(block_table), max_pages, page, n_pages, B, Hkv, d, on.handle)
    return out


def wp_pages_update(refs: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, parent: torch.Tensor,
                    keep: torch.Tensor, new_lens: torch.Tensor, page_size: int, workspace: torch.Tensor | None = None,
                    stream=None):
    """One transaction on the pages of a batch (fork, grow, copy on write,
    free): row b goes on from row parent[b] with its first keep[b] tokens and
    room for new_lens[b]. All int32 on the device: refs [n_pages], block_table
    [B,max_pages], the others [B]. Returns new tensors (refs, block_table,
    lens, copies [B,3], info [4]); info[0] is PAGES_OK, or PAGES_SHORT /
    PAGES_BAD_ARGUMENT with everything as it was."""
    _tensor(refs, "refs", torch.int32, 1)
    device = refs.device
    _tensor(block_table, "block_table", torch.int32, 2, device)
    B, max_pages = block_table.shape
    for t, name in ((lens, "lens"), (parent, "parent"), (keep, "keep"), (new_lens, "new_lens")):
        _tensor(t, name, torch.int32, 1, device)
        if t.shape[0] != B:
            raise ValueError(f"{name} must be [B]")
    on = _On(device, stream)
    n = refs.shape[0]
    out = [on.empty(s, torch.int32) for s in ((n,), (B, max_pages), (B,), (B, 3), (4,))]
    if workspace is None:
        need = int(_base().load_library().wp_pages_update_workspace_bytes(B, n))
        workspace = on.empty(max(need, 1), torch.uint8)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    with on.guard:
        _call("wp_pages_update", _ptr(refs), _ptr(block_table), _ptr(lens), _ptr(parent), _ptr(keep), _ptr(new_lens),
              *(_ptr(t) for t in out), B, max_pages, int(page_size), n, _ptr(workspace),
              workspace.numel() * workspace.element_size(), on.handle)
    return tuple(out)


def wp_pages_copy(k_pages: torch.Tensor, v_pages: torch.Tensor, copies: torch.Tensor, stream=None) -> None:
    """Copy rows between pages of a K and a V pool: copies int32 [n,3] (device),
    each source page, target page, rows; entries of -1 copy nothing."""
    _tensor(copies, "copies", torch.int32, 2)
    if copies.shape[1] != 3:
        raise ValueError("copies must be [n, 3]")
    klay, _, _, _, page, n_pages, Hkv, d = _cache(k_pages, v_pages, copies, copies.device)
    on = _On(copies.device, stream)
    with on.guard:
        _call("wp_pages_copy", _ptr(k_pages), klay, _ptr(v_pages), _ptr(copies), copies.shape[0], n_pages, page, Hkv, d,
              on.handle)
