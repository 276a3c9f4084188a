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

import ctypes
from array import array

import numpy as np
import torch

P, I, L, D, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_float, ctypes.c_size_t

PAGES_OK, PAGES_SHORT, PAGES_BAD_ARGUMENT = range(3)
TREE_MAX_NODES = 64

SIGNATURES = {  # a wp_rows argument is passed by the address of its four 64-bit words
    "wp_cutoffs_partial": (I, [I, I, D, P, D, D, I, P, P]),
    "wp_rope_scaling": (I, [I, D, D, I, D, D, P, P]),
    "wp_rope_qk": (I, [P, P, I, P, P, I, I, I, I, I, P, I, D, P, D, D, I, I, P]),
    "wp_rope_append": (I, [P, P, I, P, P, I, I, I, I, P, P, P, P, I, P, I, I, P, I, I, I, D, P, D, D, I, P]),
    "wp_decode_tree_workspace_bytes": (S, [I, I, I, I, I, I]),
    "wp_decode_tree": (I, [P, P, I, P, P, P, P, I, I, P, I, I, I, I, I, I, I, P, F, P, P, P, S, P]),
    "wp_kv_compact": (I, [P, I, P, P, P, I, P, P, I, P, I, I, I, I, I, I, P]),
    "wp_pages_update_workspace_bytes": (S, [I, I]),
    "wp_pages_update": (I, [P] * 11 + [I, I, I, I, P, S, P]),
    "wp_pages_copy": (I, [P, I, P, P, I, I, I, I, I, P]),
}

# These calls last a few microseconds on the device at their smallest, so the
# marshalling counts: one compound test per tensor (the message is looked for
# only when it fails), tensor addresses as plain integers, no numpy on the way.
BF16, I32, F32 = torch.bfloat16, torch.int32, torch.float32
_lib = None


def declare(lib):
    """Result and argument types of this module's C calls."""
    global _lib
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _lib = lib


def _load():
    if _lib is None:
        import rope_period_truncated_b200 as base
        base.load_library()
    return _lib


def _fail(name, code):
    from rope_period_truncated_b200 import WavePruneError
    raise WavePruneError(name, code)


def _complain(t, name, dtype, ndim, device, contiguous):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")


def _device(t, name, dtype, ndim, contiguous=True):
    """Device index of the call's first tensor, the tensor checked."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not dtype or t.dim() != ndim or (
            contiguous and not t.is_contiguous()):
        _complain(t, name, dtype, ndim, None, contiguous)
    return t.get_device()


def _check(t, name, dtype, ndim, device, contiguous=True):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.dim() != ndim or t.get_device() != device or (
            contiguous and not t.is_contiguous()):
        _complain(t, name, dtype, ndim, device, contiguous)


def _current(device):
    return torch.cuda.current_stream(device).cuda_stream


# the handle without a Stream object around it, where torch offers that
_current = getattr(torch._C, "_cuda_getCurrentRawStream", _current)


class _Call:
    """Device and stream of one call: the given stream, or the current one of
    the tensors' device. Buffers that the call allocates are marked as used on
    a stream that is not the current one."""
    __slots__ = ("device", "stream", "handle", "elsewhere")

    def __init__(self, device, stream):
        self.device = device
        self.stream = stream
        self.handle = _current(device)
        self.elsewhere = False
        if stream is not None:
            if stream.device_index != device:
                raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors on cuda:{device}")
            self.elsewhere = stream.cuda_stream != self.handle
            self.handle = stream.cuda_stream

    def own(self, t):
        if self.elsewhere:
            t.record_stream(self.stream)
        return t

    def __call__(self, name, *args):
        fn = getattr(_load(), name)
        if torch.cuda.current_device() == self.device:
            code = fn(*args, self.handle)
        else:
            with torch.cuda.device(self.device):
                code = fn(*args, self.handle)
        if code:
            _fail(name, code)


def _freqs(scale, n):
    """(what keeps the values alive, their address)"""
    if scale is None:
        return None, None
    a = array("d", scale.tolist() if hasattr(scale, "tolist") else scale)
    if len(a) != n:
        raise ValueError(f"freq_scale must have {n} entries (rot_dim/2)")
    return a, a.buffer_info()[0]


def _cuts(group_cut, n):
    if group_cut is None:
        return None, None
    a = array("i", group_cut.tolist() if hasattr(group_cut, "tolist") else group_cut)
    if len(a) != n:
        raise ValueError(f"group_cut must have {n} entries (d/16)")
    return a, a.buffer_info()[0]


def _rows(*tensors):
    """wp_rows of four [B,N,H,d] or [T,H,d] tensors, dims contiguous (None: all zero): the words, the address of each."""
    words = []
    for t in tensors:
        if t is None:
            words += (0, 0, 0, 0)
            continue
        st = t.stride()
        if st[-1] != 1 and t.shape[-1] > 1:
            raise ValueError("the head dims must be contiguous")
        words += (t.data_ptr(), st[0] if len(st) == 4 else 0, st[-3], st[-2])
    keep = array("q", words)
    base = keep.buffer_info()[0]
    return keep, base, base + 32, base + 64, base + 96


def _ptr(t):
    return None if t is None else t.data_ptr()


def _cache(kcache, vcache, block_table, device, B=None, Hkv=None, d=None):
    """(k_layout, B, Lmax, max_pages, page_size, n_pages, Hkv, d) of a cache, its shapes checked."""
    _check(vcache, "vcache", BF16, 4, device)
    shape = n, H, rows, dd = vcache.shape
    if isinstance(kcache, torch.Tensor) and kcache.dim() == 5:
        _check(kcache, "kcache", BF16, 5, device)
        if kcache.shape != (n, H, dd // 16, rows, 16):
            raise ValueError("group-major K cache shape mismatch")
        layout = 1
    else:
        _check(kcache, "kcache", BF16, 4, device)
        if kcache.shape != shape:
            raise ValueError("K cache shape mismatch")
        layout = 0
    if (Hkv is not None and H != Hkv) or (d is not None and dd != d):
        raise ValueError("the cache's heads or head dim do not match")
    if block_table is None:
        if B is not None and n != B:
            raise ValueError(f"the cache holds {n} sequences, expected {B}")
        return layout, n, rows, 0, 0, 0, H, dd
    _check(block_table, "block_table", I32, 2, device)
    b, pages = block_table.shape
    if B is not None and b != B:
        raise ValueError(f"the block table has {b} rows, expected {B}")
    return layout, b, 0, pages, rows, n, H, dd


# --------------------------------------------------------------------- host

def wp_cutoffs_partial(d_h: int, rot_dim: int, theta: float, layout: int, alpha: float = 2.0, freq_scale=None,
                       scale_all: float = 1.0):
    """Integer cutoffs (chan_cut [rot_dim/2], group_cut [d_h/16]) of a model that rotates the first rot_dim dims."""
    keep, fs = _freqs(freq_scale, rot_dim // 2)
    wc = np.zeros(max(rot_dim // 2, 1), dtype=np.int32)
    wg = np.zeros(max(d_h // 16, 1), dtype=np.int32)
    code = _load().wp_cutoffs_partial(d_h, rot_dim, theta, fs, scale_all, alpha, layout, wc.ctypes.data, wg.ctypes.data)
    if code:
        _fail("wp_cutoffs_partial", code)
    return wc, wg


def wp_rope_scaling(rot_dim: int, theta: float, factor: float, original_len: int, turns_slow: float = 1.0,
                    turns_fast: float = 32.0):
    """(freq_scale [rot_dim/2] float64, amplitude) for a context ``factor`` times ``original_len``."""
    fs = np.zeros(max(rot_dim // 2, 1), dtype=np.float64)
    amp = D(0.0)
    code = _load().wp_rope_scaling(rot_dim, theta, factor, original_len, turns_slow, turns_fast, fs.ctypes.data,
                                   ctypes.addressof(amp))
    if code:
        _fail("wp_rope_scaling", code)
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
    device = _device(x, "q" if q is not None else "k", BF16, 4, False)
    B, N, H, d = x.shape
    call = _Call(device, stream)
    Hq = Hk = 0
    if q is not None:
        Hq = H
        if out_q is None:
            out_q = torch.empty_like(q)
            if call.elsewhere:
                call.own(out_q)
        else:
            _check(out_q, "out_q", BF16, 4, device, False)
            if out_q.shape != q.shape:
                raise ValueError("out_q shape mismatch")
    elif out_q is not None:
        raise ValueError("out_q without q")
    if k is not None:
        _check(k, "k", BF16, 4, device, False)
        ks = k.shape
        Hk = ks[2]
        if ks[0] != B or ks[1] != N or ks[3] != d:
            raise ValueError("q/k shape mismatch")
        if out_k is None:
            out_k = torch.empty_like(k)
            if call.elsewhere:
                call.own(out_k)
        else:
            _check(out_k, "out_k", BF16, 4, device, False)
            if out_k.shape != ks:
                raise ValueError("out_k shape mismatch")
    elif out_k is not None:
        raise ValueError("out_k without k")
    if pos is not None:
        _check(pos, "pos", I32, 2, device)
        if pos.shape != (B, N):
            raise ValueError("pos must be [B, N]")
    rot = d if rot_dim is None else int(rot_dim)
    keep_f, fs = _freqs(freq_scale, rot // 2)
    keep, pq, pqo, pk, pko = _rows(q, out_q, k, out_k)
    call("wp_rope_qk", pq, pqo, Hq, pk, pko, Hk, B, N, d, rot, _ptr(pos), int(pos0), theta, fs, scale_all, amplitude, int(layout),
         1 if inverse else 0)
    return out_q, out_k



def wp_rope_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                   pos: torch.Tensor, seq: torch.Tensor, slot: torch.Tensor, theta: float, layout: int,
                   block_table: torch.Tensor | None = None, rot_dim: int | None = None, freq_scale=None,
                   scale_all: float = 1.0, amplitude: float = 1.0, out_q: torch.Tensor | None = None, stream=None):
    """Rotate the new tokens' q [T,Hq,d] (or None) and k [T,Hkv,d] by pos [T]
    and write k and v [T,Hkv,d] into key slot[i] of sequence seq[i] of the
    cache (int32 [T], device; seq -1 = padding). Returns the rotated q."""
    device = _device(k, "k", BF16, 3, False)
    T, Hkv, d = shape = k.shape
    _check(v, "v", BF16, 3, device, False)
    if v.shape != shape:
        raise ValueError("k/v shape mismatch")
    _check(pos, "pos", I32, 1, device)
    _check(seq, "seq", I32, 1, device)
    _check(slot, "slot", I32, 1, device)
    if pos.shape[0] != T or seq.shape[0] != T or slot.shape[0] != T:
        raise ValueError("pos, seq and slot must be [T]")
    klay, B, Lmax, max_pages, page, n_pages, _, _ = _cache(kcache, vcache, block_table, device, None, Hkv, d)
    rot = d if rot_dim is None else int(rot_dim)
    call = _Call(device, stream)
    Hq = 0
    if q is not None:
        _check(q, "q", BF16, 3, device, False)
        qs = q.shape
        Hq = qs[1]
        if qs[0] != T or qs[2] != d:
            raise ValueError("q shape mismatch")
        if out_q is None:
            out_q = call.own(torch.empty_like(q))
        else:
            _check(out_q, "out_q", BF16, 3, device, False)
            if out_q.shape != qs:
                raise ValueError("out_q shape mismatch")
    elif out_q is not None:
        raise ValueError("out_q without q")
    keep_f, fs = _freqs(freq_scale, rot // 2)
    keep, pq, pqo, pk, pv = _rows(q, out_q, k, v)
    call("wp_rope_append", pq, pqo, Hq, pk, pv, Hkv, T, d, rot, pos.data_ptr(), seq.data_ptr(), slot.data_ptr(), kcache.data_ptr(),
         klay, vcache.data_ptr(), B, Lmax, _ptr(block_table), max_pages, page, n_pages, theta, fs, scale_all, amplitude, int(layout))
    return out_q



def wp_decode_tree_workspace_bytes(B: int, T: int, Hq: int, Hkv: int, d_h: int, Lmax: int) -> int:
    """Scratch bytes of wp_decode_tree; Lmax: capacity per sequence (paged: max_pages * page size)."""
    return _load().wp_decode_tree_workspace_bytes(B, T, Hq, Hkv, d_h, Lmax)



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
    device = _device(q, "q", BF16, 4)
    B, T, Hq, d = shape = q.shape
    _check(lens, "lens", I32, 1, device)
    _check(parents, "parents", I32, 2, device)
    if lens.shape[0] != B or parents.shape != (B, T):
        raise ValueError("lens must be [B] and parents [B, T]")
    if n_nodes is not None:
        _check(n_nodes, "n_nodes", I32, 1, device)
        if n_nodes.shape[0] != B:
            raise ValueError("n_nodes must be [B]")
    klay, _, Lmax, max_pages, page, n_pages, Hkv, _ = _cache(kcache, vcache, block_table, device, B, None, d)
    call = _Call(device, stream)
    if out is None:
        out = call.own(torch.empty_like(q))
    else:
        _check(out, "out", BF16, 4, device)
        if out.shape != shape:
            raise ValueError("out shape mismatch")
    if lse is not None:
        _check(lse, "lse", F32, 3, device)
        if lse.shape != (B, Hq, T):
            raise ValueError("lse must be [B, Hq, T]")
    elif want_lse:
        lse = call.own(q.new_empty((B, Hq, T), dtype=F32))
    if workspace is None:
        ws = _load().wp_decode_tree_workspace_bytes(B, T, Hq, Hkv, d, Lmax if block_table is None else max_pages * page)
        if ws:
            workspace = call.own(lens.new_empty(ws // 4))
    else:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the same device")
        ws = workspace.numel() * workspace.element_size()
    keep, cut = _cuts(group_cut, d // 16)
    call("wp_decode_tree", q.data_ptr(), kcache.data_ptr(), klay, vcache.data_ptr(), lens.data_ptr(), parents.data_ptr(), _ptr(n_nodes), T,
         Lmax, _ptr(block_table), max_pages, page, n_pages, B, Hq, Hkv, d, cut, softmax_scale, out.data_ptr(), _ptr(lse),
         _ptr(workspace), ws)
    return out, lse



def wp_kv_compact(kcache: torch.Tensor, vcache: torch.Tensor, lens: torch.Tensor, path: torch.Tensor, n_keep: torch.Tensor,
                  block_table: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """Move the rows of key lens[b] + path[b,i] to key lens[b] + i, i <
    n_keep[b] (int32 [B,A] increasing, int32 [B]; device), in place. Returns
    the new lengths int32 [B] (``out``, which may be lens; -1 where a path,
    length or page is out of range)."""
    device = _device(lens, "lens", I32, 1)
    B = lens.shape[0]
    _check(path, "path", I32, 2, device)
    _check(n_keep, "n_keep", I32, 1, device)
    rows, A = path.shape
    if rows != B or n_keep.shape[0] != B:
        raise ValueError("path must be [B, A] and n_keep [B]")
    klay, _, Lmax, max_pages, page, n_pages, Hkv, d = _cache(kcache, vcache, block_table, device, B)
    call = _Call(device, stream)
    if out is None:
        out = call.own(torch.empty_like(lens))
    else:
        _check(out, "out", I32, 1, device)
        if out.shape[0] != B:
            raise ValueError("out must be [B]")
    call("wp_kv_compact", kcache.data_ptr(), klay, vcache.data_ptr(), lens.data_ptr(), path.data_ptr(), A, n_keep.data_ptr(), out.data_ptr(),
         Lmax, _ptr(block_table), max_pages, page, n_pages, B, Hkv, d)
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
    device = _device(refs, "refs", I32, 1)
    _check(block_table, "block_table", I32, 2, device)
    B, max_pages = block_table.shape
    for t, name in ((lens, "lens"), (parent, "parent"), (keep, "keep"), (new_lens, "new_lens")):
        _check(t, name, I32, 1, device)
        if t.shape[0] != B:
            raise ValueError(f"{name} must be [B]")
    call = _Call(device, stream)
    n = refs.shape[0]
    refs_out, table_out, lens_out = torch.empty_like(refs), torch.empty_like(block_table), torch.empty_like(lens)
    copies, info = lens.new_empty((B, 3)), lens.new_empty(4)
    if workspace is None:
        ws = _load().wp_pages_update_workspace_bytes(B, n)
        workspace = call.own(lens.new_empty(ws // 4))
    else:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the same device")
        ws = workspace.numel() * workspace.element_size()
    if call.elsewhere:
        for t in (refs_out, table_out, lens_out, copies, info):
            call.own(t)
    call("wp_pages_update", refs.data_ptr(), block_table.data_ptr(), lens.data_ptr(), parent.data_ptr(), keep.data_ptr(),
         new_lens.data_ptr(), refs_out.data_ptr(), table_out.data_ptr(), lens_out.data_ptr(), copies.data_ptr(), info.data_ptr(), B,
         max_pages, int(page_size), n, workspace.data_ptr(), ws)
    return refs_out, table_out, lens_out, copies, info



def wp_pages_copy(k_pages: torch.Tensor, v_pages: torch.Tensor, copies: torch.Tensor, stream=None) -> None:
    """Copy rows between pages of a K and a V pool: copies int32 [n,3] (device),
    each source page, target page, rows; entries of -1 copy nothing."""
    device = _device(copies, "copies", I32, 2)
    n, width = copies.shape
    if width != 3:
        raise ValueError("copies must be [n, 3]")
    klay, _, _, _, page, n_pages, Hkv, d = _cache(k_pages, v_pages, copies, device)
    _Call(device, stream)("wp_pages_copy", k_pages.data_ptr(), klay, v_pages.data_ptr(), copies.data_ptr(), n, n_pages, page, Hkv, d)
