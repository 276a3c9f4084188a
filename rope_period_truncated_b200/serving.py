"""Rotary, cache-append, tree-attention, compaction and page calls (the second
half of ``include/waveprune.h``), with the package module's checks and errors.
These calls last a few microseconds on the device at their smallest, so those
with tensors are marshalled by a compiled module (``csrc/wp_torch.cpp``): a
rotation of 256 tokens takes 5.6 us a call, 15 us when marshalled in Python.

A K/V cache is given by its two tensors and, when paged, a block table:
contiguous V [B,Hkv,Lmax,d] with K the same (rows) or [B,Hkv,d/16,Lmax,16]
(group-major); paged V [n_pages,Hkv,P,d] with K the same or
[n_pages,Hkv,d/16,P,16] and ``block_table`` int32 [B,max_pages] (device).

Calls run on ``stream``, or on the current stream of the tensors' device. With
a ``stream``, the caller lets it wait for what makes the inputs, keeps the
inputs until it has read them, and waits for it before using the results, which
are allocated on ``stream`` and may be used and dropped on the current one.
"""
from __future__ import annotations

import ctypes
import os
from array import array

import numpy as np
import torch

P, I, D, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_float, ctypes.c_size_t

PAGES_OK, PAGES_SHORT, PAGES_BAD_ARGUMENT = range(3)
TREE_MAX_NODES = 64

SIGNATURES = {
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

# what the compiled module calls
DEVICE_CALLS = ("wp_rope_qk", "wp_rope_append", "wp_decode_tree_workspace_bytes", "wp_decode_tree", "wp_kv_compact",
                "wp_pages_update_workspace_bytes", "wp_pages_update", "wp_pages_copy")
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


class _Native:
    """The compiled module; loaded and given the library's functions when the first call is looked up."""

    def __getattr__(self, name):
        lib = _load()
        from . import WavePruneError
        try:
            from . import _calls
        except ImportError as e:
            from . import build
            why = f"does not load ({e})" if os.path.exists(build.BINDING) else "not built"
            raise ImportError(f"_calls.so {why}; run python -m rope_period_truncated_b200.build --force") from e
        _calls.connect({f: ctypes.cast(getattr(lib, f), P).value for f in DEVICE_CALLS}, WavePruneError)
        for f in ("rope_qk", "rope_append", "decode_tree", "kv_compact", "pages_update", "pages_copy"):
            setattr(self, f, getattr(_calls, f))
        return getattr(_calls, name)


_native = _Native()


def _fail(name, code):
    from rope_period_truncated_b200 import WavePruneError
    raise WavePruneError(name, code)


def _freqs(scale, n):
    """(what keeps the values alive, their address)"""
    if scale is None:
        return None, None
    a = array("d", scale.tolist() if hasattr(scale, "tolist") else scale)
    if len(a) != n:
        raise ValueError(f"freq_scale must have {n} entries (rot_dim/2)")
    return a, a.buffer_info()[0]


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
    return _native.rope_qk(q, k, theta, layout, pos, pos0, rot_dim, freq_scale, scale_all, amplitude, inverse, out_q, out_k, stream)


def wp_rope_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                   pos: torch.Tensor, seq: torch.Tensor, slot: torch.Tensor, theta: float, layout: int,
                   block_table: torch.Tensor | None = None, rot_dim: int | None = None, freq_scale=None,
                   scale_all: float = 1.0, amplitude: float = 1.0, out_q: torch.Tensor | None = None, stream=None):
    """Rotate the new tokens' q [T,Hq,d] (or None) and k [T,Hkv,d] by pos [T]
    and write k and v [T,Hkv,d] into key slot[i] of sequence seq[i] of the
    cache (int32 [T], device; seq -1 = padding). Returns the rotated q."""
    return _native.rope_append(q, k, v, kcache, vcache, pos, seq, slot, theta, layout, block_table, rot_dim, freq_scale, scale_all,
                               amplitude, out_q, stream)


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
    return _native.decode_tree(q, kcache, vcache, lens, parents, n_nodes, block_table, group_cut, softmax_scale, out, lse, workspace,
                               want_lse, stream)


def wp_kv_compact(kcache: torch.Tensor, vcache: torch.Tensor, lens: torch.Tensor, path: torch.Tensor, n_keep: torch.Tensor,
                  block_table: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """Move the rows of key lens[b] + path[b,i] to key lens[b] + i, i <
    n_keep[b] (int32 [B,A] increasing, int32 [B]; device), in place. Returns
    the new lengths int32 [B] (``out``, which may be lens; -1 where a path,
    length or page is out of range)."""
    return _native.kv_compact(kcache, vcache, lens, path, n_keep, block_table, out, stream)


def wp_pages_update(refs: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, parent: torch.Tensor,
                    keep: torch.Tensor, new_lens: torch.Tensor, page_size: int, workspace: torch.Tensor | None = None,
                    stream=None):
    """One transaction on the pages of a batch (fork, grow, copy on write,
    free): row b goes on from row parent[b] with its first keep[b] tokens and
    room for new_lens[b]. All int32 on the device: refs [n_pages], block_table
    [B,max_pages], the others [B]. Returns new tensors (refs, block_table,
    lens, copies [B,3], info [4]); info[0] is PAGES_OK, or PAGES_SHORT /
    PAGES_BAD_ARGUMENT with everything as it was."""
    return _native.pages_update(refs, block_table, lens, parent, keep, new_lens, page_size, workspace, stream)


def wp_pages_copy(k_pages: torch.Tensor, v_pages: torch.Tensor, copies: torch.Tensor, stream=None) -> None:
    """Copy rows between pages of a K and a V pool: copies int32 [n,3] (device),
    each source page, target page, rows; entries of -1 copy nothing."""
    _native.pages_copy(k_pages, v_pages, copies, stream)
