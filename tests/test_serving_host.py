"""Host checks of the rotary, cache-append, tree-attention, compaction and
page calls: bad arguments are refused before anything is launched, and the
host-only calls follow their formulas. No GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import rope_period_truncated_b200 as wp
from rope_period_truncated_b200 import build as wpbuild

FAKE = 1 << 20  # aligned, never dereferenced: every call below is refused
ARG, UNSUPPORTED = wp.WP_ERR_ARG, wp.WP_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    wpbuild.build()
    return wp.load_library()


def _expect(f, good, bad):
    for change, code, why in bad:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert f(*args) == code, why


def rows(data, sb, sn, sh):
    return (ctypes.c_int64 * 4)(data, sb, sn, sh)


# ------------------------------------------------------------------ host calls

@pytest.mark.parametrize("d,theta,layout,scale", [(64, 1e4, 0, 1.0), (128, 1e6, 1, 1.0), (128, 1e6, 0, 0.25), (64, 1e4, 1, 0.25)])
def test_partial_cutoffs_of_a_whole_head_are_the_cutoffs(lib, d, theta, layout, scale):
    a = wp.wp_cutoffs_partial(d, d, theta, layout, scale_all=scale)
    b = oracle.cutoffs(d, theta, layout, scale_all=scale)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("d,rot,layout", [(128, 64, 0), (128, 64, 1), (128, 48, 1), (64, 16, 0), (64, 16, 1), (128, 112, 1)])
def test_partial_cutoffs_follow_the_rotated_dims(lib, d, rot, layout):
    chan, group = wp.wp_cutoffs_partial(d, rot, 1e4, layout)
    w = [min(2 ** 31 - 1, math.floor(2 * math.pi * 1e4 ** (2.0 * c / rot))) for c in range(rot // 2)]
    assert np.array_equal(chan, w)
    for g in range(d // 16):
        dims = range(16 * g, 16 * g + 16)
        expect = max(w[k // 2 if layout == 0 else k % (rot // 2)] if k < rot else 2 ** 31 - 1 for k in dims)
        assert group[g] == expect


def test_rope_scaling_ramp(lib):
    fs, amp = wp.wp_rope_scaling(128, 1e6, 4.0, 32768)
    assert amp == pytest.approx(0.1 * math.log(4.0) + 1.0, rel=1e-15)
    turns = 32768 * 1e6 ** (-2.0 * np.arange(64) / 128) / (2 * math.pi)
    assert (fs[turns >= 32] == 1.0).all() and np.allclose(fs[turns <= 1], 0.25, rtol=1e-15)
    assert (np.diff(fs) <= 0).all() and ((fs >= 0.25) & (fs <= 1.0)).all()
    assert ((turns > 1) & (turns < 32)).any()
    mid = (turns > 1) & (turns < 32)
    keep = (turns[mid] - 1) / 31
    assert np.allclose(fs[mid], (1 - keep) / 4 + keep, rtol=1e-12)
    one, amp1 = wp.wp_rope_scaling(64, 1e4, 1.0, 4096)
    assert (one == 1.0).all() and amp1 == 1.0


def test_host_calls_reject_bad_arguments(lib):
    out = np.zeros(512, dtype=np.float64)
    p = out.ctypes.data
    _expect(lib.wp_cutoffs_partial, [128, 64, 1e4, None, 1.0, 2.0, 0, p, p], [
        ({1: 8}, ARG, "rot_dim below 16"), ({1: 40}, ARG, "rot_dim not a multiple of 16"), ({1: 144}, ARG, "rot_dim above d_h"),
        ({0: 100}, ARG, "d_h"), ({2: 1.0}, ARG, "theta"), ({4: 0.0}, ARG, "scale"), ({5: 0.0}, ARG, "alpha"),
        ({6: 2}, ARG, "the paired layout is interleaved here")])
    nan = float("nan")
    _expect(lib.wp_rope_scaling, [128, 1e6, 4.0, 4096, 1.0, 32.0, p, p], [
        ({0: 8}, ARG, "rot_dim"), ({1: 1.0}, ARG, "theta"), ({2: 0.5}, ARG, "factor below 1"), ({2: nan}, ARG, "factor"),
        ({3: 0}, ARG, "length"), ({4: 32.0}, ARG, "empty ramp"), ({4: -1.0}, ARG, "negative turns"), ({5: nan}, ARG, "turns"),
        ({6: None}, ARG, "no output"), ({7: None}, ARG, "no amplitude")])


# ---------------------------------------------------------------------- rotary

def test_rope_qk_rejects_bad_arguments(lib):
    B, N, Hq, Hk, d = 2, 5, 4, 2, 128
    q, qo = rows(FAKE, N * Hq * d, Hq * d, d), rows(FAKE + (1 << 20), N * Hq * d, Hq * d, d)
    k, ko = rows(FAKE + (2 << 20), N * Hk * d, Hk * d, d), rows(FAKE + (3 << 20), N * Hk * d, Hk * d, d)
    good = [q, qo, Hq, k, ko, Hk, B, N, d, d, None, 0, 1e4, None, 1.0, 1.0, 0, 0, None]
    bad = [
        ({0: None}, ARG, "no q"), ({1: None}, ARG, "no output"), ({2: -1}, ARG, "heads"), ({2: 0, 5: 0}, ARG, "nothing to do"),
        ({6: 0}, ARG, "B"), ({7: 0}, ARG, "N"), ({8: 96, 9: 96}, UNSUPPORTED, "d_h"), ({8: 100}, ARG, "d_h"),
        ({9: 24}, ARG, "rot_dim"), ({9: 144}, ARG, "rot_dim"), ({10: FAKE + 2}, ARG, "positions misaligned"), ({12: 1.0}, ARG, "theta"),
        ({14: 0.0}, ARG, "scale"), ({15: float("inf")}, ARG, "amplitude"), ({16: 3}, ARG, "layout"),
        ({2: 1 << 17}, UNSUPPORTED, "heads"), ({6: 1 << 16, 7: 1 << 16}, UNSUPPORTED, "tokens"),
        ({0: rows(FAKE + 8, N * Hq * d, Hq * d, d)}, ARG, "q misaligned"),
        ({0: rows(FAKE, N * Hq * d, Hq * d + 4, d)}, ARG, "stride not a multiple of 8"),
        ({0: rows(FAKE, -N * Hq * d, Hq * d, d)}, ARG, "negative stride"),
        ({1: rows(FAKE + (1 << 20), N * Hq * d, 0, d)}, ARG, "broadcast output"),
        ({1: rows(FAKE + (1 << 20), N * Hq * d, Hq * d, d - 8)}, ARG, "output heads overlap"),
        ({1: rows(FAKE + 64, N * Hq * d, Hq * d, d)}, ARG, "output half over its input"),
        ({4: qo}, ARG, "both outputs in one place"),
        ({1: k}, ARG, "q's output over k"),
        ({1: q, 16: 2}, ARG, "the paired layout in place"),
    ]
    _expect(lib.wp_rope_qk, good, bad)


def test_rope_qk_slices_of_one_projection(lib):
    """In place on a fused [B, N, Hq + 2 Hk, d] buffer: no overlap is seen where there is none (the call then gets as far as
    the launch, which has no GPU here), and a slice that runs into the next one is refused."""
    B, N, Hq, Hk, d = 2, 7, 4, 2, 64
    H = Hq + 2 * Hk
    at = lambda h: rows(FAKE + 2 * h * d, N * H * d, H * d, d)  # noqa: E731
    args = [at(0), at(0), Hq, at(Hq), at(Hq), Hk, B, N, d, d, None, 0, 1e4, None, 1.0, 1.0, 1, 0, None]
    if not torch.cuda.is_available():
        assert lib.wp_rope_qk(*args) == wp.WP_ERR_CUDA
    args[3] = args[4] = at(Hq - 1)
    assert lib.wp_rope_qk(*args) == ARG


def test_rope_append_rejects_bad_arguments(lib):
    T, Hq, Hkv, d, B, Lmax = 6, 4, 2, 128, 3, 100
    M = 1 << 20
    q, qo, k, v = (rows(FAKE + i * M, 0, H * d, d) for i, H in ((1, Hq), (2, Hq), (3, Hkv), (4, Hkv)))
    kc, vc = FAKE + 8 * M, FAKE + 16 * M
    good = [q, qo, Hq, k, v, Hkv, T, d, d, FAKE, FAKE, FAKE, kc, 0, vc, B, Lmax, None, 0, 0, 0, 1e4, None, 1.0, 1.0, 0, None]
    paged = {17: FAKE, 18: 4, 19: 32, 20: 50}
    _expect(lib.wp_rope_append, good, [
        ({6: 0}, ARG, "T"), ({9: None}, ARG, "positions"), ({10: None}, ARG, "sequences"), ({11: FAKE + 1}, ARG, "slots misaligned"),
        ({12: None}, ARG, "K cache"), ({12: kc + 8}, ARG, "K cache misaligned"), ({13: 2}, UNSUPPORTED, "windowed"), ({13: 3}, ARG, "layout"),
        ({15: 0}, ARG, "B"), ({16: 0}, ARG, "Lmax"), ({7: 96, 8: 96}, UNSUPPORTED, "d_h"), ({8: 20}, ARG, "rot_dim"),
        ({25: 5}, ARG, "rotation layout"), ({24: float("nan")}, ARG, "amplitude"), ({3: None}, ARG, "no k"), ({4: None}, ARG, "no v"),
        ({1: None}, ARG, "no q output"), ({14: kc}, ARG, "K and V in one cache"), ({3: rows(kc, 0, Hkv * d, d)}, ARG, "k inside the cache"),
        ({1: rows(vc, 0, Hq * d, d)}, ARG, "q's output inside the cache"), ({1: k}, ARG, "q's output over k"),
        ({1: q, 25: 2}, ARG, "paired in place"), ({16: 1 << 30, 15: 1}, ARG, "caches that overlap"), ({16: (1 << 30) + 1}, UNSUPPORTED, "Lmax"),
        ({**paged, 19: 24}, ARG, "page size"), ({**paged, 19: 8}, ARG, "page size"), ({**paged, 18: 0}, ARG, "max_pages"),
        ({**paged, 20: 0}, ARG, "n_pages"), ({**paged, 17: FAKE + 2}, ARG, "block table misaligned"),
        ({**paged, 18: 1 << 26, 19: 32}, UNSUPPORTED, "capacity")])


# ------------------------------------------------------------------------ tree

def test_decode_tree_rejects_bad_arguments(lib):
    T, B, Hq, Hkv, d, Lmax = 8, 2, 8, 2, 128, 5000
    ws = lib.wp_decode_tree_workspace_bytes(B, T, Hq, Hkv, d, Lmax)
    cut = (ctypes.c_int32 * 8)(*([5] * 7 + [-1]))
    good = [FAKE, FAKE, 0, FAKE, FAKE, FAKE, None, T, Lmax, None, 0, 0, 0, B, Hq, Hkv, d, None, 0.0, FAKE, None, FAKE, ws, None]
    paged = {9: FAKE, 10: 8, 11: 64, 12: 30}
    assert ws > 0
    _expect(lib.wp_decode_tree, good, [
        ({0: None}, ARG, "q"), ({0: FAKE + 8}, ARG, "q misaligned"), ({1: None}, ARG, "K"), ({3: None}, ARG, "V"), ({4: None}, ARG, "lens"),
        ({4: FAKE + 2}, ARG, "lens misaligned"), ({5: None}, ARG, "parents"), ({5: FAKE + 1}, ARG, "parents misaligned"),
        ({6: FAKE + 2}, ARG, "n_nodes misaligned"), ({2: 2}, UNSUPPORTED, "windowed"), ({2: 9}, ARG, "K layout"), ({7: 0}, ARG, "T"),
        ({7: 65}, UNSUPPORTED, "T above 64"), ({8: 0}, ARG, "Lmax"), ({13: 0}, ARG, "B"), ({14: 7}, ARG, "heads"), ({15: 0}, ARG, "KV heads"),
        ({14: 34, 15: 2}, UNSUPPORTED, "17 query heads per KV head"), ({16: 96}, UNSUPPORTED, "d_h"), ({16: 20}, ARG, "d_h"),
        ({17: ctypes.addressof(cut)}, ARG, "negative cutoff"), ({18: float("nan")}, ARG, "scale"), ({19: None}, ARG, "o"),
        ({19: FAKE + 8}, ARG, "o misaligned"), ({20: FAKE + 2}, ARG, "lse misaligned"), ({21: None}, ARG, "workspace"),
        ({21: FAKE + 128}, ARG, "workspace misaligned"), ({22: ws - 1}, ARG, "workspace too small"),
        ({**paged, 11: 24}, ARG, "page size"), ({**paged, 12: 0}, ARG, "pool"), ({**paged, 10: 1 << 25}, UNSUPPORTED, "capacity")])
    assert lib.wp_decode_tree_workspace_bytes(B, T, Hq, Hkv, d, 500) == 0  # short caches need none
    for change in ((0, 0), (1, 0), (1, 65), (2, 0), (3, 0), (4, 0), (5, 0)):
        args = [B, T, Hq, Hkv, d, Lmax]
        args[change[0]] = change[1]
        assert lib.wp_decode_tree_workspace_bytes(*args) == 0


# --------------------------------------------------------------------- compact

def test_kv_compact_rejects_bad_arguments(lib):
    good = [FAKE, 0, FAKE, FAKE, FAKE, 8, FAKE, FAKE, 100, None, 0, 0, 0, 2, 2, 128, None]
    _expect(lib.wp_kv_compact, good, [
        ({0: None}, ARG, "K"), ({2: FAKE + 4}, ARG, "V misaligned"), ({1: 2}, UNSUPPORTED, "windowed"), ({3: None}, ARG, "lens"),
        ({4: None}, ARG, "path"), ({4: FAKE + 2}, ARG, "path misaligned"), ({5: 0}, ARG, "A"), ({5: 1025}, UNSUPPORTED, "A"),
        ({6: None}, ARG, "n_keep"), ({7: None}, ARG, "lens_out"), ({8: 0}, ARG, "Lmax"), ({13: 0}, ARG, "B"), ({14: 0}, ARG, "heads"),
        ({15: 80}, UNSUPPORTED, "d_h"), ({9: FAKE, 10: 2, 11: 17, 12: 4}, ARG, "page size")])


# ----------------------------------------------------------------------- pages

def test_pages_update_rejects_bad_arguments(lib):
    B, MP, P, n = 4, 10, 16, 100
    ws = lib.wp_pages_update_workspace_bytes(B, n)
    at = [FAKE + i * (1 << 16) for i in range(12)]
    good = at[:11] + [B, MP, P, n, at[11], ws, None]
    bad = [({i: None}, ARG, f"pointer {i}") for i in range(11)] + [({i: at[i] + 2}, ARG, f"pointer {i} misaligned") for i in range(11)]
    bad += [({11: 0}, ARG, "B"), ({12: 0}, ARG, "max_pages"), ({13: 8}, ARG, "page size"), ({13: 24}, ARG, "page size"), ({14: 0}, ARG, "pool"),
            ({15: None}, ARG, "workspace"), ({15: at[11] + 4}, ARG, "workspace misaligned"), ({16: ws - 1}, ARG, "workspace too small"), ({12: 1 << 27}, UNSUPPORTED, "capacity"),
            ({6: at[0]}, ARG, "counts in place"), ({7: at[1]}, ARG, "table in place"), ({8: at[2]}, ARG, "lengths in place"),
            ({9: at[7] + 4 * B * MP - 4}, ARG, "copies inside the table"), ({15: at[6]}, ARG, "workspace over an output")]
    _expect(lib.wp_pages_update, good, bad)
    assert lib.wp_pages_update_workspace_bytes(0, n) == 0 and lib.wp_pages_update_workspace_bytes(B, 0) == 0


def test_pages_copy_rejects_bad_arguments(lib):
    good = [FAKE, 0, FAKE, FAKE, 4, 100, 16, 2, 128, None]
    _expect(lib.wp_pages_copy, good, [
        ({0: None}, ARG, "K"), ({2: None}, ARG, "V"), ({3: None}, ARG, "copies"), ({3: FAKE + 2}, ARG, "copies misaligned"), ({4: 0}, ARG, "n"),
        ({5: 0}, ARG, "pool"), ({6: 20}, ARG, "page size"), ({7: 0}, ARG, "heads"), ({8: 96}, UNSUPPORTED, "d_h"), ({1: 2}, UNSUPPORTED, "windowed"),
        ({1: -1}, ARG, "layout")])


# ----------------------------------------------------------- the Python binding

def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        wp.wp_rope_qk(x, x, 1e4, 0)
    with pytest.raises(ValueError):
        wp.wp_rope_qk(None, None, 1e4, 0)
    with pytest.raises(TypeError):
        wp.wp_rope_append(None, x[0], x[0], x, x, i, i, i, 1e4, 0)
    with pytest.raises(TypeError):
        wp.wp_decode_tree(x, x, x, i, i)
    with pytest.raises(TypeError):
        wp.wp_kv_compact(x, x, i, i, i)
    with pytest.raises(TypeError):
        wp.wp_pages_update(i, i, i, i, i, i, 16)
    with pytest.raises(TypeError):
        wp.wp_pages_copy(x, x, i)


# --------------------------------------------------------- arguments that meet

def test_outputs_that_meet_other_arguments_are_refused(lib):
    """What one block writes while another still reads it."""
    M = 1 << 24
    at = [FAKE + i * M for i in range(12)]
    B, T, Hq, Hkv, d, Lmax, A = 2, 8, 8, 2, 128, 5000, 8
    q, kc, vc, lens, parents, nodes, o, lse, ws = at[:9]
    need = lib.wp_decode_tree_workspace_bytes(B, T, Hq, Hkv, d, Lmax)
    tree = [q, kc, 0, vc, lens, parents, nodes, T, Lmax, None, 0, 0, 0, B, Hq, Hkv, d, None, 0.0, o, lse, ws, need, None]
    oq, cache = B * T * Hq * d * 2, B * Hkv * Lmax * d * 2
    _expect(lib.wp_decode_tree, tree, [
        ({19: q}, ARG, "o over q"), ({19: q + oq - 16}, ARG, "o into q's end"), ({19: vc + cache - 16}, ARG, "o in V"), ({20: lens}, ARG, "lse over lens"),
        ({20: o + oq - 4}, ARG, "lse in o"), ({21: kc}, ARG, "workspace in K"), ({21: parents}, ARG, "workspace over parents"),
        ({21: lse}, ARG, "workspace over lse"), ({20: nodes}, ARG, "lse over the node counts"),
        ({9: at[9], 10: 4, 11: 64, 12: 9, 20: at[9] + 28}, ARG, "lse over the block table"), ({18: 3e38}, ARG, "a scale beyond 32 bits")])
    path, keep, out = at[4], at[5], at[6]
    compact = [kc, 0, vc, lens, path, A, keep, out, 100, None, 0, 0, 0, B, Hkv, d, None]
    _expect(lib.wp_kv_compact, compact, [
        ({7: path + 4 * A}, ARG, "lens_out in path"), ({7: keep}, ARG, "lens_out over n_keep"), ({7: lens + 4}, ARG, "lens_out beside lens"),
        ({2: kc}, ARG, "K and V in one pool"), ({2: kc + 16}, ARG, "K and V overlap"), ({3: kc}, ARG, "lens in K")])
    _expect(lib.wp_pages_copy, [kc, 0, vc, lens, 4, 100, 16, Hkv, d, None], [({2: kc}, ARG, "K and V in one pool"), ({3: vc + 64}, ARG, "copies in V")])
    if not torch.cuda.is_available():  # as far as the launch, which has no GPU here
        assert lib.wp_kv_compact(*(compact[:7] + [lens] + compact[8:])) == wp.WP_ERR_CUDA


def test_limits_of_the_page_transaction(lib):
    M = 1 << 40
    at = [FAKE + i * M for i in range(12)]
    for B, n in ((65536, 100), (4, (1 << 30) + 1)):
        assert lib.wp_pages_update(*at[:11], B, 10, 16, n, at[11], lib.wp_pages_update_workspace_bytes(B, n), None) == UNSUPPORTED


def test_an_amplitude_beyond_32_bits_is_refused(lib):
    q, qo = rows(FAKE, 256, 128, 64), rows(FAKE + (1 << 20), 256, 128, 64)
    assert lib.wp_rope_qk(q, qo, 2, None, None, 0, 1, 2, 64, 64, None, 0, 1e4, None, 1.0, 1e39, 0, 0, None) == ARG
