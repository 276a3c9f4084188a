"""Arguments that the serving calls' contracts exclude and that only a sum over
several of them shows: tensors that meet across tokens, index arrays inside what
is written, sizes whose products leave 32 bits. No GPU."""
import pytest
import torch

import rope_period_truncated_b200 as wp
from rope_period_truncated_b200 import build as wpbuild
from test_serving_host import ARG, FAKE, UNSUPPORTED, _expect, rows

M = 1 << 24


@pytest.fixture(scope="module")
def lib():
    wpbuild.build()
    return wp.load_library()


def _accepted(f, args):
    """As far as the launch, which has no GPU here."""
    if not torch.cuda.is_available():
        assert f(*args) == wp.WP_ERR_CUDA


# ------------------------------------------------- tensors that meet across tokens

@pytest.mark.parametrize("swap", [False, True])
def test_tensors_that_meet_across_tokens_are_refused(lib, swap):
    """One head of 64 dims each, y 64 elements after x, two batches of two tokens: 128 elements from token to token, and from
    batch to batch 192, where x of the next token's place is y's, or 256, where all lie apart. And the same with the two
    strides exchanged."""
    d = 64

    def at(where, outer, after=0):
        sb, sn = (128, outer) if swap else (outer, 128)
        return rows(where + 2 * after, sb, sn, d)

    call = lambda q, qo, k, ko: [q, qo, 1, k, ko, 1, 2, 2, d, d, None, 0, 1e4, None, 1.0, 1.0, 0, 0, None]  # noqa: E731
    far = [at(FAKE + i * M, 256) for i in range(4)]
    for outer, code in ((192, ARG), (256, None)):
        for args in (call(far[0], at(FAKE + 5 * M, outer), far[1], at(FAKE + 5 * M, outer, 64)),  # the two outputs
                     call(far[0], at(FAKE + 5 * M, outer, 64), at(FAKE + 5 * M, outer), far[1])):  # q's output and k
            if code is None:
                _accepted(lib.wp_rope_qk, args)
            else:
                assert lib.wp_rope_qk(*args) == code


# ------------------------------------------------------ index arrays and outputs

def test_index_arrays_inside_what_is_written_are_refused(lib):
    """Positions, sequences, slots and block table against the outputs and the caches, first and last element."""
    B, N, Hq, Hk, d = 2, 5, 4, 2, 64
    at = [FAKE + i * M for i in range(16)]
    q, qo = rows(at[0], N * Hq * d, Hq * d, d), rows(at[1], N * Hq * d, Hq * d, d)
    k, ko = rows(at[2], N * Hk * d, Hk * d, d), rows(at[3], N * Hk * d, Hk * d, d)
    good = [q, qo, Hq, k, ko, Hk, B, N, d, d, at[4], 0, 1e4, None, 1.0, 1.0, 0, 0, None]
    _expect(lib.wp_rope_qk, good, [
        ({10: at[1]}, ARG, "pos over q's output"), ({10: at[1] + B * N * Hq * d * 2 - 4}, ARG, "pos over its last element"),
        ({10: at[3] - B * N * 4 + 4}, ARG, "pos runs into k's output"), ({10: at[3] + B * N * Hk * d * 2 - 4}, ARG, "pos in k's output"),
        ({10: at[0], 1: q}, ARG, "pos in q rotated in place")])
    _accepted(lib.wp_rope_qk, good)
    _accepted(lib.wp_rope_qk, [{10: at[1] + B * N * Hq * d * 2}.get(i, x) for i, x in enumerate(good)])  # right behind
    _accepted(lib.wp_rope_qk, [{10: at[0]}.get(i, x) for i, x in enumerate(good)])  # in an input that nobody writes
    T, Lmax, P, MP, n = 6, 100, 16, 8, 20
    q, qo, k, v = (rows(at[i], 0, H * d, d) for i, H in enumerate((Hq, Hq, Hk, Hk)))
    pos, seq, slot, table, kc, vc = at[4:10]
    good = [q, qo, Hq, k, v, Hk, T, d, d, pos, seq, slot, kc, 0, vc, B, Lmax, None, 0, 0, 0, 1e4, None, 1.0, 1.0, 0, None]
    paged = {17: table, 18: MP, 19: P, 20: n}
    bytes_of = {"contiguous": B * Hk * Lmax * d * 2, "paged": n * Hk * P * d * 2}
    bad = []
    for name, i in (("pos", 9), ("seq", 10), ("slot", 11)):
        for where, first, size in (("q's output", at[1], T * Hq * d * 2), ("K", kc, bytes_of["contiguous"]), ("V", vc, bytes_of["contiguous"])):
            bad += [({i: first}, ARG, f"{name} over {where}"), ({i: first + size - 4}, ARG, f"{name} over the end of {where}"),
                    ({i: first - 4 * T + 4}, ARG, f"{name} runs into {where}")]
    for first, size in ((at[1], T * Hq * d * 2), (kc, bytes_of["paged"]), (vc, bytes_of["paged"])):
        bad += [({**paged, 17: first}, ARG, "block table over it"), ({**paged, 17: first + size - 4}, ARG, "block table over its end"),
                ({**paged, 17: first - B * MP * 4 + 4}, ARG, "block table runs into it")]
    _expect(lib.wp_rope_append, good, bad)
    _accepted(lib.wp_rope_append, good)
    _accepted(lib.wp_rope_append, [paged.get(i, x) for i, x in enumerate(good)])
    _accepted(lib.wp_rope_append, [{9: pos, 10: seq, 11: pos}.get(i, x) for i, x in enumerate(good)])  # one array for both


# -------------------------------------------------------- sizes beyond 32 bits

def test_a_block_table_beyond_32_bits_is_refused(lib):
    """The pages that all rows need together stay within 32 bits: a table of 2^31 entries or more is not taken, one of
    2^31 - 32 is."""
    at = [FAKE + (i << 40) for i in range(12)]
    n = 100
    call = lambda B, MP: lib.wp_pages_update(*at[:11], B, MP, 16, n, at[11], lib.wp_pages_update_workspace_bytes(B, n), None)  # noqa: E731
    for B, MP in ((32, 1 << 26), (65535, 1 << 26), (65535, 32769), (1 << 15, 1 << 16)):
        assert call(B, MP) == UNSUPPORTED
    if not torch.cuda.is_available():
        assert call(32, (1 << 26) - 1) == wp.WP_ERR_CUDA and call(65535, 32768) == wp.WP_ERR_CUDA


def test_page_copies_beyond_32_bits_are_refused(lib):
    """The pieces of a page are counted in 32 bits: pages of 2^27 rows of 128 would have copied nothing."""
    call = lambda P, d: lib.wp_pages_copy(FAKE, 0, FAKE + (1 << 50), FAKE + (1 << 52), 4, 2, P, 1, d, None)  # noqa: E731
    for P, d in ((1 << 27, 128), (1 << 28, 64), ((1 << 26) + 16, 128), (1 << 30, 64)):
        assert call(P, d) == UNSUPPORTED
    if not torch.cuda.is_available():
        assert call(1 << 26, 128) == call(1 << 27, 64) == wp.WP_ERR_CUDA
