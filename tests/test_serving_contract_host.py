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
