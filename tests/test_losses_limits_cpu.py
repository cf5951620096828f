"""Limits of the losses over sequences and of the embedding, on the host."""
import ctypes

import pytest

import linear_cross_entropy_forward_gb300 as flce
from linear_cross_entropy_forward_gb300 import _binding as B

BAD_SHAPE = 2
INT_MAX = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    from linear_cross_entropy_forward_gb300.build import build
    build()
    return flce.load_library()


def batches(pieces):
    """Batches of about as many pieces: one per row, and packed without a token."""
    yield B.FlceSeqs(B=pieces & ~1, S=1, dtype=1), pieces & ~1
    yield B.FlceSeqs(B=(pieces - 1) & ~1, S=0, cu_kind=1, cu_seqlens=0x10000, dtype=1), \
        ((pieces - 1) & ~1) + 1


@pytest.mark.parametrize("pieces", [INT_MAX, INT_MAX - 300, INT_MAX - 4864, INT_MAX - 20000,
                                    INT_MAX - 32766, INT_MAX - 32770, INT_MAX - 40000])
def test_piece_numbers_do_not_wrap(lib, pieces):
    """A warp's next piece is its last one plus the number of warps, 32 for each of up to 1024
    blocks, and a thread's next piece of a sequence 1024 further: within 32 bits in every batch
    that is taken."""
    for seqs, n in batches(pieces):
        pol = B.FlcePolicyParams(seqs=seqs, clip_low=0.2, clip_high=0.2, scale=1.0, kl=3)
        pre = B.FlcePreferenceParams(seqs=seqs, beta=0.1, reduction=1)
        want = 0 if n - 1 + 32 * 1024 <= INT_MAX - 1 else BAD_SHAPE
        assert lib.flce_policy_check_params(ctypes.byref(pol)) == want, n
        assert lib.flce_preference_check_params(ctypes.byref(pre)) == want, n


def test_a_negative_padding_row_is_refused():
    """The C struct's -1 means none; in Python that is None, and -1 is neither that nor the last
    row."""
    assert flce.embedding_params(4, 8, 10).padding_idx == -1
    assert flce.embedding_params(4, 8, 10, padding_idx=9).padding_idx == 9
    for padding in (-1, -2, -10):
        with pytest.raises(ValueError, match="padding_idx"):
            flce.embedding_params(4, 8, 10, padding_idx=padding)
