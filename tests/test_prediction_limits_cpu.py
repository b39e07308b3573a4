"""Where the limits of rotary positions, attention with decay and the loss over a table's
rows lie, without a GPU."""
from sparse_spatial_hashing_amd import prediction

LIB = prediction._lib
EINVAL = -1


def test_rotation_refuses_pairs_past_64_bits():
    """As many pairs as overflow their number of elements; no tokens, so that nothing is read."""
    for axes, pairs in ((1, 2**62), (2, 2**61), (2, 2**61 + 4), (3, 2**62), (1, 2**63 - 1), (3, (2**64 + 8) // 6)):
        assert LIB.tok_rotate(None, 0, 4, 64, 256, 64, 1, None, axes, 1, axes, None, pairs, 0, 0, None, None) == EINVAL, \
            (axes, pairs)
    for axes, pairs in ((1, 32), (2, 16), (3, 10)):
        assert LIB.tok_rotate(None, 0, 4, 64, 256, 64, 1, None, axes, 1, axes, None, pairs, 0, 0, None, None) == 0
