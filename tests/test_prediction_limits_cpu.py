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


def test_workspaces_of_the_loss():
    """Of any number of tokens: x laid out once (a width over 128 as whole 256s) and, of gradients, once in
    float32; of the table's, sums of each 2^19 tokens (an eighth of x at most); 12 bytes a token; and what
    does not grow with them."""
    mib = 1 << 20
    for t in (1, 16, 17, 256, 257, 4096, 20000, 120000, 1 << 19, (1 << 19) + 1, 1 << 20, 3 << 20, 1 << 22, 1 << 25):
        for rows in (4, 300, 13391, 214272, 1 << 24):
            for width in (8, 40, 128, 136, 512, 1024, 4096):
                laid = 2 * t * (width + (-width % 256 if width > 128 else 0)) + 12 * t
                assert LIB.tok_row_loss_workspace_bytes(t, rows, width) <= laid + 8 * mib, (t, rows, width)
                assert LIB.tok_row_loss_grad_workspace_bytes(t, rows, width) <= \
                    laid + 4 * t * width + t * width // 4 + 768 * mib, \
                    (t, rows, width)
    # where x is small
    assert LIB.tok_row_loss_grad_workspace_bytes(1 << 20, 4, 8) < 321 * mib
    assert LIB.tok_row_loss_grad_workspace_bytes(1 << 22, 4, 8) < 513 * mib
