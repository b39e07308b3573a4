"""Where the limits of rotary positions, attention with decay and the loss over a table's
rows lie, without a GPU."""
import ctypes

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
    for t, rows, width in ((64, 487505351, 59096), (257, 1 << 24, 65536), (4096, 214272, 32768), (16, 1 << 20, 65536)):
        assert LIB.tok_row_loss_grad_workspace_bytes(t, rows, width) <= 7 * t * (width + 256) + 3 * 768 * mib
    # where x is small
    assert LIB.tok_row_loss_grad_workspace_bytes(1 << 20, 4, 8) < 321 * mib
    assert LIB.tok_row_loss_grad_workspace_bytes(1 << 22, 4, 8) < 513 * mib


def _states_kept(t, docs, heads, width):
    strides = (heads * width, width)
    return LIB.tok_decay_carry_rows(ctypes.byref(prediction._Decay(
        dtype=1, heads=heads, kv_heads=heads, width=width, t=t, docs=docs, offsets=4096, decay=4096, scale=1.0,
        q_stride=strides, k_stride=strides, v_stride=strides, g_stride=strides)))


def test_more_segments_where_documents_end_in_them():
    """Twice as many where that evens out what documents' ends leave: not from a number of documents on."""
    each = lambda heads, width: 512 * 128 // width // heads
    for t, docs, heads, width in ((136000, 16, 8, 64), (163000, 16, 8, 64), (136000, 64, 8, 64), (34000, 64, 8, 64),
                                  (136000, 24, 8, 128), (136000, 256, 2, 64)):
        assert _states_kept(t, docs, heads, width) > 1.2 * each(heads, width), (t, docs, heads, width)
    for t, docs, heads, width in ((34000, 16, 8, 64), (136000, 16, 2, 64), (136000, 128, 8, 64), (136000, 4, 8, 64),
                                  (144001, 4, 8, 32), (136000, 64, 2, 64), (34000, 24, 8, 64), (100, 1, 8, 64)):
        assert _states_kept(t, docs, heads, width) <= each(heads, width), (t, docs, heads, width)
