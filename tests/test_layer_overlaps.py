"""What the matrix products and the cross attention accept in place, on the CPU: the
errors of the C ABI come before anything is launched."""
import ctypes

import pytest

from test_block_args import INVALID, lib, ptr  # noqa: F401
from test_layer_args import cross_args, tok


@pytest.mark.parametrize("rows,heads,d", [(96, 96, 64), (6, 6, 128)])
def test_output_over_transposed_queries(lib, rows, heads, d):  # noqa: F811
    """As many rows as heads: O laid out by heads over q laid out by rows names the same
    bytes, but another element's at each place."""
    q = tok(0, token_stride=heads * d, head_stride=d)
    O = tok(0, token_stride=d, head_stride=rows * d)
    for one, other in ((q, O), (O, q)):
        a = cross_args(rows=rows, rows_per_group=rows, heads=heads, kv_heads=3, head_dim=d, q=one, O=other)
        assert lib.bss_cross_attention(ctypes.byref(a), None) == INVALID
        assert b"O overlaps q" in lib.bss_last_error_message()
