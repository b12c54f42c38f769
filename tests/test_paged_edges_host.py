"""Paged cache, without a GPU: the ends of the ranges, what the binding keeps
between calls, and the host-side parts of the kernels' bookkeeping (every
pointer below is fake and never dereferenced).
"""

import ctypes

from test_paged_host import _attend, _desc, _lib


def test_rows_that_a_loop_of_32_bits_cannot_count_are_refused():
    """Sq * Hq from 2^31 - 2^15 on: a row index steps past its last value."""
    b, L = _lib()
    for Sq, Hq in ((16383, 131079), (13902, 154473), (16383, 131088)):
        assert (1 << 31) - (1 << 15) <= Sq * Hq
        d = _desc(b, B=1, Sq=Sq, Hq=Hq, d=32)
        assert L.pi_attn_paged_workspace_bytes(ctypes.byref(d)) == 0
        assert _attend(L, d) == b.PI_ERR_UNSUPPORTED
