"""CPU test of the largest table that fattn_kv_fork takes."""
from tests.test_search_boundary import UNSUPPORTED, fork, lib  # noqa: F401


def test_tables_beyond_32_bits_are_refused(lib):  # noqa: F811
    """The pages that all sequences lack, at most B max_pages, are added up in 32
    bits, and the sum is where in the list of free pages a sequence's begin."""
    for B, cols in ((1 << 17, 1 << 14), (2, 1 << 26), (1 << 26, 32)):
        got = fork(lib, B=B, max_pages=cols, row=cols, orow=cols)
        assert (got == UNSUPPORTED) == (B * cols > 2 ** 31 - 1)
