"""Sizes at the limits of the few-token operators, without a GPU: what the kernels' 32-bit
indexes cannot hold is refused before any device call."""

import pytest

from test_few_refusals import UNSUPPORTED, lib, mem  # noqa: F401  (fixtures)


@pytest.mark.parametrize("d,refused", [(2**31 - 264, True), (2**31 - 2048, True), (2**31 - 8184, True),
                                       (2**31 - 8192, False)])
def test_route_columns_stay_in_32_bits(lib, mem, d, refused):  # noqa: F811
    """The column loop steps by up to 2048 columns, two steps at a time, past the last one."""
    x, w, i, g, ws = mem[:5]
    # the regions are far smaller than such an x: what is not refused for its size is refused for overlaps
    st = lib.dg_moe_route(1, d, 8, 2, 0, 1.0, x, w, i, g, ws, 1 << 16, None)
    assert st != 0 and (st == UNSUPPORTED) == refused, lib.dg_last_error()
