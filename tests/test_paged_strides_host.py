"""Strides of the append's arguments (no GPU: no token, so no kernel)."""

import pytest

from test_paged_host import _append, lib  # noqa: F401

REPEATED = [0, 1024, 128]  # one sequence's rows for the whole batch


@pytest.mark.parametrize("H,status", [(0, 0), (16, -2)])
def test_strides_of_queries_count_only_with_queries(lib, H, status):  # noqa: F811
    """K and V may repeat rows; Qo, which is written, may not. Without queries their
    strides are not used."""
    some = {} if H else {"q": None, "qo": None}
    assert _append(lib, some, H=H, M=0, strides=4 * REPEATED) == status
    assert _append(lib, some, H=H, M=0, strides=3 * REPEATED + [8192, 1024, 128]) == 0
    assert _append(lib, some, H=H, M=0, strides=[4, 1024, 128] + 3 * [8192, 1024, 128]) == -6
