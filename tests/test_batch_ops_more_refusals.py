"""More that the calls of several sequences refuse on the host, before any launch
(no GPU needed)."""

import pytest

from tests.test_batch_ops_refusals import ATTN, INVALID, lib  # noqa: F401


@pytest.mark.parametrize("scale", [2.5e38, -2.5e38, 3.4e38, float("inf"), float("-inf")])
def test_scales_whose_multiple_of_log2_e_is_not_finite(lib, scale):  # noqa: F811
    assert lib.ssd_op_cache_attention(*{**ATTN, "scale": scale}.values()) == INVALID
    assert b"scale" in lib.ssd_ops_last_error()
    # (2^127 passes that check: the workspace's size is the next refusal)
    assert lib.ssd_op_cache_attention(*{**ATTN, "scale": 2.0 ** 127, "ws_bytes": 0}.values()) == 3
