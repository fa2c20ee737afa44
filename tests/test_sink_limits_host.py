"""CPU check that sizes whose launches would not fit 31 bits are refused as unsupported
by both directions, before any of them is launched."""

import pytest

UNSUPPORTED, BF16 = -2, 1


@pytest.mark.parametrize("batch,heads,n", [(1, 32, 900_000_000), (60_000, 7, 65_500), (1, 13, 2_140_000_000)])
@pytest.mark.parametrize("window,sinks", [(28, 4), (4096, 4)])  # all rows see few keys, or not
def test_rows_beyond_the_grid(built_lib, batch, heads, n, window, sinks):
    shape = (batch, heads, 1, n, 64, window, sinks, BF16)
    rows = batch * heads * (n + 127)
    blocks = rows // 64 + (rows // 16 if window + sinks <= 32 else 0)
    assert blocks > 2 ** 31 - 1 or window + sinks > 32
    assert built_lib.nb_attn_sink_fwd(16, 16, 16, 16, None, None, *shape, None) == UNSUPPORTED
    assert built_lib.nb_attn_sink_bwd_workspace_size(*shape) == 0
    assert built_lib.nb_attn_sink_bwd(*[16] * 6, None, *[16] * 3, 256, 2 ** 60, *shape, None) == UNSUPPORTED


def test_rows_that_fit(built_lib):
    """The largest the limit lets through fill a grid of 31 bits."""
    n = 2_000_000_000
    assert built_lib.nb_attn_sink_bwd_workspace_size(1, 13, 1, n, 64, 28, 4, BF16) > 0
    assert 13 * (n + 127) // 64 + 13 * (n + 127) // 16 < 2 ** 31
