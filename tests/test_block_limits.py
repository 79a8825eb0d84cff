"""Sizes that a launch of the norm's backward could not hold, on the host, with
dummy pointers that nothing reads."""
import pytest

import combine_router_top_expert_amd as mok
from test_block_abi import EINVAL, L, _cfg, _norm_bwd  # noqa: F401


@pytest.mark.parametrize("T", [0, 10, 100000])
def test_norm_bwd_refuses_rows_whose_weight_gradient_no_launch_holds(L, T):  # noqa: F811
    """d_weight takes 1024 threads for 16 columns, and a launch has fewer than 2^32 threads: refused before the first
    launch, not behind it."""
    for d in (1 << 26, (1 << 31) - 64):
        assert _norm_bwd(L, _cfg(d=d), T=T) == EINVAL
    assert mok.mok_norm_bwd_ws_bytes(_cfg(d=1 << 26), 4) > 0     # without d_weight such rows are fine
