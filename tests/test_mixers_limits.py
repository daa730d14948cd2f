"""The sizes at which the linear, prompt and cache entry points begin to refuse a call, on the CPU:
sizes are checked before pointers, so a call without q is refused for its NULL where the sizes
are in range, and for its sizes where they are not.  Nothing is launched either way."""
import pytest

from tests.test_abi import BF16, ERR_NULL, ERR_SHAPE, F32, L  # noqa: F401
from tests.test_mixers_abi import lin_fwd

# B * H workgroups of two slices of 64 value columns: 512 threads each with bf16, 384 with fp32, below 2^32 in all
MOST = {BF16: (1 << 22) - 1, F32: (1 << 32) // 768}


@pytest.mark.parametrize("it", [BF16, F32])
def test_linear_forward_launch_bound(L, it):  # noqa: F811
    few = dict(it=it, T=1, H=1, dk=16, S_in=None, S_out=None, q=None)
    assert lin_fwd(L, B=MOST[it], dv=128, **few) == ERR_NULL
    assert lin_fwd(L, B=MOST[it] + 1, dv=128, **few) == ERR_SHAPE
    assert lin_fwd(L, B=(1 << 23) - 1, dv=128, **few) == ERR_SHAPE
    assert lin_fwd(L, B=(1 << 23) - 1, dv=64, **few) == ERR_NULL
