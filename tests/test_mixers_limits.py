"""The sizes at which the linear, prompt and cache entry points begin to refuse a call, on the CPU:
sizes are checked before pointers, so a call without q is refused for its NULL where the sizes
are in range, and for its sizes where they are not.  Nothing is launched either way."""
import pytest

from tests.test_abi import BF16, ERR_NULL, ERR_SHAPE, F32, L  # noqa: F401
from tests.test_mixers_abi import lin_bwd, lin_fwd

# B * H workgroups of two slices of 64 value columns: 512 threads each with bf16, 384 with fp32, below 2^32 in all
MOST = {BF16: (1 << 22) - 1, F32: (1 << 32) // 768}


@pytest.mark.parametrize("it", [BF16, F32])
def test_linear_forward_launch_bound(L, it):  # noqa: F811
    few = dict(it=it, T=1, H=1, dk=16, S_in=None, S_out=None, q=None)
    assert lin_fwd(L, B=MOST[it], dv=128, **few) == ERR_NULL
    assert lin_fwd(L, B=MOST[it] + 1, dv=128, **few) == ERR_SHAPE
    assert lin_fwd(L, B=(1 << 23) - 1, dv=128, **few) == ERR_SHAPE
    assert lin_fwd(L, B=(1 << 23) - 1, dv=64, **few) == ERR_NULL


@pytest.mark.parametrize("it", [BF16, F32])
def test_linear_backward_launch_bound(L, it):  # noqa: F811
    """One token each: a head's walks bound the launches, whichever of dk and dv they go over; a longer
    sequence's blocks (of 256 or 128 tokens) do."""
    one = dict(it=it, T=1, H=1, q=None)
    for dk, dv in ((16, 128), (128, 16), (128, 128)):
        assert lin_bwd(L, B=MOST[it], dkd=dk, dvd=dv, **one) == ERR_NULL
        assert lin_bwd(L, B=MOST[it] + 1, dkd=dk, dvd=dv, **one) == ERR_SHAPE
        assert L.kda_linear_chunk_bwd_workspace_bytes(MOST[it], 1, 1, dk, dv, it, 0) > 0
        assert L.kda_linear_chunk_bwd_workspace_bytes(MOST[it] + 1, 1, 1, dk, dv, it, 0) == 0
    block = 256 if it == BF16 else 128
    long = dict(it=it, T=block * 8, dkd=16, dvd=16, q=None)
    assert lin_bwd(L, B=(1 << 20) - 1, H=1, **long) == ERR_NULL
    assert lin_bwd(L, B=1 << 20, H=1, **long) == ERR_SHAPE
