"""CPU-only: calls that a launch cannot hold are refused on the host, in the
gradients of the delta rule (any HIP call comes after the checks)."""

import pytest

from tests.test_abi_layer import FAKE, L, _chunk_bwd  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(B=1, T=1 << 24, Hk=64, HV=64),                 # the chunks: 2^18 x 64 work-groups of 512
    dict(B=1, T=64, cu=FAKE, n=1 << 19, Hk=1, HV=8),    # the scans: one for each sequence, head, half and direction
    dict(B=1, T=1 << 24, Hk=1, HV=512),                 # the largest gradients: 2^20 quarters x 32 blocks of channels
])
def test_chunk_bwd_refuses_more_than_a_launch_holds(L, kw):  # noqa: F811
    assert _chunk_bwd(L, wsb=1 << 62, **kw) == 2
    assert b"one launch" in L.gdn_last_error()


def test_chunk_bwd_refuses_rows_past_32_bit_offsets(L):  # noqa: F811
    assert _chunk_bwd(L, wsb=1 << 62, B=1, Hk=1, HV=1 << 16) == 2
    assert b"2^23" in L.gdn_last_error()


@pytest.mark.parametrize("scale", [2.0 ** -15, -1e5, 1e30, float("inf"), float("nan")])
def test_chunk_bwd_refuses_scales_that_fp16_cannot_hold(L, scale):  # noqa: F811
    assert _chunk_bwd(L, scale=scale) == 2
    assert b"scale" in L.gdn_last_error()
    assert _chunk_bwd(L, scale=scale, dt=0, ws=None) == 4   # fp32 io goes on to the next check
