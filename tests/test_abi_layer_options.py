"""CPU-only: options or'ed into the dtype of the packed gradients' entries.  A known one
goes on to the next check (here the workspace's), anything else is an unknown dtype."""

import pytest

from gated_delta_rule_61_amd import binding
from tests.test_abi_layer import FAKE, L, _chunk_bwd, _conv_bwd, _norm  # noqa: F401

ZERO = binding.GDN_ROWS_ZERO


@pytest.mark.parametrize("call", [_chunk_bwd, _conv_bwd])
@pytest.mark.parametrize("io", [0, 1])
def test_rows_zero(L, call, io):  # noqa: F811
    assert call(L, dt=io | ZERO, ws=None) == 4
    for bad in (io | 0x1000, io | ZERO | 0x1000, 2 | ZERO, -1, ZERO << 16 | io):
        assert call(L, dt=bad, ws=None) == 1 and b"dtype" in L.gdn_last_error()


def test_not_for_the_others(L):  # noqa: F811
    assert _norm(L, True, dt=1 | ZERO) == 1 and b"dtype" in L.gdn_last_error()


def test_workspace_sizes_do_not_depend_on_it(L):  # noqa: F811
    size = L.gdn_chunk_bwd_workspace_bytes
    for io in (0, 1):
        assert size(1, 300, 2, 4, 64, 64, 3, 1, io | ZERO) == size(1, 300, 2, 4, 64, 64, 3, 1, io) > 0


def test_no_sequences(L):  # noqa: F811
    # without the option there is nothing to do; with it (and tokens) rows are written, so pointers count
    assert _chunk_bwd(L, cu=FAKE, n=0, B=1) == 0
    assert _chunk_bwd(L, cu=FAKE, n=0, B=1, dt=1 | ZERO, dq=None) == 1


@pytest.mark.parametrize("io", [0, 1])
def test_grads_f32(L, io):  # noqa: F811
    F = binding.GDN_GRADS_F32
    assert _chunk_bwd(L, dt=io | F, ws=None) == 4
    assert _chunk_bwd(L, dt=io | F | ZERO, ws=None) == 4
    assert _conv_bwd(L, dt=io | F, ws=None) == 1 and b"dtype" in L.gdn_last_error()
    size = L.gdn_chunk_bwd_workspace_bytes
    assert size(1, 300, 2, 4, 64, 64, 3, 1, io | F) == size(1, 300, 2, 4, 64, 64, 3, 1, io) > 0
