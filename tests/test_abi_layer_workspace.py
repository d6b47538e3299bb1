"""CPU-only: what the size queries of the layer operators say is enough for every
choice of wanted sums, and no byte too many where all are wanted.  A workspace that
is large enough but not aligned is refused for its alignment, so nothing is launched."""

import pytest

from tests.test_abi_layer import FAKE, L, _conv_bwd, _norm  # noqa: F401

SUMS = [(FAKE, FAKE), (FAKE, None), (None, FAKE)]


@pytest.mark.parametrize("dw,db", SUMS)
@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("G,d", [(16, 128), (16, 80), (1, 8), (4, 512), (2, 1032), (1, 8192)])
@pytest.mark.parametrize("B,T", [(1, 1), (1, 2), (1, 5), (1, 100), (1, 1001), (4, 4096)])
def test_norm_gradients(L, B, T, G, d, shared, dw, db):  # noqa: F811
    need = L.gdn_group_norm_bwd_workspace_bytes(B, T, G, d, shared)
    call = dict(B=B, T=T, G=G, d=d, sh=shared, dw=dw, db=db, gb=T * G * d, gt=G * d, xb=T * G * d, xt=G * d)
    assert need > 0
    assert _norm(L, True, ws=FAKE + 64, wsb=need, **call) == 1 and b"256-byte" in L.gdn_last_error()
    assert _norm(L, True, ws=FAKE + 64, wsb=need - 1, **call) == 4


@pytest.mark.parametrize("dw,db", SUMS)
@pytest.mark.parametrize("B,T,D,W", [(1, 1, 8, 2), (2, 3, 520, 3), (1, 100, 512, 4), (1, 16001, 8192, 4)])
def test_convolution_gradients(L, B, T, D, W, dw, db):  # noqa: F811
    need = L.gdn_conv_bwd_workspace_bytes(B, T, D, W)
    call = dict(B=B, T=T, D=D, W=W, w0=D, xb=T * D, xt=D, dw=dw, db=db)
    assert need > 0
    assert _conv_bwd(L, ws=FAKE + 64, wsb=need, **call) == 1 and b"256-byte" in L.gdn_last_error()
    assert _conv_bwd(L, ws=FAKE + 64, wsb=need - 1, **call) == 4
