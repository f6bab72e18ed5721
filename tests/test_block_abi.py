"""The operators beside the layer: exported symbols, the statuses of bad
arguments, and the binding's own checks.  Runs without a GPU: the addresses are
fake and every call but the last ones carries an error or an empty size."""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import block as B
from bit_gemm_block_amd import w4a4 as W

P = 0x10000
Q = 0x10002      # aligned to 2 bytes only
S = 0x10004      # aligned to 4 bytes only


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def changed(args, **at):
    bad = list(args)
    for k, v in at.items():
        bad[int(k[1:])] = v
    return bad


def test_exports_every_declared_symbol(lib):
    names = B.header_functions()
    assert len(names) == 4
    assert set(names) == set(B._SIGS)
    for n in names:
        assert hasattr(lib, n), n


def test_adapter_add_argument_errors(lib):
    f = lib.w4a4_adapter_add
    need = lib.w4a4_adapter_workspace_size(16, 256, 16)
    assert need >= 16 * 16 * 4
    assert lib.w4a4_adapter_workspace_size(0, 256, 16) == 0
    assert lib.w4a4_adapter_workspace_size(-1, 256, 16) == 0
    # x dt ldx At Bt L R index ranks scales M N K y ldy out ldo ws bytes stream
    ok = [P, W.F16, 256, P, P, 4, 16, P, P, P, 16, 32, 256, P, 32, P, 32, P, need, None]
    for bad in (changed(ok, _1=2), changed(ok, _2=255), changed(ok, _5=-1), changed(ok, _6=0),
                changed(ok, _10=-1), changed(ok, _11=-1), changed(ok, _12=0), changed(ok, _14=31),
                changed(ok, _16=31), changed(ok, _0=None), changed(ok, _3=None),
                changed(ok, _4=None), changed(ok, _7=None), changed(ok, _15=None),
                changed(ok, _17=None), changed(ok, _14=40)):
        assert f(*bad) == W.ERR_INVALID_ARG, bad
    for bad in (changed(ok, _12=96, _2=256), changed(ok, _12=16448, _2=16448), changed(ok, _6=12),
                changed(ok, _6=264), changed(ok, _1=W.F32, _6=257)):
        assert f(*bad) == W.ERR_UNSUPPORTED, bad
    for bad in (changed(ok, _0=S), changed(ok, _2=257), changed(ok, _3=S), changed(ok, _4=S),
                changed(ok, _17=S), changed(ok, _7=Q), changed(ok, _8=Q), changed(ok, _9=Q),
                changed(ok, _13=Q), changed(ok, _15=Q)):
        assert f(*bad) == W.ERR_MISALIGNED, bad
    assert f(*changed(ok, _18=need - 1)) == W.ERR_WORKSPACE
    assert f(*changed(ok, _10=0, _0=None, _15=None)) == W.OK
    assert f(*changed(ok, _11=0)) == W.OK


def test_adapter_add_grid_limits(lib):
    f = lib.w4a4_adapter_add
    # The first sizes whose grids could not be launched; the limits themselves
    # pass this check and reach the next one (the workspace is too small).
    ok = [P, W.F16, 64, P, P, 4, 16, P, P, P, 16, 32, 64, P, 32, P, 32, P, 0, None]
    assert f(*changed(ok, _10=134217601)) == W.ERR_UNSUPPORTED
    assert f(*changed(ok, _10=134217600)) == W.ERR_WORKSPACE
    n = 16776960
    assert f(*changed(ok, _11=n + 1, _14=n + 1, _16=n + 1)) == W.ERR_UNSUPPORTED
    assert f(*changed(ok, _11=n, _14=n, _16=n)) == W.ERR_WORKSPACE


def test_norm_residual_argument_errors(lib):
    f = lib.w4a4_norm_residual
    # h dt ldh y dt ldy post w b gate dt ldg rows rs pre w b pdt off eps M C hout ld xout dt ld st
    ok = [P, 0, 64, P, 0, 64, 1, P, P, P, 0, 64, 1, 1.0, 1, P, P, 0, 0.0, 1e-6, 4, 64, P, 64, P, 1,
          64, None]
    for bad in (changed(ok, _1=2), changed(ok, _4=2), changed(ok, _10=2), changed(ok, _17=-1),
                changed(ok, _25=3), changed(ok, _6=3), changed(ok, _14=-1), changed(ok, _20=-1),
                changed(ok, _21=0), changed(ok, _19=-1.0), changed(ok, _19=float("nan")),
                changed(ok, _19=float("inf")), changed(ok, _2=63), changed(ok, _5=63),
                changed(ok, _11=63), changed(ok, _12=0), changed(ok, _23=63), changed(ok, _26=63),
                changed(ok, _6=0), changed(ok, _14=0), changed(ok, _3=None),
                changed(ok, _24=None), changed(ok, _0=None, _3=None, _6=0, _7=None, _8=None, _9=None),
                changed(ok, _22=None, _24=None, _14=0, _15=None, _16=None),
                changed(ok, _2=72)):                                     # in place, another distance
        assert f(*bad) == W.ERR_INVALID_ARG, bad
    assert f(*changed(ok, _21=16385, _2=16385, _5=16385, _11=16385, _23=16385, _26=16385)) == W.ERR_UNSUPPORTED
    for bad in (changed(ok, _0=Q, _22=Q), changed(ok, _3=Q), changed(ok, _9=Q),
                changed(ok, _24=P + 1), changed(ok, _7=S), changed(ok, _8=S), changed(ok, _15=S),
                changed(ok, _16=S)):
        assert f(*bad) == W.ERR_MISALIGNED, bad
    assert f(*changed(ok, _20=0, _0=None, _3=None)) == W.OK


def test_gated_activation_argument_errors(lib):
    f = lib.w4a4_gated_activation
    ok = [P, 64, P, 64, 0, 0, 4, 64, P, 64, 1, None]
    for bad in (changed(ok, _1=63), changed(ok, _3=63), changed(ok, _4=2), changed(ok, _5=4),
                changed(ok, _5=-1), changed(ok, _6=-1), changed(ok, _7=-1), changed(ok, _9=63),
                changed(ok, _10=5), changed(ok, _0=None), changed(ok, _8=None)):
        assert f(*bad) == W.ERR_INVALID_ARG, bad
    for bad in (changed(ok, _0=Q), changed(ok, _2=Q), changed(ok, _8=P + 1)):
        assert f(*bad) == W.ERR_MISALIGNED, bad
    assert f(*changed(ok, _6=0, _0=None)) == W.OK
    assert f(*changed(ok, _7=0, _0=None)) == W.OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_device_report_unsupported(lib):
    need = lib.w4a4_adapter_workspace_size(16, 256, 16)
    assert lib.w4a4_adapter_add(P, W.F16, 256, P, P, 4, 16, P, None, None, 16, 32, 256, None, 32, P,
                                32, P, need, None) == W.ERR_UNSUPPORTED
    assert lib.w4a4_norm_residual(P, 0, 64, None, 0, 64, 0, None, None, None, 0, 64, 1, 1.0, 1, P,
                                  None, 0, 0.0, 1e-6, 4, 64, None, 64, P, 1, 64,
                                  None) == W.ERR_UNSUPPORTED
    assert lib.w4a4_gated_activation(P, 64, P, 64, 0, 0, 4, 64, P, 64, 1, None) == W.ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        B.gated_activation(x, x)
    with pytest.raises(ValueError):
        B.norm_residual(x, pre_norm="rms")
    with pytest.raises(ValueError):
        B.norm_residual(None)
    with pytest.raises(ValueError):
        B.norm_residual(x, pre_norm="batch")
    with pytest.raises(ValueError):
        B.gated_activation(x, x, "swish")
    with pytest.raises(ValueError):
        B.adapter_add(None, x, torch.zeros((1, 8, 64)), torch.zeros((1, 16, 8)),
                      torch.zeros(4, dtype=torch.int32))


def test_oracle_formulas_on_hand_values():
    from oracle import block_oracle as O
    y = np.array([[1.0, 2.0]])
    x = np.array([[1.0, -1.0]])
    At = np.array([[[1.0, 0.0], [9.0, 9.0]], [[2.0, 1.0], [1.0, 3.0]]])
    Bt = np.array([[[1.0, 9.0], [2.0, 9.0]], [[1.0, 1.0], [0.0, 2.0]]])
    # adapter 0, rank 1: t = 1, adds (1, 2); adapter 1: t = (1, -2), adds (-1, -4) times 0.5
    assert np.array_equal(O.adapter_add(y, x, At, Bt, [0], [1, 2]), [[2.0, 4.0]])
    assert np.array_equal(O.adapter_add(y, x, At, Bt, [1], None, [1.0, 0.5]), [[0.5, 0.0]])
    assert np.array_equal(O.adapter_add(y, x, At, Bt, [-1]), y)
    assert np.array_equal(O.adapter_add(y, x, At, Bt, [2]), y)
    h, xo = O.norm_residual(np.array([[0.0, 4.0]]), np.array([[3.0, -3.0]]), "rms", rs=2.0, pre="layer",
                            eps=0.0)
    assert np.allclose(h, [[2.0, 2.0]]) and np.isnan(xo).all()      # an equal row has no direction
    h, xo = O.norm_residual(np.array([[1.0, 4.0]]), np.array([[3.0, -3.0]]), "rms",
                            gate=np.array([[2.0, 1.0]]), pre="layer", eps=0.0)
    assert np.allclose(h, [[3.0, 3.0]])
    assert np.allclose(O.norm(np.array([[1.0, 3.0]]), "layer", eps=0.0), [[-1.0, 1.0]])
    assert abs(O.activation(1.0, "silu") - 0.7310585786300049) < 1e-15
    assert abs(O.activation(1.0, "gelu") - 0.8413447460685429) < 1e-15
    assert abs(O.activation(1.0, "gelu_tanh") - 0.8411919906082768) < 1e-12
    assert O.activation(-2.0, "relu") == 0.0
