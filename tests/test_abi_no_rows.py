"""Null buffers are refused wherever there is a row, for every storage type
(no GPU; nothing is enqueued)."""
import ctypes

import pytest
import torch

import combine_grouped_gemm_amd as m

P = ctypes.c_void_p(4096)
ARG = m.MOE_ERR_INVALID_ARG
TYPES = [m.MOE_F32, m.MOE_BF16, m.MOE_FP8_E4M3, m.MOE_INT8]
SCALED = [m.MOE_FP8_E4M3, m.MOE_INT8]


def refused(status):
    return status == ARG and any(w in m.lib().moe_last_error() for w in (b"null", b"scale", b"needs xd_scales"))


def y_of(act):
    return m.MOE_F32 if act == m.MOE_F32 else m.MOE_BF16


def gate_up(act, cap, a=P, s=P, h=P, hs=P):
    return m.lib().moe_ffn_gate_up(a, s, P, 4, cap, 64, 64, act, P, P, P, P, act, h, hs, 0, None)


def down(act, cap, a=P, s=P, y=P):
    return m.lib().moe_ffn_down(a, s, P, 4, cap, 64, 64, act, P, P, act, y, y_of(act), 0, None)


@pytest.mark.parametrize("act", TYPES)
def test_null_rows_are_refused(act):
    assert refused(gate_up(act, 1, a=None)) and refused(gate_up(act, 1, h=None))
    assert refused(down(act, 1, a=None)) and refused(down(act, 1, y=None))
    if act in SCALED:
        assert refused(gate_up(act, 1, s=None)) and refused(down(act, 1, s=None))
    if act == m.MOE_FP8_E4M3:
        assert refused(gate_up(act, 1, hs=None))
    # weights are never empty
    assert refused(m.lib().moe_ffn_down(P, P, P, 4, 0, 64, 64, act, None, P, act, P, y_of(act), 0, None))
    if act in SCALED:
        assert refused(m.lib().moe_ffn_down(P, P, P, 4, 0, 64, 64, act, P, None, act, P, y_of(act), 0, None))


# these calls pass every check: with a device they would launch on the made-up pointers
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch")


@no_device
@pytest.mark.parametrize("act", TYPES)
def test_rows_of_nothing_pass_the_checks(act):
    """What is left is the launch, which there is no device for."""
    assert gate_up(act, 0, a=None, s=None, h=None, hs=None) != ARG
    assert down(act, 0, a=None, s=None, y=None) != ARG


def dispatch(x_dt, xd_dt, xd, s, cap):
    ptrs, rows = (ctypes.c_void_p * 1)(4096), (ctypes.c_int32 * 1)(4)
    cast = lambda a: ctypes.cast(a, ctypes.c_void_p)
    return m.lib().moe_dispatch(cast(ptrs), cast(rows), 1, x_dt, 64, P, 2, xd, xd_dt, s, cap, None)


def combine(dt, y, cap, out):
    return m.lib().moe_combine(y, dt, cap, P, P, 4, 2, 64, out, dt, None)


DISPATCHES = [(m.MOE_F32, m.MOE_F32), (m.MOE_BF16, m.MOE_BF16), (m.MOE_BF16, m.MOE_FP8_E4M3), (m.MOE_BF16, m.MOE_INT8)]


def test_dispatch_and_combine_refuse_null_rows():
    for x_dt, xd_dt in DISPATCHES:
        assert refused(dispatch(x_dt, xd_dt, None, P, 1))
        if xd_dt in SCALED:
            assert refused(dispatch(x_dt, xd_dt, P, None, 1))
    for dt in (m.MOE_F32, m.MOE_BF16):
        assert refused(combine(dt, None, 1, P)) and refused(combine(dt, None, 0, None))


@no_device
def test_dispatch_and_combine_take_no_rows():
    for x_dt, xd_dt in DISPATCHES:
        assert dispatch(x_dt, xd_dt, None, None, 0) != ARG
    for dt in (m.MOE_F32, m.MOE_BF16):
        assert combine(dt, None, 0, P) != ARG
