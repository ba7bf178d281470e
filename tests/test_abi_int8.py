"""Refusals of the scored router, the int8 quantisation and the int8 FFN calls,
on the host, before any HIP call (no GPU; no pointer is dereferenced)."""
import ctypes

import pytest
import torch

import combine_grouped_gemm_amd as m

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)          # 8-byte aligned only
NONE = None
ARG, UNSUP = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED


def err():
    return m.lib().moe_last_error().decode()


def scored(logits=P, dt=m.MOE_F32, bias=NONE, B=4, E=16, K=2, score=m.MOE_SCORE_SIGMOID, groups=4, keep=2, top=2,
           renorm=1, scale=1.0, pmap=NONE, shared=0, ids=P, w=P):
    return m.lib().moe_route_scored(logits, dt, bias, B, E, K, score, groups, keep, top, renorm, scale, pmap, shared,
                                    ids, w, None)


BAD_SCORED = [
    (dict(B=-1), ARG, "B must be"), (dict(E=0), ARG, "E must be"), (dict(E=1025, groups=1, keep=1), ARG, "E must be"),
    (dict(K=0), ARG, "K must be"), (dict(K=17), ARG, "K must be"), (dict(groups=0), ARG, "n_groups"),
    (dict(groups=3), ARG, "n_groups must divide"), (dict(groups=-4), ARG, "n_groups"), (dict(keep=0), ARG, "topk_groups"),
    (dict(keep=5), ARG, "topk_groups"), (dict(top=0), ARG, "group_top"), (dict(top=3), ARG, "group_top"),
    (dict(K=9), ARG, "exceeds"), (dict(scale=float("nan")), ARG, "scale"), (dict(scale=float("inf")), ARG, "scale"),
    (dict(shared=-1), ARG, "n_shared"), (dict(shared=1009), ARG, "n_shared"), (dict(shared=2**31 - 1), ARG, "n_shared"),
    (dict(logits=NONE), ARG, "null"), (dict(ids=NONE), ARG, "null"), (dict(w=NONE), ARG, "null"),
    (dict(dt=m.MOE_FP8_E4M3), UNSUP, "logits_dt"), (dict(dt=m.MOE_INT8), UNSUP, "logits_dt"), (dict(dt=42), UNSUP, "42"),
    (dict(score=2), UNSUP, "score"), (dict(score=-1), UNSUP, "score"),
    (dict(B=1 << 28, K=8, groups=1, keep=1), ARG, "int32"),
]


@pytest.mark.parametrize("kw,status,msg", BAD_SCORED)
def test_route_scored_rejects(kw, status, msg):
    assert scored(**kw) == status
    assert msg in err()


def test_route_scored_empty_batch_is_noop():
    assert scored(logits=NONE, ids=NONE, w=NONE, B=0) == m.MOE_OK


Q = ctypes.c_void_p(1 << 20)


def quant(x=P, dt=m.MOE_BF16, rows=P, E=4, cap=8, cols=64, q=Q, s=P, masked=False):
    fn = m.lib().moe_quant_rows_masked if masked else m.lib().moe_quant_rows
    return fn(x, dt, rows, E, cap, cols, q, s, None)


BAD_QUANT = [
    (dict(dt=m.MOE_FP8_E4M3), UNSUP, "x_dt"), (dict(dt=m.MOE_INT8), UNSUP, "x_dt"), (dict(cap=-1), ARG, "cap"),
    (dict(cols=0), ARG, "multiple of 16"), (dict(cols=72), ARG, "multiple of 16"),
    (dict(cols=131072), ARG, "131056"), (dict(E=0), ARG, "E_local"), (dict(E=1025), ARG, "E_local"),
    (dict(x=NONE), ARG, "null"), (dict(q=NONE), ARG, "null"), (dict(s=NONE), ARG, "null"),
    (dict(x=ODD), ARG, "16-byte"), (dict(q=ODD), ARG, "16-byte"),
    (dict(q=P), ARG, "overlap"), (dict(q=ctypes.c_void_p(4096 + 1008)), ARG, "overlap"),
    (dict(q=ctypes.c_void_p(4096 - 496)), ARG, "overlap"),
]


@pytest.mark.parametrize("kw,status,msg", BAD_QUANT)
def test_quant_rows_rejects(kw, status, msg):
    assert quant(**kw) == status
    assert msg in err()


def test_quant_rows_masked_rejects():
    assert quant(masked=True, cap=0) == ARG and "cap_per_expert" in err()
    assert quant(masked=True, rows=NONE) == ARG and "null m" in err()
    assert quant(masked=True, E=1024, cap=1 << 22) == ARG and "int32" in err()
    assert quant(masked=True, E=0) == ARG and "E_local" in err()


def test_quant_rows_of_nothing_is_noop():
    assert quant(x=NONE, q=NONE, s=NONE, cap=0) == m.MOE_OK


def dispatch(x_dt=m.MOE_BF16, H=128, xd=P, scales=P, row_of=P):
    ptrs, rows = (ctypes.c_void_p * 1)(4096), (ctypes.c_int32 * 1)(4)
    cast = lambda a: ctypes.cast(a, ctypes.c_void_p)
    return m.lib().moe_dispatch(cast(ptrs), cast(rows), 1, x_dt, H, row_of, 2, xd, m.MOE_INT8, scales, 8, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(H=200), ARG, "multiple of 16"), (dict(H=131072), ARG, "131056"), (dict(scales=NONE), ARG, "int8 dispatch"),
    (dict(x_dt=m.MOE_FP8_E4M3), UNSUP, "dispatch"), (dict(x_dt=m.MOE_INT8), UNSUP, "dispatch"),
    (dict(xd=ODD), ARG, "aligned"), (dict(row_of=NONE), ARG, "null")])
def test_int8_dispatch_rejects(kw, status, msg):
    assert dispatch(**kw) == status
    assert msg in err()


def gate_up(xd=P, xs=P, H=128, I=128, act=m.MOE_INT8, wg=P, wu=P, gs=P, us=P, w_dt=m.MOE_INT8, h=P, hs=NONE, cap=64):
    return m.lib().moe_ffn_gate_up(xd, xs, P, 8, cap, H, I, act, wg, wu, gs, us, w_dt, h, hs, 0, None)


def down(h=P, hs=P, H=128, I=128, wd=P, ds=P, w_dt=m.MOE_INT8, y=P, y_dt=m.MOE_BF16):
    return m.lib().moe_ffn_down(h, hs, P, 8, 64, H, I, m.MOE_INT8, wd, ds, w_dt, y, y_dt, 0, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(H=200), ARG, "multiples of 16"), (dict(I=136), ARG, "multiples of 16"), (dict(H=131072), ARG, "131056"),
    (dict(I=131072), ARG, "131056"), (dict(xs=NONE), ARG, "scale pointers"), (dict(gs=NONE), ARG, "scale pointers"),
    (dict(us=NONE), ARG, "scale pointers"), (dict(w_dt=m.MOE_BF16), UNSUP, "w_dt"),
    (dict(w_dt=m.MOE_FP8_E4M3), UNSUP, "w_dt"), (dict(act=m.MOE_BF16), UNSUP, "w_dt"),
    (dict(xd=ODD), ARG, "16-byte"), (dict(wg=ODD), ARG, "16-byte"), (dict(h=ODD), ARG, "16-byte"),
    (dict(h=NONE), ARG, "null"), (dict(xd=NONE), ARG, "null")])
def test_int8_gate_up_rejects(kw, status, msg):
    assert gate_up(**kw) == status
    assert msg in err()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(hs=NONE), ARG, "scale pointers"), (dict(ds=NONE), ARG, "scale pointers"),
    (dict(y_dt=m.MOE_INT8), UNSUP, "y_dt"), (dict(y_dt=m.MOE_FP8_E4M3), UNSUP, "y_dt"),
    (dict(w_dt=m.MOE_F32), UNSUP, "w_dt"), (dict(y=ODD), ARG, "16-byte"), (dict(I=100), ARG, "multiples of 16")])
def test_int8_down_rejects(kw, status, msg):
    assert down(**kw) == status
    assert msg in err()


def test_int8_grouped_ffn_checks_everything_first():
    L = m.lib()
    need = L.moe_ffn_workspace_bytes(64, 128, m.MOE_INT8)
    assert need == 64 * 128 * 2 + 64 * 128 + 256
    big = ctypes.c_size_t(need)

    def call(wd=P, ds=P, y=P, ws=P, n=big):
        return L.moe_grouped_ffn(P, P, P, 8, 64, 128, 128, m.MOE_INT8, P, P, wd, P, P, ds, m.MOE_INT8, y, m.MOE_BF16,
                                 ws, n, 0, None)

    assert call(ws=NONE) == ARG and "null workspace" in err()
    assert call(n=ctypes.c_size_t(need - 1)) == ARG and "too small" in err()
    assert call(ws=ctypes.c_void_p(4096 + 16)) == ARG and "256-byte" in err()
    # what only the last of the three calls reads is refused before the first is enqueued
    assert call(wd=NONE) == ARG and "null" in err()
    assert call(ds=NONE) == ARG and "scale pointers" in err()
    assert call(y=ODD) == ARG and "16-byte" in err()


def test_int8_weights_pack_at_the_byte_pitch():
    assert [m.moe_weight_ld(c, "int8") for c in (2880, 4096, 7168, 2048, 16)] == [2944, 4224, 7168, 2048, 128]
    assert m.moe_packed_weight_bytes(3, 5, 2880, "int8") == 3 * 5 * 2944


def test_layer_refuses_unknown_router_options():
    with pytest.raises(ValueError, match="n_group"):
        m.MoELayer((4,), 8, 2, 16, 16, 0, 8, "bf16", "bf16", "bf16", device="cpu", router=dict(n_group=2))


def test_binding_refuses_host_tensors_and_other_types():
    with pytest.raises(ValueError, match="device tensor"):
        m.moe_route_scored(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match="device tensor"):
        m.moe_quant_rows(torch.zeros(4, 16))
