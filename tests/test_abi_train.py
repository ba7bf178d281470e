"""Refusals of the training step's calls, on the host, before any HIP call (no GPU; no
pointer is dereferenced), and what the binding checks before it calls."""
import ctypes

import pytest
import torch

import combine_grouped_gemm_amd as m
import test_binding_streams as tbs
from test_binding_streams import bf, f32, i8, i32, on_host, recorder  # noqa: F401  (fixtures)

V = ctypes.c_void_p
P, Q, S = V(1 << 20), V(1 << 30), V(1 << 40)         # far apart
ODD, HALF8 = V((1 << 20) + 4), V((1 << 20) + 8)
NONE = None
ARG, UNSUP = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED
F32, BF16 = m.MOE_F32, m.MOE_BF16


def err():
    return m.lib().moe_last_error().decode()


def rows(x=P, dt=BF16, off=P, E=4, cap=8, cols=64, q=Q, s=S):
    return m.lib().moe_checkpoint_rows(x, dt, off, E, cap, cols, q, s, None)


def values(q=Q, s=S, off=P, E=4, cap=8, cols=64, x=P, dt=BF16):
    return m.lib().moe_checkpoint_values(q, s, off, E, cap, cols, x, dt, None)


BAD_CKPT = [
    (dict(dt=m.MOE_INT8), UNSUP, "_dt"), (dict(dt=m.MOE_CKPT8), UNSUP, "_dt"), (dict(dt=77), UNSUP, "77"),
    (dict(cap=-1), ARG, "cap"), (dict(cols=0), ARG, "multiple of 8"), (dict(cols=68), ARG, "multiple of 8"),
    (dict(cols=(1 << 24) + 8), ARG, "at most"), (dict(E=0), ARG, "E_local"), (dict(E=1025), ARG, "E_local"),
    (dict(x=NONE), ARG, "null"), (dict(q=NONE), ARG, "null"), (dict(s=NONE), ARG, "null"),
    (dict(x=HALF8), ARG, "16-byte"), (dict(q=V((1 << 30) + 4)), ARG, "8-byte"), (dict(q=P), ARG, "overlap"),
    (dict(q=V((1 << 20) + 1016)), ARG, "overlap"),
]


@pytest.mark.parametrize("call", [rows, values])
@pytest.mark.parametrize("kw,status,msg", BAD_CKPT)
def test_checkpoints_reject(call, kw, status, msg):
    assert call(**kw) == status
    assert msg in err()


def test_checkpoints_of_no_rows_are_noops():
    assert rows(x=NONE, q=NONE, s=NONE, cap=0) == m.MOE_OK
    assert values(x=NONE, q=NONE, s=NONE, cap=0) == m.MOE_OK


def gate_up(xd=P, off=P, E=4, cap=8, H=64, I=64, dt=BF16, wg=P, wu=P, w_dt=None, h=Q, gq=V(1 << 31), gs=Q, uq=V(1 << 32), us=Q):
    return m.lib().moe_ffn_gate_up_train(xd, off, E, cap, H, I, dt, wg, wu, dt if w_dt is None else w_dt, h, gq, gs, uq,
                                         us, 0, None)


BAD_GATE_UP = [
    (dict(dt=m.MOE_FP8_E4M3), UNSUP, "training"), (dict(dt=m.MOE_INT8), UNSUP, "training"), (dict(w_dt=F32), UNSUP, "training"),
    (dict(off=NONE), ARG, "null"), (dict(E=0), ARG, "E_local"), (dict(cap=-1), ARG, "cap_rows"), (dict(H=60), ARG, "multiples of 8"),
    (dict(I=0), ARG, "multiples of 8"), (dict(xd=NONE), ARG, "null"), (dict(wg=NONE), ARG, "null"), (dict(wu=NONE), ARG, "null"),
    (dict(h=NONE), ARG, "null"), (dict(gq=NONE), ARG, "null"), (dict(us=NONE), ARG, "null"), (dict(xd=HALF8), ARG, "16-byte"),
    (dict(uq=HALF8), ARG, "16-byte"), (dict(h=ODD), ARG, "16-byte"), (dict(H=(1 << 24) + 8), ARG, "at most"),
    (dict(I=(1 << 24) + 8, cap=1), ARG, "at most"), (dict(h=P), ARG, "overlap"), (dict(gq=V((1 << 30) + 1008)), ARG, "overlap"),
    (dict(uq=V((1 << 31) + 496)), ARG, "overlap"), (dict(uq=P), ARG, "overlap"),
]


@pytest.mark.parametrize("kw,status,msg", BAD_GATE_UP)
def test_gate_up_train_rejects(kw, status, msg):
    assert gate_up(**kw) == status
    assert msg in err()


def swiglu(dh=P, dt=BF16, gq=P, gs=P, uq=P, us=P, cap=8, I=64, row_of=P, w=P, B=4, K=2, dg=V(1 << 32), du=V(1 << 33),
           hw=V(1 << 34), dw=S):
    return m.lib().moe_swiglu_backward(dh, dt, gq, gs, uq, us, cap, I, row_of, w, B, K, dg, du, hw, dw, None)


BAD_SWIGLU = [
    (dict(dt=m.MOE_CKPT8), UNSUP, "training"), (dict(B=-1), ARG, "B >= 0"), (dict(K=0), ARG, "K"), (dict(K=1025), ARG, "K"),
    (dict(B=1 << 30, K=4), ARG, "int32"), (dict(cap=-1), ARG, "cap_rows"), (dict(I=12), ARG, "multiple of 8"),
    (dict(dh=NONE), ARG, "null"), (dict(us=NONE), ARG, "null"), (dict(hw=NONE), ARG, "null"), (dict(row_of=NONE), ARG, "null"),
    (dict(dw=NONE), ARG, "null"), (dict(dg=HALF8), ARG, "16-byte"), (dict(gq=HALF8), ARG, "16-byte"), (dict(dg=P), ARG, "overlap"),
    (dict(du=V((1 << 32) + 1008)), ARG, "overlap"), (dict(hw=V((1 << 20) + 496)), ARG, "overlap"),
]


@pytest.mark.parametrize("kw,status,msg", BAD_SWIGLU)
def test_swiglu_backward_rejects(kw, status, msg):
    assert swiglu(**kw) == status
    assert msg in err()


def dgrad(dy=P, dy2=P, src=P, per=2, src_rows=8, off=P, E=4, cap=8, N=64, M=64, dt=BF16, w=P, w2=P, w_dt=None, dx=Q):
    return m.lib().moe_ffn_dgrad(dy, dy2, src, per, src_rows, off, E, cap, N, M, dt, w, w2, dt if w_dt is None else w_dt, dx,
                                 0, None)


BAD_DGRAD = [
    (dict(dt=m.MOE_INT8), UNSUP, "training"), (dict(w_dt=m.MOE_FP8_E4M3), UNSUP, "training"), (dict(per=0), ARG, "slots_per_token"),
    (dict(per=1025), ARG, "slots_per_token"), (dict(src_rows=-1), ARG, "src_rows"), (dict(off=NONE), ARG, "null"),
    (dict(E=1025), ARG, "E_local"), (dict(cap=-1), ARG, "cap_rows"), (dict(N=4), ARG, "multiples of 8"),
    (dict(M=100), ARG, "multiples of 8"), (dict(dy=NONE), ARG, "null dy"), (dict(dy2=NONE), ARG, "together"),
    (dict(w2=NONE), ARG, "together"), (dict(w=NONE), ARG, "null"), (dict(dx=NONE), ARG, "null"), (dict(dx=HALF8), ARG, "16-byte"),
    (dict(w2=HALF8), ARG, "16-byte"), (dict(dx=P), ARG, "overlap"), (dict(dx=V((1 << 20) + 1008)), ARG, "overlap"),
    (dict(cap=2**31 - 1, M=1 << 20), ARG, "too large"), (dict(N=(1 << 24) + 8), ARG, "at most"),
    (dict(M=(1 << 24) + 8), ARG, "at most"),
]


@pytest.mark.parametrize("kw,status,msg", BAD_DGRAD)
def test_dgrad_rejects(kw, status, msg):
    assert dgrad(**kw) == status
    assert msg in err()


def test_dgrad_of_no_rows_is_a_noop():
    assert dgrad(dy=NONE, dy2=NONE, src=NONE, cap=0, dx=NONE) == m.MOE_OK


def wgrad(dy=P, dy2=P, x=P, x_dt=BF16, xs=NONE, src=P, per=2, src_rows=8, gather=m.MOE_GATHER_X, off=P, E=4, cap=8, N=64,
          M=64, dt=BF16, base=NONE, base2=NONE, dw=Q, dw2=S, dw_dt=F32):
    return m.lib().moe_ffn_wgrad(dy, dy2, x, x_dt, xs, src, per, src_rows, gather, off, E, cap, N, M, dt, base, base2, dw,
                                 dw2, dw_dt, 0, None)


DW = 4 * 64 * 64 * 4
BAD_WGRAD = [
    (dict(dt=m.MOE_FP8_E4M3), UNSUP, "training"), (dict(x_dt=F32), UNSUP, "x_dt"), (dict(x_dt=m.MOE_INT8), UNSUP, "x_dt"),
    (dict(dw_dt=m.MOE_INT8), UNSUP, "dw_dt"), (dict(dt=F32, x_dt=F32, dw_dt=BF16), UNSUP, "dw_dt"), (dict(gather=3), ARG, "gather"),
    (dict(gather=-1), ARG, "gather"), (dict(src=NONE), ARG, "src_of"), (dict(per=0), ARG, "slots_per_token"),
    (dict(src_rows=-2), ARG, "src_rows"), (dict(off=NONE), ARG, "null"), (dict(E=0), ARG, "E_local"), (dict(cap=-1), ARG, "cap_rows"),
    (dict(N=0), ARG, "multiples of 8"), (dict(M=7), ARG, "multiples of 8"), (dict(dy=NONE), ARG, "null"), (dict(x=NONE), ARG, "null"),
    (dict(dw=NONE), ARG, "null dw"), (dict(dw2=NONE), ARG, "together"), (dict(dy2=NONE), ARG, "together"),
    (dict(x_dt=m.MOE_CKPT8), ARG, "scales"), (dict(dw2=NONE, dy2=NONE, base2=P), ARG, "base2"), (dict(dw=HALF8), ARG, "16-byte"),
    (dict(x=HALF8), ARG, "16-byte"), (dict(dw2=Q), ARG, "overlap"), (dict(dw2=V((1 << 30) + DW - 16)), ARG, "overlap"),
    (dict(N=(1 << 24) + 8), ARG, "at most"), (dict(M=(1 << 24) + 8), ARG, "at most"), (dict(base=V((1 << 30) + 16)), ARG, "base"), (dict(base=Q, base2=Q), ARG, "base"), (dict(base=S), ARG, "base"), (dict(base2=Q), ARG, "base"), (dict(dw=P), ARG, "overlap"),
]


@pytest.mark.parametrize("kw,status,msg", BAD_WGRAD)
def test_wgrad_rejects(kw, status, msg):
    assert wgrad(**kw) == status
    assert msg in err()


def route(logits=P, dt=F32, ids=P, dw=P, B=4, E=16, K=2, score=m.MOE_SCORE_SIGMOID, renorm=1, scale=1.0, pmap=NONE, shared=0,
          out=P):
    return m.lib().moe_route_backward(logits, dt, ids, dw, B, E, K, score, renorm, scale, pmap, shared, out, None)


BAD_ROUTE = [
    (dict(B=-1), ARG, "B must"), (dict(E=1025), ARG, "E must"), (dict(K=17), ARG, "K must"), (dict(K=0), ARG, "K must"),
    (dict(dt=m.MOE_INT8), UNSUP, "logits_dt"), (dict(score=3), UNSUP, "score"), (dict(score=-1), UNSUP, "score"),
    (dict(score=m.MOE_SCORE_PICKS, dt=BF16), UNSUP, "fp32"), (dict(score=m.MOE_SCORE_PICKS, scale=2.0), ARG, "scale"),
    (dict(scale=float("nan")), ARG, "scale"), (dict(scale=float("inf")), ARG, "scale"), (dict(shared=-1), ARG, "n_shared"),
    (dict(shared=1009), ARG, "n_shared"), (dict(logits=NONE), ARG, "null"), (dict(ids=NONE), ARG, "null"),
    (dict(dw=NONE), ARG, "null"), (dict(out=NONE), ARG, "null"), (dict(B=1 << 28), ARG, "int32"),
]


@pytest.mark.parametrize("kw,status,msg", BAD_ROUTE)
def test_route_backward_rejects(kw, status, msg):
    assert route(**kw) == status
    assert msg in err()


def test_route_backward_empty_batch_is_noop():
    assert route(logits=NONE, ids=NONE, dw=NONE, out=NONE, B=0) == m.MOE_OK


def test_the_new_dtype_is_refused_where_it_has_no_meaning():
    L = m.lib()
    assert L.moe_weight_ld(128, m.MOE_CKPT8) == -1 and L.moe_packed_weight_bytes(1, 8, 128, m.MOE_CKPT8) == 0
    assert L.moe_quant_rows(P, m.MOE_CKPT8, NONE, 0, 8, 64, Q, S, None) == UNSUP
    assert L.moe_combine(P, m.MOE_CKPT8, 8, P, P, 4, 2, 64, Q, BF16, None) == UNSUP
    assert L.moe_route_scored(P, F32, NONE, 4, 16, 2, m.MOE_SCORE_PICKS, 1, 1, 1, 1, 1.0, NONE, 0, P, P, None) == UNSUP


# ------------------------------------------------------------------ the binding
CALLS = {
    "moe_checkpoint_rows": (lambda **k: m.moe_checkpoint_rows(bf(4, 16), i32(3), **k), 2),
    "moe_checkpoint_values": (lambda **k: m.moe_checkpoint_values(i8(4, 16), f32(4, 1), i32(3), **k), 1),
    "moe_ffn_gate_up_train": (lambda **k: m.moe_ffn_gate_up_train(bf(4, 16), i32(3), bf(2, 24, 16), bf(2, 24, 16), **k), 5),
    "moe_swiglu_backward": (lambda **k: m.moe_swiglu_backward(bf(4, 16), i8(4, 16), f32(4, 1), i8(4, 16), f32(4, 1), i32(2, 2),
                                                              f32(2, 2), **k), 4),
    "moe_ffn_dgrad": (lambda **k: m.moe_ffn_dgrad(bf(4, 24), i32(3), bf(2, 24, 16), bf(4, 24), bf(2, 24, 16), i32(6), 2, **k), 1),
    "moe_ffn_wgrad": (lambda **k: m.moe_ffn_wgrad(bf(4, 24), i8(3, 16), i32(3), f32(3, 1), bf(4, 24), i32(4), 2, "x",
                                                  f32(2, 24, 16), f32(2, 24, 16), **k), 2),
    "moe_route_backward": (lambda **k: m.moe_route_backward(f32(4, 8), i32(4, 2), f32(4, 2), **k), 1),
}


@pytest.fixture
def train_calls(monkeypatch):
    monkeypatch.setattr(tbs, "CALLS", CALLS)


@pytest.mark.parametrize("name", CALLS)
def test_streams_and_devices(train_calls, request, name):
    """The binding's stream and device tests, for these calls."""
    for fixture, test in (("recorder", tbs.test_what_a_call_makes_belongs_to_the_stream_it_is_given),
                          ("on_host", tbs.test_the_tensors_device_is_current_during_a_call),
                          ("on_host", tbs.test_tensors_of_two_devices_are_refused),
                          ("on_host", tbs.test_a_stream_of_another_device_is_refused)):
        with pytest.MonkeyPatch.context() as patch:
            r = tbs.Recorder(m.lib())
            patch.setattr(m, "lib", lambda r=r: r)
            patch.setattr(m, "_dev", lambda t, *a, **k: t)
            if fixture == "recorder":
                patch.setattr(m, "_stream", lambda stream: stream)
            test(r, patch, name)


BAD_SHAPES = [
    (lambda: m.moe_checkpoint_rows(i8(4, 16)), "float32 or bfloat16"),
    (lambda: m.moe_checkpoint_rows(bf(4, 16), E_loc=2), "offsets"),
    (lambda: m.moe_checkpoint_rows(bf(4, 16), i32(3), E_loc=3), "offsets needs at least 4"),
    (lambda: m.moe_checkpoint_rows(bf(4, 16), i32(0)), "offsets needs at least 2"),
    (lambda: m.moe_checkpoint_rows(bf(4, 16), q=i8(3, 16)), "q must have shape"),
    (lambda: m.moe_checkpoint_rows(bf(4, 160), scales=f32(4, 1)), "scales must have shape"),
    (lambda: m.moe_checkpoint_values(i8(4, 160), f32(4, 1)), "scales must have shape"),
    (lambda: m.moe_checkpoint_values(i8(4, 16), f32(4, 1), out=i8(4, 16)), "float32 or bfloat16"),
    (lambda: m.moe_ffn_gate_up_train(bf(4, 16), i32(2), bf(2, 24, 16), bf(2, 24, 16)), "offsets needs"),
    (lambda: m.moe_ffn_gate_up_train(bf(4, 16), i32(3), bf(2, 24, 16), bf(2, 16, 16)), "w_up must"),
    (lambda: m.moe_ffn_gate_up_train(bf(4, 16), i32(3), bf(2, 24, 24), bf(2, 24, 24)), "columns"),
    (lambda: m.moe_ffn_gate_up_train(bf(4, 16), i32(3), bf(2, 24, 16), bf(2, 24, 16), up_q=i8(4, 16)), "up_q must"),
    (lambda: m.moe_swiglu_backward(bf(4, 16), i8(4, 16), f32(4, 1), i8(4, 24), f32(4, 1), i32(2, 2), f32(2, 2)), "up_q must"),
    (lambda: m.moe_swiglu_backward(bf(4, 16), i8(4, 16), f32(4), i8(4, 16), f32(4, 1), i32(2, 2), f32(2, 2)), "gate_scales must"),
    (lambda: m.moe_swiglu_backward(bf(4, 16), i8(4, 16), f32(4, 1), i8(4, 16), f32(4, 1), i32(2, 2), f32(2, 3)), "topk_w must"),
    (lambda: m.moe_ffn_dgrad(bf(4, 16), i32(3), bf(2, 24, 16)), "dy must have 24"),
    (lambda: m.moe_ffn_dgrad(bf(4, 24), i32(3), bf(2, 24, 16), dy2=bf(4, 24)), "together"),
    (lambda: m.moe_ffn_dgrad(bf(4, 24), i32(3), bf(2, 24, 16), dx=bf(4, 24)), "columns"),
    (lambda: m.moe_ffn_dgrad(bf(4, 24), i32(3), bf(2, 24, 16), src_of=i32(3), dx=bf(4, 16)), "src_of needs"),
    (lambda: m.moe_ffn_dgrad(bf(4, 24), i32(3), bf(2, 24, 16), dy2=bf(4, 24), w2=bf(2, 24, 24)), "w2 must"),
    (lambda: m.moe_ffn_wgrad(bf(4, 24), bf(5, 16), i32(3)), "same rows"),
    (lambda: m.moe_ffn_wgrad(bf(4, 24), f32(4, 16), i32(3)), "x must be"),
    (lambda: m.moe_ffn_wgrad(bf(4, 24), i8(4, 16), i32(3)), "x_scales"),
    (lambda: m.moe_ffn_wgrad(bf(4, 24), bf(4, 16), i32(3), x_scales=f32(4, 1)), "x_scales"),
    (lambda: m.moe_ffn_wgrad(bf(4, 24), bf(4, 16), i32(3), gather="x"), "src_of"),
    (lambda: m.moe_ffn_wgrad(bf(4, 24), bf(9, 16), i32(3), gather="x", src_of=i32(3)), "src_of needs"),
    (lambda: m.moe_ffn_wgrad(bf(4, 24), bf(4, 16), i32(3), gather="w"), "gather must"),
    (lambda: m.moe_ffn_wgrad(bf(4, 24), bf(4, 16), i32(3), dw2=f32(2, 24, 16)), "dy2"),
    (lambda: m.moe_ffn_wgrad(bf(4, 24), bf(4, 16), i32(3), dw=f32(2, 16, 24)), "dw must"),
    (lambda: m.moe_ffn_wgrad(bf(4, 24), bf(4, 16), i32(2), dw=f32(2, 24, 16)), "offsets needs"),
    (lambda: m.moe_route_backward(i8(4, 8), i32(4, 2), f32(4, 2)), "float32 or bfloat16"),
    (lambda: m.moe_route_backward(f32(4, 8), i32(4, 2), f32(4, 3)), "dtopk_w must"),
    (lambda: m.moe_route_backward(f32(4, 8), i32(3, 2), f32(4, 2)), "topk_ids must"),
    (lambda: m.moe_route_backward(f32(4, 8), i32(4, 2), f32(4, 2), score="tanh"), "score must"),
    (lambda: m.moe_route_backward(f32(4, 8), i32(4, 2), f32(4, 2), phys_of_logical=i32(7)), "phys_of_logical must"),
]


@pytest.mark.parametrize("k", range(len(BAD_SHAPES)))
def test_the_binding_refuses_shapes_before_the_call(on_host, k):  # noqa: F811
    call, message = BAD_SHAPES[k]
    with pytest.raises(ValueError, match=message):
        call()
    assert not on_host.launched
