"""The training step's calls refuse outputs that share memory with each other or with an
input, on the host (no GPU; no pointer is dereferenced): every such pair of every call,
with the same address and with one byte range ending inside the other."""
import ctypes

import pytest

import combine_grouped_gemm_amd as m

F32, BF16 = m.MOE_F32, m.MOE_BF16
E, CAP, N, M, B, K = 4, 8, 64, 256, 4, 2
W, ROWS_N, ROWS_M = E * N * M * 2, CAP * N * 2, CAP * M * 2
OFF, SRC, SLOTS = (E + 1) * 4, CAP * 4, B * K * 4
S_N, S_M = CAP * 4, CAP * 2 * 4                      # scales of N and of M columns


def _call(name, a):
    """One call with the addresses of `a`."""
    L, v = m.lib(), {k: ctypes.c_void_p(p) for k, p in a.items()}
    if name == "checkpoint_rows":
        return L.moe_checkpoint_rows(v["x"], BF16, v["off"], E, CAP, M, v["q"], v["s"], None)
    if name == "checkpoint_values":
        return L.moe_checkpoint_values(v["q"], v["s"], v["off"], E, CAP, M, v["x"], BF16, None)
    if name == "gate_up":
        return L.moe_ffn_gate_up_train(v["xd"], v["off"], E, CAP, M, N, BF16, v["wg"], v["wu"], BF16, v["h"], v["gq"], v["gs"],
                                       v["uq"], v["us"], 0, None)
    if name == "swiglu":
        return L.moe_swiglu_backward(v["dh"], BF16, v["gq"], v["gs"], v["uq"], v["us"], CAP, N, v["row_of"], v["w"], B, K,
                                     v["dgate"], v["dup"], v["hw"], v["dw"], None)
    if name == "dgrad":
        return L.moe_ffn_dgrad(v["dy"], v["dy2"], v["src"], K, CAP, v["off"], E, CAP, N, M, BF16, v["w"], v["w2"], BF16,
                               v["dx"], 0, None)
    if name == "wgrad":
        return L.moe_ffn_wgrad(v["dy"], v["dy2"], v["x"], m.MOE_CKPT8, v["xs"], v["src"], K, CAP, m.MOE_GATHER_X, v["off"], E,
                               CAP, N, M, BF16, None, None, v["dw"], v["dw2"], BF16, 0, None)
    return L.moe_route_backward(v["logits"], BF16, v["ids"], v["dw"], B, M, K, m.MOE_SCORE_SIGMOID, 1, 1.0, v["map"], 0,
                                v["out"], None)


# bytes of each output and each input
CALLS = {
    "checkpoint_rows": (dict(q=CAP * M, s=S_M), dict(x=ROWS_M, off=OFF)),
    "checkpoint_values": (dict(x=ROWS_M), dict(q=CAP * M, s=S_M, off=OFF)),
    "gate_up": (dict(h=ROWS_N, gq=CAP * N, gs=S_N, uq=CAP * N, us=S_N), dict(xd=ROWS_M, wg=W, wu=W, off=OFF)),
    "swiglu": (dict(dgate=ROWS_N, dup=ROWS_N, hw=ROWS_N, dw=SLOTS),
               dict(dh=ROWS_N, gq=CAP * N, gs=S_N, uq=CAP * N, us=S_N, row_of=SLOTS, w=SLOTS)),
    "dgrad": (dict(dx=ROWS_M), dict(dy=ROWS_N, dy2=ROWS_N, w=W, w2=W, src=SRC, off=OFF)),
    "wgrad": (dict(dw=W, dw2=W), dict(dy=ROWS_N, dy2=ROWS_N, x=CAP * M, xs=S_M, src=SRC, off=OFF)),
    "route": (dict(out=B * M * 4), dict(logits=B * M * 2, ids=SLOTS, dw=SLOTS, map=M * 4)),
}
PAIRS = [(name, o, other) for name, (outs, ins) in CALLS.items() for o in outs for other in (*outs, *ins) if o != other]


@pytest.mark.parametrize("name,o,other", PAIRS)
def test_overlap_is_refused(name, o, other):
    outs, ins = CALLS[name]
    sizes = {**outs, **ins}
    far = {k: (i + 1) << 24 for i, k in enumerate(sizes)}
    may_be_one = (name, o, other) == ("swiglu", "dw", "w")
    # the same address; the first bytes of one the last of the other
    ends = [far[other] + sizes[other] - 16, far[other] - sizes[o] + 16]
    for at in ([] if may_be_one else [far[other]]) + [e for e in ends if e % 16 == 0 and e != far[other]]:
        assert _call(name, {**far, o: at}) == m.MOE_ERR_INVALID_ARG, hex(at)
        assert "overlap" in m.lib().moe_last_error().decode()


def test_bf16_logits_are_not_their_gradients():
    far = {k: (i + 1) << 24 for i, k in enumerate(("out", "logits", "ids", "dw", "map"))}
    assert _call("route", {**far, "out": far["logits"]}) == m.MOE_ERR_INVALID_ARG
    assert "overlap" in m.lib().moe_last_error().decode()
