"""Plain statements of the training step: 8-bit checkpoints, SwiGLU backwards,
input and weight gradients of the grouped products, the router's gradient and the
whole layer's backward pass.

Test infrastructure, as the rest of this package.  fp64 throughout; values are
rounded only where the layer stores a narrower tensor (checkpoints; dh, dgate,
dup, hw, dxd, dx in the activations' type).  Pinned in tests/test_oracle_train.py
by torch's automatic differentiation in fp64, by central differences of the
oracle's own forward pass, and by rational arithmetic for the checkpoints.
"""
from __future__ import annotations

import numpy as np

from . import moe
from . import numerics as nx

CKPT_BLOCK = 128


def checkpoint(v, block: int = CKPT_BLOCK):
    """Codes (int8) and scales (fp32, powers of two) of the rows of v.

    Per block of 128 columns: scale = the smallest 2^e, -126 <= e <= 121, with amax <=
    127 * 2^e (1 for a block of zeros); code = v / scale to the nearest integer, ties
    to even, within +-127.  A block with a NaN or an infinity: scale NaN, codes 0.
    """
    v = np.asarray(v, dtype=np.float64)
    rows, cols = v.shape
    nb = -(-cols // block)
    codes = np.zeros((rows, cols), dtype=np.int8)
    scales = np.ones((rows, nb), dtype=np.float32)
    for b in range(nb):
        part = v[:, b * block:(b + 1) * block]
        amax = np.max(np.abs(part), axis=1)
        bad = ~np.isfinite(amax)
        safe = np.where(bad | (amax == 0), 1.0, amax)
        e = np.full(rows, -126)
        while True:                                    # smallest exponent that holds amax
            more = (safe > 127.0 * 2.0**e) & (e < 121)
            if not more.any():
                break
            e = e + more
        s = np.where(amax == 0, 1.0, 2.0**e)
        with np.errstate(invalid="ignore"):
            c = np.clip(np.rint(part / s[:, None]), -127, 127)
        codes[:, b * block:(b + 1) * block] = np.where(bad[:, None], 0, c)
        scales[:, b] = np.where(bad, np.nan, s)
    return codes, scales


def checkpoint_values(codes, scales, block: int = CKPT_BLOCK):
    return nx.dequantize_fp8_blocks(codes, scales, block)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(x, dtype=np.float64)))


def swiglu_backward(dh, gate, up, row_of, topk_w):
    """dgate, dup, hw (rows, I) and dtopk_w (B, K); rows that no slot names hold NaN."""
    dh, gate, up = (np.asarray(a, dtype=np.float64) for a in (dh, gate, up))
    B, K = row_of.shape
    out = [np.full(dh.shape, np.nan) for _ in range(3)]
    dw = np.zeros((B, K))
    for t in range(B):
        for k in range(K):
            r = int(row_of[t, k])
            if not 0 <= r < dh.shape[0]:
                continue
            w, g, u, d = float(topk_w[t, k]), gate[r], up[r], dh[r]
            sg = sigmoid(g)
            out[0][r] = w * d * u * (sg + g * sg * sigmoid(-g))
            out[1][r] = w * d * g * sg
            out[2][r] = w * g * sg * u
            dw[t, k] = np.sum(d * g * sg * u)
    return out[0], out[1], out[2], dw


def token_rows(tokens, src_of, slots_per_token):
    """Row r of the result is tokens[src_of[r] // slots_per_token], zeros where there is none."""
    tokens = np.asarray(tokens, dtype=np.float64)
    out = np.zeros((len(src_of), tokens.shape[1]))
    for r, s in enumerate(src_of):
        if s >= 0 and s // slots_per_token < tokens.shape[0]:
            out[r] = tokens[s // slots_per_token]
    return out


def dgrad(pairs, offsets, cap):
    """dx[r] = sum over (dy, W) pairs of dy[r] W_j; rows past the last expert's hold NaN."""
    dx = np.full((cap, np.asarray(pairs[0][1]).shape[2]), np.nan)
    for j in range(len(offsets) - 1):
        a, b = min(int(offsets[j]), cap), min(int(offsets[j + 1]), cap)
        dx[a:b] = sum(np.asarray(dy, np.float64)[a:b] @ np.asarray(w, np.float64)[j] for dy, w in pairs)
    return dx


def wgrad(dy, x, offsets, base=None):
    """dW_j = base_j + dY_j^T X_j over the expert's rows."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    E = len(offsets) - 1
    dw = np.zeros((E, dy.shape[1], x.shape[1])) if base is None else np.array(base, dtype=np.float64)
    for j in range(E):
        a, b = min(int(offsets[j]), len(dy)), min(int(offsets[j + 1]), len(dy))
        dw[j] += dy[a:b].T @ x[a:b]
    return dw


def route_backward(logits, ids, dw, score: str = "picks", renorm: bool = True, scale: float = 1.0, phys_of_logical=None):
    """dlogits (B, E) from the Jacobian of the weights, token by token; ids (B, K) as
    the forward call wrote them (physical under a placement map)."""
    lg = np.asarray(logits, dtype=np.float64)
    B, E = lg.shape
    inverse = np.arange(E) if phys_of_logical is None else np.argsort(np.asarray(phys_of_logical))
    out = np.zeros((B, E))
    for t in range(B):
        live = [e for e in range(E) if score == "picks" or not lg[t, e] <= moe.LOWEST_BF16]
        picks = [(int(inverse[i]), float(d)) for i, d in zip(ids[t], dw[t]) if 0 <= i < E]
        picks = [(e, d) for e, d in picks if e in live]
        if not picks:
            continue
        at = np.array([e for e, _ in picks])
        d = np.array([x for _, x in picks])
        if score == "picks":
            w = np.exp(lg[t, at] - lg[t, at].max())
            w /= w.sum()
            out[t, at] = (np.diag(w) - np.outer(w, w)) @ d
            continue
        s = np.zeros(E)
        jac = np.zeros((E, E))                                    # ds / dl
        if score == "sigmoid":
            s[live] = sigmoid(lg[t, live])
            jac[live, live] = s[live] * sigmoid(-lg[t, live])
        else:
            p = np.exp(lg[t, live] - lg[t, live].max())
            s[live] = p / p.sum()
            jac = np.diag(s) - np.outer(s, s)
        p = s[at]
        if renorm and p.sum() == 0.0:
            continue
        dp = (d * scale - (p * d * scale).sum() / p.sum()) / p.sum() if renorm else d * scale
        ds = np.zeros(E)
        ds[at] = dp
        out[t] = jac @ ds
    return out


def layer_backward(x, logits, dout, K, E, e_begin, e_end, weights, act: str, router=None, ids=None, gates=None):
    """Gradients of the layer out = sum_k w_k FFN_e(x) for one rank's experts, with the
    layer's checkpoints and roundings.  weights: (gate, up, down) arrays (E_loc, ...).
    Returns a dict: dx, dtopk_w, dlogits (routed by moe_route, or by the keywords in
    router), gate, up, down (the weights' gradients in fp64)."""
    wg, wu, wd = (np.asarray(w, np.float64) for w in weights)
    if ids is None:
        ids, gates = (moe.route(logits, K) if router is None else moe.route_scored(logits, K, **router))
    T = len(x)
    lay = moe.layout(ids, E, e_begin, e_end, T * K)
    off, row_of, src = lay["offsets"], lay["row_of"], lay["src_of"]
    R = int(off[-1])
    rnd = nx.to_f32 if act == "f32" else nx.to_bf16
    xd = token_rows(x, src, K)
    gate, up = np.zeros((T * K, wg.shape[1])), np.zeros((T * K, wg.shape[1]))
    for j in range(e_end - e_begin):
        a, b = off[j], off[j + 1]
        gate[a:b], up[a:b] = xd[a:b] @ wg[j].T, xd[a:b] @ wu[j].T
    gate, up = checkpoint_values(*checkpoint(gate)), checkpoint_values(*checkpoint(up))
    x8 = token_rows(checkpoint_values(*checkpoint(x)), src, K)
    dyd = token_rows(dout, src, K)
    dh = rnd(np.nan_to_num(dgrad([(dyd, wd)], off, T * K)))
    w32 = nx.to_f32(gates)
    dgate, dup, hw, dw = swiglu_backward(dh, gate, up, row_of, w32)
    dgate, dup, hw = (rnd(np.nan_to_num(v)) for v in (dgate, dup, hw))
    dxd = rnd(np.nan_to_num(dgrad([(dgate, wg), (dup, wu)], off, T * K)))
    dx = np.zeros(np.shape(x))
    for t in range(T):
        for k in range(K):
            if row_of[t, k] >= 0:
                dx[t] += dxd[row_of[t, k]]
    kw = {} if router is None else {k: v for k, v in router.items() if k in ("score", "renorm", "scale")}
    kw.setdefault("score", "picks" if router is None else "sigmoid")
    return {"dx": rnd(dx), "dtopk_w": dw, "dlogits": route_backward(logits, ids, dw, **kw),
            "gate": wgrad(dgate[:R], x8[:R], off), "up": wgrad(dup[:R], x8[:R], off),
            "down": wgrad(dyd[:R], hw[:R], off)}
