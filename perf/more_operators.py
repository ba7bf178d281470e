"""The training step of the MoE layer, as cases to measure: products of the
backward pass grouped by expert, activation checkpoints in 8 bits, and the
router's gradient.

Six operators that one training step uses together: 8-bit checkpoints of rows
and their values; gate/up that leaves gate and up as checkpoints beside h; SwiGLU's backward pass
from them; the input gradients (contraction over the output channels) and the
weight gradients (contraction over each expert's rows, one operand a
checkpoint or gathered from the tokens); the gradient of the routing weights
back to the logits.  With ``own`` false ``run`` is the plain form in elementary
torch operations; with ``own`` true it calls the library.

A checkpoint holds int8 codes and a power-of-two scale for each 128 columns of
a row: the smallest 2^e, -126 <= e <= 121, with amax <= 127 * 2^e (1 for a
block of zeros); code = value / scale to the nearest integer, ties to even.
code * scale has 7 significant bits, so bf16 holds it exactly: outputs held in
checkpoints are returned as those values.

Shapes are those of workloads/: the DeepSeek-V3-shaped layer (E=256, K=8,
H=7168, I=2048) as one EP=8 rank holds it, the GPT-OSS-shaped layer (E=128,
K=4, H=I=2880) and the fp32 toy layer (E=16, K=2, H=128, I=256).
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
# the lowest finite bf16 value: logits at or below it take an expert out
LOW = -(2.0 - 2.0**-7) * 2.0**127
# what one drawn case may cost at most (the largest listed ones)
MAX_WEIGHTS = 32 * 2048 * 7168
MAX_OPS = 4 * 8192 * 7168 * 2048
MAX_VALUES = 8192 * 7168


def listed():
    dsv3 = dict(E=256, K=8, local=32, H=7168, I=2048, f32=False)
    oss = dict(E=128, K=4, H=2880, I=2880, f32=False)
    toy = dict(E=16, K=2, local=16, H=128, I=256, f32=True)
    return [
        # the tokens of a training step, kept in 8 bits for the weight gradients
        dict(name="ckpt_tokens", op="ckpt", rows=8192, cols=7168, f32=False, ragged=False),
        # a few rows of a length that ends inside a block
        dict(name="ckpt_few_rows", op="ckpt", rows=16, cols=2880, f32=False, ragged=True),
        # forward of one EP=8 rank's experts, 256 rows each on average
        dict(name="gate_up_ep_share", op="gate_up", T=8192, **dsv3),
        # a short fine-tuning batch, a quarter of the experts local: the weights stream
        dict(name="gate_up_few_tokens", op="gate_up", T=64, local=32, **oss),
        # between the two input gradients of the same step
        dict(name="swiglu_ep_share", op="swiglu", T=8192, **dsv3),
        # the toy layer's, all fp32: pure latency
        dict(name="swiglu_toy", op="swiglu", T=64, **toy),
        # dh of the rank's rows from the tokens' output gradients
        dict(name="dgrad_down_ep_share", op="dgrad", T=8192, which="down", **dsv3),
        # dx of an odd number of tokens, rows of no whole number of 128-byte lines
        dict(name="dgrad_gate_up_odd", op="dgrad", T=4093, which="gate_up", local=128, **oss),
        # both weight gradients of gate/up from checkpointed tokens, in fp32
        dict(name="wgrad_gate_up_ep_share", op="wgrad", T=8192, which="gate_up", ckpt=True, base=False, dw32=True,
             **dsv3),
        # down's weight gradient added to that of the micro-batches before
        dict(name="wgrad_down_accumulate", op="wgrad", T=4096, which="down", ckpt=False, base=True, dw32=True,
             local=32, **oss),
        # the sigmoid router's logits of a training step
        dict(name="route_bwd_sigmoid", op="route_bwd", T=8192, E=256, K=8, score="sigmoid", renorm=True, scale=2.5,
             bf16=False, masked=False),
        # the toy layer's softmax over the picks
        dict(name="route_bwd_toy", op="route_bwd", T=64, E=16, K=2, score="picks", renorm=True, scale=1.0, bf16=False,
             masked=False),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(["ckpt", "gate_up", "swiglu", "dgrad", "dgrad", "wgrad", "wgrad", "route_bwd"])
    f32 = rng.random() < 0.2
    if op == "ckpt":
        rows, cols = _log_int(rng, 1, 65536), _log_int(rng, 16, 16384, 16)
        while rows * cols > MAX_VALUES // (2 if f32 else 1):
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, cols=cols, f32=f32, ragged=rng.random() < 0.5)
    E = rng.choice([1, 4, 8, 16, 60, 64, 96, 128, 160, 256])
    K = rng.randint(1, min(E, 10))
    T = _log_int(rng, 1, 8192)
    if op == "route_bwd":
        # (one expert, or one pick whose weight is 1 whatever it scores, has no gradient)
        score, E, K = rng.choice(["picks", "sigmoid", "softmax"]), max(E, 4), max(K, 2)
        return dict(op=op, T=T, E=E, K=K, score=score, renorm=score == "picks" or rng.random() < 0.6,
                    scale=1.0 if score == "picks" else rng.choice([1.0, 2.5, 16.0]),
                    bf16=score != "picks" and rng.random() < 0.4, masked=score != "picks" and rng.random() < 0.3)
    local = rng.choice([E, E, max(1, E // 8), max(1, E // 2 - 1)])
    H, I = _log_int(rng, 64, 8192, 16), _log_int(rng, 64, 8192, 16)
    if f32:                       # the fp32 layer is the small one
        T, H, I = min(T, 512), min(H, 1024), min(I, 1024)
    pairs = 2
    while local * H * I > MAX_WEIGHTS // (8 if f32 else 1):
        local = max(1, local // 2)
    while 2 * pairs * T * K * H * I > MAX_OPS // (64 if f32 else 1):
        T = max(1, T // 2)
    case = dict(op=op, T=T, E=E, K=K, local=local, H=H, I=I, f32=f32)
    if op in ("dgrad", "wgrad"):
        case["which"] = rng.choice(["down", "gate_up"])
    if op == "wgrad":
        case.update(ckpt=rng.random() < 0.5, base=rng.random() < 0.3, dw32=f32 or rng.random() < 0.6)
    return case


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)


def _routing(T, E, K, g):
    """ids (T, K) of a softly unbalanced random routing."""
    lg = torch.randn(T, E, generator=g, device="cuda")
    lg += 0.3 * torch.randn(E, generator=g, device="cuda")
    return torch.topk(lg, K, dim=1).indices


def _layout(c, g):
    """The local experts' rows of the contiguous layout: every slot if all experts are
    local, else room for three times the share that balanced routing sends (what exceeds
    it is dropped), and a few rows more, which stay as they are."""
    T, K = c["T"], c["K"]
    flat = _routing(T, c["E"], K, g).flatten()
    order = torch.sort(flat, stable=True).indices
    mean = -(-T * K * c["local"] // c["E"])
    room = min(T * K, 3 * mean + 64)
    cap = room + 37
    slots = order[flat[order] < c["local"]][:room]
    n = slots.numel()
    counts = torch.bincount(flat, minlength=c["E"])[:c["local"]].cpu()
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).clamp(max=room).to(torch.int32).cuda()
    src = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    src[:n] = slots.to(torch.int32)
    row_of = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
    row_of[slots] = torch.arange(n, dtype=torch.int32, device="cuda")
    return dict(offsets=offsets, src_of=src, row_of=row_of.view(T, K), cap=cap, used=n,
                most=max(1, int(counts.max())), expected=max(1, T * K // c["E"]))


def _type(c):
    return torch.float32 if c["f32"] else torch.bfloat16


def _values(shape, c, g, scale=1.0):
    """Rows of one scale each, from quiet to loud ones."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= scale * torch.exp(0.7 * torch.randn((shape[0], 1), generator=g, device="cuda"))
    return x.to(_type(c))


def _weights(local, rows, cols, c, g):
    w = torch.empty((local, rows, cols), dtype=_type(c), device="cuda")
    for j in range(local):
        w[j] = torch.randn((rows, cols), generator=g, device="cuda") / math.sqrt(cols)
    return w


def _checkpoint(rows, cols, g, scale=1.0):
    """Codes of normal values and scales that differ from block to block."""
    q = (torch.randn((rows, cols), generator=g, device="cuda") * 40.0).round_().clamp_(-127, 127).to(torch.int8)
    e = torch.randint(-7, -3, (rows, -(-cols // BLOCK)), generator=g, device="cuda").float()
    return q, torch.exp2(e) * scale


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    if op == "ckpt":
        n, cols = c["rows"], c["cols"]
        st = dict(c=c, x=_values((n, cols), c, g), rows=None,
                  q=torch.zeros((n, cols), dtype=torch.int8, device="cuda"),
                  s=torch.zeros((n, -(-cols // BLOCK)), dtype=torch.float32, device="cuda"),
                  out=torch.zeros((n, cols), dtype=torch.bfloat16, device="cuda"), last=n)
        if c["ragged"]:
            # two experts' rows, a tenth of the buffer behind them unused
            st["last"] = max(1, n - n // 10)
            st["rows"] = torch.tensor([0, st["last"] // 3, st["last"]], dtype=torch.int32, device="cuda")
        return st
    if op == "route_bwd":
        T, E, K = c["T"], c["E"], c["K"]
        lg = torch.randn(T, E, generator=g, device="cuda") * 1.5
        n = torch.full((T,), K, device="cuda")
        if c["masked"]:
            # drained experts, and a token with a single expert left
            gone = torch.rand(E, generator=g, device="cuda") < 0.06
            lg[:, gone] = -math.inf
            lg[T // 3, 1:] = LOW
            lg[T // 3, 0] = 0.5
            n = (lg > LOW).sum(1).clamp(max=K)
        lg = lg.to(torch.bfloat16) if c["bf16"] else lg
        ids = torch.sort(lg.float(), dim=1, descending=True, stable=True).indices[:, :K].to(torch.int32)
        ids = torch.where(torch.arange(K, device="cuda")[None, :] < n[:, None], ids, -1).to(torch.int32).contiguous()
        return dict(c=c, logits=lg, ids=ids, dw=torch.randn(T, K, generator=g, device="cuda"),
                    out=torch.zeros((T, E), dtype=torch.float32, device="cuda"))
    st = dict(c=c, **_layout(c, g))
    T, H, I, cap, local = c["T"], c["H"], c["I"], st["cap"], c["local"]

    def zeros(*shape, dtype=_type(c)):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    if op == "gate_up":
        st.update(xd=_values((cap, H), c, g), wg=_weights(local, I, H, c, g), wu=_weights(local, I, H, c, g),
                  h=zeros(cap, I), gq=zeros(cap, I, dtype=torch.int8), uq=zeros(cap, I, dtype=torch.int8),
                  gs=zeros(cap, -(-I // BLOCK), dtype=torch.float32),
                  us=zeros(cap, -(-I // BLOCK), dtype=torch.float32),
                  gate=zeros(cap, I, dtype=torch.bfloat16), up=zeros(cap, I, dtype=torch.bfloat16))
        return st
    if op == "swiglu":
        st["dh"] = _values((cap, I), c, g, 0.05)
        st["gq"], st["gs"] = _checkpoint(cap, I, g)
        st["uq"], st["us"] = _checkpoint(cap, I, g)
        st["w"] = torch.softmax(torch.randn((T, c["K"]), generator=g, device="cuda"), dim=1)
        st.update(dg=zeros(cap, I), du=zeros(cap, I), hw=zeros(cap, I), dw=zeros(T, c["K"], dtype=torch.float32))
        return st
    both = c["which"] == "gate_up"
    if op == "dgrad":
        if both:
            st.update(dy=_values((cap, I), c, g, 0.05), dy2=_values((cap, I), c, g, 0.05),
                      w=_weights(local, I, H, c, g), w2=_weights(local, I, H, c, g), out=zeros(cap, H))
        else:
            st.update(dy=_values((T, H), c, g, 0.05), dy2=None, w=_weights(local, H, I, c, g), w2=None,
                      out=zeros(cap, I))
        return st
    dt = torch.float32 if c["dw32"] else torch.bfloat16
    n, m = (I, H) if both else (H, I)
    st["dy"] = _values((cap if both else T, n), c, g, 0.05)
    st["dy2"] = _values((cap, n), c, g, 0.05) if both else None
    if c["ckpt"]:
        st["x"], st["xs"] = _checkpoint(T if both else cap, m, g)
    else:
        st["x"], st["xs"] = _values((T if both else cap, m), c, g), None
    for k in ("", "2")[:2 if both else 1]:
        st["dw" + k] = zeros(local, n, m, dtype=dt)
        st["base" + k] = 0.1 * torch.randn((local, n, m), generator=g, device="cuda") if c["base"] else None
        if c["base"] and dt != torch.float32:
            st["base" + k] = st["base" + k].to(dt)
    return st


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _blocks(v):
    """(rows, blocks, 128) of v, zeros behind the last column."""
    rows, cols = v.shape
    nb = -(-cols // BLOCK)
    return torch.cat([v, v.new_zeros(rows, nb * BLOCK - cols)], dim=1).view(rows, nb, BLOCK)


def _plain_checkpoint(v):
    """The values that the checkpoint of v (rows, cols) fp32 stands for, and its scales."""
    b = _blocks(v)
    amax = b.abs().amax(2)
    m, e = torch.frexp(amax)                                     # amax = m * 2^e, m in [0.5, 1)
    e = torch.where(m <= 127.0 / 128.0, e - 7, e - 6).clamp(-126, 121)
    s = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), 1.0)
    code = torch.round(b / s[:, :, None]).clamp(-127, 127)
    return (code * s[:, :, None]).reshape(v.shape[0], -1)[:, :v.shape[1]], s


def _decode(q, s):
    return (_blocks(q.float()) * s[:, :, None]).reshape(q.shape[0], -1)[:, :q.shape[1]]


def _places(st):
    """(local, most) row of every expert's n-th place; places without a row name row `cap`."""
    place = torch.arange(st["most"], device="cuda")[None, :]
    first, last = st["offsets"][:-1].long()[:, None], st["offsets"][1:].long()[:, None]
    return torch.where(first + place < last, first + place, st["cap"])


def _padded(t, at):
    """Rows of t in 32 bits by (expert, place); at = len(t) names a row of zeros."""
    return torch.cat([t.float(), torch.zeros_like(t[:1], dtype=torch.float32)])[at]


def _token_of(st, at):
    """The tokens of padded rows; places without a row name token T."""
    src = torch.cat([st["src_of"].long(), st["src_of"].new_full((1,), -1).long()])[at]
    return torch.where(src >= 0, src // st["c"]["K"], st["c"]["T"])


def _unpadded(st, v, at, dtype):
    out = torch.zeros((st["cap"] + 1, v.shape[2]), dtype=dtype, device="cuda")
    out[at.flatten()] = v.reshape(-1, v.shape[2]).to(dtype)
    out[st["cap"]] = 0
    return out[:st["cap"]]


def _plain_route(st):
    c, l = st["c"], st["logits"].float()
    T, E = l.shape
    ids = st["ids"].long()
    on = ids >= 0
    at = ids.clamp(min=0)
    dw = torch.where(on, st["dw"], 0.0)
    if c["score"] == "picks":
        z = l.gather(1, at)
        e = torch.exp(z - z.amax(1, keepdim=True))
        w = e / e.sum(1, keepdim=True)
        return torch.zeros_like(l).scatter_add_(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
    live = l > LOW
    if c["score"] == "sigmoid":
        s = torch.where(live, 1.0 / (1.0 + torch.exp(-l)), 0.0)
    else:
        e = torch.where(live, torch.exp(l - torch.where(live, l, -math.inf).amax(1, keepdim=True)), 0.0)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    sp = torch.where(on, s.gather(1, at), 0.0)
    if c["renorm"]:
        total = sp.sum(1, keepdim=True)
        share = torch.where(total > 0, sp / total, 0.0)
        a = torch.where(total > 0, c["scale"] / total * (dw - (share * dw).sum(1, keepdim=True)), 0.0)
    else:
        a = c["scale"] * dw
    a = torch.zeros_like(l).scatter_add_(1, at, torch.where(on, a, 0.0))
    if c["score"] == "sigmoid":
        return torch.where(live, a * s / (1.0 + torch.exp(l)), 0.0)
    return s * (a - (s * a).sum(1, keepdim=True))


def _plain_run(st):
    c = st["c"]
    op = c["op"]
    if op == "route_bwd":
        return {"dlogits": _plain_route(st)}
    if op == "ckpt":
        v, s = _plain_checkpoint(st["x"].float())
        used = (torch.arange(c["rows"], device="cuda") < st["last"])[:, None]
        return {"values": torch.where(used, v, 0.0).to(torch.bfloat16), "scales": torch.where(used, s, 0.0)}
    if op == "swiglu":
        gate, up, dh = _decode(st["gq"], st["gs"]), _decode(st["uq"], st["us"]), st["dh"].float()
        used = (torch.arange(st["cap"], device="cuda") < st["used"])[:, None]
        w = torch.where(used, st["w"].flatten()[st["src_of"].long().clamp(min=0)][:, None], 0.0)
        sg = 1.0 / (1.0 + torch.exp(-gate))
        h = gate * sg * up
        dw = torch.cat([(dh * h).sum(1), dh.new_zeros(1)])
        t = _type(c)
        return {"dgate": (w * dh * up * sg * (1.0 + gate * (1.0 - sg))).to(t), "dup": (w * dh * gate * sg).to(t),
                "hw": (w * h).to(t), "dw": dw[st["row_of"].long()]}
    at = _places(st)
    if op == "gate_up":
        x = _padded(st["xd"], at)
        gate = torch.bmm(x, st["wg"].float().transpose(1, 2))
        up = torch.bmm(x, st["wu"].float().transpose(1, 2))
        h = _unpadded(st, gate / (1.0 + torch.exp(-gate)) * up, at, _type(c))
        gate, _ = _plain_checkpoint(_unpadded(st, gate, at, torch.float32))
        up, _ = _plain_checkpoint(_unpadded(st, up, at, torch.float32))
        return {"h": h, "gate": gate.to(torch.bfloat16), "up": up.to(torch.bfloat16)}
    both = c["which"] == "gate_up"
    if op == "dgrad":
        dx = torch.bmm(_padded(st["dy"], at if both else _token_of(st, at)), st["w"].float())
        if both:
            dx = dx + torch.bmm(_padded(st["dy2"], at), st["w2"].float())
        return {"dx": _unpadded(st, dx, at, _type(c))}
    x = st["x"] if st["xs"] is None else _decode(st["x"], st["xs"])
    x = _padded(x, _token_of(st, at) if both else at)
    out = {}
    for k in ("", "2")[:2 if both else 1]:
        dw = torch.bmm(_padded(st["dy" + k], at if both else _token_of(st, at)).transpose(1, 2).contiguous(), x)
        if st["base" + k] is not None:
            dw += st["base" + k].float()
        out["dw" + k] = dw.to(st["dw" + k].dtype)
    return out


# ----------------------------------------------------------------------------
# the library's calls
# ----------------------------------------------------------------------------
def _own_run(st):
    import combine_grouped_gemm_amd as m
    c = st["c"]
    op = c["op"]
    if op == "route_bwd":
        kw = {} if c["score"] == "picks" else dict(renorm=c["renorm"], scale=c["scale"])
        return {"dlogits": m.moe_route_backward(st["logits"], st["ids"], st["dw"], score=c["score"],
                                                dlogits=st["out"], **kw)}
    if op == "ckpt":
        q, s = m.moe_checkpoint_rows(st["x"], st["rows"], q=st["q"], scales=st["s"])
        return {"values": m.moe_checkpoint_values(q, s, st["rows"], out=st["out"]), "scales": s}
    if op == "swiglu":
        dg, du, hw, dw = m.moe_swiglu_backward(st["dh"], st["gq"], st["gs"], st["uq"], st["us"], st["row_of"], st["w"],
                                               dgate=st["dg"], dup=st["du"], hw=st["hw"], dtopk_w=st["dw"])
        return {"dgate": dg, "dup": du, "hw": hw, "dw": dw}
    if op == "gate_up":
        h, (gq, gs), (uq, us) = m.moe_ffn_gate_up_train(
            st["xd"], st["offsets"], st["wg"], st["wu"], h=st["h"], gate_q=st["gq"], gate_scales=st["gs"],
            up_q=st["uq"], up_scales=st["us"], expected_rows=st["expected"])
        return {"h": h, "gate": m.moe_checkpoint_values(gq, gs, st["offsets"], out=st["gate"]),
                "up": m.moe_checkpoint_values(uq, us, st["offsets"], out=st["up"])}
    both = c["which"] == "gate_up"
    if op == "dgrad":
        rows = {} if both else dict(src_of=st["src_of"], slots_per_token=c["K"])
        return {"dx": m.moe_ffn_dgrad(st["dy"], st["offsets"], st["w"], dy2=st["dy2"], w2=st["w2"], dx=st["out"],
                                      expected_rows=st["expected"], **rows)}
    dw = m.moe_ffn_wgrad(st["dy"], st["x"], st["offsets"], x_scales=st["xs"], dy2=st["dy2"], src_of=st["src_of"],
                         slots_per_token=c["K"], gather="x" if both else "dy", base=st["base"],
                         base2=st.get("base2"), dw=st["dw"], dw2=st.get("dw2"), expected_rows=st["expected"])
    return {"dw": dw[0], "dw2": dw[1]} if both else {"dw": dw}


def run(state):
    if own:
        return _own_run(state)
    return _plain_run(state)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    c = case
    op = c["op"]
    size = 4 if c.get("f32") else 2
    if op == "ckpt":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (size + 1 + 2 + 4 / BLOCK), "flops": 4 * n}
    T, E, K = c["T"], c["E"], c["K"]
    if op == "route_bwd":
        seen = T * (E if c["score"] == "softmax" else K)
        return {"bytes": seen * (2 if c["bf16"] else 4) + 8 * T * K + 4 * T * E, "flops": 8 * T * K}
    H, I = c["H"], c["I"]
    rows = T * K * c["local"] / E                      # mean over routings
    touched = c["local"] * (1.0 - (1.0 - K / E) ** T)  # experts with a row
    some = T * (1.0 - (1.0 - c["local"] / E) ** K)     # tokens with a local slot
    if op == "gate_up":
        return {"bytes": size * (touched * 2 * H * I + rows * (H + I)) + rows * 2 * I * (1 + 2 + 4 / BLOCK),
                "flops": 4 * rows * H * I}
    if op == "swiglu":
        return {"bytes": rows * I * (4 * size + 2 + 8 / BLOCK) + 12 * T * K, "flops": 20 * rows * I}
    both = c["which"] == "gate_up"
    if op == "dgrad":
        moved = (rows * (2 * I + H) + touched * 2 * H * I) if both else (some * H + rows * I + touched * H * I)
        return {"bytes": size * moved, "flops": (4 if both else 2) * rows * H * I}
    xs = 1 + 4 / BLOCK if c["ckpt"] else size
    dw = (4 if c["dw32"] else 2) * c["local"] * H * I * (2 if c["base"] else 1)
    moved = (rows * 2 * I * size + some * H * xs + 2 * dw) if both else (some * H * size + rows * I * xs + dw)
    return {"bytes": moved, "flops": (4 if both else 2) * rows * H * I}


# ----------------------------------------------------------------------------
# 64-bit results from the definitions
# ----------------------------------------------------------------------------
def _exact_checkpoint(v):
    """What the checkpoint of v (rows, cols) in 64 bits stands for, block by block."""
    out = torch.zeros_like(v)
    scales = torch.ones((v.shape[0], -(-v.shape[1] // BLOCK)), dtype=torch.float64, device=v.device)
    for k, b in enumerate(range(0, v.shape[1], BLOCK)):
        part = v[:, b:b + BLOCK]
        amax = part.abs().max(dim=1).values
        e = torch.ceil(torch.log2(amax.clamp(min=2.0**-140) / 127.0))
        e = torch.where(amax <= 127.0 * torch.exp2(e - 1), e - 1, e)     # log2 next to a power of two
        e = torch.where(amax > 127.0 * torch.exp2(e), e + 1, e).clamp(-126, 121)
        s = torch.where(amax > 0, torch.exp2(e), 1.0)
        out[:, b:b + BLOCK] = torch.round(part / s[:, None]).clamp(-127, 127) * s[:, None]
        scales[:, k] = s
    return out, scales


def _exact_decode(q, s):
    return q.double() * s.double().repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]


def _exact_route(c, st):
    l = st["logits"].double().cpu()
    ids, dw = st["ids"].cpu(), st["dw"].double().cpu()
    out = torch.zeros_like(l)
    for t in range(c["T"]):
        k = (ids[t] >= 0).nonzero().flatten()
        e, d = ids[t][k].long(), dw[t][k]
        if not k.numel():
            continue
        if c["score"] == "picks":
            w = torch.softmax(l[t][e], dim=0)
            out[t][e] = w * (d - (w * d).sum())
            continue
        live = (l[t] > LOW).nonzero().flatten()
        s = torch.zeros(c["E"], dtype=torch.float64)
        s[live] = torch.sigmoid(l[t][live]) if c["score"] == "sigmoid" else torch.softmax(l[t][live], dim=0)
        p = s[e]
        a = c["scale"] * d
        if c["renorm"]:
            a = (a - (p / p.sum() * a).sum()) / p.sum() if p.sum() > 0 else torch.zeros_like(a)
        if c["score"] == "sigmoid":
            out[t][e] = a * p * torch.sigmoid(-l[t][e])
        else:
            out[t] = -s * (p * a).sum()
            out[t][e] += p * a
    return out


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op = c["op"]
    if op == "route_bwd":
        return {"dlogits": _exact_route(c, st)}
    if op == "ckpt":
        n = st["last"]
        v = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")
        s = torch.zeros(st["s"].shape, dtype=torch.float64, device="cuda")
        v[:n], s[:n] = _exact_checkpoint(st["x"][:n].double())
        return {"values": v, "scales": s}
    T, K, cap, n = c["T"], c["K"], st["cap"], st["used"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if op == "swiglu":
        gate, up = _exact_decode(st["gq"][:n], st["gs"][:n]), _exact_decode(st["uq"][:n], st["us"][:n])
        dh, slot = st["dh"][:n].double(), st["src_of"][:n].long()
        w = st["w"].double().flatten()[slot][:, None]
        sg = torch.sigmoid(gate)
        h = gate * sg * up
        out = {k: torch.zeros((cap, c["I"]), **f64) for k in ("dgate", "dup", "hw")}
        out["dgate"][:n] = w * dh * up * (sg + gate * sg * torch.sigmoid(-gate))
        out["dup"][:n] = w * dh * sg * gate
        out["hw"][:n] = w * h
        out["dw"] = torch.zeros(T * K, **f64)
        out["dw"][slot] = torch.linalg.vecdot(dh, h)
        out["dw"] = out["dw"].view(T, K)
        return out
    ends = st["offsets"].cpu().tolist()
    spans = [(j, a, b) for j, (a, b) in enumerate(zip(ends, ends[1:])) if b > a]
    if op == "gate_up":
        out = {k: torch.zeros((cap, c["I"]), **f64) for k in ("h", "gate", "up")}
        for j, a, b in spans:
            x = st["xd"][a:b].double()
            gate, up = x @ st["wg"][j].double().t(), x @ st["wu"][j].double().t()
            out["h"][a:b] = torch.sigmoid(gate) * gate * up
            out["gate"][a:b], out["up"][a:b] = _exact_checkpoint(gate)[0], _exact_checkpoint(up)[0]
        return out
    both = c["which"] == "gate_up"
    token = torch.div(st["src_of"][:n], K, rounding_mode="floor").long()
    dys = [st["dy"][:n], st["dy2"][:n]] if both else [st["dy"][token]]
    if op == "dgrad":
        dx = torch.zeros((cap, st["out"].shape[1]), **f64)
        for j, a, b in spans:
            for dy, w in zip(dys, (st["w"], st["w2"])):
                dx[a:b] += dy[a:b].double() @ w[j].double()
        return {"dx": dx}
    x = st["x"].double() if st["xs"] is None else _exact_decode(st["x"], st["xs"])
    x = x[token] if both else x[:n]
    out = {}
    for k, dy in zip(("", "2"), dys):
        base = st["base" + k]
        dw = torch.zeros(st["dw" + k].shape, **f64) if base is None else base.double()
        for j, a, b in spans:
            dw[j] += dy[a:b].double().t() @ x[a:b]
        out["dw" + k] = dw
    return out
