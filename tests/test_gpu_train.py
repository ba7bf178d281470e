"""GPU parity of the training step: 8-bit checkpoints, gate/up that leaves them,
SwiGLU backwards, input and weight gradients, the router's gradient, and the layer
that runs them.

Checkpoints are exact.  Tolerances, per element: a sum of n products in fp32, in
whatever order, is off by at most n * 2^-23 * S, S the sum of the products'
magnitudes (each addition rounds or truncates its partial sum by at most 2^-23 of a
value that S bounds); rounding to bf16 adds half a step, 2^-8 of the value, to fp32
2^-24.  silu and its derivative: the exponential of -g is off by (|g| + 4) * 2^-23 and
the divisions by a few last places, |g| < 60 in these tests, so 2^-17 in all."""
import numpy as np
import pytest
import torch

import oracle
from harness import has_gpu, to_np
from oracle import train as tr

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

HALF = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}
ACT = 2.0**-17
TYPES = [torch.bfloat16, torch.float32]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _near(got, ref, room, what):
    """|got - ref| <= room everywhere; NaN in the same places."""
    got, ref = got.double(), ref.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    over = ((got - ref).abs() - room).nan_to_num(0.0)
    assert over.numel() == 0 or float(over.max()) <= 1e-37, f"{what}: {float(over.max()):.3e} over the bar"


def _values(rows, cols, seed, dtype):
    g = _gen(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return (x * torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))).to(dtype)


def _weights(E, rows, cols, seed, dtype):
    return (torch.randn(E, rows, cols, generator=_gen(seed), device="cuda") / cols**0.5).to(dtype)


def _offsets(counts):
    return torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")


def _codes(rows, cols, seed):
    g = _gen(seed)
    q = (torch.randn(rows, cols, generator=g, device="cuda") * 40).round().clamp(-127, 127).to(torch.int8)
    s = torch.exp2(torch.randint(-8, -4, (rows, -(-cols // 128)), generator=g, device="cuda").float())
    return q, s


def _decoded(q, s):
    return q.double() * s.double().repeat_interleave(128, dim=1)[:, :q.shape[1]]


# row counts of the experts: none, one, less and more than any tile, all in one
COUNTS = {"mixed": [5, 0, 1, 130, 64, 0, 33, 300], "one": [1], "none": [0, 0, 0], "last": [0, 0, 700],
          "even": [128] * 4, "many": [(j * 7) % 5 for j in range(600)]}


# ------------------------------------------------------------------ checkpoints
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [8, 64, 120, 128, 136, 2048, 2880, 7168, 16392])
def test_checkpoint_rows(cols, dtype):
    import combine_grouped_gemm_amd as m
    print(f"[ckpt] cols={cols} {dtype}", flush=True)
    x = _values(37, cols, cols, dtype)
    x[1] = 0.0
    x[2] = 0.0
    x[2, 0] = 127.0
    x[2, 1::2] = 0.5
    x[2, 2::4] = 2.5
    x[3] *= 1e-37
    x[4] = 2.0**-133
    x[5] = 3.38e38
    x[6, 0], x[6, -1] = float("nan"), 1.0
    x[7, cols // 2] = float("inf")
    x[8, -1] = -float("inf")
    x[9] = -0.0
    q, s = m.moe_checkpoint_rows(x)
    rq, rs = tr.checkpoint(to_np(x))
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    want = _decoded(q, s)
    for dt in TYPES:
        back = m.moe_checkpoint_values(q, s, out_dtype=dt)
        assert back.dtype == dt and torch.equal(torch.isnan(back), torch.isnan(want))
        assert torch.equal(back.double().nan_to_num(0.0), want.nan_to_num(0.0))     # exact in bf16 too


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offsets,rows", [([0, 3, 9], range(0, 9)), ([2, 2, 5], range(2, 5)), ([0, 0, 0], range(0)),
                                          ([-3, 4, 99], range(0, 12)), ([7, 3, 1], range(0))])
def test_checkpoint_leaves_other_rows(offsets, rows, dtype):
    import combine_grouped_gemm_amd as m
    x = _values(12, 264, 3, dtype)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    q = torch.full((12, 264), 77, dtype=torch.int8, device="cuda")
    s = torch.full((12, 3), 5.0, device="cuda")
    m.moe_checkpoint_rows(x, off, q=q, scales=s)
    out = torch.full((12, 264), 9.0, dtype=dtype, device="cuda")
    m.moe_checkpoint_values(q, s, off, out=out)
    rq, rs = tr.checkpoint(to_np(x))
    for r in range(12):
        if r in rows:
            np.testing.assert_array_equal(q[r].cpu().numpy(), rq[r])
            np.testing.assert_array_equal(s[r].cpu().numpy(), rs[r])
            assert torch.equal(out[r].double(), _decoded(q[r:r + 1], s[r:r + 1])[0])
        else:
            assert bool((q[r] == 77).all()) and bool((s[r] == 5).all()) and bool((out[r] == 9).all())


def test_checkpoint_of_no_rows_and_a_part_of_a_buffer():
    import combine_grouped_gemm_amd as m
    q, s = m.moe_checkpoint_rows(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0, 1) and m.moe_checkpoint_values(q, s).shape == (0, 64)
    x = _values(7, 72, 1, torch.bfloat16)
    q, s = torch.zeros(7, 72, dtype=torch.int8, device="cuda"), torch.zeros(7, 1, device="cuda")
    for a, b in ((0, 3), (3, 3), (3, 7)):          # rows of 72 codes: the parts start at 8-byte addresses
        m.moe_checkpoint_rows(x[a:b], q=q[a:b], scales=s[a:b])
    rq, rs = tr.checkpoint(to_np(x))
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)


# ------------------------------------------------------------------ gate/up
def _check_gate_up(m, counts, H, I, dtype, hint, packed=False, seed=0):
    E, R = len(counts), sum(counts)
    cap = R + 5
    xd = _values(cap, H, seed + 1, dtype)
    xd[R:] = float("nan")                          # rows of no expert
    wg, wu = _weights(E, I, H, seed + 2, dtype), _weights(E, I, H, seed + 3, dtype)
    nb = -(-I // 128)
    h = torch.full((cap, I), 7.0, dtype=dtype, device="cuda")
    gq, uq = (torch.full((cap, I), 7, dtype=torch.int8, device="cuda") for _ in range(2))
    gs, us = (torch.full((cap, nb), 7.0, device="cuda") for _ in range(2))
    pg, pu = (m.moe_pack_weights(wg), m.moe_pack_weights(wu)) if packed else (wg, wu)
    m.moe_ffn_gate_up_train(xd, _offsets(counts), pg, pu, h=h, gate_q=gq, gate_scales=gs, up_q=uq, up_scales=us,
                            expected_rows=hint)
    for t in (h, gq, uq, gs, us):
        assert bool((t[R:] == 7).all()), "rows behind the last expert's were written"
    at = 0
    for j, n in enumerate(counts):
        if n == 0:
            continue
        x = xd[at:at + n].double()
        rows = slice(at, at + n)
        at += n
        g, u = x @ wg[j].double().t(), x @ wu[j].double().t()
        eg, eu = (H * 2.0**-23 * (x.abs() @ w[j].double().abs().t()) for w in (wg, wu))
        for what, v, e, q, s in (("gate", g, eg, gq, gs), ("up", u, eu, uq, us)):
            sc = s[rows].double().repeat_interleave(128, dim=1)[:, :I]
            _near(_decoded(q[rows], s[rows]), v, 0.5 * sc + e, what)
            pad = torch.nn.functional.pad((v.abs() + 0), (0, nb * 128 - I)).view(n, nb, 128)
            room = torch.nn.functional.pad(e, (0, nb * 128 - I)).view(n, nb, 128).amax(2)
            amax, sd = pad.amax(2), s[rows].double()
            assert bool((amax - room <= 127 * sd).all()), f"{what}: a scale too small"
            assert bool((amax + room > 127 * sd / 2).all()), f"{what}: a scale too large"
            assert torch.equal(torch.frexp(s[rows])[0], torch.full_like(s[rows], 0.5)), "scales are powers of two"
        sg = torch.sigmoid(g)
        ref = g * sg * u
        _near(h[rows], ref, (HALF[dtype] + ACT) * ref.abs() + 1.2 * (u.abs() + eu) * eg + (g * sg).abs() * eu, "h")


GATE_UP = [("mixed", 200, 136, 0), ("mixed", 64, 256, 1), ("mixed", 328, 320, 100), ("mixed", 256, 128, 300),
           ("one", 8, 8, 1), ("one", 1032, 384, 0), ("none", 64, 64, 0), ("last", 128, 264, 700), ("even", 512, 640, 128),
           ("many", 72, 144, 2), ("many", 72, 144, 80), ("many", 72, 144, 250)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name,H,I,hint", GATE_UP)
def test_gate_up_train(name, H, I, hint, dtype):
    import combine_grouped_gemm_amd as m
    print(f"[gate_up_train] {name} H={H} I={I} hint={hint} {dtype}", flush=True)
    _check_gate_up(m, COUNTS[name], H, I, dtype, hint)


@pytest.mark.parametrize("hint", [1, 40, 100, 300])
def test_gate_up_train_packed(hint):
    import combine_grouped_gemm_amd as m
    _check_gate_up(m, COUNTS["mixed"], 200, 264, torch.bfloat16, hint, packed=True)


def test_gate_up_train_of_nan_rows():
    """A row with a NaN spoils its own blocks only."""
    import combine_grouped_gemm_amd as m
    counts, H, I = [3, 40], 64, 136
    xd = _values(43, H, 1, torch.bfloat16)
    wg, wu = _weights(2, I, H, 2, torch.bfloat16), _weights(2, I, H, 3, torch.bfloat16)
    a = m.moe_ffn_gate_up_train(xd, _offsets(counts), wg, wu)
    xd[10, 5] = float("nan")
    b = m.moe_ffn_gate_up_train(xd, _offsets(counts), wg, wu)
    for x, y in zip((a[0], *a[1], *a[2]), (b[0], *b[1], *b[2])):
        assert torch.equal(torch.cat([x[:10], x[11:]]), torch.cat([y[:10], y[11:]]))
    assert bool(torch.isnan(b[0][10]).all()) and bool(torch.isnan(b[1][1][10]).all()) and not bool(b[1][0][10].any())


# ------------------------------------------------------------------ SwiGLU backwards
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,K,I,local", [(1, 1, 8, 1.0), (5, 3, 136, 0.6), (64, 8, 2048, 0.13), (33, 70, 264, 0.9),
                                         (3000, 2, 520, 0.5), (9, 4, 2880, 0.0), (20000, 8, 64, 1.0)])
def test_swiglu_backward(B, K, I, local, dtype):
    import combine_grouped_gemm_amd as m
    print(f"[swiglu] B={B} K={K} I={I} local={local} {dtype}", flush=True)
    g = _gen(B + K + I)
    n = B * K
    cap = n + 3
    perm = torch.randperm(cap, generator=g, device="cuda")[:n].to(torch.int32)
    named = torch.rand(n, generator=g, device="cuda") < local
    row_of = torch.where(named, perm, -1).to(torch.int32)
    if n > 4:
        row_of[1], named[1] = cap, False                    # no such row
        row_of[2], named[2] = 2**31 - 1, False
    gq, gs = _codes(cap, I, 1)
    uq, us = _codes(cap, I, 2)
    gs *= 16.0                                             # g up to 127: both tails of the sigmoid, and -1.28
    gs.clamp_(max=0.25)
    w = torch.rand(B, K, generator=g, device="cuda")
    dh = _values(cap, I, 3, dtype)
    outs = [torch.full((cap, I), 3.0, dtype=dtype, device="cuda") for _ in range(3)]
    dw = torch.full((B, K), 3.0, device="cuda")
    m.moe_swiglu_backward(dh, gq, gs, uq, us, row_of.view(B, K), w, *outs, dw)
    rows = row_of[named].long()
    rest = torch.ones(cap, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert all(bool((o[rest] == 3).all()) for o in outs), "rows that no slot names were written"
    assert bool((dw.flatten()[~named] == 0).all())
    gate, up, d = _decoded(gq, gs)[rows], _decoded(uq, us)[rows], dh[rows].double()
    wr, sg = w.flatten()[named].double()[:, None], torch.sigmoid(gate)
    no = torch.sigmoid(-gate)
    h = gate * sg * up
    half = HALF[dtype]
    ref = wr * d * up * (sg + gate * sg * no)
    _near(outs[0][rows], ref, half * ref.abs() + ACT * (wr * d * up).abs() * (sg + (gate * sg * no).abs()), "dgate")
    _near(outs[1][rows], wr * d * gate * sg, (half + ACT) * (wr * d * gate * sg).abs(), "dup")
    _near(outs[2][rows], wr * h, (half + ACT) * (wr * h).abs(), "hw")
    _near(dw.flatten()[named], (d * h).sum(1), (I * 2.0**-23 + ACT) * (d * h).abs().sum(1), "dtopk_w")


def test_swiglu_backward_of_specials():
    """NaN checkpoints and infinite gradients stay in their row; far gates saturate."""
    import combine_grouped_gemm_amd as m
    I = 256
    gq, uq = (torch.full((4, I), 100, dtype=torch.int8, device="cuda") for _ in range(2))
    gq[3, :128], gq[3, 128:] = 127, -127
    gs, us = torch.ones(4, 2, device="cuda"), torch.ones(4, 2, device="cuda")
    gs[0, 1] = float("nan")
    gs[3] = 2.0**100
    dh = torch.ones(4, I, dtype=torch.bfloat16, device="cuda")
    dh[1, 3] = float("inf")
    row_of = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    w = torch.ones(2, 2, device="cuda")
    dg, du, hw, dw = m.moe_swiglu_backward(dh, gq, gs, uq, us, row_of, w)
    assert bool(torch.isnan(dg[0, 128:]).all()) and bool(torch.isfinite(dg[0, :128]).all()) and bool(torch.isnan(dw[0, 0]))
    assert bool(torch.isinf(dw[0, 1])) and bool(torch.isfinite(dg[2]).all()) and float(dw[1, 0]) == pytest.approx(I * 1e4)
    assert bool((dg[3, :128] == 100).all()) and bool((dg[3, 128:] == 0).all()) and bool((hw[3, 128:] == 0).all())


# ------------------------------------------------------------------ input gradients
def _routed(counts, T, K, cap, seed):
    """src_of of rows that name slots of T tokens, -1 behind them."""
    R = sum(counts)
    src = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    src[:R] = torch.randint(0, T * K, (R,), generator=_gen(seed), device="cuda").to(torch.int32)
    return src


def _check_dgrad(m, counts, N, M, dtype, hint, two, gather, packed=False, seed=0):
    E, R, K = len(counts), sum(counts), 3
    cap, T = R + 5, 41
    src = _routed(counts, T, K, cap, seed) if gather else None
    rows = T if gather else cap
    dys = [_values(rows, N, seed + 1 + i, dtype) for i in range(1 + two)]
    ws = [_weights(E, N, M, seed + 5 + i, dtype) for i in range(1 + two)]
    if not gather:
        for dy in dys:
            dy[R:] = float("nan")
    elif R > 3:
        src[0], src[R - 1], src[R // 2] = -1, T * K, 2**31 - 1       # rows that name no token read zeros
    dx = torch.full((cap, M), 7.0, dtype=dtype, device="cuda")
    pw = [m.moe_pack_weights(w) for w in ws] if packed else ws
    m.moe_ffn_dgrad(dys[0], _offsets(counts), pw[0], dy2=dys[1] if two else None, w2=pw[1] if two else None,
                    src_of=src, slots_per_token=K, dx=dx, expected_rows=hint)
    assert bool((dx[R:] == 7).all()), "rows behind the last expert's were written"
    at = 0
    for j, n in enumerate(counts):
        ref = torch.zeros(n, M, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(ref)
        for dy, w in zip(dys, ws):
            d = dy[at:at + n].double()
            if gather:
                s = src[at:at + n].long()
                ok = (s >= 0) & (s // K < T)
                d = torch.where(ok[:, None], dy[(s // K).clamp(0, T - 1)].double(), 0.0)
            ref += d @ w[j].double()
            mag += d.abs() @ w[j].double().abs()
        _near(dx[at:at + n], ref, HALF[dtype] * ref.abs() + (1 + two) * N * 2.0**-23 * mag, f"expert {j}")
        at += n


DGRAD = [("mixed", 200, 136, 0), ("mixed", 64, 264, 1), ("mixed", 328, 320, 30), ("mixed", 256, 512, 100),
         ("mixed", 136, 776, 300), ("one", 8, 8, 1), ("one", 1032, 392, 0), ("none", 64, 64, 0), ("last", 128, 264, 700),
         ("even", 512, 640, 128), ("many", 72, 144, 2), ("many", 72, 144, 80), ("many", 72, 144, 250)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("two,gather", [(0, False), (0, True), (1, False), (1, True)])
@pytest.mark.parametrize("name,N,M,hint", DGRAD)
def test_dgrad(name, N, M, hint, two, gather, dtype):
    import combine_grouped_gemm_amd as m
    print(f"[dgrad] {name} N={N} M={M} hint={hint} two={two} gather={gather} {dtype}", flush=True)
    _check_dgrad(m, COUNTS[name], N, M, dtype, hint, two, gather)


@pytest.mark.parametrize("counts", [[128, 129, 192, 193, 16, 17, 144], [320, 321, 256, 257, 224, 33], [641, 96, 0, 384, 209]])
@pytest.mark.parametrize("out_dim", [64, 136, 584, 832])
def test_dgrad_tiles_of_every_row_count(counts, out_dim):
    """Row counts at which a tile's rings and fragments change, contractions of one to thirteen steps."""
    import combine_grouped_gemm_amd as m
    print(f"[dgrad tiles] {counts} out_dim={out_dim}", flush=True)
    _check_dgrad(m, counts, out_dim, 264, torch.bfloat16, 0, 0, False)
    _check_dgrad(m, counts, out_dim, 512, torch.bfloat16, 200, 1, True)


@pytest.mark.parametrize("hint", [1, 40, 100, 300])
@pytest.mark.parametrize("two", [0, 1])
def test_dgrad_packed(two, hint):
    import combine_grouped_gemm_amd as m
    _check_dgrad(m, COUNTS["mixed"], 200, 264, torch.bfloat16, hint, two, False, packed=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_dgrad_does_not_depend_on_the_hint(dtype):
    """Within the order of the sums: every tile shape against the first."""
    import combine_grouped_gemm_amd as m
    counts, N, M = COUNTS["mixed"], 328, 264
    dy, w = _values(sum(counts), N, 1, dtype), _weights(len(counts), N, M, 2, dtype)
    outs = [m.moe_ffn_dgrad(dy, _offsets(counts), w, expected_rows=h) for h in (1, 40, 100, 300, 1)]
    assert torch.equal(outs[0], outs[4])
    for o in outs[1:4]:
        mag = torch.cat([dy[a:b].double().abs() @ w[j].double().abs() for j, (a, b) in
                         enumerate(zip(np.cumsum([0, *counts]), np.cumsum(counts)))])
        _near(o, outs[0], 2 * HALF[dtype] * outs[0].double().abs() + 2 * N * 2.0**-23 * mag, "hint")


# ------------------------------------------------------------------ weight gradients
def _check_wgrad(m, counts, N, M, dtype, two, gather, ckpt, base, dw_dtype, hint=0, seed=0):
    E, R, K, T = len(counts), sum(counts), 3, 41
    cap = R + 5
    src = _routed(counts, T, K, cap, seed)
    dys = [_values(T if gather == "dy" else cap, N, seed + 1 + i, dtype) for i in range(1 + two)]
    xr = T if gather == "x" else cap
    x, xs = (_codes(xr, M, seed + 5) if ckpt else (_values(xr, M, seed + 5, dtype), None))
    if gather and R > 3:
        src[0], src[R - 1], src[R // 2] = -1, T * K, 2**31 - 1       # rows that add nothing
    if gather != "dy":
        for dy in dys:
            dy[R:] = float("nan")
    if gather != "x":
        if ckpt:
            xs[R:] = float("nan")
        else:
            x[R:] = float("nan")
    dws = [torch.full((E, N, M), float("nan"), dtype=dw_dtype, device="cuda") for _ in range(1 + two)]
    bases = [None] * (1 + two)
    if base:
        bases = [_weights(E, N, M, seed + 8 + i, dw_dtype) for i in range(1 + two)]
    if base == "in place":
        dws = [b.clone() for b in bases]
    kw = dict(zip(("base", "base2"), dws if base == "in place" else bases))
    kw.update(dict(zip(("dw", "dw2"), dws)))
    m.moe_ffn_wgrad(dys[0], x, _offsets(counts), x_scales=xs, dy2=dys[1] if two else None, src_of=src,
                    slots_per_token=K, gather=gather, expected_rows=hint, **kw)
    xv = _decoded(x, xs) if ckpt else x.double()
    tok = (src.long() // K).clamp(0, T - 1)
    ok = ((src >= 0) & (src // K < T))[:R, None]
    xv = torch.where(ok, xv[tok[:R]], 0.0) if gather == "x" else xv[:R]
    for dy, dw, b in zip(dys, dws, bases):
        d = torch.where(ok, dy[tok[:R]].double(), 0.0) if gather == "dy" else dy[:R].double()
        at = 0
        for j, n in enumerate(counts):
            p, q = d[at:at + n], xv[at:at + n]
            ref = p.t() @ q + (0.0 if b is None else b[j].double())
            mag = p.abs().t() @ q.abs() + (0.0 if b is None else b[j].double().abs())
            _near(dw[j], ref, HALF[dw_dtype] * ref.abs() + (n + 1) * 2.0**-23 * mag, f"expert {j}")
            at += n


WGRAD = [("mixed", 200, 136), ("mixed", 64, 264), ("mixed", 328, 320), ("one", 8, 8), ("one", 1032, 392),
         ("none", 64, 64), ("last", 128, 264), ("even", 520, 640), ("many", 72, 144)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("two", [0, 1])
@pytest.mark.parametrize("gather", [None, "x", "dy"])
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("name,N,M", WGRAD)
def test_wgrad(name, N, M, ckpt, gather, two, dtype):
    import combine_grouped_gemm_amd as m
    print(f"[wgrad] {name} N={N} M={M} ckpt={ckpt} gather={gather} two={two} {dtype}", flush=True)
    _check_wgrad(m, COUNTS[name], N, M, dtype, two, gather, ckpt, None, torch.float32)


@pytest.mark.parametrize("dw_dtype", TYPES)
@pytest.mark.parametrize("two", [0, 1])
@pytest.mark.parametrize("base", [None, "apart", "in place"])
def test_wgrad_bases_and_types(base, two, dw_dtype):
    import combine_grouped_gemm_amd as m
    _check_wgrad(m, COUNTS["mixed"], 136, 264, torch.bfloat16, two, "x", True, base, dw_dtype)
    _check_wgrad(m, COUNTS["mixed"], 520, 72, torch.bfloat16, two, "dy", False, base, dw_dtype, hint=300)
    if dw_dtype == torch.float32:
        _check_wgrad(m, COUNTS["mixed"], 72, 136, torch.float32, two, None, False, base, dw_dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("gather", ["x", "dy"])
def test_wgrad_rows_without_a_source_add_nothing_whatever_the_other_holds(gather, ckpt, dtype):
    import combine_grouped_gemm_amd as m
    counts, N, M, K, T = [70, 3], 72, 136, 2, 9
    src = _routed(counts, T, K, 73, 4)
    src[5], src[66], src[71] = -1, -1, 2**31 - 1
    keep = [r for r in range(73) if r not in (5, 66, 71)]
    dy = _values(T if gather == "dy" else 73, N, 1, dtype)
    x, xs = _codes(T if gather == "x" else 73, M, 2) if ckpt else (_values(T if gather == "x" else 73, M, 2, dtype), None)
    for r in (5, 66, 71):
        if gather == "x":
            dy[r] = float("nan")
        elif ckpt:
            xs[r] = float("nan")
        else:
            x[r] = float("inf")
    kw = dict(gather=gather, slots_per_token=K, dw_dtype=torch.float32)
    got = m.moe_ffn_wgrad(dy, x, _offsets(counts), x_scales=xs, src_of=src, **kw)
    assert bool(torch.isfinite(got).all())
    xv = (_decoded(x, xs) if ckpt else x.double()).cpu()
    d, tok = dy.double().cpu(), (src.long() // K).cpu()
    for j, rows in enumerate(([r for r in keep if r < 70], [r for r in keep if r >= 70])):
        p, q = (d[tok[rows]], xv[rows]) if gather == "dy" else (d[rows], xv[tok[rows]])
        ref, mag = p.t() @ q, p.abs().t() @ q.abs()
        _near(got[j].cpu(), ref, 2.0**-24 * ref.abs() + (len(rows) + 1) * 2.0**-23 * mag, f"expert {j}")


def test_wgrad_of_a_nan_stays_with_its_expert_and_column():
    import combine_grouped_gemm_amd as m
    counts = [40, 50, 3]
    dy, x = _values(93, 72, 1, torch.bfloat16), _values(93, 136, 2, torch.bfloat16)
    a = m.moe_ffn_wgrad(dy, x, _offsets(counts))
    x[60, 17] = float("nan")
    b = m.moe_ffn_wgrad(dy, x, _offsets(counts))
    bad = torch.isnan(b)
    assert bool(bad[1, :, 17].all()) and int(bad.sum()) == 72
    assert torch.equal(a[~bad], b[~bad])
    # a checkpoint's NaN block
    q, s = _codes(93, 136, 3)
    s[2, 1] = float("nan")
    c = m.moe_ffn_wgrad(dy, q, _offsets(counts), x_scales=s)
    assert bool(torch.isnan(c[0, :, 128:]).all()) and int(torch.isnan(c).sum()) == 72 * 8


# ------------------------------------------------------------------ router
@pytest.mark.parametrize("score,renorm,scale", [("picks", True, 1.0), ("sigmoid", True, 2.5), ("sigmoid", False, 1.0),
                                                ("softmax", True, 1.0), ("softmax", False, 16.0)])
@pytest.mark.parametrize("T,E,K,mapped,shared", [(1, 2, 1, False, 0), (67, 16, 2, False, 1), (300, 256, 8, True, 0),
                                                 (33, 60, 60, False, 0), (20, 1000, 70, True, 3), (5, 1024, 1024, False, 0),
                                                 (9000, 64, 6, False, 0)])
def test_route_backward(T, E, K, mapped, shared, score, renorm, scale):
    import combine_grouped_gemm_amd as m
    print(f"[route_bwd] T={T} E={E} K={K} {score} {renorm} mapped={mapped} shared={shared}", flush=True)
    g = _gen(T + E)
    lg = torch.randn(T, E, generator=g, device="cuda") * 3
    dtype = torch.float32 if score == "picks" or K % 2 == 0 else torch.bfloat16
    if score != "picks" and T > 2:
        lg[:, torch.rand(E, generator=g, device="cuda") < 0.1] = -float("inf")
        lg[T // 2] = -float("inf")
        lg[T // 3, 1:] = -(2.0 - 2.0**-7) * 2.0**127
    lg = lg.to(dtype)
    phys = torch.randperm(E, generator=g, device="cuda").to(torch.int32) if mapped else None
    if score == "picks":
        ids, w = m.moe_route_mapped(lg, K, phys) if mapped else m.moe_route_shared(lg, K, shared)
        if mapped and shared:
            fill = torch.full((T, shared), E, dtype=torch.int32, device="cuda")
            ids = torch.cat([ids, fill], 1).contiguous()
    else:
        ids, w = m.moe_route_scored(lg, K, score=score, renorm=renorm, scale=scale, phys_of_logical=phys, n_shared=shared)
    dw = torch.randn(T, K + shared, generator=g, device="cuda")
    dw[:, K:] = float("nan")                               # never read
    kw = {} if score == "picks" else dict(renorm=renorm, scale=scale)
    got = m.moe_route_backward(lg, ids, dw, score=score, phys_of_logical=phys, n_shared=shared,
                               dlogits=torch.full((T, E), 9.0, device="cuda"), **kw)
    # dlogits are linear in dw: the same formula on magnitudes bounds what cancels.  Each of the
    # K terms is a product of a handful of fp32 roundings (exponential 4, quotients, scale)
    n, d = ids[:, :K].cpu().numpy(), dw[:, :K].double().cpu().numpy()
    take = range(T) if T <= 300 else range(0, T, 31)
    p = None if phys is None else phys.cpu().numpy()
    l = to_np(lg)[list(take)]
    ref = tr.route_backward(l, n[list(take)], d[list(take)], score, renorm, scale, p)
    room = np.zeros_like(ref)
    big = np.abs(d[list(take)]).max(1, keepdims=True)
    for i, t in enumerate(take):
        one = tr.route_backward(l[i:i + 1], n[t:t + 1], np.ones((1, K)), score, False if score != "picks" else True, scale, p)
        s = tr.route_backward(l[i:i + 1], n[t:t + 1], np.eye(1, K), score, False if score != "picks" else True, scale, p)
        top = np.abs(one).max() + np.abs(s).max() + scale
        total = 1.0
        if renorm and score != "picks":
            picks = w[t, :K].double().cpu().numpy()
            total = _score_sum(l[i], n[t], score, p)
        room[i] = (K + 32) * 2.0**-23 * big[i] * top / max(total, 1e-30)
    _near(got[list(take)].cpu(), torch.tensor(ref), torch.tensor(room), "dlogits")


def _score_sum(l, ids, score, phys):
    """Sum of the picks' scores of one token."""
    live = l > oracle.moe.LOWEST_BF16
    s = np.zeros(len(l))
    if score == "sigmoid":
        s[live] = tr.sigmoid(l[live])
    elif live.any():
        e = np.exp(l[live] - l[live].max())
        s[live] = e / e.sum()
    inv = np.arange(len(l)) if phys is None else np.argsort(phys)
    return max(sum(s[inv[i]] for i in ids if 0 <= i < len(l)), 1e-30)


# ------------------------------------------------------------------ the layer
def _train_layer(m, T, E, K, H, I, e_begin, e_end, dtype, router=None, n_shared=0, segs=1, seed=0):
    name = {torch.float32: "f32", torch.bfloat16: "bf16"}[dtype]
    cut = [T // segs] * (segs - 1) + [T - T // segs * (segs - 1)]
    layer = m.MoELayer(cut, E, K, H, I, e_begin, e_end, name, name, name, router=router, n_shared=n_shared, train=True)
    x = list(torch.split(_values(T, H, seed + 1, dtype), cut))
    lg = torch.randn(T, E, generator=_gen(seed + 2), device="cuda")
    n = e_end - e_begin + n_shared
    w = {"gate": _weights(n, I, H, seed + 3, dtype), "up": _weights(n, I, H, seed + 4, dtype),
         "down": _weights(n, H, I, seed + 5, dtype)}
    dout = _values(T, H, seed + 6, dtype)
    return layer, [p.contiguous() for p in x], lg, w, dout


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,K,H,I,e_begin,e_end,segs,router", [
    (64, 16, 2, 128, 256, 0, 16, 8, None), (50, 8, 3, 136, 72, 2, 5, 1, None), (1, 4, 2, 64, 64, 0, 4, 1, None),
    (90, 12, 4, 200, 264, 0, 12, 3, dict(score="sigmoid", n_groups=4, topk_groups=2, scale=2.5)),
    (40, 6, 2, 64, 128, 3, 6, 2, dict(score="softmax", renorm=False))])
def test_layer_backward(T, E, K, H, I, e_begin, e_end, segs, router, dtype):
    """The whole step against the oracle's.  Both round at the same places; a sum on the
    other side of a rounding moves dh or a checkpoint by a step, so the bar is that of
    the layer's forward pass: relative L2 of 1e-2 in bf16, and in fp32 the checkpoints'
    steps on border values, 1e-3."""
    import combine_grouped_gemm_amd as m
    print(f"[layer] T={T} E={E} K={K} H={H} I={I} {router} {dtype}", flush=True)
    layer, x, lg, w, dout = _train_layer(m, T, E, K, H, I, e_begin, e_end, dtype, router, segs=segs)
    layer.forward(x, lg, w)
    grads = layer.new_grads()
    dx, dlogits = layer.backward(dout, lg, w, grads)
    ref = tr.layer_backward(to_np(torch.cat(x)), to_np(lg), to_np(dout), K, E, e_begin, e_end,
                            [to_np(w[k]) for k in ("gate", "up", "down")], "f32" if dtype == torch.float32 else "bf16",
                            router)
    bar = 1e-2 if dtype == torch.bfloat16 else 1e-3
    for what, got in (("dx", dx), ("dlogits", dlogits), ("dtopk_w", layer.dtopk_w), *grads.items()):
        r = ref[what]
        off = np.linalg.norm(to_np(got) - r)
        assert off <= bar * np.linalg.norm(r) + 1e-30, f"{what}: {off / np.linalg.norm(r):.3e}"


def test_layer_gradients_against_differences():
    """dlogits, dx and the weights' gradients of the fp32 layer against central differences
    of the oracle's forward pass in 64 bits; what separates them are the checkpoints, whose
    half steps are at most amax / 127 a value: 3 per cent of a direction's derivative."""
    import combine_grouped_gemm_amd as m
    T, E, K, H, I = 24, 4, 2, 64, 64
    layer, x, lg, w, dout = _train_layer(m, T, E, K, H, I, 0, E, torch.float32, seed=3)
    layer.forward(x, lg, w)
    grads = layer.new_grads()
    dx, dlogits = layer.backward(dout, lg, w, grads)
    values = {"x": to_np(x[0]), "lg": to_np(lg), **{k: to_np(v) for k, v in w.items()}}
    ids, _ = oracle.route(values["lg"], K)

    def loss(v):
        out = 0.0
        for t in range(T):
            s = np.exp(v["lg"][t, ids[t]] - v["lg"][t, ids[t]].max())
            s /= s.sum()
            for k in range(K):
                e = ids[t, k]
                g = v["gate"][e] @ v["x"][t]
                h = g * tr.sigmoid(g) * (v["up"][e] @ v["x"][t])
                out += s[k] * (to_np(dout)[t] @ (v["down"][e] @ h))
        return out

    g = np.random.default_rng(1)
    for name, got in (("x", dx), ("lg", dlogits), *grads.items()):
        grad = to_np(got)
        # along the gradient itself: its norm is the derivative
        step = grad / np.linalg.norm(grad) + 0.3 * g.standard_normal(grad.shape) / grad.size**0.5
        a, b = dict(values), dict(values)
        a[name], b[name] = values[name] + 1e-5 * step, values[name] - 1e-5 * step
        want = (loss(a) - loss(b)) / 2e-5
        assert abs((grad * step).sum() - want) <= 0.03 * abs(want), name


def test_layer_accumulates_over_micro_batches_and_shared_experts():
    import combine_grouped_gemm_amd as m
    layer, x, lg, w, dout = _train_layer(m, 30, 6, 2, 72, 136, 0, 6, torch.bfloat16, n_shared=1, seed=5)
    one, two = layer.new_grads(), layer.new_grads()
    layer.forward(x, lg, w)
    layer.backward(dout, lg, w, one)
    assert float(layer.dtopk_w[:, 2].abs().max()) > 0 and layer.dlogits.shape == (30, 6)
    layer.backward(dout, lg, w, two)
    for k in one:
        assert torch.equal(one[k], two[k])                 # the same from run to run
    layer.backward(dout, lg, w, two, accumulate=True)
    for k in one:
        # base + the same sum, rounded once more
        _near(two[k], 2 * one[k].double(), 40 * 2.0**-23 * (2 * one[k].double().abs() + 1), k)


def test_layer_refuses_what_it_cannot_train():
    import combine_grouped_gemm_amd as m
    for kw in (dict(layout="masked"), dict()):
        act = "bf16" if kw else "int8"
        with pytest.raises(ValueError, match="training needs"):
            m.MoELayer([4], 4, 2, 64, 64, 0, 4, act, "bf16", "bf16", train=True, **kw)
    layer = m.MoELayer([4], 4, 2, 64, 64, 0, 4, "bf16", "bf16", "bf16")
    with pytest.raises(ValueError, match="train=True"):
        layer.backward(None, None, None, None)


def test_layer_trains_on_a_side_stream_and_in_a_graph():
    """Replays, with eager work between them, equal the eager step bit for bit."""
    import combine_grouped_gemm_amd as m
    layer, x, lg, w, dout = _train_layer(m, 200, 8, 2, 264, 136, 0, 8, torch.bfloat16, seed=7)
    grads = layer.new_grads()
    names = ("out", "dx", "dlogits", "dtopk_w", "x_q", "x_s")

    def step():
        layer.forward(x, lg, w)
        layer.backward(dout, lg, w, grads)

    def seen():
        torch.cuda.synchronize()
        R = int(layer.offsets[-1])
        return ([getattr(layer, n).clone() for n in names] + [layer.gate_q[:R].clone(), layer.up_s[:R].clone()] +
                [g.clone() for g in grads.values()])

    step()
    eager = seen()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    for a, b in zip(eager, seen()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        for g in grads.values():
            g.fill_(float("nan"))
        layer.dx.fill_(1.0)
        graph.replay()
        for a, b in zip(eager, seen()):
            assert torch.equal(a, b), f"replay {i}"
        (torch.randn(512, 512, device="cuda") @ torch.randn(512, 512, device="cuda")).sum()
    # new inputs in the same buffers
    lg.copy_(torch.randn(lg.shape, generator=_gen(99), device="cuda"))
    x[0].copy_(_values(200, 264, 98, torch.bfloat16))
    graph.replay()
    replayed = seen()
    step()
    for a, b in zip(replayed, seen()):
        assert torch.equal(a, b)


def _ragged(E, most, seed):
    return [int(v) for v in np.random.default_rng(seed).integers(0, most + 1, E)]


@pytest.mark.parametrize("E,most,cols", [(70, 400, 1032), (70, 400, 2056), (200, 900, 264), (33, 100, 2048), (300, 700, 2056)])
def test_rounds_of_ragged_tiles(E, most, cols):
    """From less than one round of wide tiles to more than the last one's assignment looks back on:
    each tile is done once, whichever block gets it."""
    import combine_grouped_gemm_amd as m
    counts = _ragged(E, most, E + cols)
    print(f"[rounds] E={E} rows={sum(counts)} cols={cols}", flush=True)
    _check_dgrad(m, counts, 72, cols, torch.bfloat16, 200, 0, True)
    _check_gate_up(m, counts, 72, cols, torch.bfloat16, 200)


def test_two_layers_at_once_on_two_streams():
    import combine_grouped_gemm_amd as m
    sets = [_train_layer(m, T, 8, 2, 264, 136, 0, 8, torch.bfloat16, seed=T) for T in (300, 170)]
    grads = [s[0].new_grads() for s in sets]

    def step(k):
        layer, x, lg, w, dout = sets[k]
        layer.forward(x, lg, w)
        layer.backward(dout, lg, w, grads[k])

    def seen(k):
        return [t.clone() for t in (sets[k][0].out, sets[k][0].dx, sets[k][0].dlogits, *grads[k].values())]

    alone = []
    for k in range(2):
        step(k)
        alone.append(seen(k))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                step(k)
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in zip(alone[k], seen(k)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ far offsets
def test_wgrad_and_dgrad_past_4_gib():
    """The last expert's matrices lie beyond 2^32 bytes, and beyond 2^31 elements of dw."""
    import combine_grouped_gemm_amd as m
    E, N, M = 130, 4096, 4104
    counts = [0] * (E - 2) + [3, 5]
    dy, x = _values(8, N, 1, torch.bfloat16), _values(8, M, 2, torch.bfloat16)
    dw = m.moe_ffn_wgrad(dy, x, _offsets(counts))
    for j, (a, b) in ((E - 2, (0, 3)), (E - 1, (3, 8))):
        p, q = dy[a:b].double(), x[a:b].double()
        _near(dw[j], p.t() @ q, HALF[torch.float32] * (p.t() @ q).abs() + 8 * 2.0**-23 * (p.abs().t() @ q.abs()), "dw")
    assert not bool(dw[:E - 2].any())
    del dw
    w = torch.zeros(E, N, M, dtype=torch.bfloat16, device="cuda")
    w[-2:] = _weights(2, N, M, 3, torch.bfloat16)
    for hint in (1, 300):
        dx = m.moe_ffn_dgrad(dy, _offsets(counts), w, expected_rows=hint)
        for j, (a, b) in ((E - 2, (0, 3)), (E - 1, (3, 8))):
            ref, mag = dy[a:b].double() @ w[j].double(), dy[a:b].double().abs() @ w[j].double().abs()
            _near(dx[a:b], ref, HALF[torch.bfloat16] * ref.abs() + N * 2.0**-23 * mag, "dx")


def test_rows_past_4_gib():
    """Checkpoints, SwiGLU and gathered products whose last rows lie beyond 2^32 bytes."""
    import combine_grouped_gemm_amd as m
    cols = 4096
    cap = 2**32 // cols + 40
    x = torch.zeros(cap, cols, dtype=torch.bfloat16, device="cuda")
    x[-20:] = _values(20, cols, 1, torch.bfloat16)
    q, s = m.moe_checkpoint_rows(x)
    rq, rs = tr.checkpoint(to_np(x[-20:]))
    np.testing.assert_array_equal(q[-20:].cpu().numpy(), rq)
    np.testing.assert_array_equal(s[-20:].cpu().numpy(), rs)
    assert torch.equal(m.moe_checkpoint_values(q, s)[-20:].double(), _decoded(q[-20:], s[-20:]))
    row_of = torch.tensor([[cap - 1, cap - 7]], dtype=torch.int32, device="cuda")
    w = torch.ones(1, 2, device="cuda")
    dg, du, hw, dw = m.moe_swiglu_backward(x, q, s, q, s, row_of, w)
    g, d = _decoded(q[[-1, -7]], s[[-1, -7]]), x[[-1, -7]].double()
    ref = g * torch.sigmoid(g) * g
    _near(hw[[-1, -7]], ref, (HALF[torch.bfloat16] + ACT) * ref.abs(), "hw")
    _near(dw[0], (d * ref).sum(1), (cols * 2.0**-23 + ACT) * (d * ref).abs().sum(1), "dw")
    del dg, du, hw
    src = torch.tensor([cap - 2, cap - 11, 0, cap - 5], dtype=torch.int32, device="cuda")
    dy = _values(4, 72, 4, torch.bfloat16)
    got = m.moe_ffn_wgrad(dy, q, _offsets([1, 3]), x_scales=s, src_of=src, gather="x")
    xv = _decoded(q[src.long()], s[src.long()])
    for j, (a, b) in enumerate(((0, 1), (1, 4))):
        ref, mag = dy[a:b].double().t() @ xv[a:b], dy[a:b].double().abs().t() @ xv[a:b].abs()
        _near(got[j], ref, HALF[torch.float32] * ref.abs() + 4 * 2.0**-23 * mag, "dw")
    # the same tokens in bf16, and as gathered gradients
    for y, z, side in ((dy, x, "x"), (x, dy, "dy")):
        for dt in TYPES:
            got = m.moe_ffn_wgrad(y, z, _offsets([1, 3]), src_of=src, gather=side, dw_dtype=dt)
            a_, b_ = (v[src.long()] if v is x else v for v in (y, z))
            for j, (a, b) in enumerate(((0, 1), (1, 4))):
                ref, mag = a_[a:b].double().t() @ b_[a:b].double(), a_[a:b].double().abs().t() @ b_[a:b].double().abs()
                _near(got[j], ref, HALF[dt] * ref.abs() + 4 * 2.0**-23 * mag, f"dw, {side} gathered")
    wt = _weights(2, cols, 72, 5, torch.bfloat16)
    for hint in (1, 300):
        dx = m.moe_ffn_dgrad(x, _offsets([1, 3]), wt, src_of=src, expected_rows=hint)
        for j, (a, b) in enumerate(((0, 1), (1, 4))):
            d = x[src[a:b].long()].double()
            ref, mag = d @ wt[j].double(), d.abs() @ wt[j].double().abs()
            _near(dx[a:b], ref, HALF[torch.bfloat16] * ref.abs() + cols * 2.0**-23 * mag, "dx")


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("base", [False, True])
def test_wgrad_of_very_wide_rows(base, ckpt):
    """256 rows of dw that together pass 2^31 bytes; the last columns are 8 codes."""
    import combine_grouped_gemm_amd as m
    N, M = 16, 2**21 + 8
    dy = _values(5, N, 1, torch.bfloat16)
    x, xs = _codes(5, M, 2) if ckpt else (_values(5, M, 2, torch.bfloat16), None)
    b = torch.ones(2, N, M, device="cuda") if base else None
    dw = m.moe_ffn_wgrad(dy, x, _offsets([2, 3]), x_scales=xs, base=b)
    xv = _decoded(x, xs) if ckpt else x.double()
    for j, (r0, r1) in enumerate(((0, 2), (2, 5))):
        ref, mag = dy[r0:r1].double().t() @ xv[r0:r1] + base, dy[r0:r1].double().abs().t() @ xv[r0:r1].abs() + base
        _near(dw[j], ref, HALF[torch.float32] * ref.abs() + 4 * 2.0**-23 * mag, "dw")


def test_layer_of_no_tokens():
    import combine_grouped_gemm_amd as m
    layer, x, lg, w, dout = _train_layer(m, 0, 4, 2, 64, 72, 0, 4, torch.bfloat16)
    grads = layer.new_grads()
    layer.forward(x, lg, w)
    dx, dlogits = layer.backward(dout, lg, w, grads)
    assert dx.shape == (0, 64) and dlogits.shape == (0, 4)
    assert all(not bool(g.any()) for g in grads.values())


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_that_drops_rows(dtype):
    """A buffer shorter than the batch's rows: the dropped slots pass no gradient."""
    import combine_grouped_gemm_amd as m
    name = {torch.float32: "f32", torch.bfloat16: "bf16"}[dtype]
    T, E, K, H, I = 60, 6, 2, 72, 136
    _, x, lg, w, dout = _train_layer(m, T, E, K, H, I, 0, E, dtype, seed=11)
    layer = m.MoELayer([T], E, K, H, I, 0, E, name, name, name, cap_rows=70, train=True)
    grads = layer.new_grads()
    layer.forward(x, lg, w)
    dx, _ = layer.backward(dout, lg, w, grads)
    row_of = layer.row_of.cpu().numpy()
    assert (row_of < 0).sum() == T * K - 70
    assert bool((layer.dtopk_w[layer.row_of < 0] == 0).all())
    off = np.minimum(layer.offsets.cpu().numpy(), 70)
    src = layer.src_of.cpu().numpy()
    dh = to_np(layer.dh)
    g, u = (to_np(_decoded(q, s)) for q, s in ((layer.gate_q, layer.gate_s), (layer.up_q, layer.up_s)))
    dg, du, hw, dw = tr.swiglu_backward(dh, g, u, row_of, layer.topk_w.cpu().numpy())
    bar = 1e-2 if dtype == torch.bfloat16 else 1e-5
    xt, dt = tr.token_rows(to_np(_decoded(layer.x_q, layer.x_s)), src, K), tr.token_rows(to_np(dout), src, K)
    dxd = tr.dgrad([(dg, to_np(w["gate"])), (du, to_np(w["up"]))], off, 70)
    want = np.zeros((T, H))
    for t in range(T):
        for k in range(K):
            if row_of[t, k] >= 0:
                want[t] += dxd[row_of[t, k]]
    for what, got, ref in (("dtopk_w", layer.dtopk_w, dw), ("gate", grads["gate"], tr.wgrad(dg, xt, off)),
                           ("up", grads["up"], tr.wgrad(du, xt, off)), ("down", grads["down"], tr.wgrad(dt, hw, off)),
                           ("dx", dx, want)):
        assert np.linalg.norm(to_np(got) - ref) <= bar * np.linalg.norm(ref), what


def test_micro_batches_add_up_to_the_batch():
    """Two micro-batches on two streams, the second's gradients added to the first's."""
    import combine_grouped_gemm_amd as m
    from combine_grouped_gemm_amd.layer import MicroBatchedLayer
    whole, x, lg, w, dout = _train_layer(m, 120, 8, 2, 136, 264, 0, 8, torch.bfloat16, seed=13, segs=2)
    one = whole.new_grads()
    whole.forward(x, lg, w)
    dx, dlogits = whole.backward(dout, lg, w, one)
    halves = MicroBatchedLayer(whole.seg_rows, 8, 2, 136, 264, 0, 8, "bf16", "bf16", "bf16", train=True)
    (xa, la), (xb, lb) = halves.split_inputs(x, lg)
    oa, ob = halves.forward(x, lg, w)
    assert torch.equal(torch.cat([oa, ob]), whole.out)
    two = halves.a.new_grads()
    Ta = halves.a.T
    dxa, dla = halves.a.backward(dout[:Ta], la, w, two)
    dxb, dlb = halves.b.backward(dout[Ta:].contiguous(), lb, w, two, accumulate=True)
    assert torch.equal(torch.cat([dxa, dxb]), dx) and torch.equal(torch.cat([dla, dlb]), dlogits)
    for k in one:
        # the same products in two sums: fp32 roundings of up to 120 terms each
        _near(two[k], one[k], 2 * 121 * 2.0**-23 * (one[k].double().abs() + one[k].double().abs().amax()), k)
