"""GPU parity of the int8 expert path: dispatch with per-token quantisation,
row quantisation, grouped gate/up and down products, and the layer that runs
them with the scored router.

Codes and scales are exact.  Tolerances of the products, relative to the
value: the int32 sum is exact; its conversion to fp32 and the two scalings
round by 2^-24 each (y in fp32: 3 * 2^-24, taken as 4); bf16 adds half a step,
2^-8.  h = silu(g) u: g and u carry 3 * 2^-24 each, silu turns an error d of g
into at most (1 + |g|) d, its exponential adds |g| * 2^-23 and a few last
places, and |g| < 30 in these tests: less than 250 * 2^-24 < 2^-16 in all."""
import numpy as np
import pytest
import torch

import oracle
from harness import assert_close, has_gpu, to_np
from oracle import numerics as nx

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

HALF_BF16 = 2.0**-8
H_TOL = HALF_BF16 + 2.0**-16
Y_TOL = {torch.bfloat16: HALF_BF16 + 2.0**-21, torch.float32: 4 * 2.0**-24}


def _near(got, ref, tol, what):
    got, ref = got.double().cpu(), ref.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    off = ((got - ref).abs() - tol * ref.abs()).nan_to_num(0.0)
    assert float(off.max() if off.numel() else 0.0) <= 1e-37, f"{what}: off by {float(off.max()):.3e} over the bar"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _values(rows, cols, seed, f32=False):
    g = _gen(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 3)
    if rows > 6:
        x[1] = 0.0
        x[2] = 0.0
        x[2, 0] = 127.0
        x[2, 1:] = (torch.randint(-126, 126, (cols - 1,), generator=g) + 0.5)   # ties at scale 1
        x[3] *= 1e-37                                                          # subnormal scale territory
        x[4] = 2.0**-140
        x[5] = 3e38
    return x if f32 else x.to(torch.bfloat16)


# ------------------------------------------------------------------ row quantisation
COLS = [16, 64, 144, 208, 512, 1040, 2048, 2880, 7168, 8192, 16400, 33008]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("cols", COLS)
def test_quant_all_rows(cols, f32):
    import combine_grouped_gemm_amd as m
    print(f"[quant] cols={cols} f32={f32}", flush=True)
    x = _values(37, cols, cols, f32)
    x[8, cols - 1] = float("nan")
    x[9, cols // 2] = float("inf")
    x[10, 0] = -float("inf")
    q, s = m.moe_quant_rows(x.cuda())
    rq, rs = nx.quantize_i8_rows(to_np(x))
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)


def _counts(E, seed, most):
    c = torch.randint(0, most + 1, (E,), generator=_gen(seed))
    c[E // 2] = 0
    c[0] = min(most, 1)
    return c


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("E,most,cols", [(1, 5, 64), (7, 40, 208), (64, 3, 2048), (300, 9, 96), (1024, 4, 32)])
def test_quant_leaves_other_rows(E, most, cols, masked):
    import combine_grouped_gemm_amd as m
    print(f"[quant] E={E} most={most} cols={cols} masked={masked}", flush=True)
    c = _counts(E, E, most)
    if masked:
        cap, rows, kw = E * most, c.to(torch.int32), dict(cap_per_expert=most)
        valid = (torch.arange(most)[None] < c[:, None]).flatten().numpy()
    else:
        # the first expert need not start at row 0
        off = torch.cat([torch.zeros(1, dtype=torch.int64), c.cumsum(0)]) + 2
        cap, rows, kw = int(off[-1]) + 11, off.to(torch.int32), {}
        valid = ((torch.arange(cap) >= 2) & (torch.arange(cap) < int(off[-1]))).numpy()
    x = _values(cap, cols, 5)
    q = torch.full((cap, cols), 99, dtype=torch.int8, device="cuda")
    s = torch.full((cap,), -3.0, device="cuda")
    m.moe_quant_rows(x.cuda(), rows.cuda(), q=q, scales=s, **kw)
    rq, rs = nx.quantize_i8_rows(to_np(x))
    q, s = q.cpu().numpy(), s.cpu().numpy()
    np.testing.assert_array_equal(q[valid], rq[valid])
    np.testing.assert_array_equal(s[valid], rs[valid])
    assert (q[~valid] == 99).all() and (s[~valid] == -3.0).all()


def test_quant_clamps_row_descriptions_to_the_buffer():
    """Counts past the buffer (an overflowing layout still counts every slot)
    and negative ones."""
    import combine_grouped_gemm_amd as m
    x = _values(20, 64, 8)
    rq, rs = nx.quantize_i8_rows(to_np(x))
    q, s = m.moe_quant_rows(x.cuda(), torch.tensor([0, 9, 25, 60], dtype=torch.int32, device="cuda"))
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    q = torch.full((20, 64), 99, dtype=torch.int8, device="cuda")
    m.moe_quant_rows(x.cuda(), torch.tensor([9, -4, 2, 3], dtype=torch.int32, device="cuda"), cap_per_expert=5, q=q,
                     scales=s)
    q = q.cpu().numpy()
    for j, n in enumerate((5, 0, 2, 3)):
        np.testing.assert_array_equal(q[5 * j:5 * j + n], rq[5 * j:5 * j + n])
        assert (q[5 * j + n:5 * j + 5] == 99).all()


# ------------------------------------------------------------------ dispatch
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("segs,E,K,first,last,H", [
    ((1,), 8, 2, 0, 8, 16), ((37,), 16, 4, 4, 12, 208), ((5, 0, 60, 1), 32, 8, 0, 32, 7168), ((90,), 128, 100, 30, 99, 96),
    ((64,), 96, 64, 0, 96, 1040), ((3,), 4, 4, 1, 2, 16400), ((2,), 4, 2, 0, 4, 33008), ((50,), 128, 128, 0, 128, 32),
    ((9, 3), 8, 2, 0, 8, 8208), ((600, 30), 16, 2, 0, 16, 64), ((650,), 16, 2, 4, 12, 2080), ((600,), 64, 3, 0, 8, 7168),
    ((610,), 32, 2, 0, 4, 16384), ((603,), 128, 70, 0, 2, 33008)])
def test_dispatch(segs, E, K, first, last, H, f32):
    import combine_grouped_gemm_amd as m
    print(f"[dispatch] segs={segs} E={E} K={K} local [{first}, {last}) H={H} f32={f32}", flush=True)
    T = sum(segs)
    x = _values(T, H, T + H, f32)
    if T > 12:
        x[12, 5] = float("nan")
    ids = torch.rand(T, E, generator=_gen(T)).topk(K, 1).indices.numpy().astype(np.int32)
    ids[T // 2] = -1                                       # a token without any expert
    lay = oracle.layout(ids, E, first, last, T * K)
    cap = max(1, int(lay["offsets"][-1]) - 3)              # the last rows do not fit
    R = int(lay["offsets"][-1])
    ro = lay["row_of"].copy()
    xd = torch.full((max(cap, R) + 2, H), 55, dtype=torch.int8, device="cuda")
    sc = torch.full((max(cap, R) + 2,), 9.0, device="cuda")
    parts, at = [], 0
    for b in segs:
        parts.append(x[at:at + b].cuda())
        at += b
    m.moe_dispatch(parts, torch.from_numpy(ro).cuda(), cap, "int8", xd=xd, xd_scales=sc)
    rq, rs = oracle.dispatch(to_np(x), np.where(ro < cap, ro, -1), cap, "int8")
    used = np.zeros(xd.shape[0], bool)
    used[ro[(ro >= 0) & (ro < cap)]] = True
    xd, sc = xd.cpu().numpy(), sc.cpu().numpy()
    np.testing.assert_array_equal(xd[used], rq[used[:cap]])
    np.testing.assert_array_equal(sc[used], rs[used[:cap], 0])
    assert (xd[~used] == 55).all() and (sc[~used] == 9.0).all()


# ------------------------------------------------------------------ grouped products
class Problem:
    """Random codes and scales for E experts, rows in the contiguous or the masked layout."""

    def __init__(self, counts, K, N, seed, cap_e=None, gated=False, lead=0):
        g = _gen(seed)
        c = torch.as_tensor(counts)
        self.E, self.K, self.N, self.gated, self.cap_e = len(c), K, N, gated, cap_e
        if cap_e is None:
            off = torch.cat([torch.zeros(1, dtype=torch.int64), c.cumsum(0)]) + lead
            self.cap, self.rows = int(off[-1]) + 5, off.to(torch.int32).cuda()
            self.spans = [(int(a), int(b)) for a, b in zip(off[:-1], off[1:])]
        else:
            self.cap, self.rows = self.E * cap_e, c.to(torch.int32).cuda()
            self.spans = [(j * cap_e, j * cap_e + int(n)) for j, n in enumerate(c)]
        codes = lambda *shape: torch.randint(-127, 128, shape, generator=g, dtype=torch.int8).cuda()
        # g = silu's argument: |x w| <= 127^2 sqrt(K)-ish codes, scaled to a few units
        unit = 1.0 / (73.0 * 73.0 * max(1.0, K)**0.5)
        self.a = codes(self.cap, K)
        self.sa = (torch.rand(self.cap, generator=g) + 0.5).cuda()
        self.w = [codes(self.E, N, K) for _ in range(2 if gated else 1)]
        self.sw = [((torch.rand(self.E, N, generator=g) + 0.5) * unit).cuda() for _ in self.w]

    def reference(self):
        out = torch.zeros((self.cap, self.N), dtype=torch.float64, device="cuda")
        for j, (a, b) in enumerate(self.spans):
            if b > a:
                # the sums of integers are exact in fp64; scaled afterwards, so that a sum of zero is zero
                x = self.a[a:b].double()
                p = [(x @ w[j].double().t()) * self.sa[a:b].double()[:, None] * s[j].double()
                     for w, s in zip(self.w, self.sw)]
                out[a:b] = p[0] / (1 + torch.exp(-p[0])) * p[1] if self.gated else p[0]
        return out

    def valid(self):
        v = torch.zeros(self.cap, dtype=torch.bool)
        for a, b in self.spans:
            v[a:b] = True
        return v.cuda()

    def run(self, hint, out=None, pack=False, y_dtype=torch.bfloat16, stream=None):
        import combine_grouped_gemm_amd as m
        dt = torch.bfloat16 if self.gated else y_dtype
        if out is None:
            out = torch.full((self.cap, self.N), 7.0, dtype=dt, device="cuda")
        w = [m.moe_pack_weights(t) for t in self.w] if pack else self.w
        kw = dict(expected_rows=hint, cap_per_expert=self.cap_e, stream=stream)
        if self.gated:
            m.moe_ffn_gate_up(self.a, self.sa, self.rows, *w, *self.sw, h=out, **kw)
        else:
            m.moe_ffn_down(self.a, self.sa, self.rows, w[0], self.sw[0], y=out, **kw)
        return out

    def check(self, got, what):
        v = self.valid()
        ref = self.reference()
        _near(got[v], ref[v], H_TOL if self.gated else Y_TOL[got.dtype], what)
        assert (got[~v] == 7.0).all(), f"{what}: rows without a slot were written"


HINTS = [1, 12, 30, 64, 100, 200, 400]      # every tile shape a hint can pick
PRODUCTS = [  # counts, K, N
    ([1], 16, 16), ([0, 3, 0, 1, 17, 0], 128, 96), ([5, 0, 64, 33], 208, 144), ([15, 16, 17, 31, 32, 33], 272, 264),
    ([129, 2, 0, 320], 1040, 272), ([321, 1, 255, 257, 0], 640, 512), ([700, 0, 3], 384, 136), ([2] * 130, 256, 128),
    ([40, 90], 2880, 80), ([1, 0, 2, 7], 7168, 48),
]


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("counts,K,N", PRODUCTS, ids=[f"{len(c)}x{max(c)}-K{k}-N{n}" for c, k, n in PRODUCTS])
def test_products(counts, K, N, gated):
    N = -(-N // 16) * 16
    p = Problem(counts, K, N, seed=K + N, gated=gated, lead=3)
    ref = None
    for hint in HINTS:
        print(f"[product] counts={counts[:6]} K={K} N={N} gated={gated} hint={hint}", flush=True)
        got = p.run(hint)
        p.check(got, f"hint {hint}")
        # sums are exact, so no tile shape, nor the packed pitch, changes a bit
        if ref is None:
            ref = got
        assert torch.equal(got, ref)
        assert torch.equal(p.run(hint, pack=True), ref)
        if not gated:
            p.check(p.run(hint, y_dtype=torch.float32), f"fp32 y, hint {hint}")


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("counts,cap_e,K,N", [([3, 0, 8, 8, 1], 8, 144, 80), ([40, 64, 0, 1], 64, 512, 256),
                                              ([200, 330, 0], 330, 256, 144)])
def test_masked_products(counts, cap_e, K, N, gated):
    p = Problem(counts, K, N, seed=1 + K, cap_e=cap_e, gated=gated)
    for hint in HINTS:
        print(f"[masked] counts={counts} K={K} N={N} gated={gated} hint={hint}", flush=True)
        p.check(p.run(hint), f"hint {hint}")


@pytest.mark.parametrize("hint", HINTS)
def test_extreme_codes_and_scales(hint):
    """Sums at the int32 border (127 * 127 and -128 codes over the longest rows
    that fit), scales from subnormal to huge, NaN scales."""
    import combine_grouped_gemm_amd as m
    print(f"[extreme] hint={hint}", flush=True)
    K, N, R = m.INT8_MAX_COLS, 32, 21
    a = torch.full((R, K), -128, dtype=torch.int8, device="cuda")
    a[1] = 127
    w = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
    w[0, 1] = 127
    w[0, 2, ::2] = 127
    sa = torch.ones(R, device="cuda")
    sa[2], sa[3], sa[4] = 2.0**-126, 1e25, float("nan")
    sw = torch.ones((1, N), device="cuda")
    sw[0, 3], sw[0, 4] = 2.0**-140, 1e20
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    y = m.moe_ffn_down(a, sa, off, w, sw, y_dtype=torch.float32, expected_rows=hint)
    dot = torch.stack([(a.double() * w[0, n].double()).sum(1) for n in range(N)], 1)
    assert float(dot.abs().max()) == 16384.0 * K < 2**31
    ref = dot * sa.double()[:, None] * sw.double()
    ref = torch.where(ref.abs() > 3.4028235677973366e38, ref.sign() * float("inf"), ref)
    got = y.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isinf(got), torch.isinf(ref))
    # below the smallest normal number a step is absolute: half a step for each of the two scalings
    # (the first of which is then multiplied by a channel scale of at most 1)
    bar = Y_TOL[torch.float32] * ref.abs() + 2.0**-149
    assert bool(((got - ref).abs() <= bar)[fin].all())


def test_gate_up_saturates_like_its_formula():
    """silu far out: h is u g for large g, minus zero for very negative g."""
    import combine_grouped_gemm_amd as m
    K, N = 64, 32
    a = torch.full((4, K), 127, dtype=torch.int8, device="cuda")
    wg = torch.full((1, N, K), 127, dtype=torch.int8, device="cuda")
    wg[0, ::2] = -127
    wu = torch.full((1, N, K), 1, dtype=torch.int8, device="cuda")
    one = torch.ones(4, device="cuda")
    s = torch.full((1, N), 1e-3, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    h, hs = m.moe_ffn_gate_up(a, one, off, wg, wu, s, s)
    assert hs is None
    g, u = 127.0 * 127 * K * float(s[0, 0].double()), 127.0 * K * float(s[0, 0].double())
    assert (h[:, ::2] == 0).all()
    _near(h[:, 1::2], torch.full((4, N // 2), g * u, dtype=torch.float64), H_TOL, "h")


def test_empty_inputs_are_no_ops():
    import combine_grouped_gemm_amd as m
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt, device="cuda")
    f = torch.float32
    off = z(3, dt=torch.int32)
    h, _ = m.moe_ffn_gate_up(z(0, 32), z(0, dt=f), off, z(2, 16, 32), z(2, 16, 32), z(2, 16, dt=f), z(2, 16, dt=f))
    assert h.shape == (0, 16)
    # a buffer whose experts are all empty
    h = torch.full((6, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_ffn_gate_up(z(6, 32), z(6, dt=f), off, z(2, 16, 32), z(2, 16, 32), z(2, 16, dt=f), z(2, 16, dt=f), h=h)
    q, s = m.moe_quant_rows(h, off, q=torch.full((6, 16), 3, dtype=torch.int8, device="cuda"))
    torch.cuda.synchronize()
    assert (h == 7.0).all() and (q == 3).all()
    assert m.moe_quant_rows(z(0, 16, dt=f))[0].shape == (0, 16)
    # a batch without tokens, and one whose tokens have no local slot
    xd, xs = torch.full((4, 32), 5, dtype=torch.int8, device="cuda"), z(4, dt=f)
    m.moe_dispatch(z(0, 32, dt=f), z(0, 2, dt=torch.int32), 4, "int8", xd=xd, xd_scales=xs)
    m.moe_dispatch(z(3, 32, dt=f), z(3, 2, dt=torch.int32) - 1, 4, "int8", xd=xd, xd_scales=xs)
    torch.cuda.synchronize()
    assert (xd == 5).all() and (xs == 0).all()
    y = m.moe_grouped_ffn(z(0, 32), z(0, dt=f), off, z(2, 16, 32), z(2, 16, 32), z(2, 32, 16), z(2, 16, dt=f),
                          z(2, 16, dt=f), z(2, 32, dt=f))
    assert y.shape == (0, 32)


# ------------------------------------------------------------------ as they are used together
def _quantised_weights(E, rows, cols, seed):
    """fp32 weights, and their int8 form made by the library's own row quantisation."""
    import combine_grouped_gemm_amd as m
    w = (torch.randn(E, rows, cols, generator=_gen(seed)) / cols**0.5).cuda()
    q, s = m.moe_quant_rows(w.view(E * rows, cols))
    return w, q.view(E, rows, cols), s.view(E, rows)


LAYERS = [  # segments, E, K, H, I, first, last, layout, cap_e, shared, router, y, out
    ((40,), 32, 4, 256, 144, 0, 32, "contiguous", None, 0,
     dict(score="sigmoid", n_groups=8, topk_groups=4, scale=2.5), "bf16", "bf16"),
    ((17, 0, 30), 16, 3, 208, 96, 4, 12, "contiguous", None, 0, dict(score="softmax", renorm=False), "f32", "f32"),
    ((64,), 16, 4, 128, 64, 0, 16, "masked", 12, 0, dict(score="sigmoid", n_groups=4, topk_groups=2), "bf16", "f32"),
    ((600,), 8, 2, 320, 256, 0, 8, "contiguous", None, 1, None, "bf16", "bf16"),
    ((50,), 16, 2, 128, 64, 0, 16, "contiguous", None, 2, dict(score="sigmoid", n_groups=4, topk_groups=2), "bf16", "bf16"),
    ((1,), 256, 8, 512, 128, 0, 256, "contiguous", None, 0,
     dict(score="sigmoid", n_groups=8, topk_groups=4, scale=2.5), "bf16", "bf16"),
]


def _make_layer(cfg, seed=3):
    import combine_grouped_gemm_amd as m
    segs, E, K, H, I, first, last, layout, cap_e, shared, router, y, out = cfg
    T, n = sum(segs), last - first + shared
    layer = m.MoELayer(segs, E, K, H, I, first, last, "int8", y, out, layout=layout, cap_per_expert=cap_e,
                       n_shared=shared, router=router)
    g = _gen(seed)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    lg = torch.randn(T, E, generator=g)
    bias = None
    if router is not None and router["score"] == "sigmoid":
        bias = torch.randn(E, generator=g) * 0.1
        layer.router_bias = bias.cuda()
    if T > 20 and router is not None:
        lg[7] = -float("inf")                              # a padding token: no expert at all
        lg[9, 2:] = -float("inf")
    parts, at = [], 0
    for b in segs:
        parts.append(x[at:at + b].cuda())
        at += b
    w = {}
    for i, (name, r, c) in enumerate((("gate", I, H), ("up", I, H), ("down", H, I))):
        _, w[name], w[name + "_scale"] = _quantised_weights(n, r, c, seed + i)
    deq = {k: to_np(w[k]) * to_np(w[k + "_scale"])[..., None] for k in ("gate", "up", "down")}
    if router is None:
        routing = oracle.route_shared(lg.numpy(), K, shared)
    else:
        ids, gates = oracle.route_scored(lg.double().numpy(), K, bias=None if bias is None else bias.double().numpy(),
                                         **router)
        routing = (np.concatenate([ids, np.tile(np.arange(E, E + shared, dtype=np.int32), (T, 1))], 1),
                   np.concatenate([gates, np.ones((T, shared))], 1))
    return layer, parts, x, lg, w, deq, routing


@pytest.mark.parametrize("cfg", LAYERS, ids=[f"T{sum(c[0])}-E{c[1]}-{c[7]}-shared{c[9]}" for c in LAYERS])
def test_layer(cfg):
    """route, layout, dispatch, gate/up, quant, down and combine in a row against
    the oracle's layer on the same integer weights (bars of an 8-bit layer:
    where an h lies next to a code's border, its bf16 rounding may pick the
    neighbour)."""
    segs, E, K, H, I, first, last, layout, cap_e, shared, router, ydt, odt = cfg
    print(f"[layer] {cfg}", flush=True)
    layer, parts, x, lg, w, deq, routing = _make_layer(cfg)
    names = [n for n, _ in layer.stages(parts, lg.cuda(), w)]
    assert names == ["route", "layout", "dispatch", "ffn_gate_up", "quant_h", "ffn_down", "combine"]
    out = layer.forward(parts, lg.cuda(), w)
    torch.cuda.synchronize()
    ids, gates = routing
    np.testing.assert_array_equal(layer.topk_ids.cpu().numpy(), ids)
    wof = lambda j: tuple(deq[k][j] for k in ("gate", "up", "down"))
    if layout == "masked":
        lay = oracle.layout_masked(ids, E, first, last, cap_e)
        np.testing.assert_array_equal(layer.row_of.cpu().numpy(), lay["row_of"])
        xd, xs = oracle.dispatch(to_np(x), lay["row_of"], layer.cap, "int8")
        y = oracle.grouped_ffn_masked(xd * xs, lay["m"], cap_e, wof, "int8", ydt)
        ref = oracle.combine(y, lay["row_of"], nx.to_f32(gates), odt)
    else:
        o = oracle.layer(to_np(x), lg.numpy(), K, E, first, last, wof, "int8", ydt, odt, n_shared=shared,
                         routing=routing)
        np.testing.assert_array_equal(layer.row_of.cpu().numpy(), o["row_of"])
        ref = o["out"]
    assert_close(to_np(out), ref, "bf16", "out")
    if sum(segs) > 20 and router is not None and not shared:
        assert (out[7] == 0).all()


def test_grouped_ffn_is_the_three_calls():
    import combine_grouped_gemm_amd as m
    for masked in (False, True):
        layer, parts, _, lg, w, _, _ = _make_layer(LAYERS[2] if masked else LAYERS[0])
        layer.forward(parts, lg.cuda(), w)
        need = m.moe_ffn_workspace_bytes(layer.cap, layer.I, "int8")
        ws = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device="cuda")
        y = torch.zeros_like(layer.y)
        layer.y.zero_()
        layer.down(w)
        m.moe_grouped_ffn(layer.xd, layer.xd_scales, layer.rows, w["gate"], w["up"], w["down"], w["gate_scale"],
                          w["up_scale"], w["down_scale"], y=y, ws=ws[:need], expected_rows=layer.expected_rows,
                          cap_per_expert=layer.cap_e)
        torch.cuda.synchronize()
        assert torch.equal(y, layer.y)
        assert (ws[need:] == 0xAB).all()
        y32 = m.moe_grouped_ffn(layer.xd, layer.xd_scales, layer.rows, w["gate"], w["up"], w["down"], w["gate_scale"],
                                w["up_scale"], w["down_scale"], y=torch.zeros(y.shape, device="cuda"),
                                cap_per_expert=layer.cap_e)
        assert torch.equal(y32.to(torch.bfloat16), y)


@pytest.mark.parametrize("i", [0, 2, 5])
def test_layer_graph_replay(i):
    layer, parts, x, lg, w, _, _ = _make_layer(LAYERS[i])
    lgd = lg.cuda()
    layer.forward(parts, lgd, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        layer.forward(parts, lgd, w)
        with torch.cuda.graph(g, stream=s):
            layer.forward(parts, lgd, w)
    torch.cuda.synchronize()
    for rep in range(4):
        new = torch.randn(lg.shape, generator=_gen(100 + rep))
        lgd.copy_(new)
        for b in parts:
            b.mul_(-1.25)
        layer.out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        got = layer.out.clone()
        layer.forward(parts, lgd, w)
        torch.cuda.synchronize()
        assert torch.equal(got, layer.out), f"replay {rep}"


def test_micro_batches_match_the_single_batch():
    import combine_grouped_gemm_amd as m
    cfg = LAYERS[0]
    layer, parts, x, lg, w, _, _ = _make_layer(cfg)
    ref = layer.forward(parts, lg.cuda(), w).clone()
    mb = m.layer.MicroBatchedLayer([40], 32, 4, 256, 144, 0, 32, "int8", "bf16", "bf16", router=cfg[10])
    mb.a.router_bias = mb.b.router_bias = layer.router_bias
    for _ in range(3):
        a, b = mb.forward(parts, lg.cuda(), w)
        torch.cuda.synchronize()
        assert torch.equal(torch.cat([a, b]), ref)


def test_layer_with_a_placement_map():
    """The scored router through a placement map: experts renumbered, weights moved
    along, the same tokens out."""
    cfg = LAYERS[0]
    layer, parts, x, lg, w, _, _ = _make_layer(cfg)
    ref = layer.forward(parts, lg.cuda(), w).clone()
    ids = layer.topk_ids.clone()
    perm = torch.randperm(32, generator=_gen(8)).cuda()
    layer.expert_map = perm.to(torch.int32)
    back = torch.argsort(perm)
    moved = {k: v[back].contiguous() for k, v in w.items()}
    out = layer.forward(parts, lg.cuda(), moved)
    torch.cuda.synchronize()
    assert torch.equal(layer.topk_ids, torch.where(ids >= 0, perm[ids.clamp(min=0).long()].to(torch.int32), -1))
    # the same products and gates, added per token in the same slot order
    assert torch.equal(out, ref)


def test_two_streams_at_once():
    """The same operands on two streams, outputs apart."""
    p = Problem([100, 3, 0, 260], 512, 256, 4, gated=True)
    d = Problem([100, 3, 0, 260], 512, 256, 5)
    rp, rd = p.run(100), d.run(100)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.full_like(rp, 7.0) for _ in range(4)], [torch.full_like(rd, 7.0) for _ in range(4)]
    torch.cuda.synchronize()
    for i in range(4):
        p.run(100, out=outs[0][i], stream=s1)
        d.run(100, out=outs[1][i], stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(o, rp) for o in outs[0]) and all(torch.equal(o, rd) for o in outs[1])


def test_rows_past_four_gigabytes():
    """Buffers whose byte offsets pass 32 bits: dispatch, quantisation and a product
    that touch only the last rows."""
    import combine_grouped_gemm_amd as m
    cap, H, n = 70000, 65536, 6
    x = _values(n, H, 3)
    xd = torch.zeros((cap, H), dtype=torch.int8, device="cuda")
    sc = torch.zeros(cap, device="cuda")
    row_of = torch.arange(cap - n, cap, dtype=torch.int32, device="cuda").view(n, 1)
    m.moe_dispatch(x.cuda(), row_of, cap, "int8", xd=xd, xd_scales=sc)
    rq, rs = nx.quantize_i8_rows(to_np(x))
    np.testing.assert_array_equal(xd[cap - n:].cpu().numpy(), rq)
    np.testing.assert_array_equal(sc[cap - n:].cpu().numpy(), rs)
    assert not xd[cap - n - 3:cap - n].any()
    off = torch.tensor([cap - n, cap - 2, cap], dtype=torch.int32, device="cuda")
    w = torch.randint(-127, 128, (2, 16, H), dtype=torch.int8, generator=_gen(1)).cuda()
    y = m.moe_ffn_down(xd, sc, off, w, torch.ones((2, 16), device="cuda"), y_dtype=torch.float32)
    for j, (a, b) in enumerate(((cap - n, cap - 2), (cap - 2, cap))):
        ref = (xd[a:b].double() @ w[j].double().t()) * sc[a:b].double()[:, None]
        _near(y[a:b], ref, Y_TOL[torch.float32], "y")
    del xd, y
    xb = torch.zeros((cap, H), dtype=torch.bfloat16, device="cuda")
    xb[cap - n:] = x.cuda()
    q, s = m.moe_quant_rows(xb, off)
    np.testing.assert_array_equal(q[cap - n:].cpu().numpy(), rq)
    np.testing.assert_array_equal(s[cap - n:].cpu().numpy(), rs)
    del xb, q
    torch.cuda.empty_cache()


def test_outputs_allocated_on_the_given_stream():
    """Outputs that a call makes itself belong to the stream it runs on: memory that
    the current stream has freed but still uses is not handed to another one."""
    import combine_grouped_gemm_amd as m
    x = torch.randn(2000, 512, generator=_gen(2)).to(torch.bfloat16).cuda()
    rq, rs = m.moe_quant_rows(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        junk = torch.empty((2000, 512), dtype=torch.int8, device="cuda")
        big = torch.randn(2048, 2048, device="cuda")
        for _ in range(4):
            big = big @ big                                # keeps the current stream busy
        junk.fill_(1)                                      # runs late, on the current stream
        del junk
        q, s = m.moe_quant_rows(x, stream=side)
        side.synchronize()
        early = q.clone()
        torch.cuda.synchronize()
        assert torch.equal(q, rq) and torch.equal(s, rs) and torch.equal(early, rq)
    q, s = m.moe_quant_rows(x, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(q, rq)


def test_binding_refusals():
    import combine_grouped_gemm_amd as m
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt, device="cuda")
    f, i32 = torch.float32, torch.int32
    xd, xs, off = z(8, 64), z(8, dt=f), z(5, dt=i32)
    w, s = z(4, 32, 64), z(4, 32, dt=f)
    up = lambda **k: m.moe_ffn_gate_up(**{**dict(xd=xd, xd_scales=xs, offsets=off, w_gate=w, w_up=w, w_gate_scales=s,
                                                 w_up_scales=s), **k})
    for kw, msg in ((dict(xd_scales=None), "row scales"), (dict(xd_scales=z(7, dt=f)), "scales"),
                    (dict(w_gate_scales=None), "w_gate_scales"), (dict(w_up_scales=z(4, 31, dt=f)), "w_up_scales"),
                    (dict(w_up_scales=z(4, 32, dt=torch.bfloat16)), "w_up_scales"), (dict(h=z(8, 32)), "h must be"),
                    (dict(h=z(7, 32, dt=torch.bfloat16)), "h needs"), (dict(w_up=z(4, 32, 48)), "w_up"),
                    (dict(w_gate=z(4, 32, 64, dt=torch.bfloat16)), "w_gate"), (dict(offsets=z(4, dt=i32)), "offsets"),
                    (dict(w_scales_pow2=True), "pow2"), (dict(xd_scales=torch.zeros(8)), "device tensor")):
        with pytest.raises(ValueError, match=msg):
            up(**kw)
    h, hs, wd, ds = z(8, 32), z(8, dt=f), z(4, 64, 32), z(4, 64, dt=f)
    dn = lambda **k: m.moe_ffn_down(**{**dict(h=h, h_scales=hs, offsets=off, w_down=wd, w_down_scales=ds), **k})
    for kw, msg in ((dict(h_scales=None), "row scales"), (dict(w_down_scales=None), "w_down_scales"),
                    (dict(w_down_scales=z(4, 63, dt=f)), "w_down_scales"), (dict(y=z(8, 63, dt=f)), "y needs")):
        with pytest.raises(ValueError, match=msg):
            dn(**kw)
    with pytest.raises(m.MoeError, match="y_dt"):
        dn(y=z(8, 64))
    x = z(8, 64, dt=torch.bfloat16)
    for kw, msg in ((dict(q=z(8, 63)), "q must"), (dict(scales=z(7, dt=f)), "scales needs"),
                    (dict(cap_per_expert=2), "masked"), (dict(rows=z(4, dt=i32), cap_per_expert=3), "rows"),
                    (dict(rows=z(4, dt=torch.int64)), "offsets"), (dict(q=z(8, 64, dt=torch.uint8)), "q must")):
        with pytest.raises(ValueError, match=msg):
            m.moe_quant_rows(x, **kw)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        m.moe_quant_rows(h)
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_quant_rows(x[:, ::2])
    with pytest.raises(m.MoeError, match="multiple of 16"):
        m.moe_quant_rows(z(8, 24, dt=f))
    with pytest.raises(ValueError, match="xd_scales"):
        m.moe_dispatch(x, z(8, 2, dt=i32), 16, "int8", xd_scales=z(15, dt=f))
    with pytest.raises(ValueError, match="xd must"):
        m.moe_dispatch(x, z(8, 2, dt=i32), 16, "int8", xd=z(16, 64, dt=f))


@pytest.mark.parametrize("rows,error,msg", [
    ([0, 4, 8], TypeError, "offsets must be a torch.Tensor"),
    ("cpu", ValueError, "device tensor"),
    ("2-D", ValueError, "1 dims"),
    ("empty", ValueError, "at least 2"),
])
def test_quant_rows_refuses_bad_row_descriptions(rows, error, msg):
    import combine_grouped_gemm_amd as m
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    rows = {"cpu": torch.zeros(3, dtype=torch.int32), "2-D": torch.zeros(1, 3, dtype=torch.int32, device="cuda"),
            "empty": torch.zeros(0, dtype=torch.int32, device="cuda")}.get(rows, rows) if isinstance(rows, str) else rows
    with pytest.raises(error, match=msg):
        m.moe_quant_rows(x, rows)


def test_dispatch_of_more_tokens_than_one_launch_takes():
    """64 threads a token: as one grid the batch has 2^32 threads; its segments meet inside
    a launch's share of it."""
    import combine_grouped_gemm_amd as m
    B, H = 2**26 + 128, 16
    few = torch.randn(64, H, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    x = few.repeat(B // 64, 1)
    cut = 2**22 + 5
    rows = torch.arange(B - 1, -1, -1, dtype=torch.int32, device="cuda").view(B, 1)
    q, s = m.moe_dispatch([x[:cut], x[cut:]], rows, B, "int8")
    wq, ws = m.moe_quant_rows(few)
    assert bool((q.view(-1, 64, H) == wq.flip(0)).all()) and bool((s.view(-1, 64) == ws.flip(0)).all())


@pytest.mark.parametrize("cols", [1024, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 16384, 16400, 32768, 32784, 65552])
@pytest.mark.parametrize("f32", [False, True])
def test_quant_row_widths(cols, f32):
    """Both sides of every width at which the row's share of a lane changes; rows that
    are no numbers among them; fewer rows than blocks, and more."""
    import combine_grouped_gemm_amd as m
    for rows in (1, 5, 67):
        x = _values(rows, cols, cols + rows, f32)
        x[0, cols - 1] = -x[0, cols - 1].abs() - 3
        if rows > 5:
            x[3, cols - 1] = float("nan")
            x[4, cols // 3] = -float("inf")
            x[5] = 0.0
        q, s = m.moe_quant_rows(x.cuda())
        rq, rs = nx.quantize_i8_rows(to_np(x))
        np.testing.assert_array_equal(q.cpu().numpy(), rq)
        np.testing.assert_array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("cols,per_cu", [(1040, 8), (2064, 16), (4112, 0)])
@pytest.mark.parametrize("more", [0, 1, 9])
def test_quant_row_counts_where_the_split_changes(cols, per_cu, more):
    """As many rows as go to blocks and a few more, in either layout; the rows behind
    them are left as they were."""
    import combine_grouped_gemm_amd as m
    few = max(per_cu, 8) * torch.cuda.get_device_properties(0).multi_processor_count
    n, E = few + more, 16
    x = _values(n + 5, cols, more).cuda()
    rq, rs = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in nx.quantize_i8_rows(to_np(x)))
    q = torch.full((n + 5, cols), 99, dtype=torch.int8, device="cuda")
    s = torch.full((n + 5,), -3.0, device="cuda")
    m.moe_quant_rows(x, torch.tensor([0, 3, n], dtype=torch.int32, device="cuda"), q=q, scales=s)
    assert bool((q[:n] == rq[:n]).all()) and bool((s[:n] == rs[:n]).all())
    assert bool((q[n:] == 99).all()) and bool((s[n:] == -3.0).all())
    # masked: experts with few rows, with few / E of them, and with more
    cap = few // E + 12
    counts = torch.tensor([few // E, few // E + 1, few // E + more, 0, 1, 2, cap, few // E - 1] * (E // 8), dtype=torch.int32)
    x = x[:cap].repeat(E, 1)
    q = torch.full((E * cap, cols), 99, dtype=torch.int8, device="cuda")
    s = torch.full((E * cap,), -3.0, device="cuda")
    m.moe_quant_rows(x, counts.cuda(), cap_per_expert=cap, q=q, scales=s)
    valid = torch.arange(cap, device="cuda")[None] < counts.cuda()[:, None]
    want = torch.where(valid[..., None], rq[None, :cap], torch.tensor(99, dtype=torch.int8, device="cuda"))
    assert bool((q.view(E, cap, cols) == want).all())
    assert bool((s.view(E, cap) == torch.where(valid, rs[None, :cap], torch.tensor(-3.0, device="cuda"))).all())


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("counts,K,N", PRODUCTS, ids=[f"{len(c)}x{max(c)}-K{k}-N{n}" for c, k, n in PRODUCTS])
def test_products_in_large_tiles(counts, K, N, gated):
    """Expected rows past what one round of small tiles holds."""
    N = -(-N // 16) * 16
    p = Problem(counts, K, N, seed=K + N, gated=gated, lead=3)
    ref = p.run(1)
    p.check(ref, "small tiles")
    for hint in (10**6, 2**31 - 1):
        print(f"[product] counts={counts[:6]} K={K} N={N} gated={gated} hint={hint}", flush=True)
        assert torch.equal(p.run(hint), ref)
        assert torch.equal(p.run(hint, pack=True), ref)
        if not gated:
            p.check(p.run(hint, y_dtype=torch.float32), f"fp32 y, hint {hint}")


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("K,N", [(128, 2048), (384, 1040), (640, 1552), (400, 1040), (256, 2000)])
def test_products_of_many_experts(K, N, gated):
    """Large tiles at ordinary hints, with weights read either way; ranks of experts
    with equal, no and many rows."""
    counts = [0, 33, 257, 64, 1, 33, 256, 0, 129, 300, 7, 33] * 8
    p = Problem(counts, K, N, seed=K + N, gated=gated, lead=5)
    ref = p.run(1)
    p.check(ref, "small tiles")
    for hint in (32, 40, 100, 191, 192, 600):
        print(f"[product] K={K} N={N} gated={gated} hint={hint}", flush=True)
        assert torch.equal(p.run(hint), ref)
    if not gated:
        p.check(p.run(100, y_dtype=torch.float32), "fp32 y")


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7, 8, 9, 10])
def test_products_by_number_of_steps(steps):
    """Every remainder of the k-loop's turns, with a whole and a partial last step."""
    for K in (128 * steps, 128 * steps - 48):
        for gated in (True, False):
            p = Problem([5, 0, 70, 200, 1], K, 208, seed=K, gated=gated, lead=1)
            ref = p.run(1)
            p.check(ref, f"K={K} gated={gated}")
            assert torch.equal(p.run(100), ref) and torch.equal(p.run(10**6), ref)


def test_extreme_codes_and_scales_in_large_tiles():
    test_extreme_codes_and_scales(10**6)


@pytest.mark.parametrize("cols", [512, 2048, 4096])
def test_quant_rows_past_four_gigabytes(cols):
    """The last rows of a long buffer, however a row is shared out."""
    import combine_grouped_gemm_amd as m
    cap, n = 2**32 // cols + 5000, 4500
    x = torch.zeros((cap, cols), dtype=torch.bfloat16, device="cuda")
    x[cap - n:] = torch.randn(n, cols, generator=_gen(cols)).to(torch.bfloat16).cuda()
    rq, rs = nx.quantize_i8_rows(to_np(x[cap - n:]))
    for first in (cap - n, cap - 9):
        q, s = m.moe_quant_rows(x, torch.tensor([first, cap], dtype=torch.int32, device="cuda"))
        np.testing.assert_array_equal(q[first:].cpu().numpy(), rq[first - cap:])
        np.testing.assert_array_equal(s[first:].cpu().numpy(), rs[first - cap:])
    del x, q
    torch.cuda.empty_cache()


def test_small_tiles_past_four_gigabytes():
    import combine_grouped_gemm_amd as m
    cap, H, n = 70000, 65536, 6
    a = torch.zeros((cap, H), dtype=torch.int8, device="cuda")
    a[cap - n:] = torch.randint(-127, 128, (n, H), dtype=torch.int8, generator=_gen(4)).cuda()
    off = torch.tensor([cap - n, cap - 2, cap], dtype=torch.int32, device="cuda")
    w = torch.randint(-127, 128, (2, 16, H), dtype=torch.int8, generator=_gen(1)).cuda()
    sa, sw = torch.full((cap,), 2.0**-7, device="cuda"), torch.ones((2, 16), device="cuda")
    y = m.moe_ffn_down(a, sa, off, w, sw, y_dtype=torch.float32, expected_rows=3)
    h, _ = m.moe_ffn_gate_up(a, sa, off, w, w, sw, sw, expected_rows=3)
    for j, (b, e) in enumerate(((cap - n, cap - 2), (cap - 2, cap))):
        ref = (a[b:e].double() @ w[j].double().t()) * 2.0**-7
        _near(y[b:e], ref, Y_TOL[torch.float32], "y")
        _near(h[b:e], ref / (1 + torch.exp(-ref)) * ref, H_TOL, "h")
    del a, y, h
    torch.cuda.empty_cache()
