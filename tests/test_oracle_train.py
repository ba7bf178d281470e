"""Pins of the training step's oracle: torch's automatic differentiation in fp64,
central differences of the oracle's own forward pass, rational arithmetic for the
checkpoints.  CPU only."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import numerics as nx
from oracle import train as tr


def _rng(seed):
    return np.random.default_rng(seed)


def test_checkpoint_against_rational_arithmetic():
    g = _rng(0)
    v = nx.to_f32(g.standard_normal((9, 200)) * np.exp(3 * g.standard_normal((9, 1))))
    v[1] = 0.0
    v[2, :128] = 127.0
    v[3, 0] = 127.0 + 2.0**-16                   # one step above a border
    v[3, 1:128] = (np.arange(127) - 63) * 1.5 + 0.75
    v[4] = 2.0**-149
    v[5, :4] = [3.4028234663852886e38, -3.4e38, 127 * 2.0**121, 1.0]
    v[6, 0], v[6, 1:128] = 2.0**-120, 2.0**-127
    codes, scales = tr.checkpoint(v)
    for r in range(v.shape[0]):
        for b in range(2):
            part = [Fraction(float(x)) for x in v[r, b * 128:(b + 1) * 128]]
            amax = max(abs(x) for x in part)
            if amax == 0:
                want = Fraction(1)
            else:
                e = next((e for e in range(-126, 122) if amax <= 127 * Fraction(2)**e), 121)
                want = Fraction(2)**e
            assert Fraction(float(scales[r, b])) == want
            for i, x in enumerate(part):
                c = max(-127, min(127, round(x / want)))      # Fraction rounds half to even
                assert codes[r, b * 128 + i] == c, (r, b, i)
    # bf16 holds every value
    back = tr.checkpoint_values(codes, scales)
    np.testing.assert_array_equal(nx.to_bf16(back), back)
    assert np.all(np.abs(back - v) <= 0.5 * np.repeat(scales, 128, 1)[:, :200] * (1 + (np.abs(v) > 127 * 2.0**121)))


def test_checkpoint_of_specials():
    v = np.ones((3, 130))
    v[0, 5], v[1, 129], v[2, 0] = np.nan, np.inf, -np.inf
    codes, scales = tr.checkpoint(v)
    assert np.isnan(scales[[0, 1, 2], [0, 1, 0]]).all() and np.isfinite(scales[[0, 1, 2], [1, 0, 1]]).all()
    assert not codes[0, :128].any() and not codes[1, 128:].any() and codes[0, 128:].all()


def test_swiglu_backward_against_autograd():
    g = _rng(1)
    R, I, B, K = 7, 24, 4, 3
    gate, up, dh = (torch.tensor(g.standard_normal((R, I)) * s, requires_grad=s != 1.0) for s in (4.0, 2.0, 1.0))
    row_of = np.array([[0, -1, 3], [6, 2, 99], [-1, -1, 5], [1, 4, -1]])
    w = torch.tensor(g.random((B, K)), requires_grad=True)
    total = 0.0
    for t in range(B):
        for k in range(K):
            r = row_of[t, k]
            if 0 <= r < R:
                h = torch.nn.functional.silu(gate[r]) * up[r]
                total = total + w[t, k] * (dh[r] * h).sum()
    total.backward()
    dg, du, hw, dw = tr.swiglu_backward(dh.numpy(), gate.detach().numpy(), up.detach().numpy(), row_of,
                                        w.detach().numpy())
    np.testing.assert_allclose(dg, gate.grad.numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(du, up.grad.numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(hw[6], (w[1, 0] * torch.nn.functional.silu(gate[6]) * up[6]).detach().numpy(), rtol=1e-12)


ROUTERS = [("picks", True, 1.0), ("sigmoid", True, 2.5), ("sigmoid", False, 1.0), ("softmax", True, 1.0),
           ("softmax", False, 16.0)]


@pytest.mark.parametrize("score,renorm,scale", ROUTERS)
def test_route_backward_against_differences_of_the_forward_call(score, renorm, scale):
    """The weights of a fixed choice, moved by every logit in turn."""
    g = _rng(2)
    B, E, K, d = 5, 9, 3, 1e-6
    lg = g.standard_normal((B, E)) * 2
    if score != "picks":
        lg[1, 2:7] = -np.inf
        lg[2, 1:] = moe_low = oracle.moe.LOWEST_BF16
        assert moe_low < 0
    dw = g.standard_normal((B, K))

    def forward(l):
        if score == "picks":
            return oracle.route(l, K)
        return oracle.route_scored(l, K, score, renorm=renorm, scale=scale)

    ids, _ = forward(lg)
    got = tr.route_backward(lg, ids, dw, score, renorm, scale)
    want = np.zeros((B, E))
    for e in range(E):
        sides = []
        for step in (d, -d):
            l = lg.copy()
            ok = l[:, e] > oracle.moe.LOWEST_BF16
            l[ok, e] += step
            i, w = forward(l)
            np.testing.assert_array_equal(i, ids)
            sides.append((w * dw).sum(1))
        want[:, e] = (sides[0] - sides[1]) / (2 * d)
    # truncation d^2 |f'''| and cancellation 2^-52 |w| / d, both below 1e-8 times the scale
    np.testing.assert_allclose(got, want, atol=1e-8 * scale)


def test_route_backward_under_a_map_and_dropped_slots():
    g = _rng(3)
    lg = g.standard_normal((4, 6))
    phys = g.permutation(6)
    ids, _ = oracle.route(lg, 2)
    dw = g.standard_normal((4, 2))
    np.testing.assert_allclose(tr.route_backward(lg, phys[ids], dw, phys_of_logical=phys), tr.route_backward(lg, ids, dw))
    assert not tr.route_backward(lg, np.full((4, 2), -1), dw).any()


def _layer_loss(x, lg, dout, K, e_begin, e_end, weights, ids):
    """sum(out * dout) of the layer without roundings, in torch fp64, for a fixed choice of experts."""
    wg, wu, wd = weights
    w = torch.softmax(torch.gather(lg, 1, ids), dim=1)
    total = 0.0
    for t in range(x.shape[0]):
        for k in range(K):
            e = int(ids[t, k])
            if e_begin <= e < e_end:
                j = e - e_begin
                h = torch.nn.functional.silu(wg[j] @ x[t]) * (wu[j] @ x[t])
                total = total + w[t, k] * torch.dot(dout[t], wd[j] @ h)
    return total


@pytest.mark.parametrize("e_begin,e_end", [(0, 5), (1, 3)])
def test_layer_backward_against_autograd(monkeypatch, e_begin, e_end):
    """With exact checkpoints and no roundings the layer's gradients are the loss's."""
    monkeypatch.setattr(tr, "checkpoint", lambda v: (np.asarray(v), np.ones((len(v), 1))))
    monkeypatch.setattr(tr, "checkpoint_values", lambda c, s: c)
    monkeypatch.setattr(nx, "to_f32", lambda v: np.asarray(v, np.float64))
    g = _rng(4)
    T, E, K, H, I = 6, 5, 2, 8, 16
    n = e_end - e_begin
    t64 = lambda *s: torch.tensor(g.standard_normal(s), requires_grad=True)
    x, lg, wg, wu, wd = t64(T, H), t64(T, E), t64(n, I, H), t64(n, I, H), t64(n, H, I)
    dout = torch.tensor(g.standard_normal((T, H)))
    ids, _ = oracle.route(lg.detach().numpy(), K)
    _layer_loss(x, lg, dout, K, e_begin, e_end, (wg, wu, wd), torch.tensor(ids).long()).backward()
    got = tr.layer_backward(x.detach().numpy(), lg.detach().numpy(), dout.numpy(), K, E, e_begin, e_end,
                            [w.detach().numpy() for w in (wg, wu, wd)], "f32")
    for name, leaf in (("dx", x), ("dlogits", lg), ("gate", wg), ("up", wu), ("down", wd)):
        np.testing.assert_allclose(got[name], leaf.grad.numpy(), rtol=1e-10, atol=1e-12, err_msg=name)


def test_layer_backward_stays_near_the_exact_one_with_checkpoints():
    """Half a step of the checkpoints, at most amax / 127 each, moves the gradients by
    about a hundredth."""
    g = _rng(5)
    T, E, K, H, I = 24, 4, 2, 128, 128
    x, lg = g.standard_normal((T, H)), g.standard_normal((T, E))
    ws = [g.standard_normal(s) / np.sqrt(s[2]) for s in ((E, I, H), (E, I, H), (E, H, I))]
    dout = g.standard_normal((T, H))
    leaves = [torch.tensor(v, requires_grad=True) for v in (x, lg, *ws)]
    ids, _ = oracle.route(lg, K)
    _layer_loss(leaves[0], leaves[1], torch.tensor(dout), K, 0, E, leaves[2:], torch.tensor(ids).long()).backward()
    got = tr.layer_backward(x, lg, dout, K, E, 0, E, ws, "f32")
    for name, leaf in zip(("dx", "dlogits", "gate", "up", "down"), leaves):
        want = leaf.grad.numpy()
        assert np.linalg.norm(got[name] - want) <= 0.03 * np.linalg.norm(want), name


# each mistake below trips a pin that a correct implementation passes
@pytest.mark.parametrize("mistake", ["silu", "swap", "weight"])
def test_planted_mistakes_show(mistake):
    g = _rng(6)
    gate, up, dh = (g.standard_normal((3, 8)) for _ in range(3))
    row_of, w = np.array([[0, 1, 2]]), g.random((1, 3)) + 0.1
    dg, du, hw, dw = tr.swiglu_backward(dh, gate, up, row_of, w)
    sg = tr.sigmoid(gate)
    wrong = {"silu": w[0][:, None] * dh * up * sg, "swap": du, "weight": dg / w[0][:, None]}[mistake]
    d = 1e-6
    h = lambda a: (a * tr.sigmoid(a) * up * dh * w[0][:, None])
    numeric = (h(gate + d) - h(gate - d)) / (2 * d)
    np.testing.assert_allclose(dg, numeric, rtol=1e-6, atol=1e-8)
    assert not np.allclose(wrong, numeric, rtol=1e-3, atol=1e-6)
