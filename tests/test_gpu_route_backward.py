"""The router's gradient where scores are too small for 32 bits, though their shares
are not: picks far below zero (sigmoid), or far below the row's largest logit
(softmax).

Tolerance, in eps = 2^-24: a share t / sum t has t = e^(l - max) (1 + e^l)^-1 with the
exponent's difference rounded once (|l - max| <= D) and a handful of roundings
more, K additions and a quotient: within (2 D + K + 16) eps.  sum share dw adds K
more of |dw| <= big, and scale * share * (dw - sum) * rest a handful:
|error| <= scale share rest big (6 D + 8 K + 64) eps."""
import numpy as np
import pytest
import torch

from harness import has_gpu, to_np
from oracle import train as tr

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

EPS = 2.0**-24


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _case(T, E, K, score, low, spread, dtype, seed):
    """Logits whose K best by the bias lie around `low` (softmax: beside others around 0)."""
    g = _gen(seed)
    picks = torch.rand(T, E, generator=g, device="cuda").topk(K, 1).indices
    lg = torch.randn(T, E, generator=g, device="cuda") + (2 * low if score == "sigmoid" else 0.0)
    mine = low + spread * (torch.rand(T, K, generator=g, device="cuda") - 0.5)
    lg.scatter_(1, picks, mine)
    return lg.to(dtype), picks.to(torch.int32).contiguous()


def _shares(l, picks):
    """64-bit shares of the picks' scores and 1 - s of the sigmoid, from differences."""
    x = np.take_along_axis(l, picks, 1)
    d = x - x.max(1, keepdims=True)
    return x, np.exp(d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low", [-20.0, -60.0, -69.5, -89.0, -90.0, -103.0, -110.0, -300.0, -500.0, -690.0])
@pytest.mark.parametrize("T,E,K", [(65, 16, 2), (130, 256, 8), (9, 130, 70)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_renormalised_weights_of_small_scores(score, T, E, K, low, dtype):
    import combine_grouped_gemm_amd as m
    print(f"[low scores] {score} T={T} E={E} K={K} low={low} {dtype}", flush=True)
    spread, scale = 3.0, 2.5
    lg, ids = _case(T, E, K, score, low, spread, dtype, int(-low) + E)
    dw = torch.randn(T, K, generator=_gen(3), device="cuda")
    got = to_np(m.moe_route_backward(lg, ids, dw, score=score, renorm=True, scale=scale)).astype(np.float64)
    assert np.isfinite(got).all()
    l, n, d = to_np(lg).astype(np.float64), ids.cpu().numpy().astype(np.int64), dw.double().cpu().numpy()
    x, share = _shares(l, n)
    rest = np.ones_like(x)
    if score == "sigmoid":
        rest = 1.0 / (1.0 + np.exp(x))
        share = share * rest
    share /= share.sum(1, keepdims=True)
    ref = scale * share * (d - (share * d).sum(1, keepdims=True)) * rest
    big = np.abs(d).max(1, keepdims=True)
    D = spread + 8.0                                   # (bf16 logits are rounded by up to 2)
    room = scale * share * rest * big * (6 * D + 8 * K + 64) * EPS
    here = np.take_along_axis(got, n, 1)
    assert (np.abs(here - ref) <= room + 1e-37).all(), f"{(np.abs(here - ref) - room).max():.3e} over"
    other = got.copy()
    np.put_along_axis(other, n, 0.0, 1)
    assert not other.any()                             # the weights depend on the picks alone
    # the Jacobian in 64 bits, which cancels to K 2^-53 of scale * dw
    jac = tr.route_backward(l, n, d, score, True, scale)
    full = np.zeros_like(jac)
    np.put_along_axis(full, n, room, 1)
    assert (np.abs(got - jac) <= full + K * 2.0**-50 * scale * big).all()


@pytest.mark.parametrize("low", [-88.0, -100.0, -400.0])
def test_gradient_against_differences_of_the_forward_call(low):
    """Along steps of +-h in every logit: the weights' third derivative along them is at
    most 8 scale a weight, their rounding 2^-24 scale."""
    import combine_grouped_gemm_amd as m
    T, E, K, scale, h = 40, 32, 4, 2.5, 2.0**-6
    lg, _ = _case(T, E, K, "sigmoid", low, 3.0, torch.float32, 7)
    lg = (lg * 64).round() / 64                        # steps of h are exact
    ids, w = m.moe_route_scored(lg, K, score="sigmoid", renorm=True, scale=scale)
    dw = torch.randn(T, K, generator=_gen(4), device="cuda")
    grad = m.moe_route_backward(lg, ids, dw, score="sigmoid", renorm=True, scale=scale).double()
    assert float(w.sum(1).min()) > 0.99 * scale
    big = dw.abs().double().amax(1)
    for seed in range(6):
        v = torch.randint(0, 2, (T, E), generator=_gen(seed), device="cuda") * 2.0 - 1.0

        def loss(x):
            # the picks' weights, whichever order the call names them in
            i, z = m.moe_route_scored(x, K, score="sigmoid", bias=None, renorm=True, scale=scale)
            full = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, i.long(), z.double())
            return (full.gather(1, ids.long()) * dw).sum(1), torch.equal(i.sort(1).values, ids.sort(1).values)

        (a, same_a), (b, same_b) = loss(lg + h * v), loss(lg - h * v)
        assert same_a and same_b                       # the picks lie far above the others
        room = K * scale * big * (8 * h * h / 6 + 4 * EPS / h)
        assert bool((((a - b) / (2 * h) - (grad * v).sum(1)).abs() <= room).all())


@pytest.mark.parametrize("low", [-89.0, -90.0, -200.0])
def test_a_single_live_pick_passes_nothing(low):
    """Its renormalised weight is constant."""
    import combine_grouped_gemm_amd as m
    lg = torch.full((3, 8), -float("inf"), device="cuda")
    lg[:, 5] = low
    for score in ("sigmoid", "softmax"):
        ids, w = m.moe_route_scored(lg, 2, score=score, scale=2.5)
        assert bool((w[:, 0] == 2.5).all()) and bool((ids[:, 1] == -1).all())
        dw = torch.tensor([[1.0, 7.0]] * 3, device="cuda")
        assert not bool(m.moe_route_backward(lg, ids, dw, score=score, scale=2.5).any())


@pytest.mark.parametrize("score,low,dead", [("sigmoid", -709.75, False), ("sigmoid", -709.8, True), ("sigmoid", -5000.0, True),
                                            ("sigmoid", -3e38, True), ("softmax", -740.0, False), ("softmax", -760.0, True),
                                            ("softmax", -3e38, True)])
def test_sums_that_are_zero_in_64_bits_pass_nothing(score, low, dead):
    """The forward call's weights are zeros there, constants."""
    import combine_grouped_gemm_amd as m
    lg = torch.zeros(2, 8, device="cuda")
    bias = torch.zeros(8, device="cuda")
    lg[:, :2], bias[:2] = low, 5.0
    ids, w = m.moe_route_scored(lg, 2, score=score, bias=bias)
    assert bool((ids < 2).all()) and bool((w == 0).all()) == dead
    dw = torch.tensor([[1.0, -1.0]] * 2, device="cuda")
    got = m.moe_route_backward(lg, ids, dw, score=score)
    assert bool((got == 0).all()) == dead and bool(torch.isfinite(got).all())


def test_gradient_in_place_of_its_logits():
    """dlogits may be the logits themselves."""
    import combine_grouped_gemm_amd as m
    for score, renorm in (("picks", True), ("sigmoid", True), ("softmax", True), ("softmax", False)):
        lg = torch.randn(77, 200, generator=_gen(1), device="cuda")
        ids = m.moe_route(lg, 6)[0]
        dw = torch.randn(77, 6, generator=_gen(2), device="cuda")
        want = m.moe_route_backward(lg, ids, dw, score=score, renorm=renorm)
        assert torch.equal(m.moe_route_backward(lg, ids, dw, score=score, renorm=renorm, dlogits=lg), want)
