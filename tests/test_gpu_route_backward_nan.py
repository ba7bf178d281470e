"""A NaN logit makes the forward call's weights NaN; the gradients of those weights are
NaN too, not the numbers of a row without it."""
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

MASKED = -float("inf")


def _grads(score, renorm, lg, K=3, dtype=torch.float32):
    import combine_grouped_gemm_amd as m
    lg = torch.tensor(lg, device="cuda").to(dtype)
    ids, w = m.moe_route_scored(lg, K, score=score, renorm=renorm)
    dw = torch.tensor([[1.0, -2.0, 0.5]] * len(lg), device="cuda")
    return torch.isnan(w).tolist(), ids.tolist(), m.moe_route_backward(lg, ids, dw, score=score, renorm=renorm)


NAN = float("nan")
# three unmasked experts of five, the second row without a NaN
ROWS = [[2.0, NAN, MASKED, 0.5, MASKED], [2.0, 1.0, MASKED, 0.5, MASKED]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sigmoid(dtype):
    bad, ids, got = _grads("sigmoid", False, ROWS, dtype=dtype)
    assert bad == [[i == 1 for i in ids[0]], [False] * 3]
    assert torch.isnan(got).tolist() == [[False, True, False, False, False], [False] * 5]
    bad, ids, got = _grads("sigmoid", True, ROWS, dtype=dtype)
    assert bad == [[True] * 3, [False] * 3]            # the sum is NaN
    assert torch.isnan(got).tolist() == [[True, True, False, True, False], [False] * 5]
    assert bool((got[:, [2, 4]] == 0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("far", [0.0, 800.0])
def test_softmax_over_all(far, renorm, dtype):
    """Also where the NaN's expert is not picked, and where the picks are too small."""
    low = [[2.0, NAN, MASKED, 0.5, 0.25], [2.0, 1.0, MASKED, 0.5, 0.25]]
    low = [[v - far for v in r] for r in low]
    bad, ids, got = _grads("softmax", renorm, low, dtype=dtype)
    assert bad == [[True] * 3, [False] * 3]
    assert torch.isnan(got).tolist() == [[True, True, False, True, True], [False] * 5]
    assert bool((got[:, 2] == 0).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_nan_beside_a_sum_of_zero(score):
    """Picks whose scores are zero in 64 bits, and a NaN: the sum is NaN, not zero."""
    import combine_grouped_gemm_amd as m
    lg = torch.tensor([[-3000.0, NAN, 0.0, -3000.0]], device="cuda")
    if score == "softmax":
        lg[0, 1], lg[0, 3] = -3000.0, NAN
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    got = m.moe_route_backward(lg, ids, torch.tensor([[1.0, -2.0]], device="cuda"), score=score)
    want = [True, True, False, False] if score == "sigmoid" else [True] * 4
    assert torch.isnan(got).tolist() == [want]


def test_an_infinite_logit():
    """Sigmoid: a score of one; softmax over all: NaN weights, and gradients."""
    inf = float("inf")
    bad, _, got = _grads("sigmoid", True, [[inf, 1.0, MASKED, 0.5, MASKED]])
    assert not any(bad[0]) and bool(torch.isfinite(got).all()) and float(got[0, 0]) == 0.0
    bad, _, got = _grads("softmax", True, [[inf, 1.0, MASKED, 0.5, MASKED]])
    assert all(bad[0]) and torch.isnan(got).tolist() == [[True, True, False, True, False]]
