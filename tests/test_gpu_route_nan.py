"""Scored routing of tokens with a logit or bias that is no ordinary number, at
every expert in turn, so in every lane and place of a lane: NaN ranks behind
every number, and every slot is written."""
import numpy as np
import pytest
import torch

import oracle
from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

SHAPES = [  # E, K, n_groups, topk_groups, group_top
    (8, 2, 1, 1, 2), (16, 3, 1, 1, 2), (29, 3, 1, 1, 2), (59, 6, 1, 1, 2), (60, 4, 4, 2, 2), (64, 8, 8, 3, 1),
    (128, 12, 1, 1, 2), (250, 8, 1, 1, 1), (256, 8, 8, 4, 2), (256, 8, 1, 1, 2), (256, 1, 16, 1, 2), (384, 10, 1, 1, 2),
    (512, 8, 2, 1, 2), (512, 12, 1, 1, 2), (256, 13, 1, 1, 2), (96, 6, 3, 2, 2), (600, 8, 1, 1, 2)]


def _check(lg, K, score, bias, kw, what):
    import combine_grouped_gemm_amd as m
    print(f"[nan] {what}", flush=True)
    T = lg.shape[0]
    ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), -7.0, device="cuda")
    m.moe_route_scored(lg.cuda(), K, score=score, bias=None if bias is None else bias.cuda(), topk_ids=ids, topk_w=w, **kw)
    with np.errstate(all="ignore"):
        ri, rw = oracle.route_scored(lg.double().numpy(), K, score, bias=None if bias is None else bias.double().numpy(),
                                     **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), ri)
    got = w.cpu().double().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(rw))
    # the weight is computed in 64 bits and rounded to fp32 once
    off = np.abs(got - rw) - 2.0**-23 * np.abs(rw)
    assert not (off > 2.0**-149).any()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,K,G,keep,top", SHAPES)
def test_a_nan_logit_at_every_expert(E, K, G, keep, top, score, bf16):
    g = torch.Generator().manual_seed(E + K)
    kw = dict(n_groups=G, topk_groups=keep, group_top=top)
    # no two scores within fp64's reach of each other: the order is the logits'
    lg = torch.stack([torch.randperm(E, generator=g) for _ in range(E)]).float() / 64 - 2
    lg[torch.arange(E), torch.arange(E)] = float("nan")
    if bf16:
        lg = lg.to(torch.bfloat16).float()                 # ties among the small steps: the lower id
    for bias in (None, torch.randperm(E, generator=g).float() / 37):
        # softmax: every weight of such a token is NaN, and the experts rank by id
        _check(lg.to(torch.bfloat16) if bf16 else lg, K, score, bias, kw, f"E={E} K={K} {score} bias={bias is not None}")


@pytest.mark.parametrize("E,K,G,keep,top", SHAPES)
def test_a_nan_bias_at_every_expert(E, K, G, keep, top):
    g = torch.Generator().manual_seed(E)
    lg = torch.stack([torch.randperm(E, generator=g) for _ in range(8)]).float() / 64 - 2
    for e in range(0, E, max(1, E // 24)):
        bias = torch.randperm(E, generator=g).float() / 37
        bias[e] = float("nan")
        _check(lg, K, "sigmoid", bias, dict(n_groups=G, topk_groups=keep, group_top=top), f"E={E} K={K} bias NaN at {e}")


@pytest.mark.parametrize("value", [float("inf"), 3e38, -3e38, 1e30, -1e30])
@pytest.mark.parametrize("E,K,G,keep,top", SHAPES)
def test_a_logit_far_out_at_every_expert(E, K, G, keep, top, value):
    """Finite ones and +inf score 1 or 0; two of them, and a NaN beside them."""
    g = torch.Generator().manual_seed(E)
    t = torch.arange(E)
    lg = torch.stack([torch.randperm(E, generator=g) for _ in range(E)]).float() / 64 - 2
    lg[t, t] = value
    lg[t[::2], (t[::2] + E // 2) % E] = value
    lg[t[::3], (t[::3] + E // 3) % E] = float("nan")
    _check(lg, K, "sigmoid", None, dict(n_groups=G, topk_groups=keep, group_top=top), f"E={E} K={K} value={value}")


def test_only_nan():
    for E, K, G, keep, top in SHAPES:
        lg = torch.full((9, E), float("nan"))
        lg[3, E // 2] = 1.0
        for score in ("sigmoid", "softmax"):
            _check(lg, K, score, None, dict(n_groups=G, topk_groups=keep, group_top=top), f"E={E} {score}")
