"""GPU parity of the scored router against the 64-bit oracle.

ids are exact (scores are compared in 64 bits on both sides; the inputs hold
exact ties, which go to the lower id, but no two scores nearer than the last
places of 64 bits).  Weights: computed in 64 bits and rounded once, 2^-24
relative; the bar of 4 * 2^-24 leaves room for one fp32 operation on each of a
weight's two factors and their quotient.  Below 2^-126 fp32 has the fixed step
2^-149, so a correctly rounded weight is off by up to 2^-150 there whatever its
size (1.4e-87 is stored as 0): the absolute bar."""
import numpy as np
import pytest
import torch

import oracle
from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

LOW = oracle.moe.LOWEST_BF16
RTOL = 4 * 2.0**-24


def _inputs(B, E, seed, bf16=False, mask=0.0, ties=False, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    lg = torch.randn(B, E, generator=g) * spread
    if ties:
        # equal logits and equal biases tie exactly; the shift keeps opposite logits
        # apart, whose sigmoids would add up to 1 and tie two groups but for rounding
        lg = torch.round(lg * 2) / 2 + 0.3
    if mask:
        lg[torch.rand(B, E, generator=g) < mask] = -float("inf")
        lg[torch.rand(B, E, generator=g) < mask / 4] = torch.finfo(torch.float32).min
        lg[B // 2] = LOW
    bias = torch.randn(E, generator=g) * 0.1
    if ties:
        bias = torch.full((E,), 0.125)
    return (lg.to(torch.bfloat16) if bf16 else lg), bias


def _check(lg, K, score, bias=None, stream=None, **kw):
    import combine_grouped_gemm_amd as m
    print(f"[scored] B={lg.shape[0]} E={lg.shape[1]} K={K} {score} {lg.dtype} bias={bias is not None} {kw}", flush=True)
    ids, w = m.moe_route_scored(lg.cuda(), K, score=score, bias=None if bias is None else bias.cuda(), **kw)
    torch.cuda.synchronize()
    rid, rw = oracle.route_scored(lg.double().numpy(), K, score, None if bias is None else bias.double().numpy(), **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=RTOL, atol=2.0**-150)
    return ids, w


SHAPES = [  # B, E, K, groups, keep, group_top
    (1, 256, 8, 8, 4, 2), (129, 256, 8, 8, 4, 2), (300, 256, 8, 8, 4, 1), (5, 1, 1, 1, 1, 2), (33, 7, 7, 1, 1, 1),
    (64, 8, 2, 4, 1, 2), (17, 60, 4, 1, 1, 2), (40, 64, 6, 8, 3, 2), (21, 96, 10, 16, 16, 2), (30, 128, 4, 1, 1, 1),
    (19, 160, 6, 8, 3, 1), (12, 384, 8, 8, 2, 2), (9, 512, 22, 4, 2, 2), (7, 1000, 100, 4, 3, 2), (6, 1024, 16, 32, 8, 2),
    (4, 1024, 1024, 1, 1, 1), (8, 1024, 70, 1024, 100, 2), (6, 1024, 3, 512, 2, 2), (11, 72, 65, 3, 3, 2),
    (10, 130, 64, 2, 1, 2), (3, 1024, 512, 2, 1, 1), (50, 31, 3, 31, 5, 2), (15, 24, 5, 3, 2, 2),
]


@pytest.mark.parametrize("B,E,K,G,keep,top", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_parity(B, E, K, G, keep, top, score):
    kw = dict(n_groups=G, topk_groups=keep, group_top=top)
    lg, bias = _inputs(B, E, B + E + K)
    _check(lg, K, score, bias, renorm=True, scale=2.5, **kw)
    _check(lg, K, score, None, renorm=False, **kw)
    lg, bias = _inputs(B, E, B + E + K + 1, bf16=True, ties=True)
    _check(lg, K, score, bias, renorm=True, **kw)
    lg, bias = _inputs(B, E, B + E + K + 2, mask=0.3)
    bias[::5] = -float("inf")
    _check(lg, K, score, bias, renorm=True, scale=16.0, **kw)
    lg, _ = _inputs(B, E, B + E + K + 3, mask=0.7, bf16=True)
    _check(lg, K, score, None, renorm=False, scale=0.5, **kw)


@pytest.mark.parametrize("E", [2, 3, 8, 15, 17, 60, 127, 129, 250, 255, 257, 500, 511, 513])
def test_expert_counts_without_groups(E):
    for K in {1, min(2, E), min(12, E), min(13, E)}:
        for score in ("sigmoid", "softmax"):
            lg, bias = _inputs(37, E, E + K)
            _check(lg, K, score, bias)
            lg, bias = _inputs(37, E, E + K + 1, bf16=True, ties=True, mask=0.2)
            _check(lg, K, score, None, renorm=False)
            _check(lg, K, score, bias, n_groups=E, topk_groups=E, group_top=1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_neighbours_that_fp32_scores_cannot_tell_apart(score):
    """Logits one fp32 step apart, on the flat parts of the score: neighbours
    differ by far less than an fp32 score's last place."""
    B, E = 64, 256
    for centre in (0.0, 3.0, 9.0, 14.0, -9.0):
        # one fp32 step at the centre (2^-22 near 3, 2^-20 near 9 and 14; around 0 a step of 2^-26)
        step = 2.0**-26 if centre == 0.0 else float(np.spacing(np.float32(abs(centre))))
        g = torch.Generator().manual_seed(int(centre) + 50)
        order = torch.stack([torch.randperm(E, generator=g) for _ in range(B)]).double()
        lg = (centre + order * step).float()
        assert (torch.sort(lg, 1).values.diff(dim=1) > 0).all()
        _check(lg, 8, score, None)
        # groups by their best alone (sums of two evenly spaced neighbours would tie)
        _check(lg, 8, score, None, n_groups=8, topk_groups=4, group_top=1)
        # and with biases that are equal: the same order
        _check(lg, 8, score, torch.full((E,), 0.25), n_groups=8, topk_groups=4, group_top=1)


@pytest.mark.parametrize("E,G,keep", [(256, 16, 5), (256, 2, 1), (256, 4, 3), (512, 16, 9), (512, 8, 4), (16, 8, 4), (32, 16, 16),
                                       (240, 8, 2), (528, 8, 4), (64, 1, 1)])
def test_candidate_counts_and_groups(E, G, keep):
    """K on both sides of the shapes that a row of lanes can hold, with more
    ties at the cut than it has candidates for."""
    for K in (1, 2, 11, 12, 13, 16):
        if K > keep * (E // G):
            continue
        for score in ("sigmoid", "softmax"):
            kw = dict(n_groups=G, topk_groups=keep)
            lg, bias = _inputs(70, E, E + K)
            _check(lg, K, score, bias, **kw)
            lg = torch.round(lg) + 0.3                    # a handful of values: long runs of ties
            _check(lg, K, score, None, **kw)
            _check(lg, K, score, torch.full((E,), -0.7), renorm=False, **kw)


def test_biases_that_cancel_scores():
    """c near zero and of both signs: the error of a score no longer shrinks with it."""
    for seed in range(3):
        lg, _ = _inputs(200, 256, seed, spread=0.3)
        g = torch.Generator().manual_seed(seed)
        bias = -torch.sigmoid(torch.randn(256, generator=g) * 0.3)
        for top in (1, 2):
            _check(lg, 8, "sigmoid", bias, n_groups=8, topk_groups=4, group_top=top)
        _check(lg, 8, "softmax", bias / 128, n_groups=8, topk_groups=4, group_top=2)
        _check(lg, 8, "sigmoid", bias * 1e4, n_groups=8, topk_groups=4, group_top=2)
        _check(lg, 8, "sigmoid", bias * 1e33, n_groups=8, topk_groups=4, group_top=2)


@pytest.mark.parametrize("E,G,keep,crowd", [(256, 8, 4, 0), (256, 16, 3, 0), (128, 4, 2, 0), (512, 2, 1, 0), (256, 8, 4, 6),
                                             (64, 8, 1, 0), (240, 8, 5, 4)])
def test_groups_that_fp32_cannot_tell_apart(E, G, keep, crowd):
    """Every group holds the same pattern of logits, each group's a few fp32 steps
    above the last one's, in an order of its own for every token: group scores
    differ by less than an fp32 score's error.  crowd: that many more experts of
    each group lie as near to its second best."""
    S = E // G
    g = torch.Generator().manual_seed(E + G)
    pattern = torch.cat([torch.tensor([1.5, 1.25]), torch.randn(S - 2, generator=g) * 0.3]).clamp(max=1.5)
    for i in range(crowd):
        pattern[2 + i] = 1.25 - (i + 1) * 2.0**-21
    lg = torch.empty(48, G, S)
    for t in range(48):
        order = torch.randperm(G, generator=g).float()
        # steps of 2^-23 are exact between 1 and 2
        lg[t] = pattern[None, torch.randperm(S, generator=g)] + order[:, None] * 2.0**-22
    lg = lg.view(48, E)
    for score in ("sigmoid", "softmax"):
        for top in (1, 2):
            for bias in (None, torch.full((E,), -0.8)):
                _check(lg, min(8, keep * S), score, bias, n_groups=G, topk_groups=keep, group_top=top)


def test_misaligned_rows():
    """Contiguous tensors that start in the middle of a 16-byte piece."""
    for E in (256, 128):
        for dt in (torch.float32, torch.bfloat16):
            lg, bias = _inputs(21, E, 5, bf16=dt == torch.bfloat16)
            import combine_grouped_gemm_amd as m
            x = torch.empty(21 * E + 1, dtype=dt, device="cuda")[1:].view(21, E)
            x.copy_(lg)
            b = torch.empty(E + 3, device="cuda")[3:]
            b.copy_(bias)
            for xx, bb in ((x, b), (lg.cuda(), b), (x, bias.cuda())):
                ids, w = m.moe_route_scored(xx, 8, bias=bb, n_groups=8, topk_groups=4)
                rid, rw = oracle.route_scored(lg.double().numpy(), 8, "sigmoid", bias.double().numpy(), 8, 4)
                np.testing.assert_array_equal(ids.cpu().numpy(), rid)
                np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=RTOL)


def test_extreme_logits():
    """Saturated sigmoids tie (lower id), scores that underflow are zero, and a
    sum of zero gives zero weights."""
    lg = torch.zeros(4, 64)
    lg[0, 10:20] = torch.arange(100, 1100, 100)           # sigmoid 1 for all
    lg[1] = -1000.0                                       # sigmoid underflows to 0
    lg[2, 5:] = -3e38                                     # far below, not masked
    lg[3] = torch.linspace(-800, 800, 64)
    for renorm in (True, False):
        for score in ("sigmoid", "softmax"):
            _check(lg, 8, score, renorm=renorm, n_groups=4, topk_groups=2)
            _check(lg, 8, score, torch.linspace(0, 1, 64), renorm=renorm, n_groups=4, topk_groups=2)


def test_nan_logits():
    lg, bias = _inputs(12, 40, 3)
    lg[3, 7] = float("nan")
    lg[4, :35] = float("nan")
    lg[5] = float("nan")
    lg[6, 2], lg[6, 3] = float("inf"), -float("inf")
    for kw in (dict(), dict(n_groups=5, topk_groups=2)):
        _check(lg, 6, "sigmoid", bias, **kw)
    # softmax: the whole row is NaN; ids stay distinct and in range
    import combine_grouped_gemm_amd as m
    ids, w = m.moe_route_scored(lg.cuda(), 6, score="softmax")
    ids, w = ids.cpu(), w.cpu()
    for t in (3, 4, 5):
        assert len(set(ids[t].tolist())) == 6 and 0 <= int(ids[t].min()) and int(ids[t].max()) < 40
        assert torch.isnan(w[t]).all()
    ok = [t for t in range(12) if t not in (3, 4, 5, 6)]
    rid, rw = oracle.route_scored(lg[ok].double().numpy(), 6, "softmax")
    np.testing.assert_array_equal(ids[ok].numpy(), rid)
    np.testing.assert_allclose(w[ok].numpy(), rw, rtol=RTOL)


def test_map_and_shared_slots():
    import combine_grouped_gemm_amd as m
    lg, bias = _inputs(37, 48, 9, mask=0.9)
    perm = torch.randperm(48, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    rid, rw = oracle.route_scored(lg.double().numpy(), 5, "sigmoid", bias.double().numpy(), 6, 3)
    ids, w = m.moe_route_scored(lg.cuda(), 5, bias=bias.cuda(), n_groups=6, topk_groups=3, phys_of_logical=perm.cuda(),
                                n_shared=2)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    np.testing.assert_array_equal(ids[:, :5], np.where(rid >= 0, perm.numpy()[rid], -1))
    np.testing.assert_array_equal(ids[:, 5:], np.tile([48, 49], (37, 1)))
    np.testing.assert_allclose(w[:, :5], rw, rtol=RTOL)
    assert (w[:, 5:] == 1.0).all()
    assert (rid < 0).any()


def test_output_rows_and_nothing_else_are_written():
    """Outputs inside larger buffers: what lies behind the last row stays."""
    import combine_grouped_gemm_amd as m
    lg, _ = _inputs(6, 64, 4)
    ids = torch.full((9, 4), 77, dtype=torch.int32, device="cuda")
    w = torch.full((9, 4), 77.0, device="cuda")
    m.moe_route_scored(lg.cuda(), 4, topk_ids=ids[:6], topk_w=w[:6])
    m.moe_route_scored(torch.empty(0, 64, device="cuda"), 4)
    torch.cuda.synchronize()
    assert (ids[6:] == 77).all() and (w[6:] == 77.0).all() and (ids[:6] < 64).all()


def test_side_stream_and_graph():
    """Two calls at once on two streams, and a captured call replayed on new inputs."""
    import combine_grouped_gemm_amd as m
    lg, bias = _inputs(500, 256, 11)
    kw = dict(n_groups=8, topk_groups=4, scale=2.5)
    x, b = lg.cuda(), bias.cuda()
    ref = m.moe_route_scored(x, 8, bias=b, **kw)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for s in (s1, s2):
        with torch.cuda.stream(s):
            outs.append(m.moe_route_scored(x, 8, bias=b, **kw))
    outs.append(m.moe_route_scored(x, 8, bias=b, stream=s1, **kw))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], ref[0]) and torch.equal(o[1], ref[1])
    ids, w = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    static = x.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_route_scored(static, 8, bias=b, topk_ids=ids, topk_w=w, **kw)
    for rep in range(3):
        new = _inputs(500, 256, 20 + rep)[0].cuda()
        static.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        eager = m.moe_route_scored(new, 8, bias=b, **kw)
        torch.cuda.synchronize()
        assert torch.equal(ids, eager[0]) and torch.equal(w, eager[1])


def test_binding_refusals():
    import combine_grouped_gemm_amd as m
    lg = torch.zeros(4, 16, device="cuda")
    t = lambda shape, dt=torch.float32: torch.zeros(shape, dtype=dt, device="cuda")
    for kw, msg in ((dict(bias=t(15)), "bias"), (dict(bias=t(16, torch.bfloat16)), "bias"),
                    (dict(bias=torch.zeros(16)), "device tensor"), (dict(score="tanh"), "score"),
                    (dict(topk_ids=t((4, 3), torch.int32)), "topk_ids"), (dict(topk_w=t((3, 2))), "topk_w"),
                    (dict(phys_of_logical=t(8, torch.int32)), "phys_of_logical")):
        with pytest.raises(ValueError, match=msg):
            m.moe_route_scored(lg, 2, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_route_scored(t((4, 32))[:, ::2], 2)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        m.moe_route_scored(lg.half(), 2)
    for kw, msg in ((dict(n_groups=3), "divide"), (dict(n_groups=4, topk_groups=5), "topk_groups"),
                    (dict(group_top=3), "group_top"), (dict(n_groups=8, topk_groups=1, group_top=1, K=3), "exceeds")):
        with pytest.raises(m.MoeError, match=msg):
            m.moe_route_scored(lg, kw.pop("K", 2), **kw)


@pytest.mark.parametrize("B,E,K", [(2**28 + 64, 1, 1), (2**26 + 192, 16, 13)])
def test_batches_of_more_tokens_than_one_launch_takes(B, E, K):
    """16 and 64 threads a token: as one grid either batch has 2^32 threads or more."""
    import combine_grouped_gemm_amd as m
    few = _inputs(64, E, 5, bf16=True)[0].cuda()
    ids, w = m.moe_route_scored(few.repeat(B // 64, 1), K)
    first = m.moe_route_scored(few, K)
    assert bool((ids.view(-1, 64, K) == first[0]).all()) and bool((w.view(-1, 64, K) == first[1]).all())
    _check(few.cpu(), K, "sigmoid")


@pytest.mark.parametrize("E,G,keep", [(60, 4, 2), (60, 2, 1), (8, 8, 3), (8, 4, 2), (8, 2, 1), (2, 2, 1), (72, 8, 5), (24, 8, 7),
                                       (500, 4, 3), (504, 8, 2), (510, 2, 1), (130, 2, 1), (36, 4, 1), (40, 8, 1)])
def test_groups_that_do_not_fill_their_lanes(E, G, keep):
    """Lanes behind a group's last expert hold nothing; a group may be smaller than its lanes."""
    test_candidate_counts_and_groups(E, G, keep)
    S = E // G
    for seed, score in ((1, "sigmoid"), (2, "softmax")):
        for B in (1, 63):
            lg, bias = _inputs(B, E, seed, mask=0.4, bf16=B == 1)
            bias[::4] = -float("inf")
            for top in (1, 2):
                _check(lg, min(8, keep * S), score, bias, n_groups=G, topk_groups=keep, group_top=top)
                _check(lg, min(8, keep * S), score, None, n_groups=G, topk_groups=keep, group_top=top, renorm=False)
    if S >= 2:
        test_groups_that_fp32_cannot_tell_apart(E, G, keep, min(3, S - 2))


@pytest.mark.parametrize("E", [64, 192, 320, 384, 512])
def test_misaligned_rows_of_other_lane_shares(E):
    import combine_grouped_gemm_amd as m
    for dt in (torch.float32, torch.bfloat16):
        lg, bias = _inputs(35, E, 8, bf16=dt == torch.bfloat16, mask=0.1)
        x = torch.empty(35 * E + 1, dtype=dt, device="cuda")[1:].view(35, E)
        x.copy_(lg)
        b = torch.empty(E + 3, device="cuda")[3:]
        b.copy_(bias)
        rid, rw = oracle.route_scored(lg.double().numpy(), 8, "softmax", bias.double().numpy(), 4, 2)
        for xx, bb in ((x, b), (lg.cuda(), b), (x, bias.cuda()), (lg.cuda(), bias.cuda())):
            ids, w = m.moe_route_scored(xx, 8, score="softmax", bias=bb, n_groups=4, topk_groups=2)
            np.testing.assert_array_equal(ids.cpu().numpy(), rid)
            np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=RTOL, atol=2.0**-150)
