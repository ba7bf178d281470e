"""The 256 x 256 int8 tiles, whose experts are ranked by rows, on the masked layout.

They are taken when expected rows >= 32 and the 64 x 128 tiles number more than
two a CU, E * ceil(expected / 64) * ceil(N / 128) (gate/up: / 64): on this
layout's small test shapes only expected rows far past the block reach them, with
many experts ordinary ones do."""
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]


def _large(E, hint, N, gated):
    small = E * -(-hint // 64) * -(-N // (64 if gated else 128))
    return hint >= 32 and small > 2 * torch.cuda.get_device_properties(0).multi_processor_count


def _check(p, hints, what):
    assert all(_large(p.E, h, p.N, p.gated) for h in hints)
    ref = p.run(1)
    p.check(ref, f"{what}, small tiles")
    for hint in hints:
        print(f"[masked] {what} hint={hint}", flush=True)
        got = p.run(hint)
        p.check(got, f"{what}, hint {hint}")             # rows without a slot among them
        assert torch.equal(got, ref)
        assert torch.equal(p.run(hint, pack=True), ref)
        if not p.gated:
            p.check(p.run(hint, y_dtype=torch.float32), f"{what}, fp32 y, hint {hint}")


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("counts,cap_e,K,N", [
    ([3, 0, 8, 8, 1], 8, 144, 80),                        # full, empty and one-row blocks
    ([256, 600, 0, 257, 511], 600, 272, 272),             # more rows than a tile, an expert's rows split evenly
    ([0, 0, 0], 64, 128, 64), ([0, 0, 1], 1, 1040, 528), ([513], 700, 400, 1552)])
def test_expected_rows_past_the_block(counts, cap_e, K, N, gated):
    from test_gpu_int8 import Problem
    p = Problem(counts, K, N, seed=K + N, cap_e=cap_e, gated=gated)
    _check(p, (10**6, 2**31 - 1), f"counts={counts} K={K} N={N} gated={gated}")


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("K,N", [(128, 2048), (384, 1040), (400, 1552)])
def test_ordinary_expected_rows_of_many_experts(K, N, gated):
    from test_gpu_int8 import Problem
    counts = [0, 33, 257, 64, 1, 33, 256, 0, 129, 300, 7, 33] * 8
    p = Problem(counts, K, N, seed=K + N, cap_e=300, gated=gated)
    _check(p, (40, 100, 192, 300), f"96 experts K={K} N={N} gated={gated}")


@pytest.mark.parametrize("gated", [True, False])
def test_counts_past_the_block_and_below_zero(gated):
    """A block's count is cut to its rows, a negative one is none."""
    from test_gpu_int8 import Problem
    counts, cap_e = [70, 0, 12, 70, 0], 70
    p = Problem(counts, 256, 144, seed=9, cap_e=cap_e, gated=gated)
    ref = p.run(1)
    p.rows = torch.tensor([71, -3, 12, 2**31 - 1, -2**31], dtype=torch.int32, device="cuda")
    for hint in (1, 10**6):
        got = p.run(hint)
        p.check(got, f"hint {hint}")
        assert torch.equal(got, ref)


def test_the_masked_layer_with_many_rows_an_expert():
    """route to combine with expected rows that take the large tiles, against the
    contiguous layout: the same products, so the same bits."""
    import combine_grouped_gemm_amd as m
    T, E, K, H, I = 3000, 32, 4, 256, 1024
    g = torch.Generator().manual_seed(3)
    x, lg = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(), torch.randn(T, E, generator=g).cuda()
    w = {}
    for name, r, c in (("gate", I, H), ("up", I, H), ("down", H, I)):
        q, s = m.moe_quant_rows((torch.randn(E * r, c, generator=g) / c**0.5).cuda())
        w[name], w[name + "_scale"] = q.view(E, r, c), s.view(E, r)
    outs = []
    for layout, cap in (("contiguous", None), ("masked", 700)):
        layer = m.MoELayer((T,), E, K, H, I, 0, E, "int8", "bf16", "bf16", layout=layout, cap_per_expert=cap,
                           router=dict(score="sigmoid"))
        assert _large(E, layer.expected_rows, I, True)
        outs.append(layer.forward([x], lg, w).clone())
        assert int(layer.counts.max()) <= 700
    assert torch.equal(*outs)
