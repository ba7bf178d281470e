"""The training layer's segments as any iterable that moe_dispatch takes, one that can be
walked once included."""
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]


@pytest.mark.parametrize("kind", [list, tuple, iter])
def test_segments_of_any_kind(kind):
    import combine_grouped_gemm_amd as m
    seg, E, K, H, I = [3, 0, 5], 4, 2, 64, 72
    layer = m.MoELayer(seg, E, K, H, I, 0, E, "bf16", "bf16", "bf16", train=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randn(n, H, generator=g, device="cuda").bfloat16() for n in seg]
    lg = torch.randn(8, E, generator=g, device="cuda")
    w = {k: torch.randn(E, *s, generator=g, device="cuda").bfloat16()
         for k, s in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I)))}
    layer.x_q.fill_(77)
    layer.x_s.fill_(7.0)
    layer.forward(kind(x), lg, w)
    q, s = m.moe_checkpoint_rows(torch.cat(x))
    assert torch.equal(layer.x_q, q) and torch.equal(layer.x_s, s)
