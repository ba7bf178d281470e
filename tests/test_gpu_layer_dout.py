"""The layer's backward pass refuses a dout that lacks rows of its tokens, which would
count as zeros; rows behind them change nothing."""
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]


def _layer(m):
    T, E, K, H, I = 6, 4, 2, 64, 72
    layer = m.MoELayer([T], E, K, H, I, 0, E, "bf16", "bf16", "bf16", train=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, lg = (torch.randn(T, n, generator=g, device="cuda") for n in (H, E))
    w = {k: torch.randn(E, *s, generator=g, device="cuda").bfloat16()
         for k, s in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I)))}
    layer.forward([x.bfloat16()], lg, w)
    return layer, lg, w, layer.new_grads()


@pytest.mark.parametrize("shape", [(5, 64), (0, 64), (6, 72), (7, 72), (384,)])
def test_dout_of_another_shape(shape):
    import combine_grouped_gemm_amd as m
    layer, lg, w, grads = _layer(m)
    dout = torch.ones(shape, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: layer.backward(dout, lg, w, grads), lambda: layer.dgrad_down(dout, w),
                 lambda: layer.wgrad_down(dout, grads)):
        with pytest.raises(ValueError, match="dout must have shape"):
            call()


def test_rows_behind_the_tokens():
    import combine_grouped_gemm_amd as m
    layer, lg, w, grads = _layer(m)
    dout = torch.full((9, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    dout[:6] = torch.randn(6, 64, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    seen = []
    for d in (dout[:6].contiguous(), dout):
        dx, dlogits = layer.backward(d, lg, w, grads)
        seen.append([t.clone() for t in (dx, dlogits, layer.dtopk_w, *grads.values())])
    for a, b in zip(*seen):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)


def test_dout_that_is_no_tensor():
    import combine_grouped_gemm_amd as m
    layer, lg, w, grads = _layer(m)
    with pytest.raises(TypeError, match="dout must be a torch.Tensor"):
        layer.backward([[0.0] * 64] * 6, lg, w, grads)
