"""A training layer whose buffer holds no rows: every slot is dropped, so no gradient
comes from what the buffers held before."""
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_capacity(dtype):
    import combine_grouped_gemm_amd as m
    T, E, K, H, I = 6, 4, 2, 64, 72
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    layer = m.MoELayer([T], E, K, H, I, 0, E, dtype, dtype, dtype, cap_rows=0, train=True)
    for name in ("xd", "h", "dh", "dgate", "dup", "hw", "dxd", "gate_q", "up_q", "gate_s", "up_s"):
        getattr(layer, name).fill_(1)
    layer.src_of.zero_()
    x, lg, dout = (torch.ones(T, n, device="cuda") for n in (H, E, H))
    w = {k: torch.ones(E, *s, dtype=dt, device="cuda") for k, s in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I)))}
    out = layer.forward([x.to(dt)], lg, w)
    assert layer.offsets.tolist() == [0, 6, 12, 12, 12] and not bool(out.any())
    grads = layer.new_grads()
    for g in grads.values():
        g.fill_(float("nan"))
    dx, dlogits = layer.backward(dout.to(dt), lg, w, grads)
    assert not bool(dx.any()) and not bool(dlogits.any()) and not bool(layer.dtopk_w.any())
    assert all(not bool(g.any()) for g in grads.values())
    for g in grads.values():
        g.fill_(3.0)
    layer.backward(dout.to(dt), lg, w, grads, accumulate=True)
    assert all(bool((g == 3.0).all()) for g in grads.values())
