"""Calls on a stream other than the current one: what they make themselves is
theirs until they end."""
import pytest
import torch

import oracle
from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]


def _busy():
    """A few milliseconds of work on the current stream."""
    big = torch.full((2048, 2048), 2.0**-6, device="cuda")
    for _ in range(8):
        big = big @ big
    return big


@pytest.mark.parametrize("masked", [False, True])
def test_layout_on_a_side_stream(masked):
    """Workspace (three kernels use it in turn) and outputs made by the call, while the
    current stream frees memory that it still writes and allocates what the call's
    workspace would leave."""
    import combine_grouped_gemm_amd as m
    T, K, E, cap = 4000, 8, 64, 600
    ids = torch.rand(T, E, generator=torch.Generator().manual_seed(1)).topk(K, 1).indices.to(torch.int32)
    ref = oracle.layout_masked(ids.numpy(), E, 0, E, cap) if masked else oracle.layout(ids.numpy(), E, 0, E, T * K)
    dev = ids.cuda()
    side = torch.cuda.Stream()
    need = m.moe_layout_workspace_bytes(T, K, E)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        for _ in range(3):
            junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (need, T * K * 4, E * 4, 4 * (E + 1))]
            keep = _busy()
            for t in junk:
                t.fill_(1)                                 # runs late, on the current stream
            del junk, t
            if masked:
                lay = m.moe_layout_masked(dev, E, 0, E, cap, stream=stream)
            else:
                lay = m.moe_layout(dev, E, 0, E, T * K, stream=stream)
            after = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            for k in ("counts", "row_of", "src_of", "m" if masked else "offsets"):
                assert torch.equal(lay[k].cpu(), torch.from_numpy(ref[k]).to(torch.int32)), k
            del after, keep


def test_layer_calls_on_a_side_stream():
    """route to combine with every output made by the calls, on a side stream."""
    import combine_grouped_gemm_amd as m
    T, E, K, H, I = 512, 16, 4, 256, 128
    g = torch.Generator().manual_seed(2)
    lg = torch.randn(T, E, generator=g).cuda()
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    w = [(torch.randn(E, *s, generator=g) / s[1]**0.5).to(torch.bfloat16).cuda() for s in ((I, H), (I, H), (H, I))]

    def chain(stream):
        ids, gates = m.moe_route(lg, K, stream=stream)
        lay = m.moe_layout(ids, E, 0, E, T * K, stream=stream)
        xd, _ = m.moe_dispatch(x, lay["row_of"], T * K, stream=stream)
        wp = [m.moe_pack_weights(t, stream=stream) for t in w]
        h, _ = m.moe_ffn_gate_up(xd, None, lay["offsets"], wp[0], wp[1], stream=stream)
        y = m.moe_ffn_down(h, None, lay["offsets"], wp[2], stream=stream)
        return m.moe_combine(y, lay["row_of"], gates, stream=stream)

    ref = chain(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        keep = _busy()
        junk = torch.empty(T * K * H, dtype=torch.bfloat16, device="cuda").fill_(1)
        del junk
        out = chain(side)
        side.synchronize()
        early = out.cpu()
        torch.cuda.synchronize()
        assert torch.equal(early, ref.cpu()) and torch.equal(out, ref)
        del keep
