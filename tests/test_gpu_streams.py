"""Calls on a stream other than the current one: what they make themselves is
theirs until they end."""
import pytest
import torch

import oracle
from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]


def _busy(products=8):
    """Milliseconds of work on the current stream."""
    big = torch.full((2048, 2048), 2.0**-6, device="cuda")
    for _ in range(products):
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


@pytest.mark.parametrize("raw", [False, True])
def test_a_dropped_output_is_not_reused_while_the_current_stream_reads_it(raw):
    """The output of a call on a side stream belongs to that stream; the current stream
    waits for it, reads it late and drops it.  The side stream's next call waits for
    nothing, so it has to get other memory."""
    import combine_grouped_gemm_amd as m
    rows, cols = 3000, 512
    x = [torch.full((rows, cols), v, dtype=torch.bfloat16, device="cuda") for v in (1.0, -1.0)]
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    torch.cuda.synchronize()
    for _ in range(4):
        q, s = m.moe_quant_rows(x[0], stream=stream)
        side.synchronize()
        keep = _busy()
        read = q.clone()                                   # late, on the current stream
        at = q.data_ptr()
        del q, s
        again, _ = m.moe_quant_rows(x[1], stream=stream)
        assert again.data_ptr() != at
        torch.cuda.synchronize()
        assert bool((read == 127).all()) and bool((again == -127).all())
        del keep, read, again, _


def test_workspaces_of_a_side_stream_are_reused_while_the_current_stream_is_busy():
    """The current stream never reads a workspace, so it does not hold one up."""
    import combine_grouped_gemm_amd as m
    T, K, E = 20000, 8, 1024
    ids = torch.rand(T, E, generator=torch.Generator().manual_seed(1)).topk(K, 1).indices.to(torch.int32).cuda()
    out = m.moe_layout(ids, E, 0, E, T * K)
    side = torch.cuda.Stream()
    _busy(2)
    m.moe_layout(ids, E, 0, E, T * K, **out, stream=side)
    torch.cuda.synchronize()
    before, need = torch.cuda.memory_reserved(), m.moe_layout_workspace_bytes(T, K, E)
    keep = _busy(200)
    for _ in range(100):
        m.moe_layout(ids, E, 0, E, T * K, **out, stream=side)
    assert torch.cuda.memory_reserved() - before < 50 * need
    torch.cuda.synchronize()
    del keep


def test_a_captured_graph_with_a_forked_stream():
    """Outputs made inside a capture, on a stream that forks from it, and dropped there."""
    import combine_grouped_gemm_amd as m
    x = torch.randn(700, 256, device="cuda")
    main, side, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    m.moe_quant_rows(x)
    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        q, s = m.moe_quant_rows(x, stream=side)
        main.wait_stream(side)
        a = q.to(torch.float32) * s[:, None]
        del q, s
        side.wait_stream(main)
        q, s = m.moe_quant_rows(a, stream=side)
        main.wait_stream(side)
        b = q.to(torch.float32) * s[:, None]
        del q, s
    for _ in range(4):
        x.copy_(torch.randn(700, 256, device="cuda"))
        a.zero_()
        b.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        q, s = m.moe_quant_rows(x)
        want = q.to(torch.float32) * s[:, None]
        q, s = m.moe_quant_rows(want)
        assert torch.equal(a, want) and torch.equal(b, q.to(torch.float32) * s[:, None])


def test_streams_given_by_number():
    """The null stream and another one by their handles, from inside either."""
    import combine_grouped_gemm_amd as m
    lg = torch.randn(50, 16, device="cuda")
    want = m.moe_route(lg, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (0, side.cuda_stream, side, torch.cuda.default_stream()):
        for inside in (torch.cuda.default_stream(), side):
            with torch.cuda.stream(inside):
                got = m.moe_route(lg, 2, stream=stream)
                lay = m.moe_layout(got[0], 16, 0, 16, 100, stream=stream)
                assert torch.cuda.current_stream() == inside
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert int(lay["offsets"][-1]) == 100
