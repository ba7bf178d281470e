"""Which stream and device the binding's calls use, on the CPU: the library is
replaced by a recorder and no kernel runs."""
import pytest
import torch

import combine_grouped_gemm_amd as m

HOST_QUERIES = ("moe_layout_workspace_bytes", "moe_ffn_workspace_bytes", "moe_weight_ld", "moe_packed_weight_bytes")


class Recorder:
    """Stands for the loaded library: host queries answer, launches are written down."""

    def __init__(self, real):
        self.real, self.launched = real, []

    def __getattr__(self, name):
        if name in HOST_QUERIES:
            return getattr(self.real, name)
        return lambda *args: self.launched.append((name, args)) or 0


i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
f32 = lambda *s: torch.zeros(s)
bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
i8 = lambda *s: torch.zeros(s, dtype=torch.int8)
fp8 = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn)

# call, tensors it makes itself
CALLS = {
    "moe_route": (lambda **k: m.moe_route(f32(4, 8), 2, **k), 2),
    "moe_route_mapped": (lambda **k: m.moe_route_mapped(f32(4, 8), 2, i32(8), **k), 2),
    "moe_route_shared": (lambda **k: m.moe_route_shared(f32(4, 8), 2, 1, **k), 2),
    "moe_route_scored": (lambda **k: m.moe_route_scored(f32(4, 8), 2, **k), 2),
    "moe_layout": (lambda **k: m.moe_layout(i32(4, 2), 8, 0, 8, 8, **k), 5),
    "moe_layout_noalloc": (lambda **k: m.moe_layout_noalloc(i32(4, 2), 8, 0, 8, 8, **k), 4),
    "moe_layout_masked": (lambda **k: m.moe_layout_masked(i32(4, 2), 8, 0, 8, 3, **k), 5),
    "moe_dispatch bf16": (lambda **k: m.moe_dispatch(bf(4, 16), i32(4, 2), 8, **k), 1),
    "moe_dispatch fp8": (lambda **k: m.moe_dispatch(bf(4, 16), i32(4, 2), 8, "fp8", **k), 2),
    "moe_dispatch int8": (lambda **k: m.moe_dispatch(bf(4, 16), i32(4, 2), 8, "int8", **k), 2),
    "moe_quant_rows": (lambda **k: m.moe_quant_rows(bf(4, 16), **k), 2),
    "moe_quant_rows_masked": (lambda **k: m.moe_quant_rows_masked(bf(4, 16), i32(2), 2, **k), 2),
    "moe_pack_weights": (lambda **k: m.moe_pack_weights(bf(2, 16, 24), **k), 1),
    "moe_ffn_gate_up": (lambda **k: m.moe_ffn_gate_up(bf(4, 16), None, i32(3), bf(2, 24, 16), bf(2, 24, 16), **k), 1),
    "moe_ffn_gate_up fp8": (lambda **k: m.moe_ffn_gate_up(fp8(4, 16), f32(4, 1), i32(3), fp8(2, 16, 16), fp8(2, 16, 16),
                                                          f32(2, 16, 1), f32(2, 16, 1), **k), 2),
    "moe_ffn_gate_up int8": (lambda **k: m.moe_ffn_gate_up(i8(4, 16), f32(4), i32(3), i8(2, 16, 16), i8(2, 16, 16),
                                                           f32(2, 16), f32(2, 16), **k), 1),
    "moe_ffn_down": (lambda **k: m.moe_ffn_down(bf(4, 24), None, i32(3), bf(2, 16, 24), **k), 1),
    "moe_ffn_down_masked": (lambda **k: m.moe_ffn_down_masked(bf(4, 24), None, i32(2), 2, bf(2, 16, 24), **k), 1),
    "moe_grouped_ffn": (lambda **k: m.moe_grouped_ffn(bf(4, 16), None, i32(3), bf(2, 24, 16), bf(2, 24, 16),
                                                      bf(2, 16, 24), **k), 2),
    "moe_combine": (lambda **k: m.moe_combine(bf(8, 16), i32(4, 2), f32(4, 2), **k), 1),
}


@pytest.fixture
def recorder(monkeypatch):
    r = Recorder(m.lib())
    monkeypatch.setattr(m, "lib", lambda: r)
    monkeypatch.setattr(m, "_dev", lambda t, *a, **k: t)       # host tensors stand for device ones
    monkeypatch.setattr(m, "_stream", lambda stream: stream)
    return r


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_makes_belongs_to_the_stream_it_is_given(recorder, monkeypatch, name):
    """Outputs and workspaces: allocated for another stream, their memory may be in use
    there, and a workspace freed on return goes to that stream while the call runs."""
    call, made = CALLS[name]
    empty, got = torch.empty, []

    def new(shape, dtype, device, stream):
        got.append(stream)
        return empty(shape, dtype=dtype, device=device)

    monkeypatch.setattr(m, "_new", new)
    monkeypatch.setattr(m, "_call", lambda fn, t, stream, *args: fn(*args, stream))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: pytest.fail("allocated on the current stream"))
    for stream in (77, None):
        del got[:], recorder.launched[:]
        call(stream=stream)
        assert got == [stream] * made
        assert [args[-1] for _, args in recorder.launched] == [stream]
