"""Which stream and device the binding's calls use, on the CPU: the library is
replaced by a recorder and no kernel runs."""
import pytest
import torch

import combine_grouped_gemm_amd as m

HOST_QUERIES = ("moe_layout_workspace_bytes", "moe_ffn_workspace_bytes", "moe_weight_ld", "moe_packed_weight_bytes")


class Recorder:
    """Stands for the loaded library: host queries answer, launches are written down."""

    def __init__(self, real):
        self.real, self.launched, self.on_launch = real, [], lambda: None

    def __getattr__(self, name):
        if name in HOST_QUERIES:
            return getattr(self.real, name)
        return lambda *args: self.launch(name, args)

    def launch(self, name, args):
        self.launched.append((name, args))
        self.on_launch()
        return m.MOE_OK


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

    def new(shape, dtype, device, stream, scratch=False):
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


class Devices:
    """Two devices, the first one current; every tensor says it is on `where`."""

    def __init__(self, monkeypatch, where):
        self.current = 0
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: where())
        monkeypatch.setattr(m, "_current_device", lambda: self.current)
        monkeypatch.setattr(m, "_raw_stream", lambda index: 1000 + index)
        devices = self

        class device:
            def __init__(self, index):
                self.index = index

            def __enter__(self):
                self.before, devices.current = devices.current, self.index

            def __exit__(self, *exc):
                devices.current = self.before

        monkeypatch.setattr(torch.cuda, "device", device)


@pytest.fixture
def on_host(monkeypatch):
    r = Recorder(m.lib())
    monkeypatch.setattr(m, "lib", lambda: r)
    monkeypatch.setattr(m, "_dev", lambda t, *a, **k: t)
    return r


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_device_is_current_during_a_call(on_host, monkeypatch, name):
    """Launches go to the tensors' device, on that device's current stream."""
    d = Devices(monkeypatch, lambda: 1)
    during = []
    on_host.on_launch = lambda: during.append(d.current)
    CALLS[name][0]()
    assert during == [1] and d.current == 0
    assert [args[-1] for _, args in on_host.launched] == [1001]
    # the current device needs no switch
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda index: pytest.fail("device switched"))
    CALLS[name][0]()
    assert during == [1, 0] and on_host.launched[1][1][-1] == 1000


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_two_devices_are_refused(on_host, monkeypatch, name):
    """A kernel would read the other device's memory, or fault on it."""
    seen = []
    Devices(monkeypatch, lambda: seen.append(0) or min(len(seen) - 1, 1))
    with pytest.raises(ValueError, match="all tensors must be on"):
        CALLS[name][0]()
    assert not on_host.launched


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(on_host, monkeypatch, name):
    class Stream:
        def __init__(self, index):
            self.device_index, self.cuda_stream = index, 500 + index

    Devices(monkeypatch, lambda: 1)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(m, "_new", lambda shape, dtype, *a, **k: torch.empty(shape, dtype=dtype))
    CALLS[name][0](stream=Stream(1))
    assert [args[-1] for _, args in on_host.launched] == [501]
    with pytest.raises(ValueError, match="stream must be"):
        CALLS[name][0](stream=Stream(0))
    assert len(on_host.launched) == 1
