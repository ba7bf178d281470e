"""Buffers of no rows, which have no address: every storage type, through the
binding (an empty tensor's pointer is null), with row descriptions that claim
rows all the same."""
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

E, H, I, T, K = 3, 64, 32, 5, 2
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


def _z(*s, dt=torch.float32):
    return torch.zeros(s, dtype=torch.uint8, device="cuda").view(dt) if dt == torch.float8_e4m3fn else torch.zeros(
        s, dtype=dt, device="cuda")


def _scales(act, *s):
    """Scales of an (..., cols) tensor of this type, None where it has none."""
    if act == "fp8":
        return _z(*s[:-1], -(-s[-1] // 128))
    return _z(*s[:-1]) if act == "int8" else None


@pytest.mark.parametrize("hint", [0, 10**6])
@pytest.mark.parametrize("counts", [(0, 0, 0), (4, 0, 2)])
@pytest.mark.parametrize("act", list(DT))
def test_ffn_of_no_rows(act, counts, hint):
    import combine_grouped_gemm_amd as m
    dt = DT[act]
    off = torch.tensor([0, counts[0], counts[0] + counts[1], sum(counts)], dtype=torch.int32, device="cuda")
    wg, wd = _z(E, I, H, dt=dt), _z(E, H, I, dt=dt)
    sg, sd = _scales(act, E, I, H), _scales(act, E, H, I)
    xd, xs = _z(0, H, dt=dt), _scales(act, 0, H)
    assert xd.data_ptr() == 0
    h, hs = m.moe_ffn_gate_up(xd, xs, off, wg, wg, sg, sg, expected_rows=hint)
    assert h.shape == (0, I) and (hs is None) == (act != "fp8")
    hd, hds = _z(0, I, dt=dt), _scales(act, 0, I)
    y = m.moe_ffn_down(hd, hds, off, wd, sd, expected_rows=hint)
    assert y.shape == (0, H)
    y = m.moe_grouped_ffn(xd, xs, off, wg, wg, wd, sg, sg, sd, expected_rows=hint)
    torch.cuda.synchronize()
    assert y.shape == (0, H)


@pytest.mark.parametrize("act", list(DT))
def test_layer_calls_of_a_buffer_without_rows(act):
    """A rank whose buffer holds nothing: every slot is dropped, the partial sum is zero."""
    import combine_grouped_gemm_amd as m
    x = _z(T, H, dt=torch.float32 if act == "f32" else torch.bfloat16) + 1
    ids = torch.tensor([[0, 1], [2, 0], [1, 2], [0, 2], [1, 0]], dtype=torch.int32, device="cuda")
    lay = m.moe_layout(ids, E, 0, E, 0)
    assert lay["offsets"].tolist() == [0, 4, 7, 10] and bool((lay["row_of"] == -1).all())
    xd, xs = m.moe_dispatch(x, lay["row_of"], 0, act, xd=_z(0, H, dt=DT[act]), xd_scales=_scales(act, 0, H))
    for ydt, odt in (((torch.float32, torch.float32),) if act == "f32" else
                     ((torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32))):
        out = torch.full((T, H), 7.0, dtype=odt, device="cuda")
        m.moe_combine(_z(0, H, dt=ydt), lay["row_of"], torch.ones(T, K, device="cuda"), out)
        # a row number all the same
        out2 = torch.full((T, H), 7.0, dtype=odt, device="cuda")
        m.moe_combine(_z(0, H, dt=ydt), lay["row_of"] + 1, torch.ones(T, K, device="cuda"), out2)
        assert (out == 0).all() and (out2 == 0).all()
