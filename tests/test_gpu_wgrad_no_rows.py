"""Weight gradients of a pair without rows: both are written, with zeros or their bases."""
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("base", [None, "apart", "in place"])
@pytest.mark.parametrize("gather,rows,tokens", [(None, 0, 0), ("x", 0, 5), ("x", 7, 0), ("dy", 7, 0), ("dy", 0, 5)])
def test_pair_of_no_rows(gather, rows, tokens, base, ckpt, dtype):
    import combine_grouped_gemm_amd as m
    E, N, M = 3, 72, 136
    gen = torch.Generator(device="cuda").manual_seed(1)
    ny, nx = (tokens if gather == "dy" else rows), (tokens if gather == "x" else rows)
    dy = torch.ones(ny, N, dtype=dtype, device="cuda")
    x = torch.ones(nx, M, device="cuda").to(torch.int8 if ckpt else dtype)
    xs = torch.ones(nx, 2, device="cuda") if ckpt else None
    src = torch.arange(max(rows, 1), dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 2, 9], dtype=torch.int32, device="cuda")
    bases = [torch.randn(E, N, M, generator=gen, device="cuda") if base else None for _ in range(2)]
    want = [torch.zeros(E, N, M, device="cuda") if b is None else b.clone() for b in bases]
    dws = bases if base == "in place" else [torch.full((E, N, M), float("nan"), device="cuda") for _ in range(2)]
    m.moe_ffn_wgrad(dy, x, off, x_scales=xs, dy2=dy.clone(), src_of=src if gather else None, slots_per_token=1,
                    gather=gather, base=bases[0], base2=bases[1], dw=dws[0], dw2=dws[1])
    for got, ref in zip(dws, want):
        assert torch.equal(got, ref)
