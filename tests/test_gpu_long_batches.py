"""Batches whose grid, at 64 threads a token, has 2^32 threads or more: such a
grid is cut without an error, so they take several launches.  A block of 64
tokens is repeated; every repetition has to come out like the first."""
import numpy as np
import pytest
import torch

import oracle
from harness import has_gpu, to_np

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

REPS = 2**20 + 2
B = 64 * REPS                    # 2^26 + 128 tokens


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _same_everywhere(got, want):
    """got (B, n): 64 rows repeated."""
    return bool((got.view(REPS, 64, -1) == want.cuda()[None]).all())


@pytest.mark.parametrize("kind", ["plain", "mapped", "shared"])
def test_route(kind):
    import combine_grouped_gemm_amd as m
    E, K, shared = 4, 2, 1 if kind == "shared" else 0
    few = torch.randn(64, E, generator=_gen(1))
    lg = few.cuda().repeat(REPS, 1)
    ids = torch.full((B, K + shared), -7, dtype=torch.int32, device="cuda")
    w = torch.full((B, K + shared), -7.0, device="cuda")
    perm = torch.tensor([2, 0, 3, 1], dtype=torch.int32)
    call = {"plain": lambda x, i, g: m.moe_route(x, K, i, g),
            "mapped": lambda x, i, g: m.moe_route_mapped(x, K, perm.cuda(), i, g),
            "shared": lambda x, i, g: m.moe_route_shared(x, K, shared, i, g)}[kind]
    call(lg, ids, w)
    ri, rw = oracle.route_shared(few.numpy(), K, shared) if shared else oracle.route(few.numpy(), K)
    ri = torch.from_numpy(ri)
    assert _same_everywhere(ids, perm[ri.long()] if kind == "mapped" else ri)
    one, gates = torch.empty(64, K + shared, dtype=torch.int32, device="cuda"), torch.empty(64, K + shared, device="cuda")
    call(few.cuda(), one, gates)
    # fp32 gates: expf, a sum of K and a division, a few steps of 2^-24 each
    assert float((gates.cpu().double() - torch.from_numpy(rw)).abs().max()) < 2.0**-20
    assert _same_everywhere(w, gates)


@pytest.mark.parametrize("xdt,dt,H", [(torch.bfloat16, "bf16", 8), (torch.float32, "f32", 8), (torch.bfloat16, "fp8", 16)])
def test_dispatch(xdt, dt, H):
    """Two segments that meet inside a launch's share of the tokens; rows in reverse."""
    import combine_grouped_gemm_amd as m
    few = torch.randn(64, H, generator=_gen(2)).to(xdt)
    x = few.cuda().repeat(REPS, 1)
    cut = 2**22 + 5
    rows = torch.arange(B - 1, -1, -1, dtype=torch.int32, device="cuda").view(B, 1)
    xd, sc = m.moe_dispatch([x[:cut], x[cut:]], rows, B, dt)
    rx, rs = oracle.dispatch(to_np(few), np.arange(63, -1, -1, dtype=np.int32)[:, None], 64, dt)
    got = (xd[:64].float() if dt == "fp8" else xd[:64]).double().cpu().numpy()
    np.testing.assert_array_equal(got, rx)
    same = xd.view(torch.uint8) if dt == "fp8" else xd
    assert _same_everywhere(same, same[:64])
    if dt == "fp8":
        np.testing.assert_array_equal(sc[:64].cpu().numpy(), rs)
        assert _same_everywhere(sc, sc[:64])


@pytest.mark.parametrize("ydt,odt,K", [(torch.bfloat16, torch.bfloat16, 2), (torch.float32, torch.float32, 2),
                                       (torch.bfloat16, torch.float32, 3)])
def test_combine(ydt, odt, K):
    import combine_grouped_gemm_amd as m
    g = _gen(3)
    H, R = 8, 50
    y = torch.randn(R, H, generator=g).to(ydt)
    rows = torch.randint(-1, R, (64, K), generator=g, dtype=torch.int32)
    w = torch.rand(64, K, generator=g)
    out = torch.full((B, H), -7.0, dtype=odt, device="cuda")
    m.moe_combine(y.cuda(), rows.cuda().repeat(REPS, 1), w.cuda().repeat(REPS, 1), out)
    picked = torch.where((rows >= 0)[..., None], y.double()[rows.clamp(min=0).long()], 0.0)
    ref = (picked * w.double()[..., None]).sum(1)
    # fp32 fused multiply-adds of K terms, each off by half a step of a partial sum of at most sum |w y|
    bar = K * 2.0**-24 * (picked * w.double()[..., None]).abs().sum(1)
    if odt == torch.bfloat16:
        bar += 2.0**-8 * (ref.abs() + bar)
    assert bool(((out[:64].cpu().double() - ref).abs() <= bar).all())
    assert _same_everywhere(out, out[:64])


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T", [3, 3000])
def test_layout_of_a_buffer_of_two_to_the_31_rows(T, masked):
    """One launch and three; the padding of the last rows, whose number plus the grid's
    step passes 2^31."""
    import combine_grouped_gemm_amd as m
    cap, E, K = 2**31 - 1, 4, 2
    ids = torch.rand(T, E, generator=_gen(4)).topk(K, 1).indices.to(torch.int32)
    src = torch.full((cap,), 5, dtype=torch.int32, device="cuda")
    if masked:                                             # the second expert's block is the whole buffer
        ref = oracle.layout_masked(ids.numpy(), E, 1, 2, 4 * T)
        lay = m.moe_layout_masked(ids.cuda(), E, 1, 2, cap, src_of=src)
        n = int(ref["m"][0])
        assert lay["m"].tolist() == [n]
    else:
        ref = oracle.layout(ids.numpy(), E, 0, E, T * K)
        lay = m.moe_layout(ids.cuda(), E, 0, E, cap, src_of=src)
        n = T * K
        np.testing.assert_array_equal(lay["offsets"].cpu().numpy(), ref["offsets"])
    np.testing.assert_array_equal(lay["row_of"].cpu().numpy(), ref["row_of"])
    np.testing.assert_array_equal(src[:n].cpu().numpy(), ref["src_of"][:n])
    assert bool((src[n:] == -1).all())
