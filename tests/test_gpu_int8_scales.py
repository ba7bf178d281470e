"""int8 products whose scales are far apart: a result that fp32 can hold is
reached although acc * scale of one operand alone would overflow, on either
side, in both tile shapes.

Tolerances: the int32 sum's conversion and the two scalings round by 2^-24
each, taken as 4 * 2^-24; below the smallest normal number a rounding is half
of 2^-149 (two of them).  h = silu(g) u with |g| < 30: less than 250 * 2^-24 <
2^-16 before bf16's 2^-8 (an error d of g changes silu by at most (1 + |g|) d)."""
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

Y_TOL = {torch.float32: 4 * 2.0**-24, torch.bfloat16: 2.0**-8 + 2.0**-21}
H_TOL = 2.0**-8 + 2.0**-16
SMALL, LARGE = 1, 10**6          # expected rows that take the 64 x 128 and the 256 x 256 tiles
E, K, N = 3, 128, 192
COUNTS = [5, 0, 70]


def _problem(n_weights=1, seed=1):
    g = torch.Generator().manual_seed(seed)
    R = sum(COUNTS)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, dtype=torch.int8).cuda()
    off = torch.tensor([0, *torch.tensor(COUNTS).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    return codes(R, K), [codes(E, N, K) for _ in range(n_weights)], off


def _sums(a, w, off):
    out = torch.zeros((a.shape[0], N), dtype=torch.float64)
    o = off.tolist()
    for j in range(E):
        out[o[j]:o[j + 1]] = a[o[j]:o[j + 1]].cpu().double() @ w[j].cpu().double().t()
    return out


def _scaled(acc, rs, cs, off):
    """acc * row scale * channel scale in 64 bits."""
    per_row = cs.cpu().double().repeat_interleave(torch.tensor(COUNTS), 0)
    return acc * rs.cpu().double()[:, None] * per_row


def _near(got, ref, tol, least=0.0):
    got = got.cpu().double()
    top = torch.finfo(torch.float32).max
    inf = ref.abs() > top
    assert not torch.isnan(got[~torch.isnan(ref)]).any(), "NaN where the formula has a number"
    assert torch.equal(torch.isinf(got), inf), "infinite in other places"
    assert torch.equal(got[inf].sign(), ref[inf].sign())
    assert bool(((got - ref).abs() <= tol * ref.abs() + least)[~inf].all())


# row scale, channel scale: results about 1e37, 1, or subnormal
SCALES = [(2e36, 1e-4), (1e-4, 2e36), (2.6e36, 2.0**-140), (2.0**-140, 2.6e36), (2.0**-126, 1e38), (1e38, 2.0**-126),
          (2.0**-126, 2.0**-12), (2.0**-12, 2.0**-126), (3e38, 1e-30), (1e-30, 3e38), (1e-3, 1e-3)]


@pytest.mark.parametrize("hint", [SMALL, LARGE])
@pytest.mark.parametrize("row,channel", SCALES)
def test_finite_products_stay_finite(row, channel, hint):
    import combine_grouped_gemm_amd as m
    print(f"[scales] row={row} channel={channel} hint={hint}", flush=True)
    a, (w,), off = _problem()
    g = torch.Generator().manual_seed(2)
    rs = (row * (0.25 + 0.75 * torch.rand(a.shape[0], generator=g))).to(torch.float32).cuda()
    cs = (channel * (0.25 + 0.75 * torch.rand((E, N), generator=g))).to(torch.float32).cuda()
    ref = _scaled(_sums(a, w, off), rs, cs, off)
    # the sums reach past 170, so the larger scale alone overflows; the results do not
    assert ref.abs().max() < 3e38
    for dt in (torch.float32, torch.bfloat16):
        y = m.moe_ffn_down(a, rs, off, w, cs, y_dtype=dt, expected_rows=hint)
        # a bf16 output is rounded once more below the smallest normal number: half of 2^-133
        _near(y, ref, Y_TOL[dt], 2.0**-149 + (2.0**-134 if dt == torch.bfloat16 else 0.0))


@pytest.mark.parametrize("hint", [SMALL, LARGE])
def test_gate_and_up_stay_finite(hint):
    """g and u of a few units from row scales near fp32's end, whose product with the
    sum alone is infinite (and silu of -inf times anything was NaN)."""
    import combine_grouped_gemm_amd as m
    a, (wg, wu), off = _problem(2, 3)
    g = torch.Generator().manual_seed(4)
    rs = (2e36 * (0.5 + torch.rand(a.shape[0], generator=g))).cuda()
    cs = [(4e-41 * (0.5 + torch.rand((E, N), generator=g))).cuda() for _ in range(2)]
    gate, up = (_scaled(_sums(a, w, off), rs, c, off) for w, c in ((wg, cs[0]), (wu, cs[1])))
    gate_only = gate.abs() < 30
    ref = gate / (1 + torch.exp(-gate)) * up
    h, _ = m.moe_ffn_gate_up(a, rs, off, wg, wu, *cs, expected_rows=hint)
    got = h.cpu().double()
    assert not torch.isnan(got).any()
    assert bool(((got - ref).abs() <= H_TOL * ref.abs() + 2.0**-133)[gate_only].all()) and gate_only.float().mean() > 0.9


@pytest.mark.parametrize("hint", [SMALL, LARGE])
def test_gate_past_fp32_has_silus_limit(hint):
    """g below fp32's range: silu's limit is zero, not -inf * 0; above it: infinite."""
    import combine_grouped_gemm_amd as m
    a, (wg, wu), off = _problem(2, 5)
    R = a.shape[0]
    rs = torch.full((R,), 1e36, device="cuda")
    gate, up = _sums(a, wg, off) * 1e36 * 1e3, _sums(a, wu, off)
    h, _ = m.moe_ffn_gate_up(a, rs, off, wg, wu, torch.full((E, N), 1e3, device="cuda"),
                             torch.full((E, N), 1e-40, device="cuda"), expected_rows=hint)
    got = h.cpu().double()
    low, high = gate < -3.5e38, (gate > 3.5e38) & (up != 0)
    assert low.any() and high.any()
    assert (got[low] == 0).all()
    assert torch.isinf(got[high]).all() and torch.equal(got[high].sign(), up[high].sign())


@pytest.mark.parametrize("hint", [SMALL, LARGE])
def test_nan_scales_reach_their_row_and_channel_only(hint):
    import combine_grouped_gemm_amd as m
    nan = float("nan")
    a, (w,), off = _problem(1, 6)
    rs, cs = torch.full((a.shape[0],), 2e36, device="cuda"), torch.full((E, N), 1e-4, device="cuda")
    rs[7], cs[2, 11] = nan, nan
    y = m.moe_ffn_down(a, rs, off, w, cs, y_dtype=torch.float32, expected_rows=hint).cpu()
    want = torch.zeros(y.shape, dtype=torch.bool)
    want[7] = True
    want[COUNTS[0] + COUNTS[1]:, 11] = True
    assert torch.equal(torch.isnan(y), want)
    h, _ = m.moe_ffn_gate_up(a, rs, off, w, w, cs, cs, expected_rows=hint)
    assert torch.isnan(h.cpu()[want]).all()


def test_loud_rows_through_the_chain():
    """Rows of 3e38 through dispatch's quantisation and the product: finite outputs stay
    finite, as the formula's."""
    import combine_grouped_gemm_amd as m
    g = torch.Generator().manual_seed(7)
    T, H = 9, 256
    x = (torch.rand((T, H), generator=g) * 2 - 1) * 3e38
    rows = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    xd, xs = m.moe_dispatch(x.cuda(), rows, T, "int8")
    w = torch.randn((N, H), generator=g) * 1e-5
    wq, ws = m.moe_quant_rows(w.cuda())
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    y = m.moe_ffn_down(xd, xs, off, wq.view(1, N, H), ws.view(1, N), y_dtype=torch.float32)
    ref = (xd.cpu().double() @ wq.cpu().double().t()) * xs.cpu().double()[:, None] * ws.cpu().double()
    _near(y, ref, Y_TOL[torch.float32])
