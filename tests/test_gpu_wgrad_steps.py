"""bf16 weight gradients of experts with many rows: several 64-row steps a tile, more rows than
are listed at a time (1024), in every kernel variant (256 x 256 tiles, 128 x 128 tiles, 64-bit
addresses), with rows that name no token in any of their steps.

Tolerance, per element: a sum of n products in fp32, in whatever order, is off by at most
(n + 1) 2^-23 of the products' magnitudes (a base counts as one); rounding the result adds
half a step."""
import numpy as np
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

HALF = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(n, cols, seed):
    return torch.randn(n, cols, generator=_gen(seed), device="cuda").bfloat16()


def _codes(n, cols, seed):
    q = torch.randint(-127, 128, (n, cols), generator=_gen(seed), device="cuda").to(torch.int8)
    return q, torch.exp2(torch.randint(-8, -4, (n, -(-cols // 128)), generator=_gen(seed + 1), device="cuda").float())


def _values(x, xs, rows):
    """The rows of x (checkpoint: decoded) in 64 bits."""
    v = x[rows].double()
    return v if xs is None else v * xs[rows].double().repeat_interleave(128, dim=1)[:, :x.shape[1]]


def _check(counts, N, M, two, gather, ckpt, base, dw_dtype, holes=(), T=500, seed=0):
    import combine_grouped_gemm_amd as m
    E, R, K = len(counts), sum(counts), 3
    cap = R + 7
    src = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    src[:R] = torch.randint(0, T * K, (R,), generator=_gen(seed), device="cuda").to(torch.int32)
    at = torch.tensor(sorted(h for h in holes if h < R), dtype=torch.long, device="cuda")
    src[at] = torch.tensor([(-1, T * K, 2**31 - 1)[i % 3] for i in range(len(at))], dtype=torch.int32, device="cuda")
    dys = [_rows(T if gather == "dy" else cap, N, seed + 1 + i) for i in range(1 + two)]
    xr = T if gather == "x" else cap
    x, xs = _codes(xr, M, seed + 5) if ckpt else (_rows(xr, M, seed + 5), None)
    # rows behind the last expert's, and those of the other operand that name no token, hold NaN
    lost = torch.arange(R, cap, device="cuda") if gather is None else torch.cat([torch.arange(R, cap, device="cuda"), at])
    if gather != "dy":
        for dy in dys:
            dy[lost] = float("nan")
    if gather != "x":
        (xs if ckpt else x)[lost] = float("nan")
    off = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
    bases = [torch.randn(E, N, M, generator=_gen(seed + 8 + i), device="cuda").to(dw_dtype) if base else None
             for i in range(1 + two)]
    dws = [b.clone() if base == "in place" else torch.full((E, N, M), float("nan"), dtype=dw_dtype, device="cuda")
           for b in bases]
    given = dws if base == "in place" else bases
    kw = dict(zip(("base", "base2"), given))
    kw.update(dict(zip(("dw", "dw2"), dws)))
    m.moe_ffn_wgrad(dys[0], x, off, x_scales=xs, dy2=dys[1] if two else None, src_of=src if gather else None,
                    slots_per_token=K, gather=gather, **kw)
    first = 0
    for j, n in enumerate(counts):
        r = torch.arange(first, first + n, device="cuda")
        first += n
        if gather:
            r = r[(src[r] >= 0) & (src[r] // K < T)]
        tok = src[r].long() // K
        xv = _values(x, xs, tok if gather == "x" else r)
        for dy, dw, b in zip(dys, dws, bases):
            d = dy[tok if gather == "dy" else r].double()
            ref, mag = d.t() @ xv, d.abs().t() @ xv.abs()
            if b is not None:
                ref, mag = ref + b[j].double(), mag + b[j].double().abs()
            room = HALF[dw_dtype] * ref.abs() + (n + 1) * 2.0**-23 * mag
            worst = ((dw[j].double() - ref).abs() - room).max()
            assert float(worst) <= 1e-37, f"expert {j} of {n} rows: {float(worst):.3e} over"


# 5 x 5 tiles of 256 x 256 an expert: more of them than the card has CUs, each with 2 to 11 steps
LARGE = [65, 128, 0, 700, 129, 1, 300, 192, 511, 66, 640, 257, 90, 0, 405, 64]
HOLES = [0, 63, 64, 70, 200, 250, 893, 1100, 1500, 2400, 3547]


@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("base", [None, "apart", "in place"])
@pytest.mark.parametrize("gather", [None, "x", "dy"])
@pytest.mark.parametrize("ckpt", [False, True])
def test_large_tiles_of_several_steps(ckpt, gather, base, dw_dtype):
    print(f"[wgrad steps] ckpt={ckpt} gather={gather} base={base} {dw_dtype}", flush=True)
    _check(LARGE, 1032, 1032, 0, gather, ckpt, base, dw_dtype, HOLES)


@pytest.mark.parametrize("gather", [None, "x", "dy"])
@pytest.mark.parametrize("ckpt", [False, True])
def test_large_tiles_of_a_pair(ckpt, gather):
    _check(LARGE[:11], 1032, 1032, 1, gather, ckpt, "in place", torch.float32, HOLES, seed=20)


# on either side of the rows that are listed at a time; holes on either side of row 1024 of
# each expert, in a whole step, and in the last rows
LONG = [1024, 1025, 0, 1088, 2500, 63, 2999]
STARTS = [0, *np.cumsum(LONG)]
LONG_HOLES = sorted({int(s) + h for s in STARTS[:-1] for h in (0, 1022, 1023, 1024, 1025, 1087, 2047, 2048, 2499)} |
                    {int(STARTS[4]) + 1152 + i for i in range(64)})


@pytest.mark.parametrize("N,M", [(72, 136), (1544, 1800)])
@pytest.mark.parametrize("gather", [None, "x", "dy"])
@pytest.mark.parametrize("ckpt", [False, True])
def test_experts_of_more_rows_than_a_list(ckpt, gather, N, M):
    """Small tiles, and 7 x 8 large ones an expert."""
    print(f"[wgrad lists] ckpt={ckpt} gather={gather} N={N} M={M}", flush=True)
    _check(LONG, N, M, int(N < 100), gather, ckpt, "apart", torch.float32, LONG_HOLES, T=1500)


@pytest.mark.parametrize("ckpt", [False, True])
def test_64_bit_addresses_of_several_steps(ckpt):
    """Rows of dw so wide that 256 of them pass 2^31 bytes; tokens gathered, some named nowhere."""
    _check([70, 0, 131], 16, 2**21 + 8, 0, "x", ckpt, None, torch.float32, [3, 64, 69, 70, 150, 200], T=90)


@pytest.mark.parametrize("ckpt", [False, True])
def test_64_bit_addresses_of_more_rows_than_a_list(ckpt):
    """Tokens' gradients that together pass 2^31 bytes, gathered by 1100 rows and more."""
    _check([1100, 70, 2100], 4096, 264, 0, "dy", ckpt, "in place", torch.bfloat16, [5, 1023, 1024, 1099, 1169, 2200, 3269],
           T=2**18 + 50)
