"""Operands of the training step's calls that lie one behind the other in one buffer, and the
inputs that an output may be: the same results as apart."""
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]


class Buffer:
    """Tensors cut from one buffer without gaps (sizes here are multiples of 16 bytes)."""

    def __init__(self):
        self.raw, self.at = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda"), 0

    def __call__(self, like):
        n = like.numel() * like.element_size()
        assert n % 16 == 0
        t = self.raw[self.at:self.at + n].view(like.dtype).view(like.shape)
        self.at += n
        return t.copy_(like)


def _sets(make):
    """Operands apart, and the same in one buffer."""
    yield make(lambda t: t.clone())
    yield make(Buffer())


def _same(results):
    for a, b in zip(*results):
        assert torch.equal(a, b)


def _rand(*shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


E, CAP, N, M, T, K = 3, 16, 64, 256, 8, 2
OFF = [0, 5, 5, 16]                                    # 16 bytes
ZERO = dict(device="cuda")


def _off():
    return torch.tensor(OFF, dtype=torch.int32, device="cuda")


def test_checkpoints():
    import combine_grouped_gemm_amd as m

    def run(put):
        x, q, s, off = put(_rand(CAP, M)), put(torch.zeros(CAP, M, dtype=torch.int8, **ZERO)), put(torch.zeros(CAP, 2, **ZERO)), put(_off())
        out = put(torch.zeros(CAP, M, dtype=torch.bfloat16, **ZERO))
        m.moe_checkpoint_rows(x, off, q=q, scales=s)
        m.moe_checkpoint_values(q, s, off, out=out)
        return q, s, out
    _same(list(_sets(run)))


def test_gate_up():
    import combine_grouped_gemm_amd as m

    def run(put):
        xd, wg, wu, off = put(_rand(CAP, M)), put(_rand(E, N, M)), put(_rand(E, N, M)), put(_off())
        outs = [put(torch.zeros(CAP, n, dtype=d, **ZERO)) for n, d in ((N, torch.bfloat16), (N, torch.int8), (1, torch.float32),
                                                                       (N, torch.int8), (1, torch.float32))]
        m.moe_ffn_gate_up_train(xd, off, wg, wu, *outs)
        return outs
    _same(list(_sets(run)))


@pytest.mark.parametrize("in_place", [False, True])
def test_swiglu_with_its_weights_gradient_in_place(in_place):
    import combine_grouped_gemm_amd as m
    row_of = torch.randperm(CAP, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.int32)
    row_of[3] = -1

    def run(put):
        dh, r, w = put(_rand(CAP, N)), put(row_of.view(T, K)), put(_rand(T, K, dtype=torch.float32))
        codes = [put((_rand(CAP, N, dtype=torch.float32) * 30).clamp(-127, 127).to(torch.int8)) for _ in range(2)]
        scales = [put(torch.full((CAP, 1), 0.125, **ZERO)) for _ in range(2)]
        outs = [put(torch.zeros(CAP, N, dtype=torch.bfloat16, **ZERO)) for _ in range(3)]
        dw = w if in_place and isinstance(put, Buffer) else put(torch.zeros(T, K, **ZERO))
        m.moe_swiglu_backward(dh, codes[0], scales[0], codes[1], scales[1], r, w, *outs, dw)
        return (*outs, dw)
    _same(list(_sets(run)))


def test_input_and_weight_gradients():
    import combine_grouped_gemm_amd as m
    src = torch.arange(CAP, dtype=torch.int32, device="cuda")

    def run(put):
        dy, dy2, w, w2 = (put(_rand(*s)) for s in ((T, N), (T, N), (E, N, M), (E, N, M)))
        s, off, dx = put(src), put(_off()), put(torch.zeros(CAP, M, dtype=torch.bfloat16, **ZERO))
        m.moe_ffn_dgrad(dy, off, w, dy2=dy2, w2=w2, src_of=s, slots_per_token=K, dx=dx)
        x, xs = put((_rand(CAP, M, dtype=torch.float32) * 30).clamp(-127, 127).to(torch.int8)), put(torch.ones(CAP, 2, **ZERO))
        dw, dw2 = (put(torch.zeros(E, N, M, **ZERO)) for _ in range(2))
        m.moe_ffn_wgrad(dy, x, off, x_scales=xs, dy2=dy2, src_of=s, slots_per_token=K, gather="dy", dw=dw, dw2=dw2)
        return dx, dw, dw2
    _same(list(_sets(run)))


def test_router():
    import combine_grouped_gemm_amd as m

    def run(put):
        lg = put(_rand(T, 64, dtype=torch.float32))
        ids = put(m.moe_route(lg, K)[0])
        dw, out = put(_rand(T, K, dtype=torch.float32)), put(torch.zeros(T, 64, **ZERO))
        m.moe_route_backward(lg, ids, dw, score="sigmoid", dlogits=out)
        return (out,)
    _same(list(_sets(run)))
