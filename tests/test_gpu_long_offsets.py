"""Row descriptions in a buffer longer than the call's experts, as one sized for
more of them: the int8 chain quantises the rows its products read."""
import pytest
import torch

from harness import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

E, H, I = 4, 64, 96


def _operands(cap, seed):
    g = torch.Generator().manual_seed(seed)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, dtype=torch.int8).cuda()
    scales = lambda *s: ((torch.rand(s, generator=g) + 0.5) / 600).cuda()
    return codes(cap, H), scales(cap) * 600, [codes(E, I, H), codes(E, I, H), codes(E, H, I)], [scales(E, I), scales(E, I),
                                                                                                scales(E, H)]


# what an old or a cleared buffer holds behind the experts' entries
@pytest.mark.parametrize("tail", [(0, 0, 0), (3, 1), (1000,), (-5, 2**31 - 1)])
@pytest.mark.parametrize("masked", [False, True])
def test_the_chain_on_a_longer_buffer(masked, tail):
    import combine_grouped_gemm_amd as m
    cap_e, counts = 9, [5, 0, 9, 3]
    cap = E * cap_e
    head = counts if masked else [2, 7, 7, 16, 19]
    rows = torch.tensor([*head, *tail], dtype=torch.int32, device="cuda")
    exact = rows[:len(head)].clone()
    kw = dict(cap_per_expert=cap_e) if masked else {}
    a, sa, (wg, wu, wd), (sg, su, sd) = _operands(cap, len(tail))
    valid = torch.zeros(cap, dtype=torch.bool, device="cuda")
    for j, n in enumerate(counts):
        start = j * cap_e if masked else head[j]
        valid[start:start + n] = True

    def chain(r, **quant):
        h = torch.full((cap, I), 7.0, dtype=torch.bfloat16, device="cuda")
        q = torch.full((cap, I), 99, dtype=torch.int8, device="cuda")
        s = torch.full((cap,), -3.0, device="cuda")
        y = torch.full((cap, H), 7.0, dtype=torch.bfloat16, device="cuda")
        m.moe_ffn_gate_up(a, sa, r, wg, wu, sg, su, h=h, **kw)
        m.moe_quant_rows(h, r, q=q, scales=s, **kw, **quant)
        m.moe_ffn_down(q, s, r, wd, sd, y=y, **kw)
        return h, q, s, y

    want, got = chain(exact), chain(rows, E_loc=E)
    for w, g in zip(want, got):
        assert torch.equal(w, g)
    assert (got[1][~valid] == 99).all() and (got[2][~valid] == -3.0).all() and (got[3][~valid] == 7.0).all()
    y = torch.full((cap, H), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_grouped_ffn(a, sa, rows, wg, wu, wd, sg, su, sd, y=y, **kw)
    assert torch.equal(y, want[3])


def test_refusals():
    import combine_grouped_gemm_amd as m
    x = torch.zeros((8, 16), device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    for kw, msg in ((dict(rows=off, E_loc=5), "offsets needs at least 6"), (dict(rows=off, E_loc=0), "E_loc must"),
                    (dict(rows=off, E_loc=-1), "E_loc must"), (dict(E_loc=2), "E_loc needs the layout"),
                    (dict(rows=off, cap_per_expert=2, E_loc=6), "m needs at least 6"),
                    (dict(rows=off, cap_per_expert=2, E_loc=3), "needs E_loc"),
                    (dict(rows=off[:1], cap_per_expert=None), "at least 2"), (dict(rows=off[:0]), "at least 2"),
                    (dict(rows=off[:0], cap_per_expert=8), "at least 1")):
        with pytest.raises(ValueError, match=msg):
            m.moe_quant_rows(x, **kw)
