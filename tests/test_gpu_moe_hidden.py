"""What the expert layer keeps of h between its two products: integer layers whose
h needs more significant bits than one bf16 holds, compared bit for bit."""
import numpy as np
import pytest
import torch

import autotuning_tcgen05_tmem_gb300 as g
import few_token_util as ref

pytestmark = pytest.mark.gpu


def one_hot_tokens(gen, T, H):
    x = torch.zeros(T, H)
    x[torch.arange(T), torch.randint(0, H, (T,), generator=gen)] = 1.0
    return x.bfloat16()


def choices(gen, T, E, k):
    return torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).int()


def integer_layer(x, ids, gate_up, down):
    """Σ_j relu(x·Gate)·(x·Up)·Down in 64 bits for integer weights [E, K, N] of any float type."""
    y = torch.zeros(x.shape[0], down.shape[2], dtype=torch.float64)
    for t in range(x.shape[0]):
        for e in ids[t].tolist():
            gate, up = ref.gate_up(x[t:t + 1].double() @ gate_up[e].double())
            y[t] += ((gate.clamp_min(0) * up) @ down[e].double())[0]
    return y


@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 32, 2, 1), (3, 200, 96, 3, 2), (12, 128, 64, 2, 2), (24, 72, 160, 4, 3),
                                       (32, 64, 64, 1, 1), (40, 136, 64, 2, 2), (64, 64, 96, 8, 2), (64, 256, 128, 1, 1)])
def test_bf16_experts_keep_16_bits(T, H, I, E, k):
    """Gates and ups are integers of 8 bits, so h is an integer of up to 16; |y| stays
    below 2^24 and every sum in 32 bits is exact."""
    gen = torch.Generator().manual_seed(T + I)
    gu = torch.randint(-255, 256, (E, H, 2 * I), generator=gen).bfloat16()
    dn = torch.randint(-1, 2, (E, I, H), generator=gen).bfloat16()
    x, ids = one_hot_tokens(gen, T, H), choices(gen, T, E, k)
    want = integer_layer(x, ids, gu, dn)
    assert float(want.abs().max()) < 2 ** 24
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    with g.moe_plan(H, I, E, k, act="reglu") as p:
        p.run_routed(x.cuda(), ids.cuda(), torch.ones(T, k).cuda(), gu.cuda(), dn.cuda(), y)
        torch.cuda.synchronize()
        assert p.status() == 0
    assert np.array_equal(ref.bits(y), ref.bits(ref.rounded(want)))


def test_bf16_experts_finite_h_above_the_largest_bf16():
    """h = (181/128)^2 · 2^127 is finite in 32 bits; the nearest bf16 is infinite."""
    H = I = 64
    gu = torch.full((1, H, 2 * I), 181.0 / 128 * 2.0 ** 63)
    gu[0, :, 32:64] *= 2
    gu[0, :, 96:] *= 2
    dn = torch.zeros(1, I, H)
    dn[0, 5] = 2.0 ** -20
    x = torch.zeros(1, H)
    x[0, 3] = 1.0
    y = torch.empty(1, H, dtype=torch.bfloat16, device="cuda")
    with g.moe_plan(H, I, 1, 1, act="reglu") as p:
        p.run_routed(x.bfloat16().cuda(), torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.ones(1, 1).cuda(),
                     gu.bfloat16().cuda(), dn.bfloat16().cuda(), y)
        torch.cuda.synchronize()
    want = torch.full((1, H), (181.0 / 128) ** 2 * 2.0 ** 107, dtype=torch.float64)
    assert np.array_equal(ref.bits(y), ref.bits(ref.rounded(want)))


@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 32, 2, 1), (3, 200, 96, 3, 2), (7, 320, 288, 9, 1), (12, 128, 64, 2, 2),
                                       (24, 72, 160, 4, 2), (40, 136, 64, 2, 2), (64, 64, 96, 8, 2), (64, 520, 224, 1, 1)])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (256, False), (0, True)])
def test_4bit_experts_keep_11_bits(T, H, I, E, k, group, zeros):
    """Gates and ups are integers up to 45, so h is one of up to 11 bits, in rows whose 64s
    have different largest values; |y| stays below 2^24 and every sum in 32 bits is exact."""
    gen = torch.Generator().manual_seed(T + I + group)

    def weight(K, N, scale):
        codes, _, z = ref.random_weight(gen, K, N, group, zeros)
        ng = 1 if group == 0 else -(-K // group)
        return codes, scale(ng, N).bfloat16(), z
    gu = [weight(H, 2 * I, lambda ng, N: torch.randint(0, 4, (ng, N // 64), generator=gen).repeat_interleave(64, 1))
          for _ in range(E)]
    dn = [weight(I, H, lambda ng, N: torch.ones(ng, N)) for _ in range(E)]
    x, ids = one_hot_tokens(gen, T, H), choices(gen, T, E, k)
    want = integer_layer(x, ids, torch.stack([ref.dequant(*w, 2 * I, group) for w in gu]),
                         torch.stack([ref.dequant(*w, H, group) for w in dn]))
    assert float(want.abs().max()) < 2 ** 24

    def packed(ws, N, gated):
        return g.wq_pack(*(None if ws[0][i] is None else torch.stack([w[i] for w in ws]).cuda() for i in range(3)), N, group,
                         gated=gated)
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    with g.moe_plan(H, I, E, k, act="reglu", weights="wq", group=group, zeros=zeros) as p:
        for _ in range(2):
            p.run_routed(x.cuda(), ids.cuda(), torch.ones(T, k).cuda(), packed(gu, 2 * I, True), packed(dn, H, False), y)
        torch.cuda.synchronize()
        assert p.status() == 0
    assert np.array_equal(ref.bits(y), ref.bits(ref.rounded(want)))


@pytest.mark.parametrize("T", [1, 12, 40])
def test_4bit_experts_rows_of_many_sizes(T):
    """Rows of h whose 64s are as far apart as 2^80, and 64s of nothing: what is small beside
    another 64 of its row still counts to 11 bits of that one's neighbourhood."""
    H, I, group = 128, 320, 64
    gen = torch.Generator().manual_seed(T)
    codes, _, _ = ref.random_weight(gen, H, 2 * I, group, False)
    power = torch.tensor([0.0, 2.0 ** -40, 2.0 ** 20, 2.0 ** -20, 1.0]).repeat_interleave(128)
    gu = (codes, power.expand(2, 2 * I).bfloat16().contiguous(), None)
    dn = ref.random_weight(gen, I, H, group, False)
    x = torch.randn(T, H, generator=gen).bfloat16()
    ids, w = torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1)
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    with g.moe_plan(H, I, 1, 1, act="reglu", weights="wq", group=group) as p:
        p.run_routed(x.cuda(), ids.cuda(), w.cuda(), g.wq_pack(*(None if t is None else t.cuda() for t in gu), 2 * I, group, gated=True),
                     g.wq_pack(*(None if t is None else t.cuda() for t in dn), H, group), y)
        torch.cuda.synchronize()
        assert p.status() == 0
    ref.within(y, *ref.experts(x, ids, w, [ref.dequant(*gu, 2 * I, group)], [ref.dequant(*dn, H, group)], "reglu", None, group))
