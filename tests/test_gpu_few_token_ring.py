"""Many laps of the copy ring with fewer tokens than converting warps: most of those
warps have nothing to convert in a step, and still may not lose count of the laps."""
import pytest
import torch

import autotuning_tcgen05_tmem_gb300 as g
import few_token_util as ref

pytestmark = pytest.mark.gpu


def weights_of(gen, K, N, group, zeros, patterns):
    parts = [ref.random_weight(gen, K, N, group, zeros) for _ in range(patterns)]
    return parts, [ref.dequant(*p, N, group) for p in parts]


def packed(parts, N, group, gated, E):
    """E experts, expert e holding the pattern e % len(parts)."""
    return torch.cat([g.wq_pack(*(None if t is None else t.cuda() for t in parts[e % len(parts)]), N, group, gated=gated)
                      for e in range(E)])


@pytest.mark.parametrize("T,E,group,zeros", [(64, 64, 128, True), (64, 256, 32, True), (33, 64, 256, False), (20, 40, 64, True),
                                             (16, 32, 128, True), (1, 16, 128, False), (3, 16, 64, True)])
def test_experts_of_one_token(T, E, group, zeros):
    """Every token has an expert of its own; above 32 tokens the ring has two slots."""
    H, I, patterns = 1536, 1024, 3
    gen = torch.Generator().manual_seed(T + E)
    gu, gu64 = weights_of(gen, H, 2 * I, group, zeros, patterns)
    dn, dn64 = weights_of(gen, I, H, group, zeros, patterns)
    gate_up, down = packed(gu, 2 * I, group, True, E), packed(dn, H, group, False, E)
    x = torch.randn(T, H, generator=gen).bfloat16()
    ids = torch.randperm(E, generator=gen)[torch.arange(T) % E].int()[:, None].contiguous()
    w = torch.rand(T, 1, generator=gen)
    want, bound = ref.experts(x, ids % patterns, w, gu64, dn64, "swiglu", None, group)
    xd, idd, wd = x.cuda(), ids.cuda(), w.cuda()
    with g.moe_plan(H, I, E, 1, weights="wq", group=group, zeros=zeros) as p:
        ys = [torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(20)]
        for y in ys:
            p.run_routed(xd, idd, wd, gate_up, down, y)
        torch.cuda.synchronize()
        assert p.status() == 0, g.last_error()
    ref.within(ys[0], want, bound)
    assert all(torch.equal(y, ys[0]) for y in ys)


@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("K,N", [(14336, 640), (8192, 20000)])
def test_products_of_few_tokens(T, K, N):
    gen = torch.Generator().manual_seed(T + K)
    (parts,), (W,) = weights_of(gen, K, N, 128, True, 1)
    x = torch.randn(T, K, generator=gen).bfloat16()
    weight = packed([parts], N, 128, False, 1)
    xd = x.cuda()
    with g.wq_plan(K, N, 128, True) as p:
        ys = [torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(20)]
        for y in ys:
            p.run(xd, weight, None, y)
        torch.cuda.synchronize()
        assert p.status() == 0, g.last_error()
    ref.within(ys[0], *ref.product(x, W, None, None, "none", 128))
    assert all(torch.equal(y, ys[0]) for y in ys)
