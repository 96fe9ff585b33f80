"""Infinities and NaN among the activations of 4-bit products: each output is what the
definition gives, an infinity of the right sign, NaN or a number, for every token count."""
import pytest
import torch

import autotuning_tcgen05_tmem_gb300 as g
import few_token_util as ref

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# (K index, value) of one token; K blocks are 256 wide, groups 32 to 256
PATTERNS = [[(3, INF)], [(3, -INF)], [(40, INF), (41, INF)], [(40, INF), (44, -INF)], [(0, INF), (200, INF)], [(10, INF), (300, INF)],
            [(10, -INF), (300, INF)], [(499, INF)], [(5, NAN)], [(5, NAN), (6, INF)], [(70, INF), (71, INF), (72, INF), (75, -INF)],
            [(k, INF) for k in range(500)], [(6, NAN), (7, NAN)], [(130, INF), (450, NAN)]]


def by_definition(x, W):
    """Σ_k x·W in 64 bits, product by product: 0·inf and inf - inf are NaN."""
    return torch.stack([(row[:, None] * W).sum(0) for row in x.double()])


def same_kind(got, want):
    got = got.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf])


def poison(x, rows):
    for t, p in zip(rows, PATTERNS):
        for k, v in p:
            x[t, k] = v
    return x


@pytest.mark.parametrize("T", [1, 6, 8, 12, 20, 40, 64])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (256, True), (0, False)])
def test_products(T, group, zeros):
    K, N = 504, 160
    gen = torch.Generator().manual_seed(T + group)
    codes, scales, z = ref.random_weight(gen, K, N, group, zeros)
    W = ref.dequant(codes, scales, z, N, group)
    packed = g.wq_pack(*(None if t is None else t.cuda() for t in (codes, scales, z)), N, group)
    clean = torch.randn(T, K, generator=gen).bfloat16()
    runs = -(-len(PATTERNS) // max(1, T // 2))
    with g.wq_plan(K, N, group, zeros) as p:
        for i in range(runs):
            mine = PATTERNS[i * max(1, T // 2):(i + 1) * max(1, T // 2)]
            x = clean.clone()
            for t, pattern in enumerate(mine):
                for k, v in pattern:
                    x[min(2 * t, T - 1), k] = v
            y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
            p.run(x.cuda(), packed, None, y)
            torch.cuda.synchronize()
            assert p.status() == 0
            want = by_definition(x, W)
            same_kind(y, want)
            good = torch.isfinite(x.double()).all(1)
            if bool(good.any()):
                ref.within(y[good.cuda()], *ref.product(x[good], W, None, None, "none", group))


@pytest.mark.parametrize("T", [2, 14, 30, 60])
@pytest.mark.parametrize("weights,group,zeros", [("bf16", 0, False), ("wq", 32, False), ("wq", 128, True)])
def test_experts(T, weights, group, zeros):
    """Infinite tokens, and finite ones whose h overflows, through both products."""
    H, I, E = 504, 96, 3
    gen = torch.Generator().manual_seed(T + group)
    if weights == "wq":
        gu = [ref.random_weight(gen, H, 2 * I, group, zeros) for _ in range(E)]
        dn = [ref.random_weight(gen, I, H, group, zeros) for _ in range(E)]
        gu64, dn64 = [ref.dequant(*w, 2 * I, group) for w in gu], [ref.dequant(*w, H, group) for w in dn]

        def packed(ws, N, gated):
            return g.wq_pack(*(None if ws[0][i] is None else torch.stack([w[i] for w in ws]).cuda() for i in range(3)), N,
                             group, gated=gated)
        gate_up, down = packed(gu, 2 * I, True), packed(dn, H, False)
    else:
        gu64 = (torch.randn(E, H, 2 * I, generator=gen) * H ** -0.5).bfloat16()
        dn64 = (torch.randn(E, I, H, generator=gen) * I ** -0.5).bfloat16()
        dn64[:, ::7, ::5] = 0.0             # times an infinity
        gate_up, down = gu64.cuda(), dn64.cuda()
        gu64, dn64 = list(gu64.double()), list(dn64.double())
    x = poison(torch.randn(T, H, generator=gen).bfloat16(), range(0, T, 2))
    x[1] *= 2.0 ** 66                       # h beyond the largest number
    ids = torch.randint(0, E, (T, 1), generator=gen, dtype=torch.int32)
    ids[1:2] = 1
    w = torch.full((T, 1), 0.5)
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    with g.moe_plan(H, I, E, 1, act="reglu", weights=weights, group=group, zeros=zeros) as p:
        p.run_routed(x.cuda(), ids.cuda(), w.cuda(), gate_up, down, y)
        torch.cuda.synchronize()
        assert p.status() == 0
    want = torch.empty(T, H, dtype=torch.float64)
    for t in range(T):
        e = int(ids[t])
        gate, up = ref.gate_up(by_definition(x[t:t + 1], gu64[e]))
        h = torch.where(gate > 0, gate, torch.where(gate != gate, gate, torch.zeros_like(gate))) * up
        h = h.float()                       # sums are held in 32 bits
        want[t] = 0.5 * by_definition(h, dn64[e])[0]
    same_kind(y, want)


@pytest.mark.parametrize("epi", ["relu_residual", "swiglu", "gelu", "bias_residual"])
@pytest.mark.parametrize("T", [3, 24])
@pytest.mark.parametrize("division", [0, 1, 2])
def test_epilogues_and_divisions(T, epi, division):
    """Resolved sums go through the epilogue like any other, in place on the residual too."""
    K, N, group = 2056, 640, 64
    gen = torch.Generator().manual_seed(T)
    codes, scales, z = ref.random_weight(gen, K, N, group, True)
    W = ref.dequant(codes, scales, z, N, group)
    x = torch.randn(T, K, generator=gen).bfloat16()
    x[0, 2055], x[1, 1000], x[2, 7], x[2, 2000] = INF, -INF, INF, NAN
    bias = torch.randn(N, generator=gen).bfloat16()
    out = N // 2 if epi in ref.GLU else N
    R = torch.randn(T, out, generator=gen).bfloat16() if epi.endswith("residual") else None
    v = by_definition(x, W) + bias.double()
    if epi in ref.GLU:
        gate, up = ref.gate_up(v)
        want = ref.act(gate, epi) * up
    else:
        want = ref.act(v, epi)
    if R is not None:
        want = want + R.double()
    packed = g.wq_pack(codes.cuda(), scales.cuda(), z.cuda(), N, group, gated=epi in ref.GLU)
    y = torch.empty(T, out, dtype=torch.bfloat16, device="cuda") if R is None else R.cuda()
    g.debug_set(16, division)
    try:
        with g.wq_plan(K, N, group, True, epi) as p:
            p.run(x.cuda(), packed, bias.cuda(), y, residual=None if R is None else y)
            torch.cuda.synchronize()
            assert p.status() == 0
    finally:
        g.debug_set(16, 0)
    same_kind(y, want)
    good = torch.isfinite(want)
    ref.within(y.cpu()[3:], *(t[3:] for t in ref.product(x, W, bias, R, epi, group))) if T > 3 else None
    assert float((y.cpu().double()[good] - want[good]).abs().max() if bool(good.any()) else 0) < 0.1
