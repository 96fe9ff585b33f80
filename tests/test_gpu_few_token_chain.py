"""Calls of one product plan queued behind one another: what a call keeps in the plan's
memory (converted activations, pieces, counts) is its own, whatever the last one left."""
import numpy as np
import pytest
import torch

import autotuning_tcgen05_tmem_gb300 as g
import few_token_util as ref

pytestmark = pytest.mark.gpu

COUNTS = [64, 9, 33, 1, 16, 64, 2, 40, 9, 17, 8]


@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("K,N", [(2304, 640), (1032, 9000)])
def test_other_tokens_each_call(K, N, early):
    gen = torch.Generator().manual_seed(K)
    codes, scales, z = ref.random_weight(gen, K, N, 128, True)
    W = ref.dequant(codes, scales, z, N, 128)
    packed = g.wq_pack(codes.cuda(), scales.cuda(), z.cuda(), N, 128)
    xs = [torch.randn(T, K, generator=gen).bfloat16() for T in COUNTS]
    xd = [x.cuda() for x in xs]
    ys = [torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for T in COUNTS]
    torch.cuda.synchronize()
    with g.wq_plan(K, N, 128, True, max_tokens=64) as p:
        p.set_independent_weights(early)
        for x, y in zip(xd, ys):
            p.run(x, packed, None, y)
        torch.cuda.synchronize()
        assert p.status() == 0
    for x, y in zip(xs, ys):
        ref.within(y, *ref.product(x, W, None, None, "none", 128))


@pytest.mark.parametrize("T", [7, 12, 50])
def test_replays_on_changed_tokens(T):
    """A captured call reads its activations anew at every replay, and is right behind
    work that writes them."""
    K, N = 1032, 1280
    gen = torch.Generator().manual_seed(T)
    codes, scales, z = ref.random_weight(gen, K, N, 64, True)
    W = ref.dequant(codes, scales, z, N, 64)
    packed = g.wq_pack(codes.cuda(), scales.cuda(), z.cuda(), N, 64)
    xs = [torch.randn(T, K, generator=gen).bfloat16() for _ in range(4)]
    xd, sources = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda"), [x.cuda() for x in xs]
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    with g.wq_plan(K, N, 64, True) as p:
        p.run(xd, packed, None, y)
        torch.cuda.synchronize()
        p.set_independent_weights()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                p.run(xd, packed, None, y)
        got = []
        for s in sources:
            xd.copy_(s)
            graph.replay()
            got.append(y.clone())
        torch.cuda.synchronize()
        assert p.status() == 0
    for x, out in zip(xs, got):
        ref.within(out, *ref.product(x, W, None, None, "none", 64))


def test_experts_other_tokens_each_call():
    """The same of an expert layer: routing, h and counts of each call are its own."""
    from test_gpu_moe import Layer
    for weights, group in (("bf16", 0), ("wq", 64)):
        L = Layer(264, 160, 8, weights, group, weights == "wq", seed=3)
        xs = [torch.randn(T, 264, generator=L.gen).bfloat16() for T in COUNTS]
        r = L.router.cuda()
        with L.plan(3, max_tokens=64) as p:
            outs = []
            for x in xs:
                T = x.shape[0]
                y = torch.empty(T, 264, dtype=torch.bfloat16, device="cuda")
                ids, w = torch.empty(T, 3, dtype=torch.int32, device="cuda"), torch.empty(T, 3, device="cuda")
                p.run(x.cuda(), r, L.gate_up, L.down, y, ids=ids, weights=w)
                outs.append((y, ids, w))
            torch.cuda.synchronize()
            assert p.status() == 0
        for x, (y, ids, w) in zip(xs, outs):
            ref.within(y, *ref.experts(x, ids.cpu(), w.cpu(), L.gate_up64, L.down64, "swiglu", None, L.group))


@pytest.mark.parametrize("K,N,group", [(128, 64, 32), (256, 264, 64), (300, 40, 256), (64, 7, 32)])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_of_tiny_weights(K, N, group, zeros):
    """Groups whose scale is so small that its reciprocal may not be finite, beside ordinary ones."""
    from test_gpu_wq import plain_quantize
    gen = torch.Generator().manual_seed(K + N)
    W = torch.randn(K, N, generator=gen)
    W[:, ::3] *= 1e-36
    W[:, 1::6] *= 1e-38                   # scales among the subnormal numbers
    W = W.bfloat16()
    codes, scales, z = g.wq_quantize(W.cuda(), group, zeros)
    c, s, zz = plain_quantize(W, group, zeros)
    assert np.array_equal(scales.float().cpu().numpy(), s)
    assert np.array_equal(ref.unpack(codes.cpu(), N).numpy(), c)
    assert (z is None) if not zeros else np.array_equal(z.cpu().numpy(), zz)
