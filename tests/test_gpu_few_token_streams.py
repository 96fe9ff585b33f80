"""Few-token plans on streams of their own: what a plan sets up is there when it is
handed out, whatever the default stream is busy with."""
import pytest
import torch

import autotuning_tcgen05_tmem_gb300 as g
import few_token_util as ref

pytestmark = pytest.mark.gpu

BUSY = 200_000_000   # clock cycles of work queued on the default stream: a tenth of a second


@pytest.mark.parametrize("make", [lambda: g.wq_plan(512, 4096, 128), lambda: g.moe_plan(256, 128, 8, 2)], ids=["product", "experts"])
def test_plan_is_set_up_when_it_is_returned(make):
    """A stream that does not wait for the default one may run the plan at once."""
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.default_stream()):
        torch.cuda._sleep(BUSY)
        with make():
            assert torch.cuda.default_stream().query(), "the plan's memory is still to be cleared"


def test_product_on_a_stream_beside_a_busy_default():
    T, K, N = 3, 2048, 20000
    gen = torch.Generator().manual_seed(1)
    codes, scales, zeros = ref.random_weight(gen, K, N, 128, True)
    x = torch.randn(T, K, generator=gen).bfloat16()
    packed = g.wq_pack(codes.cuda(), scales.cuda(), zeros.cuda(), N, 128)
    xd, y = x.cuda(), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    dirty = torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    del dirty
    torch.cuda.empty_cache()         # the plan's memory may be what this left
    torch.cuda._sleep(BUSY)
    with g.wq_plan(K, N, 128, True) as p:
        with torch.cuda.stream(side):
            p.run(xd, packed, None, y)
        side.synchronize()
        assert p.status() == 0
    ref.within(y, *ref.product(x, ref.dequant(codes, scales, zeros, N, 128), None, None, "none", 128))
