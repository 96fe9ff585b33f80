"""Packed weights that no kernel may be given: refused by the Python entry points
before anything is launched (no GPU needed)."""
import pytest
import torch

import autotuning_tcgen05_tmem_gb300 as g
from autotuning_tcgen05_tmem_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


class FakeCuda(torch.Tensor):
    """A host tensor that says it is on the GPU."""

    @property
    def is_cuda(self):
        return True


def fake(t):
    return t.as_subclass(FakeCuda)


@pytest.fixture
def launches(monkeypatch):
    """Counts what reaches the native entry points instead of calling them."""
    seen = []
    real = g.lib()

    class Stub:
        def __getattr__(self, name):
            if name in ("gemm_wq_run", "gemm_wq_pack", "gemm_moe_run", "gemm_moe_run_routed"):
                return lambda *a: seen.append(name) or g.OK
            return getattr(real, name)
    stub = Stub()
    monkeypatch.setattr(g, "lib", lambda: stub)
    monkeypatch.setattr(g, "_stream_handle", lambda stream: 0)
    return seen


def bad_weights(n):
    """Packed weights of n bytes that are on the host, of another type, too small, or views."""
    good = torch.zeros(n, dtype=torch.uint8)
    return {"host": good, "int32": fake(good.int()), "float": fake(good.float()), "small": fake(good[:-1]),
            "expanded": fake(torch.zeros(1, dtype=torch.uint8).expand(n)),
            "strided": fake(torch.zeros(2 * n, dtype=torch.uint8)[::2])}


@pytest.mark.parametrize("kind", ["host", "int32", "float", "small", "expanded", "strided"])
def test_product_refuses(launches, kind):
    p = g.WqPlan(0, 64, 96, 32, False, g.EPI_NONE, 4)
    x, y = fake(torch.zeros(2, 64).bfloat16()), fake(torch.zeros(2, 96).bfloat16())
    with pytest.raises(ValueError, match="packed"):
        p.run(x, bad_weights(p.packed_bytes)[kind], None, y)
    assert launches == []
    p.run(x, fake(torch.zeros(p.packed_bytes, dtype=torch.uint8)), None, y)
    assert launches == ["gemm_wq_run"]


@pytest.mark.parametrize("which", ["gate_up", "down"])
@pytest.mark.parametrize("kind", ["host", "int32", "float", "small", "expanded", "strided"])
def test_experts_refuse(launches, kind, which):
    d = g.MoeDesc(64, 32, 4, 2, 8, g.MOE_WEIGHTS["wq"], 32, 0, g.EPI_BIAS_SWIGLU, 1)
    p = g.MoePlan(0, d)
    x = fake(torch.zeros(2, 64).bfloat16())
    w = dict(zip(("gate_up", "down"), (fake(torch.zeros(n, dtype=torch.uint8)) for n in p._packed)))
    router = fake(torch.zeros(64, 4).bfloat16())
    ids, weights = fake(torch.zeros(2, 2, dtype=torch.int32)), fake(torch.zeros(2, 2))
    p.run(x, router, w["gate_up"], w["down"], x)
    assert launches == ["gemm_moe_run"]
    w[which] = bad_weights(p._packed[which == "down"])[kind]
    with pytest.raises(ValueError, match=which):
        p.run(x, router, w["gate_up"], w["down"], x)
    with pytest.raises(ValueError, match=which):
        p.run_routed(x, ids, weights, w["gate_up"], w["down"], x)
    assert launches == ["gemm_moe_run"]


@pytest.mark.parametrize("kind", ["host", "int32", "float", "small", "expanded", "strided"])
def test_pack_refuses_its_output(launches, kind):
    codes, scales = fake(torch.zeros(64, 48, dtype=torch.uint8)), fake(torch.zeros(2, 96).bfloat16())
    n = int(g.lib().gemm_wq_packed_bytes(1, 64, 96, 32, 0))
    with pytest.raises(ValueError, match="out"):
        g.wq_pack(codes, scales, None, 96, 32, out=bad_weights(n)[kind])
    assert launches == []
    g.wq_pack(codes, scales, None, 96, 32, out=fake(torch.zeros(n, dtype=torch.uint8)))
    assert launches == ["gemm_wq_pack"]


def pack(K, N, group=32, zeros=False, gated=False, lead=()):
    ng = -(-K // group) if group else 1
    scales = fake(torch.zeros(*lead, ng, N).bfloat16())
    z = fake(torch.zeros(*lead, ng, N, dtype=torch.uint8)) if zeros else None
    n = int(g.lib().gemm_wq_packed_bytes(lead[0] if lead else 1, K, N, group, zeros))
    return g.wq_pack(fake(torch.zeros(*lead, K, (N + 1) // 2, dtype=torch.uint8)), scales, z, N, group, gated=gated,
                     out=fake(torch.zeros(n, dtype=torch.uint8)))


def test_product_refuses_another_layout(launches):
    """Of the same size, but its columns, groups or zero points lie elsewhere."""
    p = g.WqPlan(0, 512, 128, 64, True, g.EPI_BIAS_SWIGLU, 4)
    x, y, bias = fake(torch.zeros(2, 512).bfloat16()), fake(torch.zeros(2, 64).bfloat16()), fake(torch.zeros(128).bfloat16())
    p.run(x, pack(512, 128, 64, True, True), bias, y)
    launches.clear()
    for other in (pack(512, 128, 64, True, False), pack(128, 512, 64, True, True), pack(512, 128, 32, True, True)):
        assert other.numel() >= p.packed_bytes
        with pytest.raises(ValueError, match="layout"):
            p.run(x, other, bias, y)
    assert "gemm_wq_run" not in launches
    column = g.WqPlan(0, 512, 128, 0, False, g.EPI_NONE, 4)
    column.run(x, pack(512, 128, 256), None, fake(torch.zeros(2, 128).bfloat16()))   # the same bytes as a column's scale
    assert launches[-1] == "gemm_wq_run"


def test_experts_refuse_another_layout(launches):
    p = g.MoePlan(0, g.MoeDesc(64, 32, 4, 2, 8, g.MOE_WEIGHTS["wq"], 32, 0, g.EPI_BIAS_SWIGLU, 1))
    x, router = fake(torch.zeros(2, 64).bfloat16()), fake(torch.zeros(64, 4).bfloat16())
    gu, dn = pack(64, 64, gated=True, lead=(4,)), pack(32, 64, lead=(4,))
    p.run(x, router, gu, dn, x)
    for a, b, name in ((pack(64, 64, lead=(4,)), dn, "gate_up"), (gu, pack(32, 64, gated=True, lead=(4,)), "down")):
        with pytest.raises(ValueError, match=name):
            p.run(x, router, a, b, x)
    assert launches.count("gemm_moe_run") == 1
