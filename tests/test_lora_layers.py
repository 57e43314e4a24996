"""The adapter layers and the new torch.library operators on the host: registration, fake implementations,
tracing, padding of the pool, and the swap."""

import pytest
import torch
from torch import nn

import bit_diffusion_transformer_act_b200 as P
from bit_diffusion_transformer_act_b200 import torch_ops as T


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_operators_registered():
    for name in ("lora_add_", "qk_norm_rope", "rope_axes_tables"):
        assert hasattr(torch.ops.svdq, name), name


def test_fake_shapes():
    q, k = torch.ops.svdq.qk_norm_rope(_meta(7, 4, 64), _meta(7, 2, 64), None, None, 0.0,
                                       _meta(7, 2, dtype=torch.int32), [32, 32], [1e4, 1e4], "half")
    assert q.shape == (7, 4, 64) and k.shape == (7, 2, 64)
    cos, sin = torch.ops.svdq.rope_axes_tables(_meta(7, 2, dtype=torch.int32), [32, 32], [1e4, 1e4], 64, 14)
    assert cos.shape == sin.shape == (32, 14) and cos.dtype == torch.float32


def _awq(K=512, N=128):
    return T.AwqLinear(torch.zeros((N, K // 2), dtype=torch.uint8), torch.zeros((N, K // 64), dtype=torch.bfloat16),
                       torch.zeros((N, K // 64), dtype=torch.bfloat16))


def _pool(K=512, N=128, ranks=(4, 16, 20)):
    return [(torch.ones((r, K), dtype=torch.bfloat16), torch.full((N, r), 2.0, dtype=torch.bfloat16)) for r in ranks]


def test_pool_is_padded_with_zero_ranks():
    layer = T.LoraLinear.from_adapters(_awq(), _pool())
    assert layer.A.shape == (3, 32, 512) and layer.B.shape == (3, 128, 32)
    assert (layer.A[0, :4] == 1).all() and (layer.A[0, 4:] == 0).all() and (layer.B[2, :, 20:] == 0).all()
    with pytest.raises(ValueError, match="rank"):
        T.LoraLinear.from_adapters(_awq(), [(torch.ones(4, 512), torch.ones(128, 5))])
    with pytest.raises(ValueError, match="do not fit"):
        T.LoraLinear(_awq(), torch.zeros(3, 16, 512), torch.zeros(3, 64, 16))


def test_attach_set_and_trace():
    model = nn.Sequential(_awq(), nn.GELU(), nn.Sequential(nn.Linear(128, 128), nn.Linear(128, 64)))
    seen = []

    def factory(name, layer):
        seen.append(name)
        return T.LoraLinear.from_adapters(layer, _pool()) if isinstance(layer, T.AwqLinear) else None

    assert T.attach_adapters(model, factory) == 1
    assert seen == ["0", "2.0", "2.1"] and isinstance(model[0], T.LoraLinear)
    assert T.attach_adapters(model, lambda name, layer: None) == 0
    plan = P.LoraPlan([0, 2, 6], [1, -1], [1.0, 1.0], 6, 3, device="cpu")
    x = torch.zeros((2, 3, 512), dtype=torch.bfloat16)

    def calls(m):
        return [str(n.target) for n in torch.export.export(m, (x,)).graph.nodes if n.op == "call_function"]

    assert not any("lora" in c for c in calls(model[0]))
    T.set_lora_plan(model, plan)
    assert any("svdq.lora_add_" in c or "auto_functionalized" in c for c in calls(model[0]))
    T.set_lora_plan(model, None)
    assert not any("lora" in c for c in calls(model[0]))


def test_state_dict_carries_the_pool():
    a, b = T.LoraLinear.from_adapters(_awq(), _pool()), T.LoraLinear.from_adapters(_awq(), _pool(ranks=(1, 1, 32)))
    b.load_state_dict(a.state_dict())
    assert torch.equal(a.A, b.A) and torch.equal(a.B, b.B)


@pytest.fixture
def host_kernel(monkeypatch):
    """The adapters' call computed on the host, behind the real operators; returns the calls' modes."""
    calls = []

    def add(X, Y, A, B, plan, out=None, workspace=None):
        calls.append("new" if out is None else "in place")
        r = Y.detach().clone()
        w = plan.words.view(torch.int32)
        assert plan.struct.tiles == 0 and plan.struct.slots == 1
        for g in w[16 + 8 * plan.struct.copy_tiles:].view(-1, 44)[: plan.struct.groups]:
            for i in range(int(g[0])):
                m, wt = int(g[12 + i]), g[28 + i: 29 + i].view(torch.float32)
                r[m] += (wt * (B[g[4]].float() @ (A[g[4]].float() @ X.detach()[m].float()))).to(torch.bfloat16)
        if out is None:
            return r
        out.detach().copy_(r)
        return out

    monkeypatch.setattr(T.ops, "svdq_lora_add", add)
    monkeypatch.setattr(T.ops, "_on_device", lambda t, name: None)
    return calls


def _linear_layer(K=64, N=128):
    torch.manual_seed(0)
    base = nn.Linear(K, N).to(torch.bfloat16)
    layer = T.LoraLinear.from_adapters(base, [(torch.randn(4, K), torch.randn(N, 4)) for _ in range(2)])
    layer.set_plan(P.LoraPlan([0, 2, 3], [1, 0], [0.5, 2.0], 4, 2, device="cpu"))
    return base, layer


@pytest.mark.parametrize("compiled", [False, True])
def test_a_backward_pass_through_adapters_raises(host_kernel, compiled):
    """It dropped the adapters' part of the gradient: the in-place sum left the base's graph as it was."""
    base, layer = _linear_layer()
    run = torch.compile(layer, fullgraph=True, backend="aot_eager") if compiled else layer
    x = torch.randn(4, 64).to(torch.bfloat16)
    with torch.no_grad():
        expect = run(x)
    assert not torch.equal(expect, base(x)) and host_kernel == ["in place"]
    for x_grad, w_grad in ((True, True), (True, False), (False, True)):
        base.requires_grad_(w_grad)
        y = run(x.clone().requires_grad_(x_grad))
        assert y.requires_grad and torch.equal(y, expect) and host_kernel[-1] == "new"
        with pytest.raises(RuntimeError, match="no gradient"):
            y.float().sum().backward()
    with torch.no_grad():
        assert torch.equal(run(x), expect) and host_kernel[-1] == "in place"


def test_the_in_place_operator_refuses_gradients(host_kernel):
    base, layer = _linear_layer()
    plan = P.LoraPlan([0, 2, 3], [1, 0], [0.5, 2.0], 4, 2, device="cpu")
    x = torch.randn(4, 64).to(torch.bfloat16)

    def add(x, y):
        torch.ops.svdq.lora_add_(x, y, layer.A, layer.B, plan.words, plan.sizes())
        return y

    with pytest.raises(RuntimeError, match="no gradient"):
        add(x, base(x))
    with pytest.raises(RuntimeError, match="no gradient"):
        add(x.clone().requires_grad_(), base(x).detach())
    assert host_kernel == []
    y = base(x).detach()
    before = y._version
    expect = add(x, y).clone()
    assert y._version > before
    with torch.no_grad():
        assert torch.equal(add(x.clone().requires_grad_(), base(x)), expect)
    with torch.inference_mode():
        assert torch.equal(add(x, base(x)), expect)


def test_calls_refuse_an_output_that_carries_gradients():
    """They write through its address: its graph would go on as if it had kept its values."""
    bf = torch.bfloat16
    plan = P.LoraPlan([0, 4], [0], [1.0], 4, 2, device="cpu")
    x, a, b = torch.zeros((4, 64), dtype=bf), torch.zeros((2, 16, 64), dtype=bf), torch.zeros((2, 128, 16), dtype=bf)
    y = torch.zeros((4, 128), dtype=bf, requires_grad=True) * 2
    with pytest.raises(ValueError, match="out carries gradients"):
        P.svdq_lora_add(x, y, a, b, plan, out=y)
    pos = torch.zeros((4, 2), dtype=torch.int32)
    q = y.view(4, 2, 64)
    with pytest.raises(ValueError, match="out_q carries gradients"):
        P.svdq_qk_norm_rope(q, None, None, None, 0.0, pos, [32, 32], 1e4, out_q=q)
    with pytest.raises(ValueError, match="out_k carries gradients"):
        P.svdq_qk_norm_rope(None, q, None, None, 0.0, pos, [32, 32], 1e4, out_k=q)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):      # past that check
        P.svdq_lora_add(x, y, a, b, plan, out=y)


def test_one_compiled_graph_serves_every_plan(host_kernel):
    """The plan's sizes were guarded on one by one: every batch compiled again, and the ninth raised."""
    base, layer = _linear_layer()
    torch._dynamo.reset()
    compiles = []

    def backend(gm, inputs):
        compiles.append(1)
        return gm.forward

    run = torch.compile(layer, fullgraph=True, backend=backend)
    x = torch.randn(40, 64).to(torch.bfloat16)
    sizes = set()
    with torch.no_grad():
        for i in range(20):
            n = 1 + i * 2 % 13
            off = [min(40, 3 * r * (1 + i % 2)) for r in range(n + 1)]
            plan = P.LoraPlan(off, [r % 3 - 1 for r in range(n)], [0.25 * i + r for r in range(n)], 40, 2, device="cpu")
            sizes.add(tuple(plan.sizes()))
            layer.set_plan(plan)
            assert torch.equal(run(x), layer(x))
        assert len(sizes) > 15 and len(compiles) == 1
        layer.set_plan(None)
        assert torch.equal(run(x), base(x)) and len(compiles) == 2


def test_unsupported_pools_are_refused_when_the_layer_is_built():
    def build(K, N, rank, dtype=torch.bfloat16):
        return T.LoraLinear(nn.Linear(K, N), torch.zeros((2, rank, K), dtype=dtype), torch.zeros((2, N, rank), dtype=dtype))

    assert build(64, 64, 128).A.shape == (2, 128, 64)
    for bad, message in (((96, 64, 16), "multiples of 64"), ((64, 100, 16), "multiples of 64"), ((64, 64, 24), "rank"),
                         ((64, 64, 144), "rank"), ((64, 64, 0), "rank"), ((64, 64, 16, torch.float32), "bfloat16")):
        with pytest.raises(ValueError, match=message):
            build(*bad)
    with pytest.raises(ValueError, match="rank"):
        T.LoraLinear.from_adapters(_awq(), _pool(ranks=(4, 129)))
    assert T.LoraLinear.from_adapters(_awq(), _pool(ranks=(4, 113))).A.shape[1] == 128


def test_plans_that_a_layer_cannot_serve_are_refused_when_they_are_set():
    model = nn.Sequential(T.LoraLinear.from_adapters(_awq(), _pool(ranks=(16, 64))),
                          T.LoraLinear.from_adapters(_awq(), _pool(ranks=(128, 4))))
    one = P.LoraPlan([0, 4], [1], [1.0], 4, 2, device="cpu")
    two = P.LoraPlan([0, 4], [[1, 0]], [[1.0, 1.0]], 4, 2, device="cpu")
    T.set_lora_plan(model, one)
    model[0].set_plan(two)
    model[0].set_plan(one)
    with pytest.raises(ValueError, match="2 slots needs adapters of rank 64"):
        T.set_lora_plan(model, two)
    assert all(m.plan_words is one.words for m in model)        # neither layer took it
    with pytest.raises(ValueError, match="3 adapters"):
        model[1].set_plan(P.LoraPlan([0, 4], [1], [1.0], 4, 3, device="cpu"))
    T.set_lora_plan(model, None)
    assert all(m.plan_words is None for m in model)


def test_a_default_device_does_not_move_the_plans_sizes():
    base, layer = _linear_layer()
    plan = P.LoraPlan([0, 4], [1], [1.0], 4, 2, device="cpu")
    with torch.device("meta"):
        layer.set_plan(plan)
    assert layer.plan_sizes.tolist() == plan.sizes()
