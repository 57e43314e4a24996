"""A block's attention input as it would be run: the quantised Q / K / V projection, each request's adapters, per-head
norm and rotary positions -- through the layers, against the float64 oracle of every step and, where no adapter
is active, against the fused projection fed with the tables; under torch.compile, in a CUDA graph."""

import numpy as np
import pytest
import torch

import synth
from oracle import adapters as oadapters
from oracle import rope_axes as orope
from oracle import svdq as osvdq

pytestmark = pytest.mark.gpu

HEADS, D, K = 2, 128, 512
N = 3 * HEADS * D
DIMS, THETA, EPS = [16, 56, 56], 10000.0, 1e-6


@pytest.fixture(scope="module")
def P(cuda_lib):
    return cuda_lib


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.fixture(scope="module")
def block(P):
    w = synth.svdq_workload(300, K, N)
    base = P.SvdqLinear.from_exported(w.R, synth.bf16_bits(w.L1), synth.bf16_bits(w.L2), synth.bf16_bits(w.bias),
                                      synth.bf16_bits(w.smooth_inv), w.g_a)
    g = torch.Generator(device="cuda").manual_seed(4)

    def normal(*shape, scale):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    pool = [(normal(r, K, scale=K ** -0.5), normal(N, r, scale=0.3)) for r in (8, 16, 30)]
    layer = P.LoraLinear.from_adapters(base, pool)
    x = torch.from_numpy(w.X).to(torch.bfloat16).cuda()
    pos = torch.stack([torch.zeros(300), torch.arange(300) // 20, torch.arange(300) % 20], 1).int().cuda()
    nq, nk = normal(D, scale=1.0), normal(D, scale=1.0)
    return w, base, layer, x, pos, nq, nk


def _attention_input(P, layer, x, pos, nq, nk):
    y = layer(x).view(-1, 3, HEADS, D)
    q, k = P.svdq_qk_norm_rope(y[:, 0], y[:, 1], nq, nk, EPS, pos, DIMS, THETA)
    return y, q, k


def test_projection_adapters_norm_and_rope(P, block):
    w, base, layer, x, pos, nq, nk = block
    off, ids, wt = [0, 1, 5, 140, 290], np.array([[0], [2], [1], [-1]]), np.array([[1.5], [0.5], [-1.0], [1.0]], np.float32)
    layer.set_plan(P.LoraPlan(off, ids, wt, 300, 3))
    y, q, k = _attention_input(P, layer, x, pos, nq, nk)
    shared = base(x)
    ref, us, ks = oadapters.forward(_np(x), _np(shared), _np(layer.A), _np(layer.B), off, ids, wt)
    got = _np(y).reshape(300, N)
    assert (np.abs(got - ref) <= oadapters.bound(ref, us, ks, K, 32)).all()
    assert torch.equal(y.reshape(300, N)[140:], shared[140:])
    # from the adapted projection (bf16) on, the norm and the rotation
    ang = orope.angles(_np(pos), DIMS, [THETA] * 3)
    for out, i, nw in ((q, 0, nq), (k, 1, nk)):
        n = orope.norm(_np(y[:, i]), _np(nw), EPS)
        r = orope.rotate(n, ang, False)
        assert (np.abs(_np(out) - r) <= orope.bound(n, r, False, 128, D)).all()
    # the whole run against the exact layer: the quantised projection's own bar
    exact = oadapters.forward(_np(x), osvdq.forward(w.X, w.smooth_inv, w.R, w.L1, w.L2, w.bias, w.g_a), _np(layer.A),
                              _np(layer.B), off, ids, wt)[0]
    assert np.linalg.norm(got - exact) <= 5e-3 * np.linalg.norm(exact)
    assert P.svdq_device_status() == 0


def test_without_adapters_the_run_is_the_fused_projection(P, block):
    """The fused call keeps the projection in fp32 until the end, the run rounds it once in between (half a bf16
    step, 2^-8, of every value of a head before the norm)."""
    w, base, layer, x, pos, nq, nk = block
    layer.set_plan(P.LoraPlan([0, 300], [-1], [1.0], 300, 3))
    _, q, k = _attention_input(P, layer, x, pos, nq, nk)
    cos, sin = P.svdq_rope_axes_tables(pos, DIMS, THETA, D)
    codes, scales, low = P.svdq_quantize_act_lowrank_down(x, base.smooth_inv, base.packed_w, base.act_global_scale)
    fused = P.svdq_w4a4_nvfp4_linear_qkv(codes, scales, low, base.act_global_scale, base.packed_w, base.w_global_scale,
                                         300, N, K, HEADS, nq, nk, EPS, cos, sin).view(300, 3, HEADS, D)
    for out, i in ((q, 0), (k, 1)):
        a, b = _np(out), _np(fused[:, i])
        assert np.linalg.norm(a - b) <= 2.0 ** -8 * 2 * np.linalg.norm(b)


def test_layers_under_compile_and_in_a_graph(P, block):
    w, base, layer, x, pos, nq, nk = block
    layer.set_plan(P.LoraPlan([0, 3, 200, 300], [0, 1, 2], [1.0, 1.0, 1.0], 300, 3))
    expect = layer(x.view(3, 100, K))
    assert expect.shape == (3, 100, N)
    compiled = torch.compile(layer, fullgraph=True, backend="aot_eager")
    assert torch.equal(compiled(x.view(3, 100, K)), expect)
    _, q, k = _attention_input(P, layer, x, pos, nq, nk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, gq, gk = _attention_input(P, layer, x, pos, nq, nk)
    graph.replay()
    assert torch.equal(gq, q) and torch.equal(gk, k)


def test_operators_agree_with_their_fakes(P, block):
    w, base, layer, x, pos, nq, nk = block
    plan = P.LoraPlan([0, 3, 200, 300], [0, 1, 2], [1.0, 1.0, 1.0], 300, 3)
    checks = ("test_schema", "test_faketensor")
    torch.library.opcheck(torch.ops.svdq.lora_add_.default, (x, base(x), layer.A, layer.B, plan.words, plan.sizes()),
                          test_utils=checks)
    q = torch.randn((300, 2, 64), device="cuda").to(torch.bfloat16)
    torch.library.opcheck(torch.ops.svdq.qk_norm_rope.default,
                          (q, q.clone(), None, None, 0.0, pos, [16, 24, 24], [1e4] * 3, "half"), test_utils=checks)
    torch.library.opcheck(torch.ops.svdq.rope_axes_tables.default, (pos, [16, 24, 24], [1e4] * 3, 64, 300),
                          test_utils=checks)


@pytest.mark.parametrize("rows", [8, 40])
def test_adapters_beside_the_awq_layer(P, rows):
    a = synth.awq_workload(rows, 512, 384)
    bf = lambda v: torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    base = P.AwqLinear(torch.from_numpy(a.qweight).cuda(), bf(a.scales), bf(a.zeros), None)
    pool = [(bf(np.random.default_rng(i).standard_normal((16, 512)) / 22),
             bf(np.random.default_rng(9 + i).standard_normal((384, 16)))) for i in range(3)]
    layer = P.LoraLinear.from_adapters(base, pool)
    ids = np.arange(rows)[:, None] % 4 - 1
    wt = np.linspace(-1, 1, rows, dtype=np.float32)[:, None]
    layer.set_plan(P.LoraPlan(list(range(rows + 1)), ids, wt, rows, 3))
    x = bf(a.X)
    ref, us, ks = oadapters.forward(_np(x), _np(base(x)), _np(layer.A), _np(layer.B), list(range(rows + 1)), ids, wt)
    assert (np.abs(_np(layer(x)) - ref) <= oadapters.bound(ref, us, ks, 512, 16)).all()


def test_adapters_read_what_the_kernel_before_them_wrote(P):
    """X comes from the call just before, whose kernel lets the next one start early: ten pairs of calls over one
    buffer, without a wait between them, against the same pairs one by one."""
    M, H = 16, 4
    g = torch.Generator(device="cuda").manual_seed(6)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    q, y = normal(10, M, H, D), normal(M, 256)
    a, b = normal(2, 16, H * D), normal(2, 256, 16)
    pos = torch.arange(3 * M, dtype=torch.int32, device="cuda").view(M, 3)
    plan = P.LoraPlan([0, 1, M], [1, 0], [0.5, 1.0], M, 2)
    x = torch.empty((M, H * D), dtype=torch.bfloat16, device="cuda")

    def pair(i):
        P.svdq_qk_norm_rope(q[i], None, None, None, 0.0, pos, DIMS, THETA, out_q=x.view(M, H, D))
        return P.svdq_lora_add(x, y, a, b, plan)

    alone = []
    for i in range(10):
        alone.append(pair(i))
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = [pair(i) for i in range(10)]
    graph.replay()
    for outs in ([pair(i) for i in range(10)], replayed):
        assert all(torch.equal(o, e) for o, e in zip(outs, alone))
    assert not torch.equal(alone[0], alone[1])


def test_writes_to_given_tensors_are_counted(P):
    """A graph that has saved a tensor notices when a call writes to it."""
    def normal(*shape):
        return torch.randn(shape, device="cuda").to(torch.bfloat16)

    plan = P.LoraPlan([0, 8], [0], [1.0], 8, 1)
    x, y, a, b = normal(8, 64), normal(8, 128), normal(1, 16, 64), normal(1, 128, 16)
    pos = torch.ones((8, 1), dtype=torch.int32, device="cuda")
    q, k = normal(8, 2, 64), normal(8, 2, 64)
    cos, sin = torch.empty((2, 32, 8), device="cuda").unbind(0)
    for write, tensors in ((lambda: P.svdq_lora_add(x, y, a, b, plan, out=y), [y]),
                           (lambda: P.svdq_qk_norm_rope(q, k, None, None, 0.0, pos, [64], 1e4, out_q=q, out_k=k), [q, k]),
                           (lambda: P.svdq_rope_axes_tables(pos, [64], 1e4, 64, 8, cos, sin), [cos, sin])):
        before = [t._version for t in tensors]
        write()
        assert all(t._version > v for t, v in zip(tensors, before))
    w = torch.randn((8, 128), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    z = w * y                                           # keeps y
    P.svdq_lora_add(x, y, a, b, plan, out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.float().sum().backward()
    with torch.inference_mode():
        t = y.clone()
        assert P.svdq_lora_add(x, t, a, b, plan, out=t) is t


def test_a_compiled_layer_over_many_plans(P, block):
    w, base, layer, x, pos, nq, nk = block
    torch._dynamo.reset()
    compiles = []

    def backend(gm, inputs):
        compiles.append(1)
        return gm.forward

    run = torch.compile(layer, fullgraph=True, backend=backend)
    for i in range(12):
        off = [0] + sorted({1 + 7 * i, 20 + 13 * i, 290 - 9 * i})
        n = len(off) - 1
        ids, wt = np.arange(i, i + n)[:, None] % 4 - 1, np.linspace(-1, 1, n, dtype=np.float32)[:, None]
        plan = P.LoraPlan(off, ids, wt, 300, 3)
        layer.set_plan(plan)
        assert torch.equal(run(x), P.svdq_lora_add(x, base(x), layer.A, layer.B, plan))
    assert len(compiles) == 1


def test_inductors_cuda_graphs_do_not_keep_a_plan(P):
    """Two plans of the same length in memory that launch different numbers of blocks."""
    torch._dynamo.reset()
    base = torch.nn.Linear(256, 192, device="cuda").to(torch.bfloat16).requires_grad_(False)
    g = torch.Generator(device="cuda").manual_seed(5)
    layer = P.LoraLinear.from_adapters(base, [(torch.randn((16, 256), generator=g, device="cuda"),
                                               torch.randn((192, 16), generator=g, device="cuda"))])
    plans = [P.LoraPlan([0, 200], [0], [1.0], 300, 1), P.LoraPlan([0, 100], [0], [1.0], 300, 1)]
    assert plans[0].nbytes == plans[1].nbytes and plans[0].struct.tiles != plans[1].struct.tiles
    run = torch.compile(layer, fullgraph=True, mode="reduce-overhead")
    with torch.no_grad():
        for i in range(8):
            x = torch.randn((300, 256), generator=g, device="cuda").to(torch.bfloat16)
            plan = plans[i // 4]
            layer.set_plan(plan)
            assert torch.equal(run(x).clone(), P.svdq_lora_add(x, base(x), layer.A, layer.B, plan))


def test_operators_that_read_a_plans_sizes_agree_with_their_fakes(P, block):
    w, base, layer, x, pos, nq, nk = block
    plan = P.LoraPlan([0, 3, 200, 300], [0, 1, 2], [1.0, 1.0, 1.0], 300, 3)
    sizes = torch.tensor(plan.sizes())
    checks = ("test_schema", "test_faketensor", "test_aot_dispatch_dynamic")
    for op in (torch.ops.svdq.lora_add_planned_, torch.ops.svdq.lora_add):
        torch.library.opcheck(op.default, (x, base(x), layer.A, layer.B, plan.words, sizes), test_utils=checks)
    y = base(x)
    out = torch.ops.svdq.lora_add(x, y, layer.A, layer.B, plan.words, sizes)
    assert torch.equal(y, base(x))
    torch.ops.svdq.lora_add_planned_(x, y, layer.A, layer.B, plan.words, sizes)
    assert torch.equal(y, out) and not torch.equal(y, base(x))
    with pytest.raises(RuntimeError, match="no gradient"):
        torch.ops.svdq.lora_add_planned_(x.clone().requires_grad_(), y, layer.A, layer.B, plan.words, sizes)
    z = torch.ops.svdq.lora_add(x.clone().requires_grad_(), y, layer.A, layer.B, plan.words, sizes)
    with pytest.raises(RuntimeError, match="no gradient"):
        z.float().sum().backward()
