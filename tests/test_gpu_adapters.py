"""Per-request low-rank adapters on the GPU against the float64 oracle: every kind of request (a row,
a few, many; none; no adapter; the same adapter in two slots), strided and in-place outputs, graphs,
streams, and a run through the layers."""

import numpy as np
import pytest
import torch

from oracle import adapters as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P(cuda_lib):
    return cuda_lib


def _np(t):
    return t.detach().double().cpu().numpy()


def _make(M, K, N, R, slots, adapters, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    return (normal(M, K), normal(M, N), normal(adapters, R, K, scale=K ** -0.5),
            normal(adapters, N, R, scale=R ** -0.5))


def _weights(ids, seed=0):
    return np.random.default_rng(seed).uniform(-1.5, 1.5, np.shape(ids)).astype(np.float32)


def _check(out, x, y, a, b, off, ids, w):
    ref, us, ks = oracle.forward(_np(x), _np(y), _np(a), _np(b), off, ids, w)
    tol = oracle.bound(ref, us, ks, x.shape[1], a.shape[1] * np.shape(ids)[1])
    bad = ~(np.abs(_np(out) - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], np.max(np.abs(_np(out) - ref) / tol))


# M, K, N, rank, slots, adapters, row offsets
CASES = [
    (1, 64, 64, 16, 1, 1, [0, 1]),
    (1, 320, 192, 48, 2, 3, [0, 1]),
    (2, 2560, 1024, 128, 1, 2, [0, 1, 2]),
    (9, 128, 128, 32, 1, 4, [0, 9]),
    (16, 576, 320, 16, 8, 5, [0, 16]),
    (17, 512, 256, 64, 2, 2, [0, 17]),
    (40, 256, 64, 16, 3, 3, list(range(41))),                       # a row per request
    (64, 1024, 448, 32, 4, 2, [0] + list(range(20, 65))),
    (127, 192, 64, 112, 1, 2, [0, 127]),
    (128, 64, 128, 32, 2, 2, [0, 128]),
    (129, 128, 192, 64, 1, 2, [0, 129]),
    (300, 448, 704, 80, 1, 3, [0, 0, 31, 31, 64, 200, 200, 298]),   # empty requests, rows behind the last
    (515, 640, 128, 48, 2, 6, [3, 20, 21, 150, 153, 400, 515]),     # rows before the first
    (700, 2560, 256, 128, 1, 2, [0, 260, 520, 690]),
    (1300, 128, 2560, 16, 1, 4, [0, 1000, 1001, 1290]),
]


def _ids(case):
    M, K, N, R, slots, adapters, off = case
    n = len(off) - 1
    ids = (np.arange(n * slots).reshape(n, slots) * 7 + 1) % adapters
    ids[2::3, 0] = -1
    if slots > 1:
        ids[1::4, 1] = ids[1::4, 0]                                 # the same adapter twice, or none twice
    return ids


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:6]))
def test_matches_the_oracle(P, case):
    M, K, N, R, slots, adapters, off = case
    x, y, a, b = _make(M, K, N, R, slots, adapters)
    ids = _ids(case)
    w = _weights(ids)
    plan = P.LoraPlan(off, ids, w, M, adapters)
    before = y.clone()
    out = P.svdq_lora_add(x, y, a, b, plan)
    _check(out, x, y, a, b, off, ids, w)
    assert torch.equal(y, before)
    assert torch.equal(out, P.svdq_lora_add(x, y, a, b, plan)), "repeat calls are bit-identical"
    in_place = y.clone()
    assert P.svdq_lora_add(x, in_place, a, b, plan, out=in_place) is in_place
    assert torch.equal(in_place, out)
    assert P.svdq_device_status() == 0


@pytest.mark.parametrize("case", [CASES[1], CASES[6], CASES[11], CASES[12]], ids=lambda c: str(c[0]))
def test_strided_rows_and_column_windows(P, case):
    M, K, N, R, slots, adapters, off = case
    x, y, a, b = _make(M, K, N, R, slots, adapters, seed=3)
    ids = _ids(case)
    w = _weights(ids)
    plan = P.LoraPlan(off, ids, w, M, adapters)
    wide_x = torch.full((M, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_x[:, 8:8 + K] = x
    wide = torch.full((M, 3 * N + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, N:2 * N] = y
    expect = P.svdq_lora_add(x, y, a, b, plan)
    # in place on the middle third of a packed projection
    P.svdq_lora_add(wide_x[:, 8:8 + K], wide[:, N:2 * N], a, b, plan, out=wide[:, N:2 * N])
    assert torch.equal(wide[:, N:2 * N], expect)
    assert (wide[:, :N] == 7).all() and (wide[:, 2 * N:] == 7).all()
    # from one window into another of the same buffer
    wide[:, N:2 * N] = y
    P.svdq_lora_add(x, wide[:, N:2 * N], a, b, plan, out=wide[:, 2 * N:3 * N])
    assert torch.equal(wide[:, 2 * N:3 * N], expect) and torch.equal(wide[:, N:2 * N], y)
    assert (wide[:, :N] == 7).all() and (wide[:, 3 * N:] == 7).all()


def test_untouched_rows_keep_their_bits(P):
    """In place, rows of no request and of no adapter are left as they were, NaN payloads included;
    out of place they are copied."""
    M, K, N = 260, 128, 192
    x, y, a, b = _make(M, K, N, 16, 1, 2)
    off, ids = [2, 4, 140, 250], np.array([[0], [-1], [1]])
    keep = [0, 1] + list(range(4, 140)) + list(range(250, 260))
    y[keep] = torch.randint(-32768, 32767, (len(keep), N), dtype=torch.int16, device="cuda").view(torch.bfloat16)
    x[keep] = float("nan")
    plan = P.LoraPlan(off, ids, np.ones((3, 1)), M, 2)
    for out in (y.clone(), None):
        src = y if out is None else out
        got = P.svdq_lora_add(x, src, a, b, plan, out=out)
        assert torch.equal(got.view(torch.int16)[keep], y.view(torch.int16)[keep])
        touched = [i for i in range(M) if i not in keep]
        assert torch.isfinite(got[touched].float()).all()


@pytest.mark.parametrize("rows", [[0, 5, 9], [0, 140, 300]])
def test_a_bad_row_stays_alone(P, rows):
    """NaN and infinity in a row of X reach that row only; an empty slot does not turn them into NaN."""
    M, K, N = rows[-1], 192, 128
    x, y, a, b = _make(M, K, N, 32, 2, 3)
    ids = np.array([[-1, -1], [0, -1]])
    w = np.ones((2, 2), np.float32)
    x[1] = float("inf")
    x[rows[1] + 1] = float("nan")
    got = P.svdq_lora_add(x, y, a, b, P.LoraPlan(rows, ids, w, M, 3))
    assert torch.equal(got[: rows[1]], y[: rows[1]])
    bad = torch.isnan(got.float()).any(1).nonzero().flatten().tolist()
    assert bad == [rows[1] + 1]
    ids = np.array([[-1, 1], [0, 2]])
    x[1] = 1.0
    got = P.svdq_lora_add(x, y, a, b, P.LoraPlan(rows, ids, w, M, 3))
    keep = [i for i in range(M) if i != rows[1] + 1]
    x[rows[1] + 1] = 0.0
    ref, us, ks = oracle.forward(_np(x), _np(y), _np(a), _np(b), rows, ids, w)
    assert (np.abs(_np(got) - ref) <= oracle.bound(ref, us, ks, K, 64))[keep].all()


def test_graph_replays_read_the_plan_again(P):
    M, K, N = 150, 256, 192
    x, y, a, b = _make(M, K, N, 32, 1, 4)
    off = [0, 1, 3, 140]
    w = _weights([[0], [0], [0]])
    ids1, ids2 = np.array([[0], [1], [2]]), np.array([[3], [2], [0]])
    p1, p2 = P.LoraPlan(off, ids1, w, M, 4), P.LoraPlan(off, ids2, -w, M, 4)
    assert p1.sizes() == p2.sizes()
    out = torch.empty_like(y)
    P.svdq_lora_add(x, y, a, b, p1, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.svdq_lora_add(x, y, a, b, p1, out=out)
    out.zero_()
    graph.replay()
    _check(out, x, y, a, b, off, ids1, w)
    p1.words.copy_(p2.words)
    x.mul_(0.5)
    graph.replay()
    _check(out, x, y, a, b, off, ids2, -w)


def test_two_streams_at_once(P):
    sets = []
    for i, (M, off) in enumerate([(600, [0, 1, 300, 600]), (48, list(range(49)))]):
        x, y, a, b = _make(M, 512, 512, 64, 1, 3, seed=i)
        ids = np.arange(len(off) - 1)[:, None] % 3
        w = _weights(ids)
        sets.append((x, y, a, b, off, ids, w, P.LoraPlan(off, ids, w, M, 3), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, (x, y, a, b, off, ids, w, plan, stream) in enumerate(sets):
            with torch.cuda.stream(stream):
                outs[i].append(P.svdq_lora_add(x, y, a, b, plan))
    torch.cuda.synchronize()
    for i, (x, y, a, b, off, ids, w, plan, _) in enumerate(sets):
        _check(outs[i][0], x, y, a, b, off, ids, w)
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])


def test_the_next_requests_nan_rows_do_not_reach_a_partial_tile(P):
    """A tile of 78 rows is loaded in slabs of 32: the rows behind it belong to the next request."""
    M, K, N = 300, 256, 192
    x, y, a, b = _make(M, K, N, 32, 1, 2)
    off, ids = [0, 78, 156, 300], np.array([[0], [1], [0]])
    w = _weights(ids)
    plan = P.LoraPlan(off, ids, w, M, 2)
    expect = P.svdq_lora_add(x, y, a, b, plan)
    x[78:156] = float("nan")
    y[156:] = float("inf")
    got = P.svdq_lora_add(x, y, a, b, plan)
    assert torch.equal(got[:78], expect[:78])
    assert torch.isnan(got[78:156].float()).all() and torch.isinf(got[156:].float()).all()


@pytest.mark.parametrize("off", [[0, 4200], [0, 4000, 4001, 4017, 4200], list(range(0, 4201, 10))])
def test_offsets_past_32_bits(P, off):
    """Rows 2^20 elements apart: the last ones start beyond 2^32 elements (and 2^33 bytes)."""
    M, K, N, ld = 4200, 64, 128, 1 << 20
    x, y, a, b = _make(M, K, N, 16, 1, 3)
    wide = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")
    wide[:, 512:512 + N] = y
    wide[:, 512 + N:1024] = 3.0
    ids = np.arange(len(off) - 1)[:, None] % 3
    w = _weights(ids)
    plan = P.LoraPlan(off, ids, w, M, 3)
    win = wide[:, 512:512 + N]
    P.svdq_lora_add(x, win, a, b, plan, out=win)
    assert torch.equal(win, P.svdq_lora_add(x, y, a, b, plan))
    assert (wide[:, 512 + N:1024] == 3).all()


def test_many_adapters_in_one_batch(P):
    """More requests than a wave has CTAs, each row its own adapter; and long requests of one row more than a
    tile."""
    M, K, N = 700, 64, 64
    x, y, a, b = _make(M, K, N, 16, 1, 700)
    off, ids = list(range(M + 1)), np.arange(M)[:, None]
    w = _weights(ids)
    _check(P.svdq_lora_add(x, y, a, b, P.LoraPlan(off, ids, w, M, M)), x, y, a, b, off, ids, w)
    off, ids = [0, 129, 258, 387, 516, 645], np.array([[5], [5], [699], [-1], [0]])
    w = _weights(ids)
    _check(P.svdq_lora_add(x, y, a, b, P.LoraPlan(off, ids, w, M, M)), x, y, a, b, off, ids, w)


@pytest.mark.parametrize("case", [
    (20011, 128, 192, 64, 2, 3, [0, 7000, 7003, 19900, 20000]),     # more tiles than SMs, slices of one
    (3001, 256, 2624, 32, 1, 3, [0, 500, 510, 2000, 2900]),         # many pieces per CTA, the last of 64 columns
], ids=["tiles", "pieces"])
def test_more_tiles_or_pieces_than_sms(P, case):
    M, K, N, R, slots, adapters, off = case
    x, y, a, b = _make(M, K, N, R, slots, adapters)
    ids = _ids(case)
    w = _weights(ids)
    plan = P.LoraPlan(off, ids, w, M, adapters)
    out = P.svdq_lora_add(x, y, a, b, plan)
    _check(out, x, y, a, b, off, ids, w)
    assert torch.equal(P.svdq_lora_add(x, y, a, b, plan, out=y), out)
    assert P.svdq_device_status() == 0


def test_the_output_carries_no_autograd_graph(P):
    """The calls are for inference, as the layers' are: their results are no part of a graph."""
    x, y, a, b = _make(20, 64, 64, 16, 1, 1)
    plan = P.LoraPlan([0, 20], [0], [1.0], 20, 1)
    out = P.svdq_lora_add(x.requires_grad_(), y, a, b, plan)
    assert not out.requires_grad


def test_device_and_stream(P):
    """On a side stream, ordered by events with the tensors' own; a plan on the host is refused."""
    x, y, a, b = _make(200, 512, 256, 32, 1, 2)
    off, ids = [0, 5, 200], np.array([[0], [1]])
    w = _weights(ids)
    plan = P.LoraPlan(off, ids, w, 200, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = P.svdq_lora_add(x, y, a, b, plan)
    torch.cuda.current_stream().wait_stream(side)
    _check(out, x, y, a, b, off, ids, w)
    with pytest.raises(ValueError, match="CUDA tensor"):
        P.svdq_lora_add(x, y, a, b, P.LoraPlan(off, ids, w, 200, 2, device="cpu"))


@pytest.mark.parametrize("rows", [17, 31, 47, 63, 97, 127])
def test_partial_slabs_through_a_turning_ring(P, rows):
    """Tiles that end inside a 32-row slab are stored row by row from a stage that TMA then refills; with more
    pieces per CTA than stages every stage is refilled.  The rows are those of whole slabs, bit for bit: a row's
    sums do not depend on its tile (as many tiles, so K is split alike)."""
    n, K, N, whole = 40, 128, 5120, (rows + 31) // 32 * 32
    x, y, a, b = _make(n * whole, K, N, 32, 1, 3)
    ids = np.arange(n)[:, None] % 3
    w = _weights(ids)
    expect = P.svdq_lora_add(x, y, a, b, P.LoraPlan(whole * np.arange(n + 1), ids, w, n * whole, 3))

    def short(t):
        return t.view(n, whole, -1)[:, :rows].reshape(n * rows, -1).contiguous()

    plan = P.LoraPlan(rows * np.arange(n + 1), ids, w, n * rows, 3)
    xs, ys = short(x), short(y)
    for _ in range(10):
        assert torch.equal(P.svdq_lora_add(xs, ys, a, b, plan), short(expect))
        in_place = ys.clone()
        assert torch.equal(P.svdq_lora_add(xs, in_place, a, b, plan, out=in_place), short(expect))
    off = rows * np.arange(n + 1)
    _check(short(expect), xs, ys, a, b, off, ids, w)
    assert P.svdq_device_status() == 0


@pytest.mark.parametrize("case", [
    (400, 192, 320, 16, 8, 5, [0, 17, 150, 390]),                   # eight slots
    (300, 128, 192, 96, 1, 3, [0, 130, 150, 300]),                  # three boxes of 32 ranks
    (300, 128, 192, 48, 2, 3, [0, 130, 150, 300]),                  # three boxes of 16 ranks, twice
    (260, 64, 64, 16, 7, 3, [0, 240, 260]),                         # 112 ranks in seven slots
], ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_ranks_and_slots_of_long_requests(P, case):
    M, K, N, R, slots, adapters, off = case
    x, y, a, b = _make(M, K, N, R, slots, adapters, seed=8)
    ids = _ids(case)
    ids[0, slots - 1] = -1
    w = _weights(ids)
    out = P.svdq_lora_add(x, y, a, b, P.LoraPlan(off, ids, w, M, adapters))
    _check(out, x, y, a, b, off, ids, w)
    assert P.svdq_device_status() == 0


@pytest.mark.parametrize("off", [[0, 3, 20], [0, 140, 300]])
def test_other_adapters_of_the_pool_are_not_read_into_a_result(P, off):
    M, K, N = off[-1], 128, 192
    x, y, a, b = _make(M, K, N, 48, 1, 3)
    a[0] = b[0] = a[2] = b[2] = float("nan")
    ids = np.array([[1], [1]])
    w = _weights(ids)
    _check(P.svdq_lora_add(x, y, a, b, P.LoraPlan(off, ids, w, M, 3)), x, y, a[1:2], b[1:2], off, ids * 0, w)


def test_a_pool_past_32_bits(P):
    """The last adapter's B starts beyond 2^31 elements."""
    adapters, N, K, R, off = 1200, 15360, 64, 128, [0, 5, 40]
    b = torch.empty((adapters, N, R), dtype=torch.bfloat16, device="cuda")
    x, y, a1, b1 = _make(off[-1], K, N, R, 1, 1)
    a = torch.zeros((adapters, R, K), dtype=torch.bfloat16, device="cuda")
    a[-1], b[-1] = a1[0], b1[0]
    assert (adapters - 1) * N * R > 2 ** 31
    w = _weights([[0], [0]])
    big = P.svdq_lora_add(x, y, a, b, P.LoraPlan(off, [adapters - 1] * 2, w.ravel(), off[-1], adapters))
    assert torch.equal(big, P.svdq_lora_add(x, y, a1, b1, P.LoraPlan(off, [0, 0], w.ravel(), off[-1], 1)))


def test_more_groups_than_a_grid_axis_of_16_bits(P):
    """A row per request and an adapter per row: 70000 groups, whose parts are formed and added at once."""
    M, K, N, R = 70000, 64, 64, 16
    x, y, a, b = _make(M, K, N, R, 1, M)
    off, ids = np.arange(M + 1), np.arange(M)[::-1].copy()
    w = _weights(ids)
    plan = P.LoraPlan(off, ids, w, M, M)
    assert plan.struct.groups == M
    out = P.svdq_lora_add(x, y, a, b, plan)
    pick = np.concatenate([[0, 1, M - 1], np.random.default_rng(0).integers(0, M, 500)])
    at = torch.from_numpy(pick).cuda()
    idt = torch.from_numpy(ids[pick]).cuda()
    _check(out[at], x[at], y[at], a[idt], b[idt], np.arange(len(pick) + 1), np.arange(len(pick))[:, None], w[pick, None])


def test_a_workspace_of_the_callers(P):
    """One workspace serves calls of one stream after another; a short or misplaced one is refused."""
    M, K, N = 300, 256, 192
    x, y, a, b = _make(M, K, N, 32, 1, 3)
    plans = [P.LoraPlan([0, 200, 204], [0, 1], [1.0, 2.0], M, 3), P.LoraPlan(list(range(41)), np.arange(40) % 3, np.ones(40), M, 3)]
    need = [P.svdq_lora_workspace_bytes(p, K, 32) for p in plans]
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    expect = [P.svdq_lora_add(x, y, a, b, p) for p in plans]
    got = [P.svdq_lora_add(x, y, a, b, p, workspace=ws) for _ in range(3) for p in plans]
    assert all(torch.equal(g, expect[i % 2]) for i, g in enumerate(got))
    with pytest.raises(ValueError, match="workspace"):
        P.svdq_lora_add(x, y, a, b, plans[0], workspace=ws[:need[0] - 16])
    with pytest.raises(ValueError, match="workspace"):
        P.svdq_lora_add(x, y, a, b, plans[0], workspace=ws.cpu())
