"""Rotary positions with several axes on the GPU: the norm-and-rotate call and the tables against the
float64 oracle, strided and in-place heads, far and fractional positions, and the fused projection fed
with the tables."""

import numpy as np
import pytest
import torch

from oracle import rope_axes as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P(cuda_lib):
    return cuda_lib


def _np(t):
    return t.detach().double().cpu().numpy()


def _positions(P_, axes, fractional, seed):
    r = np.random.default_rng(seed)
    pos = r.integers(-200, 70000, size=(P_, axes))
    pos[0] = 0
    if fractional:
        return torch.from_numpy((pos * 0.3125).astype(np.float32)).cuda()
    return torch.from_numpy(pos.astype(np.int32)).cuda()


def _check(got, x, w, eps, pos, dims, thetas, half, M):
    ang = oracle.angles(_np(pos), dims, thetas)
    ang = np.tile(ang, (M // ang.shape[0], 1))
    n = oracle.norm(_np(x), None if w is None else _np(w), eps)
    ref = oracle.rotate(n, ang, half)
    tol = oracle.bound(n, ref, half, sum(dims), x.shape[2])
    bad = ~(np.abs(_np(got) - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], np.max(np.abs(_np(got) - ref) / tol))


# M, P, q heads, k heads, D, dims, thetas
CASES = [
    (1, 1, 1, 1, 8, [8], [10000.0]),
    (1, 1, 20, 20, 128, [16, 56, 56], [10000.0] * 3),
    (3, 3, 5, 3, 128, [44, 42, 42], [10000.0, 100.0, 1e6]),
    (77, 77, 3, 1, 64, [64], [10000.0]),
    (50, 25, 4, 4, 96, [24, 36, 36], [256.0] * 3),
    (33, 11, 2, 7, 80, [16, 32, 32], [10000.0] * 3),
    (40, 40, 2, 2, 256, [32, 64, 64], [10000.0] * 3),            # 96 columns past the rotated ones
    (19, 19, 3, 3, 40, [2, 6, 16], [10000.0] * 3),               # runs of four pairs, a tail
    (21, 21, 1, 2, 248, [120, 128], [500.0, 10000.0]),
    (12, 12, 2, 1, 16, [2, 2, 2, 2, 2, 2, 2, 2], [3.0, 4.0, 5.0, 6.0, 7.0, 8.0, 9.0, 10.0]),
    (1025, 1025, 2, 2, 24, [8, 8], [10000.0] * 2),
]


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_matches_the_oracle(P, case, half):
    M, Pn, hq, hk, D, dims, thetas = case
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((M, (hq + 2 * hk) * D), generator=g, device="cuda").to(torch.bfloat16)
    q, k = qkv[:, : hq * D].view(M, hq, D), qkv[:, hq * D:(hq + hk) * D].view(M, hk, D)
    wq = torch.randn(D, generator=g, device="cuda").to(torch.bfloat16)
    wk = torch.randn(D, generator=g, device="cuda").to(torch.bfloat16)
    pos = _positions(Pn, len(dims), half, 5)
    keep = qkv.clone()
    pairing = "half" if half else "interleaved"
    theta = thetas[0] if len(set(thetas)) == 1 else thetas
    oq, ok = P.svdq_qk_norm_rope(q, k, wq, wk, 1e-6, pos, dims, theta, pairing)
    assert torch.equal(qkv, keep)
    _check(oq, q, wq, 1e-6, pos, dims, thetas, half, M)
    _check(ok, k, wk, 1e-6, pos, dims, thetas, half, M)
    # without a norm, and one of the two alone
    nq, nk = P.svdq_qk_norm_rope(q, k, None, wk, 1e-6, pos, dims, theta, pairing)
    _check(nq, q, None, 0.0, pos, dims, thetas, half, M)
    assert torch.equal(nk, ok)
    only, none = P.svdq_qk_norm_rope(None, k, None, wk, 1e-6, pos, dims, theta, pairing)[::-1]
    assert none is None and torch.equal(only, ok)
    # head-major outputs, then in place on the packed projection (v stays)
    hm = torch.zeros((hq, M, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    P.svdq_qk_norm_rope(q, None, wq, None, 1e-6, pos, dims, theta, pairing, out_q=hm)
    assert torch.equal(hm, oq)
    P.svdq_qk_norm_rope(q, k, wq, wk, 1e-6, pos, dims, theta, pairing, out_q=q, out_k=k)
    assert torch.equal(q, oq) and torch.equal(k, ok)
    assert torch.equal(qkv[:, (hq + hk) * D:], keep[:, (hq + hk) * D:])


@pytest.mark.parametrize("case", CASES + [(4096, 2048, 0, 0, 128, [16, 56, 56], [10000.0] * 3)],
                         ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_tables_match_the_oracle(P, case):
    M, Pn, _, _, D, dims, thetas = case
    for fractional in (False, True):
        pos = _positions(Pn, len(dims), fractional, 9)
        cos, sin = P.svdq_rope_axes_tables(pos, dims, thetas, D, M)
        assert cos.shape == sin.shape == (D // 2, M)
        ang = np.tile(oracle.angles(_np(pos), dims, thetas), (M // Pn, 1)).T
        # the reduced angle's rounding (at most 2^-25 half turns, times pi) and the two ulp of the
        # sine and cosine; the 64-bit angle by 2^-45 of its size
        tol = 2.0 ** -22 + np.abs(ang) * 2.0 ** -45
        n = ang.shape[0]
        assert (np.abs(_np(cos)[:n] - np.cos(ang)) <= tol).all()
        assert (np.abs(_np(sin)[:n] - np.sin(ang)) <= tol).all()
        assert (cos[n:] == 1).all() and (sin[n:] == 0).all()


def test_zero_and_infinite_rows(P):
    """A zero head stays zero (eps under the root); a NaN stays in its head; columns past the rotated
    ones are not touched by their neighbours."""
    q = torch.randn((4, 3, 64), device="cuda").to(torch.bfloat16)
    q[0, 1] = 0
    q[2, 0, 5] = float("nan")
    q[3, 2, 40] = float("inf")
    pos = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out, _ = P.svdq_qk_norm_rope(q, None, w, None, 1e-6, pos, [8, 8], 100.0)
    assert (out[0, 1] == 0).all()
    assert torch.isnan(out[2, 0].float()).all() and torch.isfinite(out[2, 1:].float()).all()
    plain, _ = P.svdq_qk_norm_rope(q, None, None, None, 0.0, pos, [8, 8], 100.0)
    assert torch.equal(plain[3, 2, 16:], q[3, 2, 16:])
    assert torch.equal(plain[:, :, 16:].view(torch.int16), q[:, :, 16:].contiguous().view(torch.int16))


def test_far_positions_keep_their_angle(P):
    """Positions near 2^31, where a product in 32 bits has no correct digit left."""
    pos = torch.tensor([[2 ** 31 - 1], [-(2 ** 31)], [2 ** 30 + 1]], dtype=torch.int32, device="cuda")
    cos, sin = P.svdq_rope_axes_tables(pos, [64], 10000.0, 64)
    ang = oracle.angles(_np(pos), [64], [10000.0]).T
    tol = 2.0 ** -22 + np.abs(ang) * 2.0 ** -45
    assert (np.abs(_np(cos) - np.cos(ang)) <= tol).all() and (np.abs(_np(sin) - np.sin(ang)) <= tol).all()


def test_offsets_past_32_bits(P):
    """Tokens 2^20 elements apart: the last ones start beyond 2^32 elements."""
    M, H, D, ld = 4200, 3, 64, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((M, H, D), generator=g, device="cuda").to(torch.bfloat16)
    wide = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")
    wide[:, 512:512 + H * D] = q.view(M, H * D)
    wide[:, 512 + H * D:1024] = 3.0
    win = wide[:, 512:512 + H * D].unflatten(1, (H, D))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    pos = _positions(M, 2, False, 1)
    expect, _ = P.svdq_qk_norm_rope(q, None, w, None, 1e-6, pos, [32, 32], 1e4)
    P.svdq_qk_norm_rope(win, None, w, None, 1e-6, pos, [32, 32], 1e4, out_q=win)
    assert torch.equal(win, expect) and (wide[:, 512 + H * D:1024] == 3).all()


def test_a_slice_of_positions_and_every_token_alone(P):
    """Positions that start anywhere in a longer list; one token at a time gives the same bits."""
    q = torch.randn((40, 20, 128), device="cuda").to(torch.bfloat16)
    k = torch.randn((40, 4, 128), device="cuda").to(torch.bfloat16)
    w = torch.randn(128, device="cuda").to(torch.bfloat16)
    for fractional in (False, True):
        pos = _positions(43, 3, fractional, 3)
        a = P.svdq_qk_norm_rope(q, k, w, w, 1e-5, pos[3:], [16, 56, 56], 1e4)
        for m in (0, 1, 17, 39):
            b = P.svdq_qk_norm_rope(q[m:m + 1], k[m:m + 1], w, w, 1e-5, pos[3 + m:4 + m], [16, 56, 56], 1e4)
            assert torch.equal(a[0][m:m + 1], b[0]) and torch.equal(a[1][m:m + 1], b[1])


def test_many_heads_and_units(P):
    """More heads than a stage holds, few and many tokens, uneven q and k."""
    g = torch.Generator(device="cuda").manual_seed(7)
    w = torch.randn(128, generator=g, device="cuda").to(torch.bfloat16)
    for M, hq, hk in ((1, 130, 1), (5, 64, 8), (600, 70, 3), (2400, 24, 24), (5000, 1, 9)):
        q = torch.randn((M, hq, 128), generator=g, device="cuda").to(torch.bfloat16)
        k = torch.randn((M, hk, 128), generator=g, device="cuda").to(torch.bfloat16)
        pos = _positions(M, 3, False, M)
        oq, ok = P.svdq_qk_norm_rope(q, k, w, None, 1e-6, pos, [44, 42, 42], 1e4)
        pick = sorted({0, M // 2, M - 1})
        for out, x, nw in ((oq, q, w), (ok, k, None)):
            _check(out[pick], x[pick], nw, 1e-6, pos[pick], [44, 42, 42], [1e4] * 3, False, len(pick))
        # all tokens against the halves' kernel on columns sorted even before odd (its sums differ in order)
        order = torch.cat([torch.arange(0, 128, 2), torch.arange(1, 128, 2)]).cuda()
        hq_, _ = P.svdq_qk_norm_rope(q[..., order].contiguous(), None, w[order].contiguous(), None, 1e-6, pos, [44, 42, 42],
                                     1e4, "half")
        d = (hq_.float() - oq[..., order].float()).abs()
        assert (d <= 2.0 ** -7 * oq[..., order].float().abs() + 2.0 ** -14).all()


def test_nan_positions_and_nothing_else(P):
    q = torch.randn((3, 2, 16), device="cuda").to(torch.bfloat16)
    pos = torch.tensor([[1.0], [float("nan")], [float("inf")]], device="cuda")
    out, _ = P.svdq_qk_norm_rope(q, None, None, None, 0.0, pos, [8], 100.0)
    assert torch.isfinite(out[0].float()).all()
    assert torch.isnan(out[1:, :, :8].float()).all() and torch.equal(out[1:, :, 8:], q[1:, :, 8:])
    cos, sin = P.svdq_rope_axes_tables(pos, [8], 100.0, 16)
    assert torch.isnan(cos[:4, 1:]).all() and torch.isnan(sin[:4, 1:]).all() and (cos[4:] == 1).all()


def test_a_graph_reads_new_positions(P):
    q = torch.randn((300, 4, 64), device="cuda").to(torch.bfloat16)
    pos, other = _positions(300, 2, False, 1), _positions(300, 2, False, 2)
    P.svdq_qk_norm_rope(q, None, None, None, 0.0, pos, [32, 32], 1e4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = P.svdq_qk_norm_rope(q, None, None, None, 0.0, pos, [32, 32], 1e4)
        cos, _ = P.svdq_rope_axes_tables(pos, [32, 32], 1e4, 64)
    pos.copy_(other)
    graph.replay()
    assert torch.equal(out, P.svdq_qk_norm_rope(q, None, None, None, 0.0, other, [32, 32], 1e4)[0])
    assert torch.equal(cos, P.svdq_rope_axes_tables(other, [32, 32], 1e4, 64)[0])
    assert P.svdq_device_status() == 0


def test_axes_given_as_tensors_are_read_at_every_call(P):
    pos = _positions(40, 2, False, 3)
    theta, dims = torch.tensor(1e4), torch.tensor([16, 8])
    first = P.svdq_rope_axes_tables(pos, dims, theta, 32)[0]
    assert torch.equal(first, P.svdq_rope_axes_tables(pos, [16, 8], 1e4, 32)[0])
    theta.fill_(100.0)
    dims.copy_(torch.tensor([8, 16]))
    assert torch.equal(P.svdq_rope_axes_tables(pos, dims, theta, 32)[0], P.svdq_rope_axes_tables(pos, [8, 16], 100.0, 32)[0])
    thetas = [theta, torch.tensor(1e3)]
    P.svdq_rope_axes_tables(pos, np.array([8, 16]), thetas, 32)
    thetas[1].fill_(10.0)
    assert torch.equal(P.svdq_rope_axes_tables(pos, [8, 16], thetas, 32)[0],
                       P.svdq_rope_axes_tables(pos, [8, 16], [100.0, 10.0], 32)[0])


@pytest.mark.parametrize("theta,d", [(1e4, 56), (1e6, 64), (1e9, 64), (256.0, 36), (3.0, 2)])
def test_small_angles_are_rounded_to_the_nearest_unit(P, theta, d):
    """The angle is rounded to 2^-32 turns (half a unit, 2^-33 turns, and 2^-64 turns per unit of position for the
    frequency); sine and cosine are off by 4.5 * 2^-24 of themselves -- the reduced angle as a float by three
    roundings, which reach them with a factor of at most 1, the polynomial's last rounding, and less than half a
    rounding of its inner terms and its remainder; the float64 angle by a few 2^-53.  Cut off instead of rounded, the
    angle is off by twice as much, which small angles show."""
    r = np.random.default_rng(0)
    near = np.array([0, 1, -1, 2, -2, 3, 17, -200, 96, 1000, 4097, 69999, -69999])
    pos = np.concatenate([near, r.integers(-200, 70000, 243)])
    width = (d + 7) // 8 * 8
    dims, thetas = ([d], [theta]) if width == d else ([d, width - d], [theta, 1e4])
    both = np.stack([pos] * len(dims), 1)
    ang = oracle.angles(both, dims, thetas).T
    for t in (torch.int32, torch.float32):
        cos, sin = P.svdq_rope_axes_tables(torch.from_numpy(both).to(t).cuda(), dims, thetas, width)
        for got, exact in ((cos, np.cos(ang)), (sin, np.sin(ang))):
            tol = 2 * np.pi * (2.0 ** -33 + np.abs(pos) * 2.0 ** -64) + 4.5 * 2.0 ** -24 * np.abs(exact) + \
                np.abs(ang) * 2.0 ** -50
            assert (np.abs(_np(got) - exact) <= tol).all()


@pytest.mark.parametrize("M", [1, 300])
def test_q_k_and_v_of_a_head_side_by_side(P, M):
    """[M, heads, 3, D] in place: as from separate tensors, v as it was."""
    g = torch.Generator(device="cuda").manual_seed(11)
    packed = torch.randn((M, 5, 3, 64), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(64, generator=g, device="cuda").to(torch.bfloat16)
    pos = _positions(M, 2, False, 4)
    keep = packed.clone()
    q, k, v = packed.unbind(2)
    eq, ek = P.svdq_qk_norm_rope(q.contiguous(), k.contiguous(), w, None, 1e-6, pos, [32, 24], 1e4)
    P.svdq_qk_norm_rope(q, k, w, None, 1e-6, pos, [32, 24], 1e4, out_q=q, out_k=k)
    assert torch.equal(q, eq) and torch.equal(k, ek) and torch.equal(v, keep[:, :, 2])
